"""CPU checks of the binding: what a call on a given stream allocates by itself belongs to that stream."""
import pytest
import torch

from expert_routed_grouped_amd import moe

T, E, K, H, I = 4, 4, 2, 128, 64
bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
f32 = lambda *s: torch.zeros(s)  # noqa: E731
MAPS = (i32(E + 1), i32(T * K), f32(T * K))

CALLS = {  # name: (tensors it allocates, the call)
    "moe_route": (2, lambda s: moe.moe_route(bf(T, H), bf(E, H), None, K, stream=s)),
    "moe_permute": (7, lambda s: moe.moe_permute(i32(T, K), f32(T, K), E, 0, E, x=bf(T, H), stream=s)),
    "moe_grouped_ffn": (1, lambda s: moe.moe_grouped_ffn(bf(T, H), *MAPS, T, T * K, bf(E, 2 * I, H), bf(E, H, I),
                                                         y=f32(T, H), stream=s)),
    "moe_quantize_mx": (2, lambda s: moe.moe_quantize_mx(bf(T, H), stream=s)),
    "moe_grouped_ffn_mx": (1, lambda s: moe.moe_grouped_ffn_mx(
        u8(T, H), u8(T, H // 32), *MAPS, T, T * K, u8(E, 256, H), u8(E, 256, H // 32), u8(E, H, 128), u8(E, H, 4),
        y=f32(T, H), stream=s)),
    "moe_combine": (1, lambda s: moe.moe_combine(f32(T * K, H), i32(T, K), f32(T, K), stream=s)),
    "moe_shared_expert": (1, lambda s: moe.moe_shared_expert(bf(T, H), bf(2 * I, H), bf(H, I), f32(T, H), stream=s)),
    "moe_pack_weights": (1, lambda s: moe.moe_pack_weights(bf(E, 2 * I, H), stream=s)),
    "moe_pack_router": (1, lambda s: moe.moe_pack_router(bf(E, H), stream=s)),
    "moe_quantize_mx4": (2, lambda s: moe.moe_quantize_mx4(bf(T, H), stream=s)),
    "moe_dequantize_mx": (1, lambda s: moe.moe_dequantize_mx(u8(T, H // 2), u8(T, H // 32), stream=s)),
    "moe_pack_mx4": (2, lambda s: moe.moe_pack_mx4(u8(E, 32, H // 2), u8(E, 32, H // 32), stream=s)),
}


@pytest.mark.parametrize("name", CALLS)
def test_own_buffers_belong_to_the_stream(name, monkeypatch):
    """Every buffer goes through ``_new`` with the stream of the call.  (Host tensors: the call ends before the library.)"""
    n, call = CALLS[name]
    made, empty, stream = [], torch.empty, object()
    monkeypatch.setattr(moe, "_new", lambda shape, dtype, device, stream: made.append(stream) or empty(shape, dtype=dtype))
    for f in ("empty", "empty_like"):
        monkeypatch.setattr(torch, f, lambda *a, **k: pytest.fail("allocated on the current stream"))
    with pytest.raises(ValueError, match="on the GPU"):
        call(stream)
    assert made == [stream] * n
