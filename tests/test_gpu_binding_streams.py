"""GPU: chains of calls on another stream that allocate their own results and workspaces, while the current stream goes on
allocating: what a call made for itself is not handed out while it is still in use."""
import pytest
import torch

from expert_routed_grouped_amd import layer as L
from expert_routed_grouped_amd import moe, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


def w4a8(dev, cfg, stream):
    ids, w = moe.moe_route(dev["x"], dev["w_router"], None, cfg.k, stream=stream)
    p = moe.moe_permute(ids, w, cfg.E, 0, cfg.E, stream=stream)
    codes, scales = moe.moe_quantize_mx(dev["x"], stream=stream)
    return moe.moe_grouped_ffn_mx4(codes, scales, p["offsets"], p["row_token"], p["row_w"], p["token_row"],
                                   dev["wgu_mx4"], dev["wd_mx4"], stream=stream)


def bf16(dev, cfg, stream):
    ids, w = moe.moe_route(dev["x"], dev["w_router"], None, cfg.k, stream=stream)
    p = moe.moe_permute(ids, w, cfg.E, 0, cfg.E, stream=stream)
    gu, dn = (moe.moe_pack_weights(dev[n], stream=stream) for n in ("w_gate_up", "w_down"))
    rows = moe._new((p["R_cap"], cfg.H), torch.float32, dev["x"].device, stream)
    moe.moe_grouped_ffn(dev["x"], p["offsets"], p["row_token"], p["row_w"], cfg.T, p["R_cap"], gu, dn, y_perm=rows,
                        packed=True, stream=stream)
    return moe.moe_combine(rows, p["token_row"], w, stream=stream)


@pytest.mark.parametrize("T", [30, 333])
@pytest.mark.parametrize("chain", [w4a8, bf16])
def test_own_buffers_on_a_stream(chain, T):
    cfg = synth.LayerConfig("streams", T=T, H=384, E=8, k=2, I=256, seed=96, w_std=0.06)
    dev = L.convert_experts_mx4(L.to_device(synth.make_inputs(cfg)))
    want = chain(dev, cfg, None)
    side = torch.cuda.Stream()
    for use in (side, side.cuda_stream):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        y = chain(dev, cfg, use)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV)
                for n in (512, 2 * T * 4, T * 384, T * 12, 2 * T * 256, 2 * T * 384 * 4, 8 * 512 * 384 * 2) for _ in range(3)]
        torch.cuda.current_stream().synchronize()
        side.synchronize()
        assert torch.equal(y, want), junk[0][0]
