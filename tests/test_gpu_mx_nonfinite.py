"""GPU: NaN and infinities in the activations of the block-scaled formats.  A block of 32 values that holds one has scale
255 and reads as NaN, in every call and on both sides of the sizes where a call changes its kernels; the token's row
is NaN and no other row is touched."""
import math

import pytest
import torch

import mx4_ref as R
from expert_routed_grouped_amd import layer as L
from expert_routed_grouped_amd import moe, synth
from test_gpu_mx4 import DEV, gen, quantize_act, setup

pytestmark = pytest.mark.gpu
BAD = [math.nan, -math.nan, math.inf, -math.inf]


@pytest.mark.parametrize("bad", BAD, ids=["nan", "-nan", "inf", "-inf"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("at", [0, 7, 8, 31])
def test_quantize_mx(bad, dtype, at):
    g = gen(1)
    x = torch.randn((5, 160), device=DEV, generator=g).to(dtype)
    x[4] = torch.finfo(dtype).max  # the largest finite values are none of it
    want, s = moe.moe_quantize_mx(x)
    assert int(s.max()) <= 254 - 7
    y = x.clone()
    y[1, 32 + at] = y[3, 128 + at] = bad
    codes, scales = moe.moe_quantize_mx(y)
    hit = torch.zeros((5, 5), dtype=torch.bool, device=DEV)
    hit[1, 1] = hit[3, 4] = True
    assert torch.equal(scales, torch.where(hit, 255, s.int()).to(torch.uint8))
    assert torch.equal(codes, torch.where(hit.repeat_interleave(32, 1), 0, want.int()).to(torch.uint8))
    assert torch.equal(moe.moe_dequantize_mx(codes, scales).isnan(), hit.repeat_interleave(32, 1))


def check_rows(y0, y1, bad):
    """Row ``bad`` of y1 is NaN throughout; every other row is y0's, bit for bit, and finite."""
    keep = torch.arange(y0.shape[0], device=DEV) != bad
    assert bool(y1[bad].isnan().all())
    assert torch.equal(y1[keep], y0[keep]) and bool(y1[keep].isfinite().all())


@pytest.mark.parametrize("T", [40, 64, 65, 300])
@pytest.mark.parametrize("act", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("bad", [math.nan, math.inf], ids=["nan", "inf"])
def test_ffn_mx4_through_the_quantiser(T, act, bad):
    s = setup(T, 4, 2, 256, 128, 0, 4, seed=21)
    p = moe.moe_permute(s["ids"], s["gates"], 4, 0, 4)
    args = (p["offsets"], p["row_token"], p["row_w"], p["token_row"], s["wgu"], s["wd"])
    y0 = moe.moe_grouped_ffn_mx4(*quantize_act(s["x"], act), *args)
    s["x"][T // 2, 77] = bad
    check_rows(y0, moe.moe_grouped_ffn_mx4(*quantize_act(s["x"], act), *args), T // 2)


@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("act", ["mxfp8", "mxfp4"])
def test_ffn_mx4_intermediate_overflow(T, act):
    """Finite activations whose silu(G) U passes the largest fp32 value."""
    s = setup(T, 4, 2, 256, 128, 0, 4, seed=22)
    p = moe.moe_permute(s["ids"], s["gates"], 4, 0, 4)
    args = (p["offsets"], p["row_token"], p["row_w"], p["token_row"], s["wgu"], s["wd"])
    y0 = moe.moe_grouped_ffn_mx4(*quantize_act(s["x"], act), *args)
    s["x"][T // 2] *= 1e30
    check_rows(y0, moe.moe_grouped_ffn_mx4(*quantize_act(s["x"], act), *args), T // 2)


@pytest.mark.parametrize("T,E", [(20, 4), (600, 4)])  # weight streaming; tiles
@pytest.mark.parametrize("kind", ["nan", "inf", "overflow"])
def test_ffn_mx_rows(T, E, kind):
    """The W8A8 FFN with MXFP8 weights, per-row outputs."""
    g = gen(23)
    H, I = 256, 128
    w = [moe.moe_quantize_mx(torch.randn((E * n, k), device=DEV, generator=g) * 0.05) for n, k in ((2 * I, H), (H, I))]
    wgu, wd = ((c.view(E, -1, k), s.view(E, -1, k // 32)) for (c, s), k in zip(w, (H, I)))
    x = torch.randn((T, H), device=DEV, generator=g).bfloat16()
    top, ids = torch.randn((T, E), device=DEV, generator=g).topk(2, 1)
    p = moe.moe_permute(ids.int().contiguous(), torch.softmax(top, 1).contiguous(), E, 0, E)

    def run():
        rows = torch.empty((2 * T, H), dtype=torch.float32, device=DEV)
        moe.moe_grouped_ffn_mx(*moe.moe_quantize_mx(x), p["offsets"], p["row_token"], p["row_w"], T, 2 * T, *wgu, *wd,
                               y_perm=rows)
        return rows
    r0 = run()
    bad = T // 2
    if kind == "overflow":
        x[bad] *= 1e30
    else:
        x[bad, 77] = math.nan if kind == "nan" else math.inf
    r1 = run()
    hit = p["row_token"] == bad
    assert int(hit.sum()) == 2
    assert bool(r1[hit].isnan().all())
    assert torch.equal(r1[~hit], r0[~hit]) and bool(r1[~hit].isfinite().all())


@pytest.mark.parametrize("T", [1, 64, 65, 150])
@pytest.mark.parametrize("act", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("bad", [math.nan, math.inf], ids=["nan", "inf"])
def test_layer(T, act, bad):
    """run_layer with MXFP4 experts: the same on both sides of 64 tokens.  All experts are local, so that the bad token
    has rows wherever its NaN logits send it; the others are held to 64 bits."""
    cfg = synth.LayerConfig("mx4", T=T, H=512, E=24, k=4, I=256, seed=95, w_std=0.06)
    dev = L.to_device(synth.make_inputs(cfg))
    dev["x"] = R.even_rows((T, 512), gen(T), DEV)
    L.convert_experts_mx4(dev)
    bufs = L.Mx4LayerBuffers(cfg, act=act)
    x = dev["x"].clone()
    dev["x"][T // 2, 300] = bad
    y = L.run_layer(dev, bufs)
    ids, w = moe.moe_route(dev["x"], dev["w_router"], None, 4)
    assert torch.equal(ids, bufs.topk_ids) and torch.equal(w.isnan(), bufs.topk_w.isnan())
    keep = torch.arange(T, device=DEV) != T // 2
    assert bool(y[T // 2].isnan().all()) and torch.equal(w[keep], bufs.topk_w[keep])
    if T == 1:
        return
    xv, _ = R.quantize(x, act)
    q = {n: R.quantize(dev[n], "mxfp4")[0] for n in ("w_gate_up", "w_down")}
    mid, rad = R.layer(xv[keep], ids[keep], w[keep], 0, 24, lambda e: q["w_gate_up"][e], lambda e: q["w_down"][e], act,
                       y.dtype, rows_rounded=True)
    R.check_interval(y[keep], mid, rad, f"layer T={T} {act}")
