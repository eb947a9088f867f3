"""GPU: the MXFP4 calls (moe_quantize_mx4, moe_dequantize_mx, moe_pack_mx4, moe_grouped_ffn_mx4) against plain
64-bit formulations (tests/mx4_ref.py), through the C ABI."""
import math

import pytest
import torch

import mx4_ref as R
from expert_routed_grouped_amd import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (7, 4096), (65, 1536), (1000, 160)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_is_exact(rows, K, dtype):
    g = gen(rows * K)
    x = torch.randn((rows, K), device=DEV, generator=g) * torch.exp2(30 * torch.randn((rows, 1), device=DEV, generator=g))
    x = x.clamp(-3e38, 3e38).to(dtype)
    v, s = R.quantize(x, "mxfp4")
    codes, scales = moe.moe_quantize_mx4(x)
    assert torch.equal(scales.long(), s)
    assert torch.equal(codes, R.codes4(v, s))
    for out in (torch.float32, torch.bfloat16):
        assert torch.equal(moe.moe_dequantize_mx(codes, scales, dtype=out), v.to(out))


def test_quantize_at_borders():
    """Every midpoint between neighbours and one fp32 step either side of it, both signs, in blocks whose
    maximum fixes the scale, from the smallest subnormal blocks to the largest finite ones."""
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 3.0, 6.0, 7.0]
    v = torch.tensor(mids, dtype=torch.float64)
    v = torch.cat([v, -v, v * (1 + 2.0 ** -22), v * (1 - 2.0 ** -22)])[:31 + 13]
    blocks = []
    for e in (-127, -126, -125, -100, -3, 0, 5, 100, 125):
        for part in (v[:31], v[13:]):
            b = torch.cat([part, torch.tensor([4.0], dtype=torch.float64)])
            blocks.append(b * 2.0 ** e)
    blocks += [torch.zeros(32, dtype=torch.float64), -torch.zeros(32, dtype=torch.float64),
               torch.full((32,), 2.0 ** -149, dtype=torch.float64)]
    x = torch.stack(blocks).float()
    want, s = R.quantize(x, "mxfp4")
    codes, scales = moe.moe_quantize_mx4(x.to(DEV))
    assert torch.equal(scales.cpu().long(), s)
    assert torch.equal(codes.cpu(), R.codes4(want, s))
    assert torch.equal(moe.moe_dequantize_mx(codes, scales).cpu().double(), want)


def test_quantize_non_finite_blocks():
    x = torch.randn((4, 96), device=DEV)
    x[0, 3], x[1, 40], x[2, 95] = math.nan, math.inf, -math.inf
    codes, scales = moe.moe_quantize_mx4(x)
    back = moe.moe_dequantize_mx(codes, scales)
    bad = torch.zeros((4, 3), dtype=torch.bool, device=DEV)
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    assert torch.equal(scales == 255, bad)
    assert torch.equal(back.isnan(), bad.repeat_interleave(32, 1))
    want, _ = R.quantize(torch.where(x.isfinite(), x, 0.0), "mxfp4")
    keep = ~bad.repeat_interleave(32, 1)
    assert torch.equal(back.double()[keep], want[keep])


def test_dequantize_every_code():
    for name, n, values in (("mxfp4", 256, R.values4), ("mxfp8", 256, R.values8)):
        codes = torch.arange(n, dtype=torch.uint8).repeat(8, 1)[:, :n]
        K = n * 2 if name == "mxfp4" else n
        s = torch.tensor([0, 1, 100, 127, 130, 200, 246, 254], dtype=torch.uint8)[:, None].expand(8, K // 32).contiguous()
        want = values(codes, s)
        got = moe.moe_dequantize_mx(codes.to(DEV), s.to(DEV))
        f = want.float()
        assert torch.equal(got.cpu().isnan(), f.isnan())
        assert torch.equal(got.cpu()[~f.isnan()], f[~f.isnan()])
        gb = moe.moe_dequantize_mx(codes.to(DEV), s.to(DEV), dtype=torch.bfloat16).cpu()
        fb = f.bfloat16()
        assert torch.equal(gb[~fb.isnan()], fb[~fb.isnan()])


def test_quantize_past_four_gigabytes():
    """Offsets past 2^32 elements' bytes: the last rows of a 5 GiB matrix."""
    rows, K = (5 << 30) // 2 // 4096, 4096
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device=DEV)
    x[-3:] = torch.randn((3, K), device=DEV).bfloat16()
    codes, scales = moe.moe_quantize_mx4(x)
    v, s = R.quantize(x[-3:], "mxfp4")
    assert torch.equal(scales[-3:].long(), s) and torch.equal(codes[-3:], R.codes4(v, s))
    assert not codes[:-3].any() and not scales[:-3].any()
    back = moe.moe_dequantize_mx(codes, scales, dtype=torch.bfloat16)
    assert torch.equal(back[-3:].double(), v) and not back[:-3].any()


@pytest.mark.parametrize("E,N,K", [(None, 16, 128), (1, 32, 384), (3, 48, 512), (2, 128, 640), (2, 16, 1536)])
def test_pack_layout(E, N, K):
    g = gen(N + K)
    lead = () if E is None else (E,)
    codes = torch.randint(0, 256, (*lead, N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    scales = torch.randint(0, 256, (*lead, N, K // 32), dtype=torch.uint8, device=DEV, generator=g)
    pc, ps = moe.moe_pack_mx4(codes, scales)
    c = codes.view(*lead, N // 16, 16, K // 128, 4, 16)  # row, block, q, byte
    assert torch.equal(pc.view(*lead, N // 16, K // 128, 4, 16, 16), c.movedim(-4, -2))
    kb = (K + 511) // 512
    s = torch.zeros((*lead, N, kb * 16), dtype=torch.uint8, device=DEV)
    s[..., :K // 32] = scales
    s = s.view(*lead, N // 16, 16, kb, 4, 4)  # row, group, step, q
    want = torch.stack([s[..., q].movedim(-3, -2) for q in range(4)], -3)  # [..., group, q, row, step]
    assert torch.equal(ps.view(*lead, N // 16, kb, 4, 16, 4), want)


# ------------------------------------------------------------------ grouped FFN
def weights(El, N, K, g, std=0.05):
    w = torch.randn((El, N, K), device=DEV, generator=g) * std
    v, s = R.quantize(w, "mxfp4")
    return R.codes4(v, s), s.to(torch.uint8), v


def routing(T, E, k, g, skew=0.0):
    logits = torch.randn((T, E), device=DEV, generator=g) - skew * torch.arange(E, device=DEV)
    top, ids = logits.topk(k, 1)
    return ids.int().contiguous(), torch.softmax(top, 1).contiguous()


def act_values(codes, scales, act):
    return R.values8(codes, scales) if act == "mxfp8" else R.values4(codes, scales)


def quantize_act(x, act):
    return moe.moe_quantize_mx(x) if act == "mxfp8" else moe.moe_quantize_mx4(x)


def setup(T, E, k, H, I, lo, hi, seed, skew=0.0, even=False):
    g = gen(seed)
    El = hi - lo
    gc, gs, gv = weights(El, 2 * I, H, g)
    dc, ds, dv = weights(El, H, I, g)
    x = R.even_rows((T, H), g, DEV) if even else torch.randn((T, H), device=DEV, generator=g).bfloat16()
    ids, gates = routing(T, E, k, g, skew)
    return dict(x=x, ids=ids, gates=gates, wgu=moe.moe_pack_mx4(gc, gs), wd=moe.moe_pack_mx4(dc, ds), gv=gv, dv=dv)


def run_ffn(s, E, lo, hi, act, dtype, **kw):
    p = moe.moe_permute(s["ids"], s["gates"], E, lo, hi)
    a, sc = quantize_act(s["x"], act)
    y = moe.moe_grouped_ffn_mx4(a, sc, p["offsets"], p["row_token"], p["row_w"], p["token_row"], s["wgu"], s["wd"],
                                dtype=dtype, **kw)
    return y, act_values(a, sc, act)


def check_ffn(T, E, k, H, I, lo, hi, act, dtype, seed, skew=0.0):
    s = setup(T, E, k, H, I, lo, hi, seed, skew, even=act == "mxfp8")
    y, av = run_ffn(s, E, lo, hi, act, dtype)
    mid, rad = R.layer(av, s["ids"], s["gates"], lo, hi - lo, lambda e: s["gv"][e], lambda e: s["dv"][e], act, dtype,
                       rows_rounded=True)
    R.check_interval(y, mid, rad, f"T={T} E={E} k={k} H={H} I={I} [{lo},{hi}) {act} {dtype}")


SHAPES = [
    # T, E, k, H, I, lo, hi, skew
    (1, 4, 2, 256, 128, 0, 4, 0.0),        # one token
    (3, 8, 8, 128, 128, 0, 8, 0.0),        # smallest widths, every expert of every token
    (17, 8, 2, 384, 256, 0, 8, 0.0),       # K not a multiple of 512, an odd row past a 16-row tile
    (33, 5, 1, 640, 384, 1, 4, 0.0),       # tokens with no local expert
    (64, 16, 4, 512, 512, 0, 16, 0.0),
    (65, 3, 2, 256, 640, 0, 3, 0.0),       # more than 64 tokens: tiles
    (200, 8, 2, 1024, 256, 0, 8, 2.0),     # a few experts hold most rows, some none
    (300, 4, 3, 384, 128, 0, 2, 0.0),
    (1100, 2, 1, 256, 384, 0, 2, 3.0),     # one expert with over 1024 rows
    (700, 40, 2, 128, 256, 3, 37, 0.0),    # odd expert range, few rows each
    (64, 33, 32, 128, 128, 0, 33, 0.0),    # the most rows a small batch can have
    (64, 1024, 2, 128, 128, 0, 1024, 0.0), # the most experts
    (2, 64, 8, 128, 512, 0, 64, 0.0),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act,dtype", [("mxfp8", torch.bfloat16), ("mxfp4", torch.bfloat16), ("mxfp8", torch.float32),
                                       ("mxfp4", torch.float32)])
def test_grouped_ffn(shape, act, dtype):
    T, E, k, H, I, lo, hi, skew = shape
    check_ffn(T, E, k, H, I, lo, hi, act, dtype, seed=T + E, skew=skew)


@pytest.mark.parametrize("act", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("T", [48, 400])
def test_grouped_ffn_full_width(T, act):
    """The widths of the 3 x 4096 x 1536 expert."""
    check_ffn(T, 8, 2, 4096, 1536, 0, 8, act, torch.bfloat16, seed=T)


@pytest.mark.parametrize("act", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("T", [600, 1300])
@pytest.mark.parametrize("n", range(1, 11))
def test_grouped_ffn_ring(n, T, act):
    """Every length of the contraction from one step of 128 to ten, with several tiles for each workgroup, in 64-row
    tiles and in larger ones: what one tile leaves in the ring the next must not see."""
    check_ffn(T, 64, 2, 128 * n, 128 * (11 - n), 0, 64, act, torch.bfloat16, seed=n)


@pytest.mark.parametrize("T", [40, 350])
def test_grouped_ffn_normal_activations(T):
    """Normal MXFP8 activations.  The matrix cores drop up to 7 * 2^-13 of the largest product of each group of
    eight; over 512 groups of a 4096-long sum that leaves G and U good to about 1e-4, and some values of h next to a
    midpoint go the other way, by a sixteenth: 2e-3 of y in the 2-norm at one in five hundred.  The two bf16
    roundings add at most 2^-8 each."""
    s = setup(T, 8, 2, 4096, 512, 0, 8, seed=T)
    y, av = run_ffn(s, 8, 0, 8, "mxfp8", torch.bfloat16)
    mid, _ = R.layer(av, s["ids"], s["gates"], 0, 8, lambda e: s["gv"][e], lambda e: s["dv"][e], "mxfp8",
                     torch.bfloat16, rows_rounded=True)
    assert float((y.double() - mid).norm() / mid.norm()) <= 2 * 2.0 ** -8 + 2e-3


@pytest.mark.parametrize("T", [40, 300])
def test_grouped_ffn_no_local_rows(T):
    """Every token routed elsewhere: y is zero, whatever was in it."""
    s = setup(T, 8, 2, 256, 128, 0, 2, seed=5)
    s["ids"] = torch.tensor([[6, 4]], dtype=torch.int32, device=DEV).repeat(T, 1)
    y = torch.full((T, 256), math.nan, dtype=torch.bfloat16, device=DEV)
    run_ffn(s, 8, 0, 2, "mxfp8", torch.bfloat16, y=y)
    assert not y.any()


@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("act", ["mxfp8", "mxfp4"])
def test_grouped_ffn_bad_token_stays_alone(T, act):
    """A token whose scales say NaN gives a NaN row; every other row is what it was, bit for bit."""
    s = setup(T, 4, 2, 256, 128, 0, 4, seed=6)
    p = moe.moe_permute(s["ids"], s["gates"], 4, 0, 4)
    a, sc = quantize_act(s["x"], act)
    args = (p["offsets"], p["row_token"], p["row_w"], p["token_row"], s["wgu"], s["wd"])
    y0 = moe.moe_grouped_ffn_mx4(a, sc, *args)
    bad = T // 2
    sc = sc.clone()
    sc[bad, 1] = 255
    y1 = moe.moe_grouped_ffn_mx4(a, sc, *args)
    keep = torch.arange(T, device=DEV) != bad
    assert y1[bad].isnan().all()
    assert torch.equal(y1[keep], y0[keep]) and not y0.isnan().any()


@pytest.mark.parametrize("T", [50, 500])
def test_grouped_ffn_repeats_bit_for_bit(T):
    """Same inputs, workspaces with other contents, several runs: the same bits (no order left to chance)."""
    s = setup(T, 16, 4, 512, 256, 0, 16, seed=7)
    ys = []
    for fill in (0, 255, 7):
        ws = moe.moe_ffn_mx4_workspace(T, 4, 16, 512, 256).fill_(fill)
        ys.append(run_ffn(s, 16, 0, 16, "mxfp8", torch.bfloat16, workspace=ws)[0])
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


@pytest.mark.parametrize("T", [30, 333])
def test_grouped_ffn_graph_and_stream(T):
    """quantise -> FFN captured on another stream; replays with new inputs between eager work match eager calls."""
    s = setup(T, 8, 2, 384, 256, 0, 8, seed=8)
    p = moe.moe_permute(s["ids"], s["gates"], 8, 0, 8)
    ws = moe.moe_ffn_mx4_workspace(T, 2, 8, 384, 256)
    codes, scales = moe.moe_quantize_mx4(s["x"])
    y = torch.empty((T, 384), dtype=torch.bfloat16, device=DEV)

    def step(st=None):
        moe.moe_quantize_mx4(s["x"], codes, scales, stream=st)
        moe.moe_grouped_ffn_mx4(codes, scales, p["offsets"], p["row_token"], p["row_w"], p["token_row"], s["wgu"],
                                s["wd"], y=y, workspace=ws, stream=st)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    g = gen(9)
    for _ in range(4):
        s["x"].copy_(torch.randn(s["x"].shape, device=DEV, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, y)


@pytest.mark.parametrize("T", [30, 333])
def test_grouped_ffn_own_buffers_on_a_stream(T):
    """What a call on another stream allocates is not handed to the current stream while the call still runs."""
    s = setup(T, 8, 2, 384, 256, 0, 8, seed=11)
    p = moe.moe_permute(s["ids"], s["gates"], 8, 0, 8)
    args = (p["offsets"], p["row_token"], p["row_w"], p["token_row"], s["wgu"], s["wd"])
    want = moe.moe_grouped_ffn_mx4(*moe.moe_quantize_mx4(s["x"]), *args)
    n = moe.moe_ffn_mx4_workspace_size(T, 2, 8, 384, 256, moe.MOE_BF16)
    side = torch.cuda.Stream()
    for use in (side, side.cuda_stream):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        a, sc = moe.moe_quantize_mx4(s["x"], stream=use)
        y = moe.moe_grouped_ffn_mx4(a, sc, *args, stream=use)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
        torch.cuda.current_stream().synchronize()
        side.synchronize()
        assert torch.equal(y, want), junk[0][0]


def test_grouped_ffn_empty_batch():
    s = setup(1, 4, 2, 256, 128, 0, 4, seed=10)
    e = lambda *shape, dt=torch.uint8: torch.empty(shape, dtype=dt, device=DEV)  # noqa: E731
    y = moe.moe_grouped_ffn_mx4(e(0, 256), e(0, 8), e(5, dt=torch.int32), e(0, dt=torch.int32), e(0, dt=torch.float32),
                                e(0, 2, dt=torch.int32), s["wgu"], s["wd"])
    assert y.shape == (0, 256)
    c, sc = moe.moe_quantize_mx4(e(0, 64, dt=torch.bfloat16))
    assert c.shape == (0, 32) and moe.moe_dequantize_mx(c, sc).shape == (0, 64)


# ------------------------------------------------------------------ the few-token layer
def check_clean(ws):
    ctl = ws[:256].view(torch.int32).cpu()
    assert int(ctl[4]) == 0, "a wait inside the kernel gave up"
    assert not ctl[:4].any(), "control words not reset"


def layer_setup(T, E, k, H, I, lo, hi, seed, even=True, bias=False):
    s = setup(T, E, k, H, I, lo, hi, seed, even=even)
    g = gen(seed + 1)
    s["wr"] = (torch.randn((E, H), device=DEV, generator=g) * 0.05).bfloat16()
    s["bias"] = torch.randn(E, device=DEV, generator=g) if bias else None
    s["router"] = moe.moe_pack_router(s["wr"])
    return s


def run_layer(s, k, lo, hi, ws, dtype=torch.bfloat16, **kw):
    return moe.moe_decode_layer_mx4(s["x"], s["router"], s["bias"], k, lo, hi, s["wgu"], s["wd"], ws, dtype=dtype, **kw)


LAYERS = [
    # T, E, k, H, I, lo, hi, bias
    (1, 8, 2, 256, 128, 0, 8, False),
    (1, 128, 8, 1024, 512, 0, 128, True),
    (2, 64, 1, 128, 128, 0, 64, False),     # one step of the contraction
    (5, 65, 8, 640, 384, 0, 65, True),      # experts past a multiple of 64, K not a multiple of 512
    (17, 16, 4, 384, 256, 3, 11, False),    # local experts, more rows than a tile
    (33, 200, 6, 512, 128, 0, 200, False),
    (64, 8, 8, 256, 256, 0, 8, True),       # every token on every expert
    (64, 256, 8, 384, 128, 64, 128, False),
    (64, 40, 32, 128, 128, 0, 40, False),   # the most rows
    (3, 1, 1, 128, 128, 0, 1, False),       # one expert
    (4, 16, 2, 8192, 128, 0, 16, False),    # the widest
]


@pytest.mark.parametrize("shape", LAYERS, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_layer(shape, dtype):
    """Routing bit for bit as moe_route; y inside the interval; the workspace's control words zero again; the
    same call again gives the same bits."""
    T, E, k, H, I, lo, hi, bias = shape
    s = layer_setup(T, E, k, H, I, lo, hi, seed=T * E + H, bias=bias)
    ids, w = moe.moe_route(s["x"], s["wr"], s["bias"], k)
    ws = moe.moe_decode_layer_mx4_workspace(T, k, hi - lo, H, I)
    y, ids2, w2 = run_layer(s, k, lo, hi, ws, dtype)
    check_clean(ws)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    xv, _ = R.quantize(s["x"], "mxfp8")
    mid, rad = R.layer(xv, ids, w, lo, hi - lo, lambda e: s["gv"][e], lambda e: s["dv"][e], "mxfp8", dtype,
                       rows_rounded=False)
    R.check_interval(y, mid, rad, str(shape))
    y2, _, _ = run_layer(s, k, lo, hi, ws, dtype)
    check_clean(ws)
    assert torch.equal(y, y2)


def test_decode_layer_full_width():
    T, E, k, H, I = 6, 32, 8, 4096, 1536
    s = layer_setup(T, E, k, H, I, 0, E, seed=3)
    ws = moe.moe_decode_layer_mx4_workspace(T, k, E, H, I)
    y, ids, w = run_layer(s, k, 0, E, ws)
    ids1, w1 = moe.moe_route(s["x"], s["wr"], s["bias"], k)
    assert torch.equal(ids, ids1) and torch.equal(w, w1)
    xv, _ = R.quantize(s["x"], "mxfp8")
    mid, rad = R.layer(xv, ids, w, 0, E, lambda e: s["gv"][e], lambda e: s["dv"][e], "mxfp8", torch.bfloat16, False)
    R.check_interval(y, mid, rad, "full width")


def test_decode_layer_routing_ties_and_zero_router():
    """Equal logits go to the lower index, also across 64-expert items; a zero router picks the first k."""
    s = layer_setup(7, 130, 5, 256, 128, 0, 130, seed=4)
    s["wr"][70] = s["wr"][3]
    s["wr"][129] = s["wr"][3]
    for wr in (s["wr"], torch.zeros_like(s["wr"])):
        s["wr"], s["router"] = wr, moe.moe_pack_router(wr)
        ws = moe.moe_decode_layer_mx4_workspace(7, 5, 130, 256, 128)
        _, ids, w = run_layer(s, 5, 0, 130, ws)
        ids1, w1 = moe.moe_route(s["x"], wr, None, 5)
        assert torch.equal(ids, ids1) and torch.equal(w, w1)
    assert torch.equal(ids.cpu(), torch.arange(5, dtype=torch.int32).repeat(7, 1))


def test_decode_layer_one_workspace_many_sizes():
    """One workspace of the largest size serves smaller calls in any order."""
    big = dict(E=24, k=4, H=512, I=256)
    ws = moe.moe_decode_layer_mx4_workspace(64, 4, 24, 512, 256)
    for T in (64, 1, 30, 2, 64):
        s = layer_setup(T, **big, lo=0, hi=24, seed=T)
        y, ids, w = run_layer(s, 4, 0, 24, ws)
        check_clean(ws)
        fresh, _, _ = run_layer(s, 4, 0, 24, moe.moe_decode_layer_mx4_workspace(T, 4, 24, 512, 256))
        assert torch.equal(y, fresh)


def test_decode_layer_no_local_rows_and_bad_token():
    s = layer_setup(9, 16, 2, 256, 128, 0, 4, seed=5)
    ws = moe.moe_decode_layer_mx4_workspace(9, 2, 4, 256, 128)
    s["bias"] = torch.zeros(16, device=DEV)
    s["bias"][8:] = 1e4  # every token on experts that are not local
    y = torch.full((9, 256), math.nan, dtype=torch.bfloat16, device=DEV)
    run_layer(s, 2, 0, 4, ws, y=y)
    check_clean(ws)
    assert not y.any()
    s["bias"] = torch.zeros(16, device=DEV)
    s["bias"][:4] = 1e4  # every token local
    y0, ids0, _ = run_layer(s, 2, 0, 4, ws)
    s["x"][4, 100] = math.inf
    y1, ids1, _ = run_layer(s, 2, 0, 4, ws)
    check_clean(ws)
    keep = torch.arange(9, device=DEV) != 4
    assert y1[4].isnan().all() and torch.equal(y1[keep], y0[keep]) and torch.equal(ids1[keep], ids0[keep])


def test_decode_layer_agrees_with_the_composed_calls():
    """moe_route, moe_permute, moe_quantize_mx and moe_grouped_ffn_mx4 one after another: same routing and
    the same products in the same order, so the same y bit for bit."""
    s = layer_setup(20, 48, 6, 1024, 512, 8, 40, seed=6, even=False)
    ws = moe.moe_decode_layer_mx4_workspace(20, 6, 32, 1024, 512)
    y, ids, w = run_layer(s, 6, 8, 40, ws)
    ids1, w1 = moe.moe_route(s["x"], s["wr"], s["bias"], 6)
    assert torch.equal(ids, ids1) and torch.equal(w, w1)
    s["ids"], s["gates"] = ids1, w1
    y1, _ = run_ffn(s, 48, 8, 40, "mxfp8", torch.bfloat16)
    assert torch.equal(y, y1)


def test_decode_layer_graph_streams_and_empty():
    """Captured and replayed with new inputs between eager calls on another workspace; two streams at once with a
    workspace each; T = 0."""
    T, E, k, H, I = 12, 32, 4, 512, 256
    s = layer_setup(T, E, k, H, I, 0, E, seed=7)
    ws, ws2 = (moe.moe_decode_layer_mx4_workspace(T, k, E, H, I) for _ in range(2))
    y = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), dtype=torch.float32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run_layer(s, k, 0, E, ws, topk_ids=ids, topk_w=w, y=y, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run_layer(s, k, 0, E, ws, topk_ids=ids, topk_w=w, y=y)
    g = gen(8)
    for _ in range(4):
        s["x"].copy_(R.even_rows((T, H), g, DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = (y.clone(), ids.clone(), w.clone())
        want = run_layer(s, k, 0, E, ws2)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):  # both streams busy at once
        a = run_layer(s, k, 0, E, ws)
        with torch.cuda.stream(side):
            b = run_layer(s, k, 0, E, ws2)
    torch.cuda.synchronize()
    check_clean(ws)
    check_clean(ws2)
    assert torch.equal(a[0], want[0]) and torch.equal(b[0], want[0])
    s["x"] = s["x"][:0]
    assert run_layer(s, k, 0, E, ws)[0].shape == (0, H)


# ------------------------------------------------------------------ together, as a layer
@pytest.mark.parametrize("T,act,wact", [(9, "mxfp8", "bf16"), (9, "mxfp4", "bf16"), (150, "mxfp8", "bf16"),
                                        (150, "mxfp4", "f32")])
@pytest.mark.parametrize("I_s", [0, 192])
def test_layer(T, act, wact, I_s):
    """convert_experts_mx4 and run_layer on a synthetic layer (an expert-parallel share, with and without a shared
    expert), called twice, against 64 bits."""
    from expert_routed_grouped_amd import layer as L
    from expert_routed_grouped_amd import synth
    cfg = synth.LayerConfig("mx4", T=T, H=512, E=24, k=4, I=256, act=wact, wdt=wact, e_begin=4, e_end=20, seed=77, w_std=0.06,
                            I_s=I_s)
    dev = L.to_device(synth.make_inputs(cfg))
    if act == "mxfp8":  # activations whose sums are exact on the matrix cores
        dev["x"] = R.even_rows((T, 512), gen(T), DEV).to(dev["x"].dtype)
    L.convert_experts_mx4(dev)
    bufs = L.Mx4LayerBuffers(cfg, act=act, dtype=torch.float32 if I_s else torch.bfloat16)
    L.run_layer(dev, bufs)
    first = bufs.y.clone()
    y = L.run_layer(dev, bufs)
    ids, w = moe.moe_route(dev["x"], dev["w_router"], None, 4)
    assert torch.equal(ids, bufs.topk_ids)
    xv, _ = R.quantize(dev["x"], act)
    q = {n: R.quantize(dev[n], "mxfp4")[0] for n in ("w_gate_up", "w_down")}
    mid, rad = R.layer(xv, ids, w, 4, 16, lambda e: q["w_gate_up"][e], lambda e: q["w_down"][e], act, y.dtype,
                       rows_rounded=True)
    if I_s:
        # the shared expert: fp32 or bf16 products (exact for bf16, one rounding each for fp32) with fp32 sums in
        # some order, h rounded to bf16 for bf16 models
        x, gu, dn = dev["x"].double(), dev["ws_gate_up"].double(), dev["ws_down"].double()
        a = x @ gu.T
        mag = x.abs() @ gu.abs().T
        G, U = a[:, :I_s], a[:, I_s:]
        n = 2 * 512 * 2.0 ** -24
        h = G * torch.sigmoid(G) * U
        dh = U.abs() * 1.1 * n * mag[:, :I_s] + (G * torch.sigmoid(G)).abs() * n * mag[:, I_s:]
        dh = dh + h.abs() * ((G.abs() + 5) * 2.0 ** -22 + (2.0 ** -8 if wact == "bf16" else 0))
        mid = mid + h @ dn.T
        rad = rad + dh @ dn.abs().T + 2 * I_s * 2.0 ** -24 * (h.abs() @ dn.abs().T) + (mid.abs() + rad) * 2.0 ** -22
    else:
        assert torch.equal(first, y)  # the shared expert's split sums are in no fixed order
    R.check_interval(y, mid, rad, f"layer T={T} {act}")


def test_layer_refusals():
    from expert_routed_grouped_amd import layer as L
    from expert_routed_grouped_amd import synth
    cfg = synth.LayerConfig("mx4", T=4, H=256, E=4, k=2, I=128, seed=78, I_s=128)
    with pytest.raises(ValueError):
        L.Mx4LayerBuffers(cfg)  # a shared expert with a bf16 y
    with pytest.raises(ValueError):
        L.Mx4LayerBuffers(cfg.replace(I_s=0), act="bf16")
    dev = L.to_device(synth.make_inputs(cfg.replace(I_s=0)))
    L.pack_weights(dev)
    with pytest.raises(ValueError):
        L.convert_experts_mx4(dev)
