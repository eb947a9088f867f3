"""GPU: the operators that train a MoE block against plain 64-bit formulations (tests/train_ref.py), one by one."""
import pytest
import torch

import train_ref as R
from expert_routed_grouped_amd import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
TYPES = [(BF, BF), (BF, F32), (F32, F32)]
NAN = float("nan")


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, device=DEV, generator=g) * std).to(dtype)


# rows per expert: empty experts, single rows, one below, at and above tile heights, one expert with most rows
COUNTS = {"one": [1], "none": [0, 0, 0], "few": [0, 1, 2, 0, 5, 1], "tiles": [63, 64, 65, 0, 31, 32, 33, 1],
          "edges": [127, 128, 129, 256, 0, 255, 257], "hot": [3, 1500, 0, 1], "many": [1] * 130 + [0] * 7 + [9]}


def grouped_rows(g, counts, width, dtype, gather, extra=5):
    """(a, index, R_cap): rows grouped by expert, or tokens and an index with repeats; NaN wherever no product reads."""
    n = sum(counts)
    cap = n + extra
    if not gather:
        a = randn(g, cap, width, dtype=dtype)
        a[n:] = NAN
        return a, None, cap
    tokens = max(3, n // 2)
    a = randn(g, tokens, width, dtype=dtype)
    a[1] = NAN  # a token that no row names
    pick = torch.randint(0, tokens - 1, (cap,), device=DEV, generator=g)
    index = torch.where(pick >= 1, pick + 1, pick).int()
    index[n:] = 1
    return a, index, cap


def check_mm(counts, N, K, types, gather, transposed, seed=0):
    g = gen(seed + N * 7 + K)
    dt, ot = types
    E = len(counts)
    off = R.offsets_of(counts)
    a, index, cap = grouped_rows(g, counts, K, dt, gather)
    w = randn(g, E, K, N, dtype=dt, std=0.3) if transposed else randn(g, E, N, K, dtype=dt, std=0.3)
    out = torch.full((cap, N), 7.0, dtype=ot, device=DEV)
    got = moe.moe_grouped_mm(a, w, off, row_index=index, transposed=transposed, out=out)
    assert got is out
    n = sum(counts)
    want, mag = R.mm(a, w, off, index, transposed)
    R.check(out[:n], want, mag * (K + 2) * R.STEP32 + want.abs() * R.half_step(ot) * 1.01, "product")
    assert (out[n:] == 7.0).all(), "rows behind the last expert's were written"


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("gather", [False, True])
def test_mm_rows(counts, gather, transposed, types):
    check_mm(COUNTS[counts], 136, 200, types, gather, transposed)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("N,K", [(1, 1), (1, 64), (64, 1), (3, 5), (8, 8), (7, 129), (129, 7), (127, 1000), (255, 64), (256, 72),
                                 (257, 520), (1024, 8), (8, 1032), (40, 2047), (384, 512), (520, 1000)])
@pytest.mark.parametrize("counts", ["few", "edges"])
def test_mm_sizes(counts, N, K, transposed, types):
    check_mm(COUNTS[counts], N, K, types, True, transposed)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 24, 31, 32, 33, 47, 64, 65, 96, 130])
def test_mm_rows_per_expert(rows, transposed):
    """Every height at which another variant or one more tile may be taken, for aligned bf16 operands."""
    check_mm([rows, 0, rows], 320, 576, (BF, BF), True, transposed)
    check_mm([rows] * 3, 1024, 256, (BF, F32), False, transposed)


# enough experts and rows that every workgroup works through several tiles, of every height, whole and short
MANY = [0, 1, 63, 64, 65, 127, 128, 129, 0, 191, 192, 193, 255, 256, 257, 300, 511, 512, 513, 700] * 6


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K", [(8, 8), (256, 64), (264, 72), (520, 136), (512, 200), (248, 584), (257, 129)])
def test_mm_many_tiles(N, K, gather, transposed, types):
    check_mm(MANY, N, K, types, gather, transposed)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts", [[5000] + [3] * 60, [40] * 200, [1] * 500 + [2000], [0] * 300 + [256] * 40 + [0] * 300, [100] * 1024])
def test_mm_uneven_loads(counts, transposed):
    check_mm(counts, 264, 128, (BF, BF), True, transposed)
    check_mm(counts, 512, 72, (BF, F32), False, transposed)


def test_mm_many_tiles_and_shorter_buffers():
    """Offsets that run past the buffers: the rows there are, nothing behind them."""
    g = gen(66)
    w = randn(g, len(MANY), 264, 64, dtype=BF)
    n = 5000
    a = randn(g, n, 64, dtype=BF)
    store = torch.full((n + 300, 264), 7.0, device=DEV, dtype=BF)
    off = R.offsets_of(MANY)
    moe.moe_grouped_mm(a, w, off, out=store[:n])
    assert (store[n:] == 7.0).all()
    want, mag = R.mm(a, w, off.clamp(max=n))
    R.check(store[:n], want, mag * 66 * R.STEP32 + want.abs() * R.half_step(BF) * 1.01)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("transposed", [False, True])
def test_mm_non_finite_values_stay_in_their_rows(types, transposed):
    dt, ot = types
    g, off = gen(5), R.offsets_of([40, 0, 70])
    a, w = randn(g, 110, 96, dtype=dt), randn(g, 3, 96, 96, dtype=dt)
    a[3, 5], a[60, 95] = NAN, float("inf")
    w[1] = NAN  # an expert without rows
    out = moe.moe_grouped_mm(a, w, off, transposed=transposed, dtype=ot)
    bad = ~torch.isfinite(out)
    assert bad[3].all() and bad[60].all()
    assert int(bad.any(1).sum()) == 2


def test_mm_without_rows_and_shorter_buffers():
    g = gen(6)
    w = randn(g, 4, 64, 32, dtype=BF)
    empty = torch.empty((0, 32), dtype=BF, device=DEV)
    assert moe.moe_grouped_mm(empty, w, R.offsets_of([0] * 4)).shape == (0, 64)
    # offsets that promise more rows than the buffers hold: the rows there are, nothing behind them
    a = randn(g, 20, 32, dtype=BF)
    store = torch.full((24, 64), 7.0, device=DEV, dtype=BF)
    moe.moe_grouped_mm(a, w, R.offsets_of([5, 9, 30, 40]), out=store[:20])
    assert (store[20:] == 7.0).all()
    want, _ = R.mm(a, w, R.offsets_of([5, 9, 6, 0]))
    assert (store[:20].double() - want).abs().max() < 0.1


@pytest.mark.parametrize("dt", [BF, F32])
def test_mm_indexes_out_of_range_read_the_nearest_row(dt):
    g, off = gen(7), R.offsets_of([3, 3])
    a, w = randn(g, 4, 64, dtype=dt), randn(g, 2, 64, 64, dtype=dt)
    bad = torch.tensor([-5, 0, 9, 2 ** 31 - 1, -2 ** 31, 3], dtype=torch.int32, device=DEV)
    assert torch.equal(moe.moe_grouped_mm(a, w, off, row_index=bad),
                       moe.moe_grouped_mm(a, w, off, row_index=bad.clamp(0, 3)))


# ------------------------------------------------------------------ weight gradient
def check_wgrad(counts, M, N, types, gather, add, seed=0):
    g = gen(seed + 3 * M + N)
    dt, ot = types
    E, n, off = len(counts), sum(counts), R.offsets_of(counts)
    a, ai, cap = grouped_rows(g, counts, M, dt, gather == "a")
    b, bi, _ = grouped_rows(g, counts, N, dt, gather == "b")
    old = randn(g, E, M, N, dtype=ot)
    out = old.clone() if add else torch.full((E, M, N), NAN, dtype=ot, device=DEV)
    assert moe.moe_grouped_wgrad(a, b, off, a_index=ai, b_index=bi, out=out, add=add) is out
    want, mag = R.wgrad(a, b, off, ai, bi)
    if add:
        want, mag = want + old.double(), mag + old.double().abs()
    most = max(counts)
    R.check(out, want, mag * (most + 3) * R.STEP32 + want.abs() * R.half_step(ot) * 1.01, "weight gradient")
    again = old.clone() if add else torch.full((E, M, N), NAN, dtype=ot, device=DEV)
    assert torch.equal(moe.moe_grouped_wgrad(a, b, off, a_index=ai, b_index=bi, out=again, add=add), out)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("gather", ["none", "a", "b"])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("counts", COUNTS)
def test_wgrad_rows(counts, gather, add, types):
    check_wgrad(COUNTS[counts], 136, 72, types, gather, add)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("M,N", [(1, 1), (1, 64), (64, 1), (3, 5), (8, 8), (7, 129), (129, 40), (127, 255), (256, 72), (257, 520),
                                 (1024, 8), (8, 1032), (384, 512)])
@pytest.mark.parametrize("counts", ["few", "edges"])
def test_wgrad_sizes(counts, M, N, types):
    check_wgrad(COUNTS[counts], M, N, types, "b", False)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("M,N", [(24, 40), (128, 256), (33, 19)])
def test_wgrad_long_sums(M, N, types):
    """Few tiles and many rows."""
    check_wgrad([4099, 1, 2500], M, N, types, "none", False)
    check_wgrad([4099, 1, 2500], M, N, types, "a", True)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("gather", ["none", "a", "b", "both"])
@pytest.mark.parametrize("add", [False, True])
def test_wgrad_many_tiles(gather, add, types):
    """Several tiles a workgroup, whole and short, with experts that have none, one, two and more steps of rows."""
    counts = [0, 1, 31, 32, 33, 64, 65, 0, 0, 96, 97, 128, 300] * 10
    for M, N in ((264, 520), (512, 256), (136, 64)):
        if gather != "both":
            check_wgrad(counts, M, N, types, gather, add)
            continue
        g = gen(M)
        dt, ot = types
        off = R.offsets_of(counts)
        a, ai, _ = grouped_rows(g, counts, M, dt, True)
        b, bi, _ = grouped_rows(g, counts, N, dt, True)
        out = randn(g, len(counts), M, N, dtype=ot)
        old = out.double()
        moe.moe_grouped_wgrad(a, b, off, a_index=ai, b_index=bi, out=out, add=add)
        want, mag = R.wgrad(a, b, off, ai, bi)
        if add:
            want, mag = want + old, mag + old.abs()
        R.check(out, want, mag * 303 * R.STEP32 + want.abs() * R.half_step(ot) * 1.01)


@pytest.mark.parametrize("types", TYPES)
def test_wgrad_in_parts_whatever_the_loads(types):
    """Averages that split the rows, with an expert that has all of them, few or none."""
    for counts in ([4096, 0, 0], [1, 4000, 30], [0, 0, 0, 5000], [600, 700, 800, 1]):
        check_wgrad(counts, 136, 264, types, "a", True)
        check_wgrad(counts, 40, 24, types, "none", False)


def test_wgrad_and_offsets_past_the_buffers():
    g = gen(67)
    counts, n = [40] * 30, 700
    a, b = randn(g, n, 256, dtype=BF), randn(g, n, 256, dtype=BF)
    off = R.offsets_of(counts)
    got = moe.moe_grouped_wgrad(a, b, off, dtype=F32)
    want, mag = R.wgrad(a, b, off.clamp(max=n))
    R.check(got, want, mag * 43 * R.STEP32)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("M,N", [(1, 1), (65, 131), (130, 5), (64, 128), (67, 777)])
def test_wgrad_of_experts_without_rows_writes_its_matrices_alone(M, N, types):
    """Zeros in every element of theirs and nowhere else; nothing at all where gradients are added to."""
    t, ot = types
    off = R.offsets_of([0, 2, 0, 0])
    g, n, pad = gen(M), 4 * M * N, 64
    a, b = randn(g, 2, M, dtype=t), randn(g, 2, N, dtype=t)
    for add in (False, True):
        whole = torch.full((n + 2 * pad,), 7.0, dtype=ot, device=DEV)
        out = whole[pad:pad + n].view(4, M, N)
        moe.moe_grouped_wgrad(a, b, off, out=out, add=add)
        assert (whole[:pad] == 7.0).all() and (whole[pad + n:] == 7.0).all()
        for e in (0, 2, 3):
            assert (out[e] == (7.0 if add else 0.0)).all(), (add, e)


def test_wgrad_non_finite_rows_stay_with_their_expert():
    g, off = gen(8), R.offsets_of([33, 0, 31])
    a, b = randn(g, 64, 64, dtype=BF), randn(g, 64, 128, dtype=BF)
    a[33], b[40, 7] = float("inf"), NAN  # both of the third expert
    out = moe.moe_grouped_wgrad(a, b, off)
    assert torch.isfinite(out[:2]).all() and (out[1] == 0).all()
    assert torch.isnan(out[2, :, 7]).all() and not torch.isfinite(out[2]).any()


# ------------------------------------------------------------------ SwiGLU
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("I", [1, 3, 8, 64, 100, 516, 1536, 2051])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("counts", [None, [0, 0], [5, 0, 1, 70]])
def test_swiglu(I, weighted, counts, dtype):
    g = gen(I)
    n, cap = (9, 9) if counts is None else (sum(counts), sum(counts) + 4)
    off = None if counts is None else R.offsets_of(counts)
    gu, dh = randn(g, cap, 2 * I, dtype=dtype, std=3.0), randn(g, cap, I, dtype=dtype)
    gu[:, 0] *= 20  # both tails of the sigmoid
    w = randn(g, cap) if weighted else None
    h, dgu = torch.full((cap, I), 7.0, dtype=dtype, device=DEV), torch.full((cap, 2 * I), 7.0, dtype=dtype, device=DEV)
    h2, dw = h.clone(), torch.full((cap,), 7.0, device=DEV)
    moe.moe_swiglu(gu, off, w, h=h)
    moe.moe_swiglu_backward(gu, dh, off, w, dgu=dgu, h=h2, d_row_w=dw if weighted else None)
    assert torch.equal(h, h2)
    for t in (h, dgu, dw):
        assert (t[n:] == 7.0).all()
    gu, dh, w = gu[:n], dh[:n], None if w is None else w[:n]
    want, half = R.swiglu(gu, w), R.half_step(dtype)
    # about ten roundings a value; the exponential of a rounded product of up to 24 * 60 / ln 2 is off by |g| steps
    g64 = gu.double().chunk(2, 1)[0]
    fp = (20 + 2 * g64.abs()) * R.STEP32
    tiny = 1e-30
    R.check(h[:n], want, want.abs() * (half * 1.01 + fp) + tiny, "h")
    dgate, sums = R.swiglu_backward(gu, dh, w)
    ww = torch.ones(n, 1, dtype=R.F64, device=DEV) if w is None else w.double()[:, None].abs()
    # 1 + g (1 - s) cancels: its terms' magnitudes, not its value, carry the error
    s, u = torch.sigmoid(g64), gu.double().chunk(2, 1)[1]
    mag = torch.cat([ww * (dh.double() * u).abs() * s * (1 + g64.abs() * (1 - s)), dgate[:, I:].abs()], 1)
    R.check(dgu[:n], dgate, dgate.abs() * half * 1.01 + mag * torch.cat([fp, fp], 1) + tiny, "dgu")
    if weighted:
        terms = (dh.double() * R.swiglu(gu)).abs()
        R.check(dw[:n], sums, terms.sum(1) * (I + 2) * R.STEP32 + (terms * fp).sum(1) + tiny, "d_row_w")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_swiglu_backward_in_place(dtype):
    g = gen(3)
    gu, dh, w = randn(g, 70, 2 * 520, dtype=dtype), randn(g, 70, 520, dtype=dtype), randn(g, 70)
    want = moe.moe_swiglu_backward(gu, dh, None, w)
    got = moe.moe_swiglu_backward(gu, dh, None, w, dgu=gu, h=dh)
    assert got[0] is gu and got[1] is dh
    for x, y in zip(got, want):
        assert torch.equal(x, y)


# ------------------------------------------------------------------ router
def routing(g, T, E, k, lo=0, hi=None, hot=False):
    ids = torch.rand((T, E), device=DEV, generator=g)
    if hot:
        ids[:, 0] += 1
    ids = ids.topk(k, 1).indices.int()
    gates = torch.softmax(randn(g, T, k), 1)
    every = moe.moe_permute(ids, gates, E, 0, E)
    local = every if hi is None else moe.moe_permute(ids, gates, E, lo, hi)
    return ids, gates, every, local


@pytest.mark.parametrize("types", [(BF, BF, BF), (BF, F32, F32), (F32, F32, F32), (F32, BF, BF)])  # x and router; rows; dx
@pytest.mark.parametrize("T,E,k,H,lo,hi", [(1, 8, 1, 64, 0, None), (1, 128, 8, 264, 0, None), (5, 3, 3, 7, 0, None),
                                           (64, 8, 2, 256, 2, 5), (300, 16, 4, 1000, 0, None), (700, 2, 1, 520, 1, 2),
                                           (33, 40, 32, 96, 3, 21), (257, 130, 6, 4096, 0, None), (3000, 4, 2, 72, 0, None)])
def test_route_backward(T, E, k, H, lo, hi, types):
    g = gen(T + E)
    dt, rt, ot = types
    ids, gates, every, local = routing(g, T, E, k, lo, hi, hot=T > 200)
    x, wr, dg = randn(g, T, H, dtype=dt), randn(g, E, H, dtype=dt), randn(g, T, k)
    n = int(local["offsets"][-1])
    rows = randn(g, local["R_cap"], H, dtype=rt)
    rows[n:] = NAN
    dx, dw, db = moe.moe_route_backward(ids, gates, dg, x, wr, every, rows=rows, token_row=local["token_row"], dtype=ot)
    dl, wx, ww, wb = R.route_backward(ids, gates, dg, x, wr, rows.nan_to_num(), local["token_row"])
    # dl: two products and a sum of k terms
    dmag = gates.double() * (dg.double().abs() + (gates * dg).double().abs().sum(1, keepdim=True))
    derr = dmag * (k + 4) * R.STEP32
    dense = lambda v: torch.zeros((T, E), dtype=R.F64, device=DEV).scatter_(1, ids.long(), v)  # noqa: E731
    part = torch.where((local["token_row"] >= 0).unsqueeze(-1), rows.nan_to_num().double()[local["token_row"].long().clamp(min=0)], 0)
    xmag = dense(dl.abs()) @ wr.double().abs() + part.abs().sum(1)
    R.check(dx, wx, dense(derr) @ wr.double().abs() + xmag * (2 * k + 2) * R.STEP32 + wx.abs() * R.half_step(ot) * 1.01, "dx")
    most = int(every["counts"].max())
    R.check(dw, ww, dense(derr).T @ x.double().abs() + (dense(dl.abs()).T @ x.double().abs()) * (most + 2) * R.STEP32, "dw")
    R.check(db, wb, dense(derr).sum(0) + dense(dl.abs()).sum(0) * (most + 2) * R.STEP32, "db")
    again = moe.moe_route_backward(ids, gates, dg, x, wr, every, rows=rows, token_row=local["token_row"], dtype=ot)
    for p, q in zip((dx, dw, db), again):
        assert torch.equal(p, q)


def test_route_backward_without_rows_and_without_tokens():
    g = gen(11)
    ids, gates, every, _ = routing(g, 40, 8, 2)
    x, wr, dg = randn(g, 40, 128), randn(g, 8, 128), randn(g, 40, 2)
    dx, dw, db = moe.moe_route_backward(ids, gates, dg, x, wr, every)
    _, wx, ww, wb = R.route_backward(ids, gates, dg, x, wr)
    for got, want in ((dx, wx), (dw, ww), (db, wb)):
        assert (got.double() - want).abs().max() <= 1e-5 * want.abs().max()
    none = {n: every[n][:0] for n in ("row_token", "token_row")} | {"offsets": torch.zeros_like(every["offsets"])}
    dx, dw, db = moe.moe_route_backward(ids[:0], gates[:0], dg[:0], x[:0], wr, none, dw_router=torch.full_like(dw, NAN),
                                        d_bias=torch.full_like(db, NAN))
    assert dx.shape == (0, 128) and (dw == 0).all() and (db == 0).all()


def test_route_backward_agrees_with_differences():
    """d/dz of sum(d * softmax over the chosen logits) by central differences of the 64-bit formula."""
    g = gen(12)
    T, E, k, H = 4, 6, 3, 16
    x, wr, b = (randn(g, *s).double() for s in ((T, H), (E, H), (E,)))
    d = randn(g, T, k).double()
    ids = (x @ wr.T + b).topk(k, 1).indices

    def loss(wr, b, x):
        return (d * torch.softmax((x @ wr.T + b).gather(1, ids), 1)).sum()

    gates = torch.softmax((x @ wr.T + b).gather(1, ids), 1).float()
    every = moe.moe_permute(ids.int(), gates, E, 0, E)
    dx, dw, db = moe.moe_route_backward(ids.int(), gates, d.float(), x.float(), wr.float(), every)
    h = 1e-5
    for got, at in ((dw, 0), (db, 1), (dx, 2)):
        args = [wr, b, x]
        flat = args[at].flatten()
        for i in range(0, flat.numel(), 7):
            e = torch.zeros_like(flat)
            e[i] = h
            hi = loss(*[v + e.view(v.shape) if j == at else v for j, v in enumerate(args)])
            lo = loss(*[v - e.view(v.shape) if j == at else v for j, v in enumerate(args)])
            # differences are off by h^2 times third derivatives of order one, the result by fp32 steps
            assert abs(float(got.flatten()[i]) - float((hi - lo) / (2 * h))) < 1e-4


# ------------------------------------------------------------------ norms
NORMS = [(True, False, None), (True, True, None), (True, True, "channel"), (True, True, "token"), (True, False, "token"),
         (True, False, "channel"), (False, False, None)]


@pytest.mark.parametrize("types", [(BF, F32, F32), (BF, BF, BF), (F32, F32, F32), (F32, BF, BF)])  # x; y; weights
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (2, 64), (5, 250), (70, 256), (4, 513), (3, 1000), (9, 2048), (2, 2049), (700, 4096),
                                 (3, 4104), (2, 8192), (2, 16383), (2, 16384)])
@pytest.mark.parametrize("has_y,post,gate_kind", NORMS)
def test_block_norm(T, H, has_y, post, gate_kind, types):
    g = gen(T * 31 + H)
    xt, yt, wt = types
    x, y = randn(g, T, H, dtype=xt, std=2.0), randn(g, T, H, dtype=yt) if has_y else None
    x[-1] = 0
    if has_y:
        y[-1] = 0  # a row of zeros: its root is that of eps
    wn, wp = randn(g, H, dtype=wt) + 1, randn(g, H, dtype=wt) + 1 if post else None
    gate = None if gate_kind is None else randn(g, *((H,) if gate_kind == "channel" else (T, 1)), dtype=wt)
    scale = 0.75 if has_y else 1.0
    s, n, rn, rp = moe.moe_block_norm(x, wn, y=y, w_post=wp, gate=gate, scale=scale, stats=True)
    lo = lambda t: None if t is None else t.double()  # noqa: E731
    ws, wnn, wrn, wrp = R.norm(lo(x), lo(wn), lo(y), lo(wp), lo(gate), scale)
    # sums of H squares, all positive: relative error H steps at most, halved by the root
    rel = (H + 8) * R.STEP32
    terms = (scale * x.double()).abs()
    if has_y:
        terms = terms + (ws - scale * x.double()).abs()
        R.check(s, ws, terms * (rel + 8 * R.STEP32) + ws.abs() * R.half_step(xt) * 1.01, "sum")
    else:
        assert s is None
    # the sum's error reaches its own root through the mean of sum * error, and n twice
    root = wrn[:, None]
    drift = (terms * ws.abs()).mean(1, keepdim=True) * root.square() * (rel + 8 * R.STEP32)
    R.check(rn, wrn, wrn * (rel + drift.squeeze(1)), "rstd_next")
    R.check(n, wnn, (terms * root * wn.double().abs()) * (rel + 8 * R.STEP32) + wnn.abs() * (drift + rel + 1.01 * R.half_step(xt)), "n")
    if post:
        R.check(rp, wrp, wrp * rel, "rstd_post")
    else:
        assert rp is None
    if has_y:  # in place, and the sum alone
        x2 = x.clone()
        moe.moe_block_norm(x2, wn, y=y, w_post=wp, gate=gate, scale=scale, x_out=x2)
        alone = moe.moe_block_norm(x, y=y, w_post=wp, gate=gate, scale=scale)
        assert torch.equal(x2, s) and torch.equal(alone[0], s) and alone[1] is None


@pytest.mark.parametrize("types", [(BF, F32, F32), (BF, BF, BF), (F32, F32, F32), (F32, BF, BF)])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (2, 64), (5, 250), (70, 256), (4, 513), (9, 2048), (2, 2049), (700, 4096),
                                 (3, 4104), (2, 8192), (1100, 40), (2, 16383), (2, 16384)])
@pytest.mark.parametrize("has_y,post,gate_kind", NORMS)
def test_block_norm_backward(T, H, has_y, post, gate_kind, types):
    g = gen(T * 37 + H)
    xt, yt, wt = types
    s, y = randn(g, T, H, dtype=xt, std=2.0), randn(g, T, H, dtype=yt) if has_y else None
    wn, wp = randn(g, H, dtype=wt) + 1, randn(g, H, dtype=wt) + 1 if post else None
    gate = None if gate_kind is None else randn(g, *((H,) if gate_kind == "channel" else (T, 1)), dtype=wt)
    ds, dn = randn(g, T, H, dtype=xt), randn(g, T, H, dtype=xt)
    scale = 0.75 if has_y else 1.0
    rn = torch.rsqrt(s.double().square().mean(1) + 1e-6).float()
    rp = torch.rsqrt(y.double().square().mean(1) + 1e-6).float() if post else None
    got = moe.moe_block_norm_backward(s, wn, rn, dn, dx_out=ds, y=y, w_post=wp, rstd_post=rp, gate=gate, scale=scale)
    S, r, d = s.double(), rn.double()[:, None], dn.double()
    xh, W = S * r, wn.double()
    c = (d * W * xh).mean(1, keepdim=True)
    cm = (d * W * xh).abs().mean(1, keepdim=True)
    D = ds.double() + r * (d * W - xh * c)
    # magnitudes of D's terms, the mean's with that of its own terms; H + 8 steps of each
    Dm = ds.double().abs() + r * ((d * W).abs() + xh.abs() * cm)
    steps = (H + 12) * R.STEP32
    R.check(got["dx"], scale * D, scale * Dm * steps + (scale * D).abs() * R.half_step(xt) * 1.01, "dx")
    R.check(got["dw_next"], (d * xh).sum(0), (d * xh).abs().sum(0) * (T + 8) * R.STEP32, "dw_next")
    if not has_y:
        assert got["dy"] is None and got["dw_post"] is None and got["dgate"] is None
        return
    q = rp.double()[:, None] if post else torch.ones((T, 1), dtype=R.F64, device=DEV)
    yh, P = y.double() * q, wp.double() if post else torch.ones(H, dtype=R.F64, device=DEV)
    G = gate.double() if gate is not None else torch.ones(1, dtype=R.F64, device=DEV)
    dv, dvm = G * D * P, G.abs() * Dm * P.abs()
    if post:
        m, mm = (dv * yh).mean(1, keepdim=True), (dvm * yh.abs()).mean(1, keepdim=True)
        dy, dym = q * (dv - yh * m), q * (dvm + yh.abs() * mm)
    else:
        dy, dym = dv, dvm
    R.check(got["dy"], dy, dym * 2 * steps + dy.abs() * R.half_step(yt) * 1.01, "dy")
    if post:
        R.check(got["dw_post"], (G * D * yh).sum(0), (G.abs() * Dm * yh.abs()).sum(0) * (T * R.STEP32 + steps), "dw_post")
    else:
        assert got["dw_post"] is None
    if gate is not None:
        axis = dict(dim=0) if gate_kind == "channel" else dict(dim=1, keepdim=True)
        n = T if gate_kind == "channel" else H
        R.check(got["dgate"], (D * yh * P).sum(**axis), (Dm * (yh * P).abs()).sum(**axis) * (n * R.STEP32 + steps), "dgate")
    else:
        assert got["dgate"] is None
    again = moe.moe_block_norm_backward(s, wn, rn, dn, dx_out=ds, y=y, w_post=wp, rstd_post=rp, gate=gate, scale=scale)
    other = moe.moe_block_norm_backward(s, wn, rn, dn, dx_out=ds, y=y, w_post=wp, rstd_post=rp, gate=gate, scale=scale,
                                        dy_dtype=BF if yt == F32 else F32)["dy"]
    assert other.dtype != yt and torch.equal(other.to(BF), got["dy"].to(BF))
    for name in got:
        assert (got[name] is None) == (again[name] is None)
        assert got[name] is None or torch.equal(got[name], again[name])


def test_block_norm_backward_parts():
    """One of the two gradients alone, results in place of an input, no tokens."""
    g = gen(21)
    s, y, ds, dn = (randn(g, 30, 264, dtype=BF) for _ in range(4))
    wn, wp, gate = (randn(g, 264) for _ in range(3))
    rn, rp = (torch.rsqrt(t.float().square().mean(1) + 1e-6) for t in (s, y))
    kw = dict(y=y, w_post=wp, rstd_post=rp, gate=gate, scale=0.5)
    both = moe.moe_block_norm_backward(s, wn, rn, dn, dx_out=ds, **kw)
    zero = torch.zeros_like(ds)
    a, b = moe.moe_block_norm_backward(s, wn, rn, dn, **kw), moe.moe_block_norm_backward(s, wn, rn, dn, dx_out=zero, **kw)
    c, d = moe.moe_block_norm_backward(s, dx_out=ds, **kw), moe.moe_block_norm_backward(s, wn, rn, zero, dx_out=ds, **kw)
    for p, q in ((a, b), (c, d)):
        for n in ("dx", "dy", "dw_post", "dgate"):
            assert torch.equal(p[n], q[n]), n
    assert c["dw_next"] is None and (d["dw_next"] == 0).all()
    for t in (ds, dn):
        keep = t.clone()
        got = moe.moe_block_norm_backward(s, wn, rn, dn, dx_out=ds, dx=t, **kw)
        assert torch.equal(got["dx"], both["dx"]) and torch.equal(got["dy"], both["dy"])
        t.copy_(keep)
    kw = dict(y=y[:0], w_post=wp, rstd_post=rp[:0], gate=gate)
    none = moe.moe_block_norm_backward(s[:0], wn, rn[:0], dn[:0], **kw)
    assert none["dx"].shape == (0, 264) and all((none[n] == 0).all() for n in ("dw_next", "dw_post", "dgate"))
    x, n, r1, r2 = moe.moe_block_norm(s[:0], wn, y=y[:0], stats=True)
    assert x.shape == n.shape == (0, 264) and r1.shape == (0,) and r2 is None


# ------------------------------------------------------------------ sizes past 32 bits
def test_rows_past_four_gigabytes():
    """Outputs and inputs of more than 2^32 bytes: the first and the last rows."""
    g, R_, N, K = gen(77), 1_100_000, 2048, 64
    off = torch.tensor([0, 1000, R_ - 700, R_], dtype=torch.int32, device=DEV)
    a, w = randn(g, R_, K, dtype=BF), randn(g, 3, N, K, dtype=BF)
    out = moe.moe_grouped_mm(a, w, off)
    for i, j, e in ((0, 300, 0), (R_ - 1000, R_ - 700, 1), (R_ - 700, R_, 2)):
        want = a[i:j].double() @ w[e].double().T
        mag = a[i:j].double().abs() @ w[e].double().abs().T
        R.check(out[i:j], want, mag * (K + 2) * R.STEP32 + want.abs() * R.half_step(BF) * 1.01)
    back = moe.moe_grouped_mm(out, w, off, transposed=True)  # rows of 4 KB each, from 4.5 GB
    i = R_ - 700
    want, mag = out[i:].double() @ w[2].double(), out[i:].double().abs() @ w[2].double().abs()
    R.check(back[i:], want, mag * (N + 2) * R.STEP32 + want.abs() * R.half_step(BF) * 1.01)
    h = moe.moe_swiglu(out, off)
    g64 = out[i:].double().chunk(2, 1)[0]
    want = R.swiglu(out[i:])
    R.check(h[i:], want, want.abs() * (1.01 * R.half_step(BF) + (20 + 2 * g64.abs()) * R.STEP32) + 1e-30)  # as in test_swiglu
    last = torch.tensor([0, 0, i, R_], dtype=torch.int32, device=DEV)
    dw = moe.moe_grouped_wgrad(out, a, last, dtype=F32)
    want, mag = out[i:].double().T @ a[i:].double(), out[i:].double().abs().T @ a[i:].double().abs()
    R.check(dw[2], want, mag * 703 * R.STEP32)
    assert (dw[0] == 0).all()


def test_tokens_past_two_gigabytes():
    """Gathered from a tensor that 31-bit offsets do not reach."""
    g, T, K = gen(78), 300_000, 4096
    a, w = torch.zeros((T, K), dtype=BF, device=DEV), randn(g, 2, 96, K, dtype=BF)
    pick = torch.tensor([0, T - 1, 262_145, T - 2, 5, 270_000], dtype=torch.int32, device=DEV)
    a[pick.long()] = randn(g, 6, K, dtype=BF)
    off = R.offsets_of([2, 4])
    want, mag = R.mm(a, w, off, pick)
    R.check(moe.moe_grouped_mm(a, w, off, row_index=pick), want, mag * (K + 2) * R.STEP32 + want.abs() * R.half_step(BF) * 1.01)
    b = randn(g, 6, 136, dtype=BF)
    want, mag = R.wgrad(b, a, off, None, pick)
    R.check(moe.moe_grouped_wgrad(b, a, off, b_index=pick, dtype=F32), want, mag * 9 * R.STEP32)


def test_norm_past_four_gigabytes():
    T, H = 530_000, 4096
    x = torch.ones((T, H), dtype=BF, device=DEV)
    x[-1] = 3
    w = torch.full((H,), 2.0, device=DEV)
    _, n, rn, _ = moe.moe_block_norm(x, w, stats=True)
    assert (n[0] == 2).all() and (n[-1] == 2).all() and abs(float(rn[-1]) * 3 - 1) < 1e-5
    # gradients in three rows alone: adding the others' zeros rounds nothing, so three terms a column.  In such a row dn w is
    # constant, so that dn w - xh mean(dn w xh) is eps-sized and dx is dx_out; half a step of its type.
    dn = torch.zeros_like(x)
    for t in (0, T - 2, T - 1):
        dn[t] = x[t]
    got = moe.moe_block_norm_backward(x, w, rn, dn, dx_out=x)
    half = R.half_step(BF)
    assert (got["dx"][-1] - 3).abs().max() <= 3 * half and (got["dx"][:-1].amax() - 1).abs() <= half
    assert (got["dx"][:-1].amin() - 1).abs() <= half
    want = 1 / (1 + 1e-6) ** 0.5 * 2 + 9 / (9 + 1e-6) ** 0.5
    assert (got["dw_next"].double() - want).abs().max() <= want * (3 + 8) * R.STEP32
