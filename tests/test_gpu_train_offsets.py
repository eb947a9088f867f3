"""GPU: grouped calls whose offsets do not fit the buffers.  The rows there are, clipped to the buffers, are computed in every
variant; nothing else is read or written."""
import pytest
import torch

import train_ref as R
from expert_routed_grouped_amd import moe
from test_gpu_train_ops import BF, DEV, F32, MANY, TYPES, gen, randn

pytestmark = pytest.mark.gpu


def check_clipped(offsets, n, N, K, types, transposed, gather, seed=0):
    """A product of n rows with these offsets, against the one with what lies in [0, n) of them."""
    g = gen(seed + N + K)
    dt, ot = types
    E = len(offsets) - 1
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    index = None
    if gather:
        index = torch.randint(0, n, (n,), device=DEV, generator=g).int()
    a = randn(g, n, K, dtype=dt)
    w = randn(g, E, K, N, dtype=dt) if transposed else randn(g, E, N, K, dtype=dt)
    store = torch.full((n + 300, N), 7.0, device=DEV, dtype=ot)
    moe.moe_grouped_mm(a, w, off, row_index=index, transposed=transposed, out=store[:n])
    assert (store[n:] == 7.0).all(), "rows behind the buffer were written"
    lo, hi = min(max(offsets[0], 0), n), min(max(offsets[-1], 0), n)
    want, mag = R.mm(a, w, off.clamp(0, n), index, transposed)
    assert (store[:lo] == 7.0).all() and (store[hi:n] == 7.0).all()
    bound = mag * (K + 2) * R.STEP32 + want.abs() * R.half_step(ot) * 1.01
    R.check(store[lo:hi], want[lo:hi], bound[lo:hi], "product")


# whole 16-byte rows and odd ones, one column of tiles and several
SIZES = [(264, 64), (264, 65), (128, 65), (257, 129), (33, 200)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K", SIZES)
def test_mm_offsets_past_the_buffers(N, K, gather, transposed, types):
    """More tiles promised than a grid for the buffers' rows has: many rows an expert, few, and one expert."""
    check_clipped(R.offsets_of(MANY, "cpu").tolist(), 5000, N, K, types, transposed, gather)
    check_clipped(R.offsets_of([40] * 30, "cpu").tolist(), 600, N, K, types, transposed, gather)
    check_clipped([0, 1024], 512, N, K, types, transposed, gather)
    check_clipped([0, 7, 1024, 1 << 30], 512, N, K, types, transposed, gather)


# ------------------------------------------------------------------ offsets from anywhere
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


def check_untouched(offsets, n, N, K, types, transposed):
    """Nothing in front of the buffer and nothing behind it."""
    dt, ot = types
    g, E, pad = gen(N + K), len(offsets) - 1, 64
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    a = randn(g, n, K, dtype=dt)
    w = randn(g, E, K, N, dtype=dt) if transposed else randn(g, E, N, K, dtype=dt)
    store = torch.full((n + 2 * pad, N), 7.0, device=DEV, dtype=ot)  # pad rows: whole 16-byte pieces
    moe.moe_grouped_mm(a, w, off, transposed=transposed, out=store[pad:pad + n])
    assert (store[:pad] == 7.0).all() and (store[pad + n:] == 7.0).all()
    return store[pad:pad + n]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("n,N,K", [(512, 264, 64), (512, 257, 65), (5000, 1536, 64), (9, 64, 64)])
def test_mm_offsets_from_anywhere(n, N, K, transposed, types):
    """Ends whose difference does not fit 32 bits, negative ones, ranges that come more than once."""
    for offsets in ([HIGH, LOW], [HIGH, -2], [LOW, LOW], [HIGH, HIGH], [n, n + 5], [-9, -2], [3, 0]):
        assert (check_untouched(offsets, n, N, K, types, transposed) == 7.0).all(), offsets
    for offsets in ([-7, 5, 20], [LOW, HIGH], [LOW, 6, HIGH], [0, 0, n, HIGH]):
        check_clipped(offsets, n, N, K, types, transposed, False)
    for offsets in ([0, n] * 40, [HIGH, LOW] * 70 + [HIGH], [5, 3, 9, -1, n]):
        check_untouched(offsets, n, N, K, types, transposed)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("n,M,N", [(512, 264, 64), (513, 37, 65), (5000, 136, 72)])
def test_wgrad_offsets_from_anywhere(n, M, N, types):
    g = gen(n + M)
    dt, ot = types
    a, b = randn(g, n, M, dtype=dt), randn(g, n, N, dtype=dt)
    index = torch.arange(n, device=DEV).int()
    for offsets in ([HIGH, LOW], [HIGH, -2, -1], [n, n + 5], [3, 0], [-7, 5, 20], [LOW, HIGH], [LOW, 6, HIGH, HIGH]):
        off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        clipped = off.clamp(0, n)
        want, mag = torch.zeros((len(offsets) - 1, M, N), dtype=R.F64, device=DEV), 0.0
        for e, i, j in R.spans(clipped):
            if j > i:
                want[e] = a[i:j].double().T @ b[i:j].double()
        mag = a.double().abs().T @ b.double().abs()
        for kw in ({}, dict(a_index=index), dict(b_index=index)):
            got = moe.moe_grouped_wgrad(a, b, off, dtype=ot, **kw)
            R.check(got, want, mag * (n + 3) * R.STEP32 + want.abs() * R.half_step(ot) * 1.01, offsets)


def test_row_wise_calls_with_offsets_from_anywhere():
    g, n, I = gen(4), 40, 72
    gu, dh = randn(g, n, 2 * I, dtype=BF), randn(g, n, I, dtype=BF)
    for last, rows in ((LOW, 0), (-1, 0), (n + 1, n), (HIGH, n), (7, 7)):
        off = torch.tensor([0, last], dtype=torch.int32, device=DEV)
        h = torch.full((n + 8, I), 7.0, dtype=BF, device=DEV)
        moe.moe_swiglu(gu, off, h=h[:n])
        assert torch.equal(h[:rows], moe.moe_swiglu(gu)[:rows]) and (h[rows:] == 7.0).all()
        dgu, d, w = torch.full((n + 8, 2 * I), 7.0, dtype=BF, device=DEV), h.clone().fill_(7.0), torch.ones(n, device=DEV)
        dw = torch.full((n + 8,), 7.0, device=DEV)
        moe.moe_swiglu_backward(gu, dh, off, w, dgu=dgu[:n], h=d[:n], d_row_w=dw[:n])
        for t in (dgu, d, dw):
            assert (t[rows:] == 7.0).all() and (rows == 0 or not (t[:rows] == 7.0).all())
    T, E, k, H = 20, 4, 2, 136
    ids = torch.rand((T, E), device=DEV, generator=g).topk(k, 1).indices.int()
    gates, dg = torch.softmax(randn(g, T, k), 1), randn(g, T, k)
    x, wr = randn(g, T, H), randn(g, E, H)
    perm = moe.moe_permute(ids, gates, E, 0, E)
    want = moe.moe_route_backward(ids, gates, dg, x, wr, perm)
    off = perm["offsets"].clone()
    off[0], off[E] = LOW, HIGH  # clipped they are what they were
    got = moe.moe_route_backward(ids, gates, dg, x, wr, dict(perm, offsets=off))
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    off = torch.tensor([HIGH, LOW, HIGH, -2, -3], dtype=torch.int32, device=DEV)
    got = moe.moe_route_backward(ids, gates, dg, x, wr, dict(perm, offsets=off))
    assert torch.equal(got[0], want[0])
    for e in (0, 2, 3):  # the second expert is given every row; none is one of the others'
        assert (got[1][e] == 0).all() and got[2][e] == 0
