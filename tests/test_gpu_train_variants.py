"""GPU: variants of the training operators' products that other sizes leave out, and rows that are not finite at the tiles of
every one of them."""
import pytest
import torch

import train_ref as R
from expert_routed_grouped_amd import moe
from test_gpu_train_ops import BF, DEV, F32, NAN, TYPES, check_mm, gen, randn

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ aligned bf16 operands in tiles of 128 rows
# too few large tiles to fill the chip, too many small ones: 3000 rows of 8 experts, 16 columns of small tiles
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32)])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K", [(1024, 1024), (1000, 520)])
@pytest.mark.parametrize("counts", [[375] * 8, [0, 1, 127, 128, 129, 1000, 700, 915]], ids=["even", "uneven"])
def test_mm_in_tiles_of_128_rows(counts, N, K, gather, transposed, types):
    check_mm(counts, N, K, types, gather, transposed)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts", [[2, 4], [200, 101]], ids=["few", "many"])
def test_mm_gathered_from_past_two_gigabytes(counts, transposed):
    """Whole 16-byte rows that 31-bit offsets do not reach, in tiles of 32 and of 128 rows."""
    T, K, N = 300_000, 4096, 96
    g, n = gen(sum(counts)), sum(counts)
    a, w = torch.zeros((T, K), dtype=BF, device=DEV), randn(g, 2, *((K, N) if transposed else (N, K)), dtype=BF)
    pick = T - 1 - 7 * torch.randperm(n, device=DEV, generator=g).int()  # the last of them, from 2.4 GB on
    pick[n // 2] = 0
    a[pick.long()] = randn(g, n, K, dtype=BF)
    off = R.offsets_of(counts)
    want, mag = R.mm(a, w, off, pick, transposed)
    got = moe.moe_grouped_mm(a, w, off, row_index=pick, transposed=transposed)
    R.check(got, want, mag * (K + 2) * R.STEP32 + want.abs() * R.half_step(BF) * 1.01, "product")


# ------------------------------------------------------------------ rows that are not finite
BAD = [NAN, float("inf"), float("-inf")]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("N,K", [(264, 200), (264, 72), (129, 65)])
@pytest.mark.parametrize("counts", [[3, 40, 0, 5], [700, 333, 0, 900], [300] * 4 + [0, 513] * 20], ids=["few", "some", "many"])
def test_mm_values_that_are_not_finite(counts, N, K, transposed, types):
    """One row of the operand and one output column of an expert's matrix, next to others at every end of a step: they reach
    their own row and column and nothing else."""
    dt, ot = types
    g, off, E = gen(N + K), R.offsets_of(counts), len(counts)
    a, w = randn(g, sum(counts), K, dtype=dt), randn(g, E, N, K, dtype=dt)
    w[1, 5], w[1, 6, 0], w[1, 4, K - 1] = NAN, float("inf"), float("-inf")
    a[2], a[0, K - 1], a[3, 0] = NAN, float("inf"), float("-inf")
    if transposed:
        w = w.transpose(1, 2).contiguous()
    out = moe.moe_grouped_mm(a, w, off, transposed=transposed, dtype=ot)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[[0, 2, 3]] = True
    bad[int(off[1]):int(off[2]), 4:7] = True
    assert torch.equal(~torch.isfinite(out), bad)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("gather", ["none", "a", "b", "both"])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("M,N", [(264, 520), (128, 64), (61, 77)])
def test_wgrad_rows_that_are_not_finite(M, N, gather, add, types):
    """Experts whose last step of rows is short, each followed by one whose first rows are not finite: the others' gradients
    are to the bit what they are with zeros in those rows."""
    dt, ot = types
    g, counts = gen(M + N), [33, 3, 0, 31, 40, 97, 5, 1, 64, 2]
    off, n, E = R.offsets_of(counts), sum(counts), len(counts)
    bad = [1, 4, 6, 9]  # experts
    rows = torch.cat([torch.arange(int(off[e]), min(int(off[e]) + 3, int(off[e + 1]))) for e in bad]).to(DEV)
    ta, tb = randn(g, n, M, dtype=dt), randn(g, n, N, dtype=dt)
    spoilt, zeroed = [], []
    for t in (ta, tb):
        s, z = t.clone(), t.clone()
        z[rows] = 0
        for i, r in enumerate(rows.tolist()):
            s[r] = BAD[i % 3]
        spoilt.append(s)
        zeroed.append(z)
    order = torch.randperm(n, device=DEV, generator=g)
    index = torch.empty_like(order)
    index[order] = torch.arange(n, device=DEV)  # row r lies at index[r]
    kw = {}
    for i, name in enumerate("ab"):
        if gather in (name, "both"):
            spoilt[i], zeroed[i] = spoilt[i][order], zeroed[i][order]
            kw[name + "_index"] = index.int()
    old = randn(g, E, M, N, dtype=ot)
    got, want = (moe.moe_grouped_wgrad(p, q, off, out=old.clone(), add=add, **kw) for p, q in (spoilt, zeroed))
    assert torch.isfinite(want).all()
    for e in range(E):
        if e in bad:
            assert not torch.isfinite(got[e]).any(), e
        else:
            assert torch.equal(got[e], want[e]), e
