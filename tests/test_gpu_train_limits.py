"""GPU: documented sizes that need more than 2^32 threads, or workgroups than one axis of a grid takes."""
import pytest
import torch

import train_ref as R
from expert_routed_grouped_amd import moe
from test_gpu_train_ops import BF, DEV, F32, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def ends(n, mark):
    """Slices at the first row, around ``mark`` and at the last."""
    return slice(0, 1000), slice(mark - 500, min(mark + 500, n)), slice(n - 1000, n)


@pytest.mark.parametrize("R_,I", [((1 << 26) + 5, 1), ((1 << 27) + 1, 8)])
def test_swiglu(R_, I):
    """One wave a row, four a workgroup."""
    gu, dh = randn(gen(1), R_, 2 * I, dtype=BF), randn(gen(2), R_, I, dtype=BF)
    h = moe.moe_swiglu(gu)
    dgu, h2, _ = moe.moe_swiglu_backward(gu, dh)
    assert torch.equal(h, h2)
    for s in ends(R_, 1 << 26):
        assert torch.equal(h[s], moe.moe_swiglu(gu[s].clone()))
        want = moe.moe_swiglu_backward(gu[s].clone(), dh[s].clone())[0]
        assert torch.equal(dgu[s], want)


@pytest.mark.parametrize("T,H,dtype", [((1 << 26) + 3, 8, BF), ((1 << 26) + 3, 1, F32), ((1 << 22) + 3, 4104, BF)])
def test_block_norm(T, H, dtype):
    """A workgroup of one wave a row, and of sixteen."""
    x = torch.ones((T, H), dtype=dtype, device=DEV)
    marks = [0, 1 << 22, T - 2, T - 1]
    x[marks] = 3
    w = torch.full((H,), 2.0, device=DEV)
    n = torch.zeros_like(x)
    _, _, rn, _ = moe.moe_block_norm(x, w, n=n, stats=True)
    rn = rn.double()
    rn[marks] *= 3
    assert (rn - (1 + 1e-6) ** -0.5).abs().max() < 1e-6  # a root of sums of up to 4104 ones is off by a few steps of 2^-23
    assert (n.amin() - 2).abs() < 1e-5 and (n.amax() - 2).abs() < 1e-5  # 2 (1 - 5e-7) in the type


def test_route_backward():
    """Four tokens to a workgroup of sixteen waves; values whose sums are exact."""
    T, E, k, H = (1 << 24) + 5, 2, 2, 8
    ids = torch.tensor([0, 1], dtype=torch.int32, device=DEV).repeat(T, 1)
    gates = torch.full((T, k), 0.5, device=DEV)
    dg = torch.zeros((T, k), device=DEV)
    marks = [0, 1, 1 << 24, T - 2, T - 1]
    dg[marks, 0] = 2.0  # dl = 0.5 (2 - 1), 0.5 (0 - 1)
    x = torch.ones((T, H), dtype=BF, device=DEV)
    wr = torch.arange(16, device=DEV).view(E, H).to(BF) / 4
    at = torch.arange(T, dtype=torch.int32, device=DEV)
    perm = dict(offsets=torch.tensor([0, T, 2 * T], dtype=torch.int32, device=DEV), row_token=torch.cat([at, at]))
    dx, dw, db = moe.moe_route_backward(ids, gates, dg, x, wr, perm)
    assert (dw[0] == 2.5).all() and (dw[1] == -2.5).all() and db.tolist() == [2.5, -2.5]
    want = 0.5 * (wr[0].float() - wr[1].float())  # -1 in every column
    assert (dx[marks].float() == want).all()
    dx[marks] = 0
    assert (dx == 0).all()


def test_mm_of_many_columns():
    """129 rows, one an expert, of 2^24 - 1 columns at odd sizes; 65 of whole pieces."""
    E, N = 129, (1 << 24) - 1
    a, w = randn(gen(3), E, 1, dtype=BF), randn(gen(4), E, N, 1, dtype=BF)
    out = moe.moe_grouped_mm(a, w, R.offsets_of([1] * E))
    assert torch.equal(out, w.view(E, N) * a)  # one product each, rounded once
    del out, w
    E, N, K = 65, (1 << 24) - 8, 8
    a, w = randn(gen(5), E, K, dtype=BF), torch.empty((E, N, K), dtype=BF, device=DEV)
    w.normal_(generator=gen(6))
    out = moe.moe_grouped_mm(a, w, R.offsets_of([1] * E))
    for e in (0, 31, 63, 64):
        want, mag = w[e].double() @ a[e].double(), w[e].double().abs() @ a[e].double().abs()
        R.check(out[e], want, mag * (K + 2) * R.STEP32 + want.abs() * R.half_step(BF) * 1.01, f"expert {e}")


def test_wgrad_of_many_columns():
    E, N = 129, (1 << 24) - 1
    a, b = randn(gen(7), E, 1, dtype=BF), randn(gen(8), E, N, dtype=BF)
    dw = moe.moe_grouped_wgrad(a, b, R.offsets_of([1] * E))
    assert torch.equal(dw.view(E, N), a * b)


def test_route_backward_of_the_weight_alone():
    """More pieces of odd rows than one row of workgroups takes, and no dx: the workgroups too many have nothing to write."""
    T, E, k, H = 32769, 1024, 32, 64 * 4096 + 1
    at = torch.arange(T, device=DEV)[:, None]
    ids = ((at + 32 * torch.arange(k, device=DEV)) % E).int()
    gates, dg = torch.full((T, k), 1 / 32, device=DEV), torch.zeros((T, k), device=DEV)
    t = T - 3
    dg[t, 0] = 32.0  # dl = (32 - 1) / 32, and (0 - 1) / 32 for the token's other experts
    x = torch.ones((T, H), dtype=BF, device=DEV)
    perm = moe.moe_permute(ids, gates, E, 0, E)
    dw, db = torch.full((E, H), 7.0, device=DEV), torch.full((E,), 7.0, device=DEV)
    p = lambda v: v.data_ptr()  # noqa: E731
    assert moe.lib().moe_route_backward(p(ids), p(gates), p(dg), T, k, E, H, p(x), None, moe.MOE_BF16, p(perm["offsets"]),
                                        p(perm["row_token"]), None, 0, None, 0, None, 0, p(dw), p(db),
                                        torch.cuda.current_stream().cuda_stream) == 0
    want = torch.zeros(E, device=DEV)
    want[ids[t].long()] = -1 / 32
    want[int(ids[t, 0])] = 31 / 32
    assert torch.equal(db, want) and torch.equal(dw, want[:, None].expand(E, H))
