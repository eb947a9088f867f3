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
