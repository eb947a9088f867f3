"""GPU: the MXFP4 expert FFN at the largest sizes it takes (operands just below 2^31 bytes)."""
import pytest
import torch

from expert_routed_grouped_amd import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("act", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("T,k,H,I", [((1 << 24) - 1, 1, 128, 128), ((1 << 20) - 1, 2, 256, 1024)])
def test_grouped_ffn_at_the_size_limit(T, k, H, I, act):
    """T * H or T * k * I one step below 2^31: rows from the start, the middle and the end are what a small call makes of
    them, bit for bit (a row's result depends on its own operands alone)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    El = 2
    gu, dn = (moe.moe_pack_mx4(*(t.view(El, n, -1) for t in moe.moe_quantize_mx4(
        torch.randn((El * n, m), device=DEV, generator=g) * 0.1))) for n, m in ((2 * I, H), (H, I)))
    x = torch.randn((T, H), dtype=torch.bfloat16, device=DEV, generator=g)
    a, s = moe.moe_quantize_mx(x) if act == "mxfp8" else moe.moe_quantize_mx4(x)
    del x
    # k == 1: the first half of the tokens on expert 0, the others on expert 1; k == 2: every token on both
    t = torch.arange(T, dtype=torch.int32, device=DEV)
    half = T // 2

    def maps(tok):
        n = tok.numel()
        if k == 2:
            order = torch.arange(n, dtype=torch.int32, device=DEV)
            row_token = torch.cat((order, order))
            token_row = torch.stack((order, order + n), 1).contiguous()
            off = [0, n, 2 * n]
        else:
            row_token = torch.arange(n, dtype=torch.int32, device=DEV)
            token_row = row_token[:, None].contiguous()
            off = [0, int((tok < half).sum()), n]
        row_w = (tok.float() % 7 + 1).repeat(k) / 8
        return torch.tensor(off, dtype=torch.int32, device=DEV), row_token, row_w.contiguous(), token_row

    y = moe.moe_grouped_ffn_mx4(a, s, *maps(t), gu, dn)
    pick = torch.cat((t[:90], t[half - 90:half + 90], t[-90:]))
    want = moe.moe_grouped_ffn_mx4(a[pick].contiguous(), s[pick].contiguous(), *maps(pick), gu, dn)
    assert torch.equal(y[pick], want) and bool(want.any(1).all())
    assert bool(y[::4097].any(1).all())
