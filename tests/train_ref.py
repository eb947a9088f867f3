"""Plain 64-bit formulations of the operators that train a MoE block, and the bounds that their tests hold results to.

Bounds: a result differs from the 64-bit value by the roundings on its way.  Each fp32 addition or multiplication is
off by at most one step of its result, 2^-23 of it (half a step when rounded to nearest; a matrix instruction may
truncate), so a sum of n products differs by at most (n + 2) 2^-23 of the sum of their magnitudes; the last rounding
adds half a step of the output's type (``half_step``)."""
import torch

F64 = torch.float64
STEP32 = 2.0 ** -23


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def offsets_of(counts, device="cuda"):
    c = torch.tensor([0] + list(counts), dtype=torch.int64).cumsum(0)
    return c.to(torch.int32).to(device)


def spans(offsets):
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1)]


def mm(a, w, offsets, index=None, transposed=False):
    """(values, sums of magnitudes) of the rows there are, fp64."""
    R = int(offsets[-1])
    src = a[index[:R].long()] if index is not None else a[:R]
    N = w.shape[2] if transposed else w.shape[1]
    out, mag = (torch.zeros((R, N), dtype=F64, device=a.device) for _ in range(2))
    for e, i, j in spans(offsets):
        m = w[e].double() if transposed else w[e].double().T
        out[i:j], mag[i:j] = src[i:j].double() @ m, src[i:j].double().abs() @ m.abs()
    return out, mag


def wgrad(a, b, offsets, ai=None, bi=None):
    R = int(offsets[-1])
    x = (a[ai[:R].long()] if ai is not None else a[:R]).double()
    y = (b[bi[:R].long()] if bi is not None else b[:R]).double()
    E = offsets.numel() - 1
    out, mag = (torch.zeros((E, a.shape[1], b.shape[1]), dtype=F64, device=a.device) for _ in range(2))
    for e, i, j in spans(offsets):
        out[e], mag[e] = x[i:j].T @ y[i:j], x[i:j].abs().T @ y[i:j].abs()
    return out, mag


def swiglu(gu, w=None):
    g, u = gu.double().chunk(2, 1)
    h = g * torch.sigmoid(g) * u
    return h if w is None else h * w.double()[:, None]


def swiglu_backward(gu, dh, w=None):
    g, u = gu.double().chunk(2, 1)
    s, d = torch.sigmoid(g), dh.double()
    ww = 1.0 if w is None else w.double()[:, None]
    dgu = torch.cat([ww * d * u * s * (1 + g * (1 - s)), ww * d * g * s], 1)
    return dgu, (d * g * s * u).sum(1)


def route_backward(ids, gates, d_gates, x, wr, rows=None, at=None):
    """dl, dx, dw, db in fp64."""
    g, d = gates.double(), d_gates.double()
    dl = g * (d - (g * d).sum(1, keepdim=True))
    dense = torch.zeros((ids.shape[0], wr.shape[0]), dtype=F64, device=x.device).scatter_(1, ids.long(), dl)
    dx = dense @ wr.double()
    if rows is not None:
        part = rows.double()[at.long().clamp(min=0)]
        dx = dx + torch.where((at >= 0).unsqueeze(-1), part, 0.0).sum(1)
    return dl, dx, dense.T @ x.double(), dense.sum(0)


def norm(x, w_next=None, y=None, w_post=None, gate=None, scale=1.0, eps=1e-6):
    """x_out, n, rstd_next, rstd_post in fp64; the leaves may require gradients."""
    rp = None
    s = x
    if y is not None:
        u = y
        if w_post is not None:
            rp = torch.rsqrt(y.square().mean(1) + eps)
            u = y * rp[:, None] * w_post
        s = scale * x + (u if gate is None else gate * u)
    rn = torch.rsqrt(s.square().mean(1) + eps)
    return s, None if w_next is None else s * rn[:, None] * w_next, rn, rp


def check(got, want, bound, what=""):
    """Every element within its bound (NaN and infinity nowhere)."""
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} elements out of bound, the worst by "
                           f"{float((err / bound.clamp(min=1e-300)).nan_to_num(nan=float('inf')).max()):.3g} times; first at "
                           f"{bad.nonzero()[0].tolist()}")
