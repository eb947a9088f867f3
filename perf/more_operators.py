"""Operators that train a MoE block, in their plain form and as the library's calls.

Five kinds of cases:

* ``mm``: products of rows grouped by expert with that expert's matrix (``moe_grouped_mm``): ``nk`` with W [E, N, K] as a
  projection multiplies, ``kn`` with W [E, K, N], the gradient of a projection's input; the rows lie in order or are
  gathered from the tokens by an index;
* ``wgrad``: the gradient of those matrices, one product over the ragged rows of each expert (``moe_grouped_wgrad``);
* ``swiglu``: the gated activation between two projections, weighted by the row's gate, and its gradient
  (``moe_swiglu``, ``moe_swiglu_backward``);
* ``route``: from the gradient of the gates to that of the router weight, its bias and the layer's input, which the
  experts' rows are summed into (``moe_route_backward``);
* ``norm``: the RMS norms after a block and before the next one with the gate and the scale of the residual between
  them (``moe_block_norm``), and the gradient (``moe_block_norm_backward``).

With ``own = False`` ``run`` computes them with elementary torch operations in 32 bits; with ``own = True`` it makes
the calls of this package.  ``exact`` computes them in 64 bits, apart from the plain form.  Rows behind the last
expert's are left as they were: zero here.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def _rows(T, E=128, k=8, lo=0, hi=None, skew=False):
    return {"T": T, "E": E, "k": k, "lo": lo, "hi": hi or E, "skew": skew}


def _m(name, w, N, K, dtype="bf16", out="bf16", gather=False, **rows):
    return {"name": name, "kind": "mm", "w": w, "N": N, "K": K, "dtype": dtype, "out": out, "gather": gather,
            **_rows(**rows)}


def _w(name, M, N, dtype="bf16", out="bf16", gather="none", add=False, **rows):
    return {"name": name, "kind": "wgrad", "M": M, "N": N, "dtype": dtype, "out": out, "gather": gather, "add": add,
            **_rows(**rows)}


def _s(name, I, dtype="bf16", weighted=True, grad=True, **rows):
    return {"name": name, "kind": "swiglu", "I": I, "dtype": dtype, "weighted": weighted, "grad": grad, **_rows(**rows)}


def _r(name, T, E=128, k=8, H=4096, dtype="bf16", out="bf16", lo=0, hi=None):
    return {"name": name, "kind": "route", "H": H, "dtype": dtype, "out": out, **_rows(T, E, k, lo, hi)}


def _n(name, T, H, dtype="bf16", ydt="f32", post=True, gate="channel", scale=1.0, grad=True):
    return {"name": name, "kind": "norm", "T": T, "H": H, "dtype": dtype, "ydt": ydt, "post": post, "gate": gate,
            "scale": scale, "grad": grad}


def listed():
    return [
        # one token's eight rows through the down projections of its experts: latency, eight matrices
        _m("mm_token", "nk", 4096, 1536, T=1),
        # a 6000-token batch through the gate projections, rows gathered from the tokens
        _m("mm_prompt", "nk", 1536, 4096, gather=True, T=6000),
        # input gradient of the down projections for a few tokens: every active matrix read once, along its rows
        _m("mm_grad_few", "kn", 1536, 4096, T=24),
        # input gradient of an up projection on one rank's 32 experts under a hot-expert load: ragged rows
        _m("mm_grad_share", "kn", 4096, 1536, T=3001, hi=32, skew=True),
        # weight gradient of the down projections of a 6000-token batch
        _w("wgrad_prompt", 4096, 1536, gather="a", T=6000),
        # a small fp32 model with odd sizes, gradients added to those of earlier batches
        _w("wgrad_f32_odd", 777, 515, dtype="f32", out="f32", add=True, T=301, E=8, k=2),
        # one token's rows, no gradient: latency
        _s("swiglu_token", 1536, grad=False, T=1),
        # a 6000-token batch, forward and gradient
        _s("swiglu_prompt", 1536, T=6000),
        # a decode-sized batch of a fine-tuning step
        _r("route_64", 64),
        # a 6000-token batch
        _r("route_prompt", 6000),
        # one token through the residual and both norms: latency
        _n("norm_token", 1, 4096, grad=False),
        # gradient of the same for a 6000-token batch
        _n("norm_grad_prompt", 6000, 4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _size(rng, lo, hi):
    """A size, a multiple of eight three times in four."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else max(8, n // 8 * 8)


def _draw_rows(rng, most=6000):
    E = _log(rng, 2, 128)
    n, k, skew = rng.choice((E, rng.randint(1, E))), rng.randint(1, min(8, E)), rng.random() < 0.3
    T = _log(rng, 1, max(1, min(most, 32000 // n) if skew else most))
    if T * k * n < 16 * E:  # a share this small might get no row at all
        n = E
    lo = 0 if skew else rng.randint(0, E - n)
    return dict(T=T, E=E, k=k, lo=lo, hi=lo + n, skew=skew)


def draw(rng):
    kind = rng.choice(("mm", "mm", "wgrad", "swiglu", "route", "norm"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    out = rng.choice(("bf16", "f32")) if dtype == "bf16" else "f32"
    if kind == "mm":
        c = _m("", rng.choice(("nk", "kn")), _size(rng, 16, 2048), _size(rng, 16, 2048), dtype, out,
               rng.random() < 0.5, **_draw_rows(rng))
    elif kind == "wgrad":
        c = _w("", _size(rng, 16, 2048), _size(rng, 16, 2048), dtype, out, rng.choice(("none", "a", "b")),
               rng.random() < 0.3, **_draw_rows(rng))
    elif kind == "swiglu":
        c = _s("", _size(rng, 16, 1536), dtype, rng.random() < 0.7, rng.random() < 0.7, **_draw_rows(rng))
    elif kind == "route":
        r = _draw_rows(rng)
        del r["skew"]
        c = _r("", H=_size(rng, 64, 4096), dtype=dtype, out=out, **r)
    else:
        c = _n("", _log(rng, 1, 6000), _size(rng, 64, 4096), dtype, rng.choice(("bf16", "f32")), rng.random() < 0.7,
               rng.choice(("none", "channel", "token")), rng.choice((1.0, 0.7071067811865476)), rng.random() < 0.7)
    del c["name"]
    return c


def _expected(c):
    """Rows of the local experts and experts with a row, for uniform routing; a skewed load puts nearly all on the
    first experts."""
    El, E, T, k = c["hi"] - c["lo"], c["E"], c["T"], c["k"]
    share = El / E if not c["skew"] else min(1.0, 4 * El / E)
    return T * k * share, El * (1 - (1 - k / E) ** T)


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["kind"] == "norm":
        n, ye = c["T"] * c["H"], 2 if c["ydt"] == "bf16" else 4
        if c["grad"]:
            return {"bytes": n * (4 * e + 2 * ye), "flops": 20 * n}
        return {"bytes": n * (3 * e + ye), "flops": 10 * n}
    R, active = _expected(c)
    if c["kind"] == "swiglu":
        n = R * c["I"]
        return {"bytes": n * e * (9 if c["grad"] else 3), "flops": n * (25 if c["grad"] else 8)}
    if c["kind"] == "route":
        T, H, E = c["T"], c["H"], c["E"]
        return {"bytes": (R + T + E) * H * e + T * H * (2 if c["out"] == "bf16" else 4) + E * H * 4 + T * c["k"] * 16,
                "flops": 4 * T * c["k"] * H + R * H}
    o = 2 if c["out"] == "bf16" else 4
    if c["kind"] == "mm":
        a = min(R, c["T"]) if c["gather"] else R
        return {"bytes": active * c["N"] * c["K"] * e + a * c["K"] * e + R * c["N"] * o, "flops": 2 * R * c["N"] * c["K"]}
    El = c["hi"] - c["lo"]
    return {"bytes": sum((min(R, c["T"]) if c["gather"] == s else R) * c[d] * e for s, d in (("a", "M"), ("b", "N")))
            + El * c["M"] * c["N"] * o * (2 if c["add"] else 1), "flops": 2 * R * c["M"] * c["N"]}


# ------------------------------------------------------------------ inputs
def _routing(c, g):
    """Top-k of random logits and the grouping of the local assignments by expert, in token order inside an expert."""
    T, E, k, lo = c["T"], c["E"], c["k"], c["lo"]
    El = c["hi"] - lo
    logits = torch.randn((T, E), device=DEV, generator=g)
    if c["skew"]:  # 2 ln of Zipf(1.2) weights
        logits = logits - 2.4 * torch.log(torch.arange(1, E + 1, device=DEV).float())
    top, ids = logits.topk(k, 1)
    s = {"ids": ids.int(), "gates": torch.softmax(top, 1)}
    loc = ids - lo
    local = (loc >= 0) & (loc < El)
    key = torch.where(local, loc, El).flatten()
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=El + 1)[:El]
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    rank = torch.empty_like(order)
    rank[order] = torch.arange(T * k, device=DEV)
    s["token_row"] = torch.where(local, rank.view(T, k), -1).int()
    s["capacity_rows"] = T * min(k, El)
    s["row_token"] = (order // k)[:s["capacity_rows"]].int().contiguous()
    s["row_w"] = s["gates"].flatten()[order][:s["capacity_rows"]].contiguous()
    s["most"] = max(1, int(counts.max()))
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    c = dict(case)
    dt = DT[c["dtype"]]

    def randn(*shape, std=1.0, dtype=dt):
        return torch.randn(shape, device=DEV, generator=g).mul_(std).to(dtype)

    if c["kind"] == "norm":
        T, H, f = c["T"], c["H"], torch.float32
        s = {"case": c, "y": randn(T, H, dtype=DT[c["ydt"]]), "w_next": randn(H, std=0.1, dtype=f) + 1,
             "w_post": randn(H, std=0.1, dtype=f) + 1 if c["post"] else None,
             "gate": None if c["gate"] == "none" else randn(*((H,) if c["gate"] == "channel" else (T, 1)), std=0.5, dtype=f)}
        if not c["grad"]:
            s["x"] = randn(T, H, std=2.0)
            return s
        # what the forward call left: the sum, and the reciprocal roots of both norms
        s["x_out"], s["dx_out"], s["dn"] = randn(T, H, std=2.0), randn(T, H, std=0.01), randn(T, H, std=0.01)
        s["rstd_next"] = (s["x_out"].double().square().mean(1) + EPS).rsqrt().float()
        s["rstd_post"] = (s["y"].double().square().mean(1) + EPS).rsqrt().float() if c["post"] else None
        return s
    s = {"case": c, **_routing(c, g)}
    El, R, T = c["hi"] - c["lo"], s["capacity_rows"], c["T"]
    if c["kind"] == "mm":
        N, K = c["N"], c["K"]
        s["a"] = randn(T if c["gather"] else R, K)
        s["weight"] = randn(*((El, N, K) if c["w"] == "nk" else (El, K, N)), std=0.02)
        s["out"] = torch.zeros((R, N), dtype=DT[c["out"]], device=DEV)
    elif c["kind"] == "wgrad":
        s["a"] = randn(T if c["gather"] == "a" else R, c["M"], std=0.1)
        s["b"] = randn(T if c["gather"] == "b" else R, c["N"])
        s["dw"] = randn(El, c["M"], c["N"], dtype=DT[c["out"]]) if c["add"] else torch.empty(
            (El, c["M"], c["N"]), dtype=DT[c["out"]], device=DEV)
    elif c["kind"] == "swiglu":
        s["gu"], s["h"] = randn(R, 2 * c["I"], std=1.5), torch.zeros((R, c["I"]), dtype=dt, device=DEV)
        s["w"] = s["row_w"] if c["weighted"] else None
        if c["grad"]:
            s["dh"] = randn(R, c["I"], std=0.1)
            s["dgu"], s["h_again"] = torch.zeros_like(s["gu"]), torch.zeros_like(s["h"])
            s["dw"] = torch.zeros(R, device=DEV) if c["weighted"] else None
    else:
        H, E = c["H"], c["E"]
        s["x"], s["w_router"], s["d_gates"] = randn(T, H), randn(E, H, std=0.02), randn(T, c["k"], dtype=torch.float32)
        s["rows"] = randn(R, H, std=0.1)
        every = dict(c, lo=0, hi=E)  # the grouping over all experts, which the router weight's gradient follows
        flat = s["ids"].long().flatten()
        order = torch.sort(flat, stable=True).indices
        counts = torch.bincount(flat, minlength=every["hi"])
        rank = torch.empty_like(order)
        rank[order] = torch.arange(flat.numel(), device=DEV)
        s["all"] = {"offsets": torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int(),
                    "row_token": (order // c["k"]).int(), "token_row": rank.view(T, c["k"]).int()}
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"mm": _own_mm, "wgrad": _own_wgrad, "swiglu": _own_swiglu, "route": _own_route,
                "norm": _own_norm}[kind](state)
    return {"mm": _plain_mm, "wgrad": _plain_wgrad, "swiglu": _plain_swiglu, "route": _plain_route,
            "norm": _plain_norm}[kind](state)


def _own_mm(s):
    from expert_routed_grouped_amd import moe
    return moe.moe_grouped_mm(s["a"], s["weight"], s["offsets"], row_index=s["row_token"] if s["case"]["gather"] else None,
                              transposed=s["case"]["w"] == "kn", out=s["out"])


def _own_wgrad(s):
    from expert_routed_grouped_amd import moe
    c = s["case"]
    return moe.moe_grouped_wgrad(s["a"], s["b"], s["offsets"], a_index=s["row_token"] if c["gather"] == "a" else None,
                                 b_index=s["row_token"] if c["gather"] == "b" else None, out=s["dw"], add=c["add"])


def _own_swiglu(s):
    from expert_routed_grouped_amd import moe
    h = moe.moe_swiglu(s["gu"], s["offsets"], s["w"], h=s["h"])
    if not s["case"]["grad"]:
        return h
    dgu, again, dw = moe.moe_swiglu_backward(s["gu"], s["dh"], s["offsets"], s["w"], dgu=s["dgu"], h=s["h_again"],
                                             d_row_w=s["dw"])
    return {"h": h, "dgu": dgu, "h_again": again, "dw": dw}


def _own_route(s):
    from expert_routed_grouped_amd import moe
    dx, dw, db = moe.moe_route_backward(s["ids"], s["gates"], s["d_gates"], s["x"], s["w_router"], s["all"],
                                        rows=s["rows"], token_row=s["token_row"], dtype=DT[s["case"]["out"]])
    return {"dx": dx, "dw": dw, "db": db}


def _own_norm(s):
    from expert_routed_grouped_amd import moe
    c = s["case"]
    if not c["grad"]:
        x, n, _, _ = moe.moe_block_norm(s["x"], s["w_next"], y=s["y"], w_post=s["w_post"], gate=s["gate"],
                                        scale=c["scale"], eps=EPS)
        return {"x": x, "n": n}
    return moe.moe_block_norm_backward(s["x_out"], s["w_next"], s["rstd_next"], s["dn"], dx_out=s["dx_out"], y=s["y"],
                                       w_post=s["w_post"], rstd_post=s["rstd_post"], gate=s["gate"], scale=c["scale"])


def _padded(s, a, index):
    """Rows grouped by expert as fp32 [E, most, width], zero behind an expert's last row."""
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["most"], device=DEV)
    inside = at < off[1:, None]
    at = at.clamp(max=s["capacity_rows"] - 1)
    rows = s["row_token"].long()[at] if index else at
    return a[rows].float().masked_fill_(~inside.unsqueeze(-1), 0.0)


def _expert_of_row(s):
    """Expert of each row and whether the row is one at all."""
    off, r = s["offsets"].long(), torch.arange(s["capacity_rows"], device=DEV)
    return torch.searchsorted(off[1:], r, right=True).clamp(max=off.numel() - 2), r < off[-1]


def _plain_mm(s):
    c = s["case"]
    e, there = _expert_of_row(s)
    if s["capacity_rows"] < c["hi"] - c["lo"]:  # fewer rows than experts: each row with its own copy of its matrix
        a = (s["a"][s["row_token"].long()] if c["gather"] else s["a"]).float()
        w = s["weight"][e].float()
        o = (torch.bmm(w, a.unsqueeze(2)).squeeze(2) if c["w"] == "nk" else torch.bmm(a.unsqueeze(1), w).squeeze(1))
    else:
        a, w = _padded(s, s["a"], c["gather"]), s["weight"].float()
        o = torch.bmm(a, w.transpose(1, 2) if c["w"] == "nk" else w)
        o = o[e, (torch.arange(s["capacity_rows"], device=DEV) - s["offsets"].long()[e]).clamp(0, s["most"] - 1)]
    return torch.where(there[:, None], o, 0.0).to(DT[c["out"]])


def _plain_wgrad(s):
    c = s["case"]
    dw = torch.bmm(_padded(s, s["a"], c["gather"] == "a").transpose(1, 2), _padded(s, s["b"], c["gather"] == "b"))
    if c["add"]:
        return s["dw"].copy_(dw.add_(s["dw"]))
    return dw.to(DT[c["out"]])


def _plain_swiglu(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    there = _expert_of_row(s)[1][:, None]
    g, u = s["gu"].float().chunk(2, 1)
    w = s["w"][:, None] if c["weighted"] else 1.0
    sig = 1 / (1 + torch.exp(-g))
    a = g * sig * u
    h = torch.where(there, a * w, 0.0).to(dt)
    if not c["grad"]:
        return h
    dh = s["dh"].float()
    dgu = torch.cat([dh * w * u * sig * (1 + g * (1 - sig)), dh * w * g * sig], 1)
    dw = torch.where(there[:, 0], (dh * a).sum(1), 0.0) if c["weighted"] else None
    return {"h": h, "dgu": torch.where(there, dgu, 0.0).to(dt), "h_again": h, "dw": dw}


def _plain_route(s):
    c = s["case"]
    g, d = s["gates"], s["d_gates"]
    dl = g * (d - (g * d).sum(1, keepdim=True))
    dense = torch.zeros((c["T"], c["E"]), device=DEV).scatter_(1, s["ids"].long(), dl)
    dx = dense @ s["w_router"].float()
    rows = s["rows"][s["token_row"].long().clamp(min=0).flatten()].float().view(c["T"], c["k"], c["H"])
    dx = dx + rows.masked_fill_((s["token_row"] < 0).unsqueeze(-1), 0.0).sum(1)
    return {"dx": dx.to(DT[c["out"]]), "dw": dense.T @ s["x"].float(), "db": dense.sum(0)}


def _plain_norm(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    y = s["y"].float()
    gate = 1.0 if s["gate"] is None else s["gate"]
    if not c["grad"]:
        if c["post"]:
            y = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * s["w_post"]
        x = c["scale"] * s["x"].float() + gate * y
        n = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s["w_next"]
        return {"x": x.to(dt), "n": n.to(dt)}
    r, dn = s["rstd_next"][:, None], s["dn"].float()
    xh = s["x_out"].float() * r
    d = s["dx_out"].float() + r * (dn * s["w_next"] - xh * (dn * s["w_next"] * xh).mean(1, keepdim=True))
    out = {"dx": (c["scale"] * d).to(dt), "dw_next": (dn * xh).sum(0)}
    du = gate * d
    if c["post"]:
        yh = y * s["rstd_post"][:, None]
        dv = du * s["w_post"]
        dy = s["rstd_post"][:, None] * (dv - yh * (dv * yh).mean(1, keepdim=True))
        out["dw_post"] = (du * yh).sum(0)
        u = yh * s["w_post"]
    else:
        dy, u, out["dw_post"] = du, y, None
    out["dgate"] = None if c["gate"] == "none" else (d * u).sum(0) if c["gate"] == "channel" else (d * u).sum(1, keepdim=True)
    out["dy"] = dy.to(DT[c["ydt"]])
    return out


# ------------------------------------------------------------------ in 64 bits
def _groups(s, e):
    """Rows of expert e, and the tokens they came from."""
    a, b = int(s["offsets"][e]), int(s["offsets"][e + 1])
    return torch.arange(a, b, device=DEV), s["row_token"].long()[a:b]


def exact(case, seed):
    s = prepare(case, seed)
    c, f = s["case"], torch.float64
    if c["kind"] == "norm":
        return _exact_norm(s)
    El, R, T = c["hi"] - c["lo"], s["capacity_rows"], c["T"]
    if c["kind"] == "mm":
        out = torch.zeros((R, c["N"]), dtype=f, device=DEV)
        for e in range(El):
            r, t = _groups(s, e)
            w = s["weight"][e].double()
            out[r] = s["a"][t if c["gather"] else r].double() @ (w.T if c["w"] == "nk" else w)
        return out
    if c["kind"] == "wgrad":
        out = torch.zeros((El, c["M"], c["N"]), dtype=f, device=DEV)
        for e in range(El):
            r, t = _groups(s, e)
            out[e] = s["a"][t if c["gather"] == "a" else r].double().T @ s["b"][t if c["gather"] == "b" else r].double()
        return out + s["dw"].double() if c["add"] else out
    if c["kind"] == "swiglu":
        n = int(s["offsets"][-1])
        gu = s["gu"].double()[:n].clone().requires_grad_(True)
        w = (s["w"][:n].double() if c["weighted"] else torch.ones(n, dtype=f, device=DEV)).clone().requires_grad_(True)
        h = torch.sigmoid(gu[:, :c["I"]]) * gu[:, :c["I"]] * gu[:, c["I"]:] * w[:, None]

        def whole(v):
            return torch.cat([v.detach(), v.new_zeros((R - n, *v.shape[1:]))])

        if not c["grad"]:
            return whole(h)
        h.backward(s["dh"].double()[:n])
        return {"h": whole(h), "dgu": whole(gu.grad), "h_again": whole(h), "dw": whole(w.grad) if c["weighted"] else None}
    x, wr = s["x"].double(), s["w_router"].double()
    ids = s["ids"].long()
    g, d = s["gates"].double(), s["d_gates"].double()
    # the gates' Jacobian diag(g) - g g^T, entry by entry
    dl = torch.bmm(torch.diag_embed(g) - g[:, :, None] * g[:, None, :], d[:, :, None]).squeeze(2)
    dx = torch.zeros((T, c["H"]), dtype=f, device=DEV)
    dw, db = torch.zeros((c["E"], c["H"]), dtype=f, device=DEV), torch.zeros(c["E"], dtype=f, device=DEV)
    for j in range(c["k"]):
        dx += dl[:, j, None] * wr[ids[:, j]]
        at = (s["token_row"][:, j] >= 0).nonzero().flatten()
        dx[at] += s["rows"][s["token_row"][at, j].long()].double()
        dw.index_add_(0, ids[:, j], dl[:, j, None] * x)
        db.index_add_(0, ids[:, j], dl[:, j])
    return {"dx": dx, "dw": dw, "db": db}


def _exact_norm(s):
    """The forward formula in 64 bits, its gradient by differentiation with the given reciprocal roots' inputs."""
    c, f = s["case"], torch.float64

    def rms(v):
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS)

    def leaf(v):
        return v.detach().to(f).clone().requires_grad_(True)

    y, wn = leaf(s["y"]), leaf(s["w_next"])
    wp = leaf(s["w_post"]) if c["post"] else None
    gate = None if s["gate"] is None else leaf(s["gate"])
    u = rms(y) * wp if c["post"] else y
    if gate is not None:
        u = u * gate
    if not c["grad"]:
        x = c["scale"] * s["x"].to(f) + u
        return {"x": x.detach(), "n": (rms(x) * wn).detach()}
    # x_out is given: the residual that it came from is what is left of it without the block's part
    x = leaf((s["x_out"].to(f) - u.detach()) / c["scale"])
    x_out = c["scale"] * x + u
    ((x_out * s["dx_out"].to(f)).sum() + (rms(x_out) * wn * s["dn"].to(f)).sum()).backward()
    return {"dx": x.grad, "dw_next": wn.grad, "dw_post": wp.grad if c["post"] else None,
            "dgate": None if gate is None else gate.grad, "dy": y.grad}
