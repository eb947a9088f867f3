"""Operators of the MXFP4 expert layer, in their plain form and as the library's calls.

Three kinds of cases:

* ``quantize``: a matrix to MXFP4 (E2M1 codes, one E8M0 scale per 32 values of a row) and back to the values
  that the codes stand for (``moe_quantize_mx4``, ``moe_dequantize_mx``);
* ``ffn``: the SwiGLU expert FFN over rows grouped by expert with MXFP4 weights, activations quantised to MXFP8
  (W4A8) or MXFP4 (W4A4) within the call, and the gate-weighted sum to token order (``moe_grouped_ffn_mx4``);
* ``layer``: a whole MoE layer for a few tokens: router, top-k, gates, grouping, expert FFN (W4A8) and the
  weighted sum (``moe_decode_layer_mx4``).

With ``own = False`` ``run`` computes them with elementary torch operations in 32 bits; with ``own = True`` it makes
the calls of this package.  ``exact`` computes them in 64 bits, apart from the plain form.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _q(name, rows, K, dtype):
    return {"name": name, "kind": "quantize", "rows": rows, "K": K, "dtype": dtype}


def _f(name, T, act, E=128, k=8, H=4096, I=1536, lo=0, hi=None, skew=False):
    return {"name": name, "kind": "ffn", "T": T, "E": E, "k": k, "H": H, "I": I, "lo": lo, "hi": hi or E,
            "act": act, "skew": skew}


def _l(name, T, E=128, k=8, H=4096, I=1536, lo=0, hi=None, bias=False):
    return {"name": name, "kind": "layer", "T": T, "E": E, "k": k, "H": H, "I": I, "lo": lo, "hi": hi or E,
            "bias": bias}


def listed():
    return [
        # the activations of seven tokens (a small decode batch): latency
        _q("quantize_tokens", 7, 4096, "bf16"),
        # the activations of a 6000-token prompt
        _q("quantize_prompt", 6000, 4096, "bf16"),
        # the down projections of 128 experts [128 * 4096, 1536], converted once when a model is loaded
        _q("quantize_weights", 128 * 4096, 1536, "f32"),
        # decode batch: 64 tokens x top-8 of 128 experts, every active expert's weights read once
        _f("ffn_decode", 64, "mxfp8"),
        # a prefill chunk of odd length: 32 rows per expert, neither weight- nor matrix-bound
        _f("ffn_chunk", 509, "mxfp4"),
        # prompts: 375 rows per expert
        _f("ffn_prompt_a8", 6000, "mxfp8"),
        _f("ffn_prompt_a4", 6000, "mxfp4"),
        # one rank's 32 experts of 128 under a hot-expert load: ragged rows, a few experts hold most of them
        _f("ffn_share_skew", 3001, "mxfp8", lo=0, hi=32, skew=True),
        # one token: latency, eight experts' weights
        _l("layer_1", 1),
        # a few tokens with a routing bias, odd count
        _l("layer_5", 5, bias=True),
        # drafted tokens of a few sequences
        _l("layer_24", 24),
        # a decode batch on one rank of four: 32 local experts, tokens with no local expert
        _l("layer_64_share", 64, lo=32, hi=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(("quantize", "ffn", "layer"))
    if kind == "quantize":
        K = 32 * _log(rng, 1, 256)
        c = _q("", _log(rng, 1, max(1, (1 << 29) // K)), K, rng.choice(("bf16", "f32")))
    else:
        E = _log(rng, 8, 128)
        k = rng.randint(1, min(8, E))
        n = rng.choice((E, rng.randint(1, E)))
        lo = rng.randint(0, E - n)
        size = dict(E=E, k=k, H=128 * rng.randint(2, 32), I=128 * rng.randint(1, 12), lo=lo, hi=lo + n)
        if kind == "ffn":
            c = _f("", _log(rng, 1, 6000), rng.choice(("mxfp8", "mxfp4")), skew=rng.random() < 0.3, **size)
        else:
            c = _l("", _log(rng, 1, 64), bias=rng.random() < 0.5, **size)
    del c["name"]
    return c


def work(case):
    c = case
    if c["kind"] == "quantize":
        n, e = c["rows"] * c["K"], 2 if c["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * e + n // 32, "flops": 0}
    H, I, El = c["H"], c["I"], c["hi"] - c["lo"]
    # the Zipf bias of a skewed load puts nearly every assignment on the first experts
    share = El / c["E"] if not c.get("skew") else min(1.0, 4 * El / c["E"])
    rows = c["T"] * c["k"] * share
    active = El * (1 - (1 - c["k"] / c["E"]) ** c["T"])  # experts with at least one row, uniform routing
    b = active * 3 * H * I * (0.5 + 1 / 32) + c["T"] * H * 4 + c["T"] * c["k"] * 8
    f = 6 * rows * H * I
    if c["kind"] == "layer":
        b += c["E"] * H * 4
        f += 2 * c["T"] * c["E"] * H
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ MX formats, plain
_tables = {}


def _table(name):
    if name not in _tables:
        if name == "pairs":  # byte -> the two E2M1 values it holds, low nibble first
            v = E2M1 + tuple(-x for x in E2M1)
            _tables[name] = torch.tensor([(v[i & 15], v[i >> 4]) for i in range(256)], device=DEV)
        elif name == "pow2":  # E8M0 byte -> 2^(byte - 127)
            _tables[name] = torch.tensor([2.0 ** (i - 127) for i in range(255)] + [math.nan], device=DEV)
    return _tables[name]


def _dequant4(codes, scales):
    """E2M1 codes [..., K/2] and E8M0 scales [..., K/32] -> fp32 [..., K]."""
    v = _table("pairs")[codes.int()].view(*scales.shape, 32)
    return v.mul_(_table("pow2")[scales.int()].unsqueeze(-1)).view(*codes.shape[:-1], -1)


def _scales(b, emax):
    """E8M0 bytes of fp32 blocks [..., 32]: floor(log2 amax) - emax, biased, 0 for a block of zeros."""
    amax = b.abs().amax(-1)
    s = (torch.frexp(amax).exponent - 1 - emax + 127).clamp_(0, 254)
    return torch.where(amax == 0, torch.zeros_like(s), s)


def _round4(v):
    """fp32 -> nearest E2M1 value, ties to the even code, magnitudes from 6 saturate."""
    a = v.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    return torch.copysign(_table("pairs")[:8, 0][code], v)


def _fake(x, fmt):
    """Quantise [..., K] to MXFP8 or MXFP4 along K and return (fp32 values, scale bytes)."""
    b = x.float().unflatten(-1, (-1, 32))
    s = _scales(b, 8 if fmt == "mxfp8" else 2)
    p = _table("pow2")
    v = b * p[254 - s].unsqueeze(-1)
    q = v.clamp(-448, 448).to(torch.float8_e4m3fn).float() if fmt == "mxfp8" else _round4(v)
    return (q * p[s].unsqueeze(-1)).flatten(-2), s


def _draw_mx4(shape, g):
    """Weights as they are loaded: N(0, 0.02) in MXFP4, codes [..., K/2] and scales [..., K/32]."""
    out_c = torch.empty((*shape[:-1], shape[-1] // 2), dtype=torch.uint8, device=DEV)
    out_s = torch.empty((*shape[:-1], shape[-1] // 32), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (shape[1] * shape[2]))
    for i in range(0, shape[0], step):
        b = torch.randn((min(step, shape[0] - i), *shape[1:]), device=DEV, generator=g).mul_(0.02).unflatten(-1, (-1, 32))
        s = _scales(b, 2)
        v = b.mul_(_table("pow2")[254 - s].unsqueeze(-1))
        a = v.abs()
        code = torch.bucketize(a, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV), out_int32=True)
        code = (code + 8 * (v < 0)).to(torch.uint8).view(*b.shape[:-2], -1, 2)
        out_c[i:i + step] = code[..., 0] | (code[..., 1] << 4)
        out_s[i:i + step] = s.to(torch.uint8)
    return out_c, out_s


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    c = dict(case)
    s = {"case": c}
    if c["kind"] == "quantize":
        # rows of differing magnitude, as activations and weight rows have
        row = torch.exp2(4 * torch.randn((c["rows"], 1), device=DEV, generator=g))
        s["x"] = (torch.randn((c["rows"], c["K"]), device=DEV, generator=g) * row).to(DT[c["dtype"]])
        return s
    T, E, k, H, I, lo, hi = (c[n] for n in ("T", "E", "k", "H", "I", "lo", "hi"))
    El = hi - lo
    s["wgu"], s["wd"] = _draw_mx4((El, 2 * I, H), g), _draw_mx4((El, H, I), g)
    x = torch.randn((T, H), device=DEV, generator=g)
    if c["kind"] == "layer":
        # activations in steps of 1/16 and router weights in steps of 1/1024: every partial sum of a logit is then
        # exact in fp32, so that each order of summation picks the same experts
        s["x"] = ((x * 16).round() / 16).bfloat16()
        s["w_router"] = ((torch.randn((E, H), device=DEV, generator=g) * 20.48).round() / 1024).bfloat16()
        s["bias"] = (torch.randn(E, device=DEV, generator=g) * 256).round() / 256 if c["bias"] else None
        if own:
            from expert_routed_grouped_amd import moe
            s["router"] = moe.moe_pack_router(s["w_router"])
            s["ws"] = moe.moe_decode_layer_mx4_workspace(T, k, El, H, I)
            s["pgu"], s["pd"] = moe.moe_pack_mx4(*s["wgu"]), moe.moe_pack_mx4(*s["wd"])
        return s
    s["x"] = x.bfloat16()
    logits = torch.randn((T, E), device=DEV, generator=g)
    if c["skew"]:  # 2 ln of Zipf(1.2) weights
        logits = logits - 2.4 * torch.log(torch.arange(1, E + 1, device=DEV).float())
    top, ids = logits.topk(k, 1)
    s["ids"], s["gates"] = ids.int(), torch.softmax(top, 1)
    # the grouping of the local assignments by expert, in token order inside an expert
    loc = ids - lo
    local = (loc >= 0) & (loc < El)
    key = torch.where(local, loc, El).flatten()
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=El + 1)[:El]
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    rank = torch.empty_like(order)
    rank[order] = torch.arange(T * k, device=DEV)
    s["token_row"] = torch.where(local, rank.view(T, k), -1).int()
    s["row_token"] = (order // k)[:T * min(k, El)].int().contiguous()
    s["row_w"] = s["gates"].flatten()[order][:T * min(k, El)].contiguous()
    s["capacity"] = max(1, int(counts.max()))
    if own:
        from expert_routed_grouped_amd import moe
        s["ws"] = moe.moe_ffn_mx4_workspace(T, k, El, H, I)
        s["pgu"], s["pd"] = moe.moe_pack_mx4(*s["wgu"]), moe.moe_pack_mx4(*s["wd"])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"quantize": _own_quantize, "ffn": _own_ffn, "layer": _own_layer}[kind](state)
    return {"quantize": _plain_quantize, "ffn": _plain_ffn, "layer": _plain_layer}[kind](state)


def _own_quantize(s):
    from expert_routed_grouped_amd import moe
    codes, scales = moe.moe_quantize_mx4(s["x"])
    return {"values": moe.moe_dequantize_mx(codes, scales, dtype=s["x"].dtype), "scales": scales}


def _own_ffn(s):
    from expert_routed_grouped_amd import moe
    a = moe.moe_quantize_mx(s["x"]) if s["case"]["act"] == "mxfp8" else moe.moe_quantize_mx4(s["x"])
    return moe.moe_grouped_ffn_mx4(*a, s["offsets"], s["row_token"], s["row_w"], s["token_row"], s["pgu"],
                                   s["pd"], workspace=s["ws"], dtype=torch.bfloat16)


def _own_layer(s):
    from expert_routed_grouped_amd import moe
    c = s["case"]
    y, ids, gates = moe.moe_decode_layer_mx4(s["x"], s["router"], s["bias"], c["k"], c["lo"], c["hi"], s["pgu"],
                                             s["pd"], s["ws"], dtype=torch.bfloat16)
    return {"y": y, "ids": ids, "gates": gates}


def _plain_quantize(s):
    values, scales = _fake(s["x"], "mxfp4")
    return {"values": values.to(s["x"].dtype), "scales": scales.to(torch.uint8)}


def _experts(a, wgu, wd, fmt):
    """SwiGLU FFN of expert-wise rows: a [E, C, H] fp32 (quantised values), weights MXFP4 -> [E, C, H] fp32."""
    gu = torch.bmm(_dequant4(*wgu), a.transpose(1, 2).contiguous())  # [E, 2I, C]
    gate, up = gu.chunk(2, 1)
    h, _ = _fake((gate / (1 + torch.exp(-gate)) * up).transpose(1, 2), fmt)
    return torch.bmm(_dequant4(*wd), h.transpose(1, 2).contiguous()).transpose(1, 2)


def _plain_ffn(s):
    c, off = s["case"], s["offsets"].long()
    C, T, k = s["capacity"], c["T"], c["k"]
    x, _ = _fake(s["x"], c["act"])
    rows = (off[:-1, None] + torch.arange(C, device=DEV)).clamp(max=s["row_token"].numel() - 1)  # experts' rows, padded
    o = _experts(x[s["row_token"].long().clamp(0, T - 1)[rows]], s["wgu"], s["wd"], c["act"])
    e = (s["ids"].long() - c["lo"]).clamp(0, c["hi"] - c["lo"] - 1)
    here = s["token_row"] >= 0
    at = torch.where(here, e * C + s["token_row"] - off[e], 0)
    gates = torch.where(here, s["gates"], 0.0)
    return (o.reshape(-1, c["H"])[at.flatten()].view(T, k, -1) * gates.unsqueeze(-1)).sum(1).bfloat16()


def _plain_layer(s):
    c = s["case"]
    T, k, El, H = c["T"], c["k"], c["hi"] - c["lo"], c["H"]
    logits = s["x"].float() @ s["w_router"].float().T
    if s["bias"] is not None:
        logits = logits + s["bias"]
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    u = torch.exp(top - top[:, :1])
    gates = u / u.sum(1, keepdim=True)
    loc = ids - c["lo"]
    here = (loc >= 0) & (loc < El)
    loc = loc.clamp(0, El - 1)
    x, _ = _fake(s["x"], "mxfp8")
    if T * k < El:  # the weights of the selected experts only, one row each
        pick = loc.flatten()
        a = x.unsqueeze(1).expand(T, k, H).reshape(T * k, 1, H)
        o = _experts(a, [w[pick] for w in s["wgu"]], [w[pick] for w in s["wd"]], "mxfp8").view(T, k, H)
    else:  # every local expert on every token, then the selected ones
        o = _experts(x.expand(El, T, H), s["wgu"], s["wd"], "mxfp8")[loc, torch.arange(T, device=DEV)[:, None]]
    y = (o * torch.where(here, gates, 0.0).unsqueeze(-1)).sum(1)
    return {"y": y.bfloat16(), "ids": ids.int(), "gates": gates}


# ------------------------------------------------------------------ in 64 bits
def _exact_mx(x, grid, emax):
    """Nearest grid value times the block's power of two, fp64; ``grid`` holds the non-negative code values in order."""
    b = x.double().reshape(-1, 32)
    amax = b.abs().max(1, keepdim=True).values
    e = torch.floor(torch.log2(torch.where(amax == 0, torch.ones_like(amax), amax)))
    e = torch.where(torch.exp2(e) > amax, e - 1, torch.where(torch.exp2(e + 1) <= amax, e + 1, e))  # log2 may round
    scale = torch.exp2(torch.where(amax == 0, torch.full_like(e, -127.0), (e - emax).clamp(-127, 127)))
    v = (b / scale).abs()
    hi = torch.searchsorted(grid, v).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    below, above = v - grid[lo], grid[hi] - v
    code = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    code = torch.where(v >= grid[-1], torch.full_like(code, grid.numel() - 1), code)
    return (torch.copysign(grid[code], b) * scale).reshape(x.shape)


def _grid(fmt):
    if fmt == "mxfp4":
        return torch.tensor(E2M1, dtype=torch.float64, device=DEV), 2
    v = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device=DEV), 8


def _exact_weights(codes, scales):
    v = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    mag = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[v & 7]
    return torch.where(v >= 8, -mag, mag) * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["kind"] == "quantize":
        x = s["x"]
        out = torch.empty(x.shape, dtype=torch.float64, device=DEV)
        step = max(1, (1 << 24) // c["K"])
        for i in range(0, c["rows"], step):
            out[i:i + step] = _exact_mx(x[i:i + step], *_grid("mxfp4"))
        return {"values": out, "scales": None}
    T, k, H, I, lo, El = c["T"], c["k"], c["H"], c["I"], c["lo"], c["hi"] - c["lo"]
    fmt = c.get("act", "mxfp8")
    grid, emax = _grid(fmt)
    if c["kind"] == "ffn":
        ids, gates = s["ids"].long(), s["gates"].double()
    else:
        logits = s["x"].double() @ s["w_router"].double().T
        if s["bias"] is not None:
            logits = logits + s["bias"].double()
        # largest first, the lower index of equal logits: sort by index within the stable descending order
        ids = torch.sort(-logits, dim=1, stable=True).indices[:, :k]
        gates = torch.softmax(logits.gather(1, ids), 1)
    x = _exact_mx(s["x"], grid, emax)
    y = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    for e in range(El):
        t, j = (ids == lo + e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        gu = x[t] @ _exact_weights(s["wgu"][0][e], s["wgu"][1][e]).T
        h = _exact_mx(gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:], grid, emax)
        y.index_add_(0, t, gates[t, j, None] * (h @ _exact_weights(s["wd"][0][e], s["wd"][1][e]).T))
    return y if c["kind"] == "ffn" else {"y": y, "ids": None, "gates": gates}
