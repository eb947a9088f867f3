"""GPU: a MoE block trained through train.py, forward and backward together, against 64-bit differentiation of the same
formulas on the routing that the library chose."""
import pytest
import torch

from expert_routed_grouped_amd import layer as L
from expert_routed_grouped_amd import moe, synth
from expert_routed_grouped_amd import train
from expert_routed_grouped_amd.synth import LayerConfig

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64


def block(cfg, post=True, gate="channel", scale=0.8, seed=0):
    dev = L.to_device(synth.make_inputs(cfg))
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = dev["x"].dtype
    dev["norm_pre"] = torch.randn(cfg.H, device=DEV, generator=g) * 0.1 + 1
    if post:
        dev["norm_post"] = torch.randn(cfg.H, device=DEV, generator=g) * 0.1 + 1
    if gate is not None:
        dev["gate"] = torch.randn(*((cfg.H,) if gate == "channel" else (cfg.T, 1)), device=DEV, generator=g)
    dev["scale"] = scale
    dev["bias"] = torch.randn(cfg.E, device=DEV, generator=g) * 0.1
    d_out = torch.randn((cfg.T, cfg.H), device=DEV, generator=g).to(dt)
    return dev, dev["x"], d_out


def reference(dev, x, d_out, ids):
    """out and gradients by autograd in fp64, with the experts chosen as in ``ids``."""
    cfg = dev["cfg"]
    leaf = lambda t: None if t is None else t.detach().to(F64).requires_grad_(True)  # noqa: E731
    p = {n: leaf(dev.get(n)) for n in ("w_gate_up", "w_down", "w_router", "bias", "norm_pre", "norm_post", "gate")}
    xx = leaf(x)
    rms = lambda v: v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731
    n = rms(xx) * p["norm_pre"]
    gates = torch.softmax((n @ p["w_router"].T + p["bias"]).gather(1, ids.long()), 1)
    y = torch.zeros_like(xx)
    for e in range(cfg.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        gu = n[t] @ p["w_gate_up"][e].T
        g, u = gu.chunk(2, 1)
        o = (g * torch.sigmoid(g) * u) @ p["w_down"][e].T
        y = y.index_add(0, t, gates[t, j, None] * o)
    u = rms(y) * p["norm_post"] if p["norm_post"] is not None else y
    out = dev["scale"] * xx + (u if p["gate"] is None else p["gate"] * u)
    out.backward(d_out.to(F64))
    return out.detach(), {"dx": xx.grad, **{n: None if t is None else t.grad for n, t in p.items()}}


CFGS = [LayerConfig("a", T=96, H=256, E=8, k=2, I=128, act="f32", wdt="f32", seed=31, w_std=0.08),
        LayerConfig("b", T=301, H=320, E=16, k=4, I=192, seed=32, w_std=0.08),
        LayerConfig("c", T=1, H=256, E=8, k=8, I=64, seed=33, w_std=0.08),
        LayerConfig("d", T=700, H=384, E=4, k=1, I=256, seed=34, w_std=0.08),
        LayerConfig("e", T=33, H=260, E=5, k=3, I=36, act="f32", wdt="f32", seed=35, w_std=0.08),
        LayerConfig("f", T=40, H=260, E=5, k=3, I=36, seed=36, w_std=0.08)]
# Relative error in the 2-norm.  fp32: some thousand roundings of 2^-24 add up to less than 2e-5 even one-sidedly.  bf16: each
# value on the way is rounded to half a step of 2^-8 at most (2^-9 rms or less); no result has more than ten roundings of
# independent values on its way (n, gu, h, out, dy, dh, dgu, dx rows, dn, dx), which in the square mean is below 10 ** 0.5 2^-8.
TOL = {torch.float32: 2e-5, torch.bfloat16: 10 ** 0.5 * 2 ** -8}


def rel(a, b):
    return float((a.double() - b).norm() / b.norm().clamp(min=1e-300))


@pytest.mark.parametrize("post,gate", [(True, "channel"), (True, "token"), (False, None), (True, None), (False, "channel")])
@pytest.mark.parametrize("cfg", CFGS, ids=lambda c: c.name)
def test_block(cfg, post, gate):
    dev, x, d_out = block(cfg, post, gate)
    out, saved = train.block_forward(dev, x)
    grads = train.block_backward(dev, saved, d_out)
    want, wg = reference(dev, x, d_out, saved["ids"])
    tol = TOL[x.dtype]
    assert rel(out, want) < tol
    for n, g in wg.items():
        if g is None:
            assert grads[n] is None
            continue
        if cfg.k == 1 and n in ("w_router", "bias"):  # the one gate is 1 whatever the router says
            assert float(grads[n].abs().max()) <= 1e-5 * float(saved["y"].abs().max()) * cfg.T
            continue
        assert rel(grads[n], g) < (tol if n not in ("w_router", "bias") else 3 * tol), n


def test_gradients_are_added():
    """A second batch's expert gradients go on top of the first's, in fp32 and in bf16."""
    cfg = CFGS[1]
    dev, x, d_out = block(cfg)
    out, saved = train.block_forward(dev, x)
    for dtype in (torch.float32, torch.bfloat16):
        one = train.block_backward(dev, saved, d_out, dtype=dtype)
        first = {n: one[n].clone() for n in ("w_gate_up", "w_down")}
        two = train.block_backward(dev, saved, d_out, grads=one, dtype=dtype)
        for n, f in first.items():
            assert two[n] is one[n] and f.dtype == dtype
            # the same sums twice: exactly double, up to half a step of the type
            assert (two[n].double() - 2 * f.double()).abs().max() <= torch.finfo(dtype).eps * f.double().abs().max()


def test_backward_agrees_with_differences():
    """The loss along a random direction of every parameter, by central differences in fp32."""
    cfg = LayerConfig("fd", T=12, H=64, E=4, k=4, I=32, act="f32", wdt="f32", seed=41, w_std=0.2)
    dev, x, d_out = block(cfg)
    out, saved = train.block_forward(dev, x)
    grads = train.block_backward(dev, saved, d_out)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)

    def loss(name, t):
        d = dict(dev, **({} if name == "dx" else {name: t}))
        return float((train.block_forward(d, t if name == "dx" else x)[0].double() * d_out.double()).sum())

    for name in ("dx", "w_gate_up", "w_down", "w_router", "bias", "norm_pre", "norm_post", "gate"):
        p = x if name == "dx" else dev[name]
        v = torch.randn(p.shape, device=DEV, generator=g)
        h = 1e-2 * float(p.norm() / v.norm())
        num = (loss(name, p + h * v) - loss(name, p - h * v)) / (2 * h)
        ana = float((grads[name].double() * v.double()).sum())
        # h^2 times the third derivative (1e-4 of the loss's scale) and the roundings of two losses divided by 2 h
        scale = float(grads[name].norm() * v.norm())
        assert abs(num - ana) < 2e-2 * abs(ana) + 2e-3 * scale, (name, num, ana)


@pytest.mark.parametrize("cfg", [CFGS[0], CFGS[1]], ids=lambda c: c.name)
def test_shares_of_the_experts_sum_to_all(cfg):
    """Two ranks' halves of the experts, each with its own maps: sums of outputs and of gradients are the whole's."""
    dev = L.to_device(synth.make_inputs(cfg))
    x = dev["x"]
    dy = torch.randn((cfg.T, cfg.H), device=DEV).to(x.dtype)
    ids, gates = moe.moe_route(x, dev["w_router"], None, cfg.k)
    parts, perms = [], []
    for lo, hi in ((0, cfg.E), (0, cfg.E // 2), (cfg.E // 2, cfg.E)):
        perm = moe.moe_permute(ids, gates, cfg.E, lo, hi)
        wgu, wd = dev["w_gate_up"][lo:hi].contiguous(), dev["w_down"][lo:hi].contiguous()
        y, saved = train.experts_forward(x, wgu, wd, perm)
        g = train.experts_backward(saved, dy, wgu, wd)
        dx, _, _ = moe.moe_route_backward(ids, gates, torch.zeros_like(gates), x, dev["w_router"],
                                          moe.moe_permute(ids, gates, cfg.E, 0, cfg.E), rows=g["dx_rows"],
                                          token_row=perm["token_row"], dtype=torch.float32)
        parts.append((y, dx, g["d_gates"], g["dw_gate_up"], g["dw_down"]))
    whole, a, b = parts
    tol = 1e-5  # fp32 sums in another order
    for i in range(3):
        assert (whole[i] - a[i] - b[i]).abs().max() <= tol * whole[i].abs().max()
    for i in (3, 4):
        assert torch.equal(whole[i], torch.cat([a[i], b[i]]))


def test_a_captured_step_replays_and_other_streams_agree():
    cfg = CFGS[1]
    dev, x, d_out = block(cfg)
    x, d_out = x.clone(), d_out.clone()

    def step(stream=None):
        out, saved = train.block_forward(dev, x, stream=stream)
        g = train.block_backward(dev, saved, d_out, stream=stream)
        return [out] + [g[n] for n in sorted(g) if g[n] is not None]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = step(s)
        side.synchronize()
        for p, q in zip(got, want):
            assert torch.equal(p, q)
    with torch.cuda.stream(side):
        step()  # outside the capture once
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for i in range(4):
        x.copy_(torch.randn_like(x.float()).to(x.dtype))
        d_out.mul_(0.5)
        for r in res:
            r.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(res, step()):
            assert torch.equal(p, q), i


def test_two_graphs_do_not_share_memory():
    """Captured apart, replayed in turn and at once on two streams."""
    cfg = CFGS[3]
    runs = []
    for seed in (1, 2):
        dev, x, d_out = block(cfg, seed=seed)
        if seed == 2:
            x = (x.float() * 0.5).to(x.dtype)

        def step(dev=dev, x=x, d_out=d_out):
            out, saved = train.block_forward(dev, x)
            g = train.block_backward(dev, saved, d_out)
            return [out, g["dx"], g["w_down"], g["norm_post"]]

        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = step()
        runs.append((graph, res, want, step))  # the step keeps its inputs alive, which the graph reads
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for at_once in (False, True):
        for _, res, _, _ in runs:
            for r in res:
                r.fill_(7.0)
        torch.cuda.synchronize()
        for (graph, _, _, _), s in zip(runs, streams):
            with torch.cuda.stream(s):
                graph.replay()
            if not at_once:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        for _, res, want, _ in runs:
            for p, q in zip(res, want):
                assert torch.equal(p, q)


@pytest.mark.parametrize("cfg", [CFGS[0], CFGS[1]], ids=["f32", "bf16"])
def test_a_block_without_tokens(cfg):
    """A rank that got no tokens: empty results, zero gradients, and what is added to is left as it was."""
    dev, x, d_out = block(cfg)
    out, saved = train.block_forward(dev, x[:0])
    assert out.shape == (0, cfg.H)
    grads = train.block_backward(dev, saved, d_out[:0])
    assert grads["dx"].shape == (0, cfg.H)
    for n, t in grads.items():
        assert t is not None and (n == "dx" or (t == 0).all()), n
    _, full = train.block_forward(dev, x)
    have = train.block_backward(dev, full, d_out)
    want = {n: have[n].clone() for n in ("w_gate_up", "w_down")}
    train.block_backward(dev, saved, d_out[:0], grads=have)
    for n, t in want.items():
        assert torch.equal(have[n], t), n
