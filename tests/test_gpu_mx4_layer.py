"""GPU: layer.run_layer with MXFP4 experts (convert_experts_mx4, Mx4LayerBuffers) in the orders and on the streams that
a program may use."""
import pytest
import torch

import mx4_ref as R
from expert_routed_grouped_amd import layer as L
from expert_routed_grouped_amd import moe, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


def model(T, seed, I_s=0, act="bf16", H=512, E=24, I=256, **kw):
    cfg = synth.LayerConfig("mx4", T=T, H=H, E=E, k=4, I=I, act=act, wdt=act, seed=seed, w_std=0.06, I_s=I_s, **kw)
    return cfg, L.to_device(synth.make_inputs(cfg))


@pytest.mark.parametrize("T,act", [(9, "mxfp8"), (9, "mxfp4"), (150, "mxfp8")])
def test_shared_expert_with_packed_weights(T, act):
    """convert_experts_mx4, then pack_weights, then run_layer gives what it gives before pack_weights.

    The two runs of the shared expert may add in another order (fp32), so that a value of its h can round to the
    neighbouring bf16: one step, 2^-7 of it; its down product and the sum into y are fp32 with at most I_s + 8 additions."""
    I_s = 192
    cfg, dev = model(T, 91, I_s=I_s, e_begin=4, e_end=20)
    L.convert_experts_mx4(dev)
    bufs = L.Mx4LayerBuffers(cfg, act=act, dtype=torch.float32)
    want = L.run_layer(dev, bufs).clone()
    gu, dn = dev["ws_gate_up"].double(), dev["ws_down"].double()
    L.pack_weights(dev)
    assert dev["packed"]
    y = L.run_layer(dev, bufs)
    a = dev["x"].double() @ gu.T
    G, U = a[:, :I_s], a[:, I_s:]
    shared = G * torch.sigmoid(G) * U
    mag = shared.abs() @ dn.abs().T
    bound = (2.0 ** -7 + 2 * (I_s + 8) * 2.0 ** -24) * mag + 2.0 ** -20 * want.abs()
    assert bool(((y - want).double().abs() <= bound).all())
    # and the bound would not let another layout pass
    assert float(bound.square().mean().sqrt()) < 0.2 * float((shared @ dn.T).square().mean().sqrt())


@pytest.mark.parametrize("mx4", [True, False])
def test_edited_router_on_another_stream(mx4):
    """w_router is edited, then the layer runs on a stream while the current one is busy, then on a third: every call
    routes with the new weight, and the current stream's new tensors do not land on a copy that is still read."""
    cfg, dev = model(9, 92)
    if mx4:
        L.convert_experts_mx4(dev)
        bufs = [L.Mx4LayerBuffers(cfg) for _ in range(2)]
    else:
        L.pack_router(dev)
        bufs = [L.LayerBuffers(cfg) for _ in range(2)]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    for _ in range(4):
        w = torch.randn(dev["w_router"].shape, device=DEV, generator=g) * 0.05
        dev["w_router"].copy_(w)
        want, gates = moe.moe_route(dev["x"], dev["w_router"], None, 4)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # the current stream is behind
        L.run_layer(dev, bufs[0], stream=a)
        L.run_layer(dev, bufs[1], stream=b)
        junk = [torch.full((512 // 4, 24, 4), 1e9, device=DEV) for _ in range(4)]
        torch.cuda.synchronize()
        for f in bufs:
            assert torch.equal(f.topk_ids, want) and torch.equal(f.topk_w, gates)
        del junk


def test_edited_router_captured():
    """A graph captured while the packed router is stale packs it for itself; calls outside pack their own."""
    cfg, dev = model(9, 93)
    L.convert_experts_mx4(dev)
    bufs, other = L.Mx4LayerBuffers(cfg), L.Mx4LayerBuffers(cfg)
    L.run_layer(dev, bufs)
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    new = lambda: torch.randn(dev["w_router"].shape, device=DEV, generator=g) * 0.05  # noqa: E731
    dev["w_router"].copy_(new())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        L.run_layer(dev, bufs)
    for _ in range(3):
        want = moe.moe_route(dev["x"], dev["w_router"], None, 4)
        L.run_layer(dev, other)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for f in (bufs, other):
            assert torch.equal(f.topk_ids, want[0]) and torch.equal(f.topk_w, want[1])
        assert torch.equal(bufs.y, other.y)
        dev["w_router"].copy_(new())


def test_graph_keeps_its_router_copy():
    """A graph captured with one router weight goes on routing with it after the weight was edited and packed again,
    whatever was allocated since."""
    cfg, dev = model(9, 94)
    L.convert_experts_mx4(dev)
    bufs, other = L.Mx4LayerBuffers(cfg), L.Mx4LayerBuffers(cfg)
    L.run_layer(dev, bufs)
    want = [t.clone() for t in (bufs.topk_ids, bufs.topk_w, bufs.y)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        L.run_layer(dev, bufs)
    for _ in range(3):
        dev["w_router"].mul_(-1.0)
        L.run_layer(dev, other)
        ids = moe.moe_route(dev["x"], dev["w_router"], None, 4)[0]
        junk = [torch.full((512 // 4, 24, 4), 1e9, device=DEV) for _ in range(8)]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(other.topk_ids, ids)
        assert all(torch.equal(a, b) for a, b in zip(want, (bufs.topk_ids, bufs.topk_w, bufs.y)))
        del junk


def test_copied_layer():
    import copy
    cfg, dev = model(9, 97)
    L.convert_experts_mx4(dev)
    bufs = L.Mx4LayerBuffers(cfg)
    y = L.run_layer(dev, bufs).clone()
    other = copy.deepcopy(dev)
    dev["w_router"].zero_()
    assert torch.equal(L.run_layer(other, bufs), y)


@pytest.mark.parametrize("T,I_s", [(9, 0), (9, 192), (150, 0), (150, 192)])
@pytest.mark.parametrize("act", ["mxfp8", "mxfp4"])
def test_captured_layer(T, I_s, act):
    """The layer captured and replayed with new tokens, eager calls on other buffers in between."""
    cfg, dev = model(T, 98, I_s=I_s, e_begin=4, e_end=20)
    L.convert_experts_mx4(dev)
    dtype = torch.float32 if I_s else torch.bfloat16
    bufs, other = (L.Mx4LayerBuffers(cfg, act=act, dtype=dtype) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    L.run_layer(dev, bufs, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        L.run_layer(dev, bufs, stream=side)
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    for _ in range(4):
        dev["x"].copy_(torch.randn(dev["x"].shape, device=DEV, generator=g))
        L.run_layer(dev, other)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs.topk_ids, other.topk_ids) and torch.equal(bufs.topk_w, other.topk_w)
        if I_s:  # the shared expert adds in no fixed order, see test_shared_expert_with_packed_weights
            gu, dn = dev["ws_gate_up"].double(), dev["ws_down"].double()
            a = dev["x"].double() @ gu.T
            h = (a[:, :I_s] * torch.sigmoid(a[:, :I_s]) * a[:, I_s:]).abs()
            bound = (2.0 ** -7 + 2 * (I_s + 8) * 2.0 ** -24) * (h @ dn.abs().T) + 2.0 ** -20 * other.y.abs()
            assert bool(((bufs.y - other.y).double().abs() <= bound).all())
        else:
            assert torch.equal(bufs.y, other.y)


@pytest.mark.parametrize("act", ["mxfp8", "mxfp4"])
def test_layer_without_tokens(act):
    cfg, dev = model(0, 99)
    L.convert_experts_mx4(dev)
    assert L.run_layer(dev, L.Mx4LayerBuffers(cfg, act=act)).shape == (0, 512)


@pytest.mark.parametrize("T,E,k,H,I", [(64, 256, 32, 1024, 256), (64, 256, 8, 8192, 128)])
def test_few_token_layer_at_its_limits(T, E, k, H, I):
    """The most tokens, experts and assignments, and the widest rows, against the separate calls bit for bit."""
    cfg = synth.LayerConfig("mx4", T=T, H=H, E=E, k=k, I=I, seed=100, w_std=0.06)
    dev = L.to_device(synth.make_inputs(cfg))
    L.convert_experts_mx4(dev)
    bufs = L.Mx4LayerBuffers(cfg)
    assert bufs.one_call
    y = L.run_layer(dev, bufs)
    ids, w = moe.moe_route(dev["x"], dev["w_router"], None, k)
    p = moe.moe_permute(ids, w, E, 0, E)
    want = moe.moe_grouped_ffn_mx4(*moe.moe_quantize_mx(dev["x"]), p["offsets"], p["row_token"], p["row_w"],
                                   p["token_row"], dev["wgu_mx4"], dev["wd_mx4"])
    assert torch.equal(ids, bufs.topk_ids) and torch.equal(w, bufs.topk_w) and torch.equal(y, want)
