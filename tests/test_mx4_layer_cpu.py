"""CPU checks of layer.run_layer with MXFP4 experts: which calls it makes, with what, and on which stream.  The
library's calls are replaced by recorders."""
import pytest
import torch

from expert_routed_grouped_amd import layer as L
from expert_routed_grouped_amd import moe
from expert_routed_grouped_amd.synth import LayerConfig


class Recorder:
    """Replaces calls of the binding: notes (name, arguments, keywords), returns what ``result`` makes of them."""

    def __init__(self, monkeypatch):
        self.calls, self.patch = [], monkeypatch

    def replace(self, name, result=lambda *a, **k: None):
        def call(*a, **k):
            self.calls.append((name, a, k))
            return result(*a, **k)
        self.patch.setattr(moe, name, call)

    def named(self, name):
        return [(a, k) for n, a, k in self.calls if n == name]


@pytest.fixture
def rec(monkeypatch):
    r = Recorder(monkeypatch)
    for name in ("moe_route", "moe_permute", "moe_quantize_mx", "moe_decode_layer_mx4", "moe_grouped_ffn_mx4",
                 "moe_shared_expert"):
        r.replace(name)
    r.replace("moe_quantize_mx4", lambda w, *a, **k: (torch.zeros((w.shape[0], w.shape[1] // 2), dtype=torch.uint8),
                                                      torch.zeros((w.shape[0], w.shape[1] // 32), dtype=torch.uint8)))
    r.replace("moe_pack_mx4", lambda c, s, **k: (c, s))
    r.replace("moe_pack_weights", lambda w, **k: w.clone())
    r.replace("moe_pack_router", lambda w, **k: w.float().view(w.shape[0], -1, 4).transpose(0, 1).contiguous())
    return r


def model(T, I_s=0, act="mxfp8"):
    cfg = LayerConfig("mx4 cpu", T=T, H=128, E=4, k=2, I=128, I_s=I_s)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    dev = dict(cfg=cfg, x=bf(T, 128), w_router=bf(4, 128), bias=None, w_gate_up=bf(4, 256, 128), w_down=bf(4, 128, 128))
    if I_s:
        dev.update(ws_gate_up=bf(2 * I_s, 128), ws_down=bf(128, I_s))
    bufs = L.Mx4LayerBuffers(cfg, device="cpu", act=act, dtype=torch.float32 if I_s else torch.bfloat16)
    return dev, bufs


@pytest.mark.parametrize("T,act", [(4, "mxfp8"), (4, "mxfp4"), (70, "mxfp8")])
@pytest.mark.parametrize("pack", [False, True])
def test_shared_expert_is_told_of_packed_weights(rec, T, act, pack):
    """convert_experts_mx4, then pack_weights (which reorders the shared expert's weights in place of the originals),
    then run_layer: the shared expert has to know the layout it is given."""
    dev, bufs = model(T, I_s=64, act=act)
    L.convert_experts_mx4(dev)
    if pack:
        L.pack_weights(dev)
    L.run_layer(dev, bufs)
    (args, kw), = rec.named("moe_shared_expert")
    assert args[1] is dev["ws_gate_up"] and kw.get("packed", False) is pack


# ------------------------------------------------------------------ the packed router and streams
class FakeEvent:
    def __init__(self, log):
        self.log = log

    def record(self, stream):
        self.log.append(("record", stream.cuda_stream, self))


class FakeStream:
    def __init__(self, at, log):
        self.cuda_stream, self.log = at, log

    def wait_event(self, event):
        self.log.append(("wait", self.cuda_stream, event))


class FakePacked:
    """What moe_pack_router returns on a GPU, as far as the layer looks at it."""
    is_cuda = True

    def __init__(self, log):
        self.log = log

    def record_stream(self, stream):
        self.log.append(("keep", stream.cuda_stream, self))


@pytest.fixture
def streams(rec, monkeypatch):
    """(log, a function that makes streams); stream 0 is the current one.  Packing notes the stream it runs on."""
    log = []
    of = lambda n: FakeStream(n, log)  # noqa: E731
    current = of(0)
    monkeypatch.setattr(torch.cuda, "Event", lambda: FakeEvent(log))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    monkeypatch.setattr(L, "_capturing", lambda t: False)

    def pack(w, stream=None):
        log.append(("pack", 0 if stream is None else stream.cuda_stream, None))
        return FakePacked(log)
    monkeypatch.setattr(moe, "moe_pack_router", pack)
    return log, of


def old_model():
    """A decode batch of the layer with bf16 experts and a packed router weight."""
    cfg = LayerConfig("bf16 cpu", T=4, H=128, E=4, k=2, I=128)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    dev = dict(cfg=cfg, x=bf(4, 128), w_router=bf(4, 128), bias=None, w_gate_up=bf(4, 256, 128), w_down=bf(4, 128, 128))
    return L.pack_router(dev), L.LayerBuffers(cfg, device="cpu")


@pytest.fixture(params=["mx4", "bf16"])
def routed(request, rec, streams):
    """(log, streams, a layer with a packed router weight, its buffers, the router weights its calls got)."""
    rec.replace("moe_route_dispatch")
    rec.replace("moe_grouped_ffn")
    if request.param == "mx4":
        dev, bufs = model(4)
        L.convert_experts_mx4(dev)
        used = lambda: rec.named("moe_decode_layer_mx4")  # noqa: E731
    else:
        dev, bufs = old_model()
        used = lambda: rec.named("moe_route_dispatch")  # noqa: E731
    return (*streams, dev, bufs, used)


def test_router_is_repacked_on_the_stream_of_the_call(routed):
    log, stream, dev, bufs, used = routed
    s = stream(7)
    dev["w_router"].add_(1.0)
    del log[:]
    L.run_layer(dev, bufs, stream=s)
    assert [e[:2] for e in log if e[0] == "pack"] == [("pack", 7)]
    (args, kw), = used()
    assert args[1] is dev["w_router_packed"] and kw["stream"] is s


def test_router_packed_on_another_stream_is_waited_for_and_kept(routed):
    """Packed on stream 0 (or, after an edit, on stream 7): a call on another stream waits for that, and the memory
    is not handed out again before the call has read it; a call on the same stream needs neither."""
    log, stream, dev, bufs, used = routed
    a, b = stream(7), stream(9)
    for s, at in ((b, 0), (a, None)):
        del log[:]
        if at is None:
            dev["w_router"].add_(1.0)
            L.run_layer(dev, bufs, stream=a)
            del log[:]
            s = b
        packed = dev["w_router_packed"]
        L.run_layer(dev, bufs, stream=s)
        assert [e[:2] for e in log] == [("wait", 9), ("keep", 9)] and log[1][2] is packed
    del log[:]
    L.run_layer(dev, bufs, stream=a)
    assert log == []


def test_router_repacked_in_a_capture_stays_in_the_graph(routed, monkeypatch):
    """A graph that is being captured packs a stale router for itself: its copy is not written before the graph runs,
    so that calls outside must not take it for theirs."""
    log, stream, dev, bufs, used = routed
    before = dev["w_router_packed"]
    dev["w_router"].add_(1.0)
    monkeypatch.setattr(L, "_capturing", lambda t: True)
    del log[:]
    s = stream(7)
    L.run_layer(dev, bufs, stream=s)
    assert [e[:2] for e in log] == [("pack", 7)]
    assert used()[-1][0][1] is not before and dev["w_router_packed"] is before
    with pytest.raises(RuntimeError, match="captur"):
        L.pack_router(dev)
    monkeypatch.setattr(L, "_capturing", lambda t: False)
    del log[:]
    L.run_layer(dev, bufs, stream=s)
    assert ("pack", 7) in [e[:2] for e in log] and used()[-1][0][1] is dev["w_router_packed"] is not before
    # and a router that is up to date is used as it is, without an event from outside the capture
    monkeypatch.setattr(L, "_capturing", lambda t: True)
    del log[:]
    L.run_layer(dev, bufs, stream=stream(9))
    assert log == []


def test_router_replaced_at_the_same_address(rec):
    """A new weight may get the memory of the one it replaces, with the same version count: it is packed all the same."""
    import numpy as np
    memory = np.zeros((4, 128), dtype=np.float32)
    dev, bufs = model(4)
    dev["w_router"] = torch.from_numpy(memory)
    L.convert_experts_mx4(dev)
    first = dev["w_router_packed"]
    at = dev["w_router"].data_ptr()
    memory[:] = 1.0
    dev["w_router"] = torch.from_numpy(memory)
    assert dev["w_router"].data_ptr() == at and dev["w_router"]._version == 0
    L.run_layer(dev, bufs)
    (args, _), = rec.named("moe_decode_layer_mx4")
    assert args[1] is not first and bool((args[1] == 1).all())


def test_router_made_in_inference_mode(rec):
    """Weights loaded under torch.inference_mode have no version counter; replacing the tensor still shows."""
    dev, bufs = model(4)
    with torch.inference_mode():
        dev["w_router"] = torch.zeros((4, 128), dtype=torch.bfloat16)
    L.convert_experts_mx4(dev)
    first = dev["w_router_packed"]
    L.run_layer(dev, bufs)
    assert rec.named("moe_decode_layer_mx4")[0][0][1] is first
    with torch.inference_mode():
        dev["w_router"] = torch.ones((4, 128), dtype=torch.bfloat16)
    L.run_layer(dev, bufs)
    assert bool((rec.named("moe_decode_layer_mx4")[1][0][1] == 1).all())


def test_router_copy_of_a_graph_outlives_a_repack(rec, routed, monkeypatch):
    """A captured call holds the address of the packed copy: packing again must not free what the graph reads."""
    import weakref
    log, stream, dev, bufs, used = routed

    def edit_and_run():
        dev["w_router"].add_(1.0)
        L.run_layer(dev, bufs)
        del rec.calls[:], log[:]  # they hold the copies too

    copy = weakref.ref(dev["w_router_packed"])
    monkeypatch.setattr(L, "_capturing", lambda t: True)
    for _ in range(3):
        L.run_layer(dev, bufs)
    monkeypatch.setattr(L, "_capturing", lambda t: False)
    edit_and_run()
    assert copy() is not None and len(dev["w_router_packed_captured"]) == 1
    unread = weakref.ref(dev["w_router_packed"])  # no graph reads this one
    edit_and_run()
    assert unread() is None


# ------------------------------------------------------------------ another device than the current one
class OnDevice:
    """A tensor's device, as far as the layer looks at it."""
    is_cuda, device = True, torch.device("cuda", 1)

    def __init__(self, shape=(4, 128)):
        self.shape, self.dtype, self._version = shape, torch.bfloat16, 0

    def data_ptr(self):
        return id(self)

    def is_inference(self):
        return False

    def reshape(self, *shape):
        return OnDevice(shape)

    view = reshape


@pytest.mark.parametrize("T", [4, 70])
@pytest.mark.parametrize("mx4", [True, False])
def test_layer_on_another_device(monkeypatch, T, mx4):
    """Every call of the layer, and of the conversion before it, is made with the tensors' device as the current one."""
    current, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *exc):
            current.pop()
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(L, "_capturing", lambda t: False)
    for name in ("moe_route", "moe_permute", "moe_quantize_mx", "moe_decode_layer_mx4", "moe_grouped_ffn_mx4",
                 "moe_shared_expert", "moe_quantize_mx4", "moe_pack_mx4", "moe_pack_router", "moe_pack_weights",
                 "moe_route_dispatch", "moe_grouped_ffn", "moe_combine"):
        result = (OnDevice(), OnDevice()) if name == "moe_quantize_mx4" else None
        monkeypatch.setattr(moe, name, lambda *a, name=name, result=result, **k: seen.append((name, current[-1])) or result)
    dev, bufs = model(T, I_s=64)
    if not mx4:
        bufs = L.LayerBuffers(dev["cfg"], device="cpu", shared_beside_router=False)
    dev.update(x=OnDevice((T, 128)), w_router=OnDevice(), w_gate_up=OnDevice((4, 256, 128)), w_down=OnDevice((4, 128, 128)),
               ws_gate_up=OnDevice(), ws_down=OnDevice())
    if mx4:
        L.convert_experts_mx4(dev)
    else:
        L.pack_weights(dev)
    L.pack_router(dev)
    L.run_layer(dev, bufs)
    assert len(seen) >= 4 and all(at == 1 for _, at in seen), seen
    assert current == [0]


def test_a_layer_with_a_packed_router_can_be_copied(routed, monkeypatch):
    """copy.deepcopy and pickle of the layer's dict: events cannot be copied, and a copy's router is packed anew."""
    import copy
    log, stream, dev, bufs, used = routed

    def refuse(self, protocol):
        raise TypeError("cannot pickle 'Event' object")
    monkeypatch.setattr(FakeEvent, "__reduce_ex__", refuse)
    del log[:]
    other = copy.deepcopy({k: v for k, v in dev.items() if k != "w_router_packed"})
    other["w_router_packed"] = dev["w_router_packed"]  # the stand-in; a tensor would be copied with the rest
    L.run_layer(other, bufs, stream=stream(9))
    assert ("pack", 9) in [e[:2] for e in log] and used()[-1][0][1] is other["w_router_packed"]
    assert other["w_router_packed"] is not dev["w_router_packed"]


@pytest.mark.parametrize("T,act", [(4, "mxfp8"), (4, "mxfp4"), (70, "mxfp8"), (70, "mxfp4")])
@pytest.mark.parametrize("shape", ["more", "fewer", "wider"])
def test_batch_that_does_not_fit_the_buffers(rec, T, act, shape):
    """The routing and the codes of more tokens than the buffers hold would be written past them: refused before any call."""
    dev, bufs = model(T, act=act)
    L.convert_experts_mx4(dev)
    del rec.calls[:]
    dev["x"] = torch.zeros({"more": (T + 1, 128), "fewer": (T - 1, 128), "wider": (T, 256)}[shape], dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="buffers"):
        L.run_layer(dev, bufs)
    assert rec.calls == []


@pytest.mark.parametrize("shape", [(5, 128), (4, 256)])
def test_batch_that_does_not_fit_the_buffers_of_the_layer(rec, shape):
    rec.replace("moe_route_dispatch")
    rec.replace("moe_grouped_ffn")
    dev, bufs = old_model()
    del rec.calls[:]
    dev["x"] = torch.zeros(shape, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="buffers"):
        L.run_layer(dev, bufs)
    assert rec.calls == []
    dev["x"] = torch.zeros((3, 128), dtype=torch.bfloat16)  # fewer tokens than the buffers were made for
    L.run_layer(dev, bufs)
    assert rec.calls
