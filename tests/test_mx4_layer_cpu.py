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
