"""CPU checks of train.py: what it refuses, before anything reaches the library."""
import pytest
import torch

from expert_routed_grouped_amd import train
from expert_routed_grouped_amd.synth import LayerConfig

GOOD = LayerConfig("t", T=4, H=64, E=4, k=2, I=32)


def dev(cfg, **kw):
    return dict({"cfg": cfg, "norm_pre": torch.ones(cfg.H), "bias": None}, **kw)


@pytest.mark.parametrize("d,match", [
    (dev(GOOD, packed=True), "row-major"), (dev(GOOD.replace(wdt="fp8")), "row-major"), (dev(GOOD.replace(act="f32")), "row-major"),
    (dev(GOOD.replace(I_s=32)), "shared expert"), (dev(GOOD.replace(e_end=2)), "all of its experts"),
])
def test_blocks_that_cannot_be_trained(d, match):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=match):
        train.block_forward(d, x)
    with pytest.raises(ValueError, match=match):
        train.block_backward(d, {"x": x}, x)


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="on the GPU"):
        train.block_forward(dev(GOOD), torch.zeros((4, 64), dtype=torch.bfloat16))
