"""GPU: gradients of a MoE block against central differences of the 64-bit block, along directions in which a missing or wrong
term shows: the gradient's own and random ones."""
import pytest
import torch

from expert_routed_grouped_amd import train
from expert_routed_grouped_amd.synth import LayerConfig
from test_gpu_train_block import DEV, F64, TOL, block, reference

pytestmark = pytest.mark.gpu
NAMES = ("dx", "w_gate_up", "w_down", "w_router", "bias", "norm_pre", "norm_post", "gate")


@pytest.mark.parametrize("gate", ["channel", "token"])
def test_backward_agrees_with_differences_of_64_bits(gate):
    cfg = LayerConfig("fd", T=12, H=64, E=4, k=4, I=32, act="f32", wdt="f32", seed=41, w_std=0.2)
    dev, x, d_out = block(cfg, gate=gate)
    _, saved = train.block_forward(dev, x)
    grads, ids = train.block_backward(dev, saved, d_out), saved["ids"]
    g = torch.Generator(device=DEV)
    g.manual_seed(5)

    def loss(name, t):
        d = dict(dev, **({} if name == "dx" else {name: t}))
        return float((reference(d, t if name == "dx" else x, d_out, ids)[0] * d_out.double()).sum())

    for name in NAMES:
        p = (x if name == "dx" else dev[name]).to(F64)
        grad = grads[name].to(F64)
        size = float(grad.norm())
        assert size > 1e-3, name
        for along in ("gradient", "random", "random"):
            v = grad if along == "gradient" else torch.randn(p.shape, device=DEV, generator=g, dtype=F64)
            v = v / v.norm()
            # The sum over the steps h and h / 2 that cancels the h^2 term: (4 D(h / 2) - D(h)) / 3 is off by h^4 times a fifth
            # derivative.  With a step of 1e-3 per value (root mean square) that is far below 1e-9 of the gradient; losses of
            # about 1e3 in 64 bits, rounded some thousand times, leave 1e-10 / h or less.
            h = 1e-3 * p.numel() ** 0.5
            diff = [(loss(name, p + s * v) - loss(name, p - s * v)) / (2 * s) for s in (h, h / 2)]
            num = (4 * diff[1] - diff[0]) / 3
            # fp32 gradients: as the block's test has it, relative in the 2-norm; projected on a unit vector the error is at most
            # that of the whole
            assert abs(num - float((grad * v).sum())) < 3 * TOL[torch.float32] * size, (name, along, num)


def test_what_is_added_to_and_what_is_of_one_call():
    """With an earlier call's dict the experts' gradients become sums in place, every other entry is this call's alone."""
    cfg = LayerConfig("acc", T=12, H=64, E=4, k=2, I=32, act="f32", wdt="f32", seed=42, w_std=0.2)
    dev, x, d_out = block(cfg)
    _, saved = train.block_forward(dev, x)
    first = train.block_backward(dev, saved, d_out)
    kept = {n: t.clone() for n, t in first.items()}
    second = train.block_backward(dev, saved, d_out, grads=first)
    for n in NAMES:
        if n in ("w_gate_up", "w_down"):
            assert second[n] is first[n] and torch.equal(second[n], 2 * kept[n])  # the same fp32 sums twice: exact
        else:
            assert second[n] is not first[n] and torch.equal(second[n], kept[n]) and torch.equal(first[n], kept[n])
