"""CPU checks of train.py on another device than the current one: every library call is made with the tensors' device as the
current one, on that device's stream.  (The tensors are stand-ins, the library calls recorded.)"""
from contextlib import nullcontext
from types import SimpleNamespace

import pytest
import torch

from expert_routed_grouped_amd import moe, train

T, K, H, I, R = 4, 2, 64, 32, 8


class OnDevice:
    """A tensor's device and shape, as far as the host code looks at them."""
    is_cuda, device, dtype = True, torch.device("cuda", 1), torch.bfloat16

    def __init__(self, *shape):
        self.shape = shape


@pytest.fixture
def calls(monkeypatch):
    """(call, current device, stream) of every library call; the streams are 100 + their device."""
    current, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *exc):
            current.pop()

    def stream_of(device=None):
        return SimpleNamespace(cuda_stream=100 + (current[-1] if device is None else device.index))
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "current_stream", stream_of)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: nullcontext())
    monkeypatch.setattr(moe, "_new", lambda shape, dtype, device, stream: torch.zeros(shape, dtype=dtype))
    monkeypatch.setattr(moe, "_ptr", lambda t: None)

    def combine(*args):
        seen.append(("moe_combine", current[-1], args[-1].value))
        return 0
    monkeypatch.setattr(moe, "lib", lambda: SimpleNamespace(moe_combine=combine))
    results = dict(moe_grouped_mm=OnDevice(R, H), moe_swiglu=OnDevice(R, I), moe_grouped_wgrad=OnDevice(2, I, H),
                   moe_swiglu_backward=(OnDevice(R, 2 * I), OnDevice(R, I), torch.zeros(R)))
    for name, result in results.items():
        monkeypatch.setattr(moe, name, lambda *a, name=name, result=result, stream=None, **k: seen.append(
            (name, current[-1], 100 + current[-1] if stream is None else stream)) or result)
    yield seen
    assert current == [0]


def perm():
    return dict(offsets=None, row_token=torch.zeros(R, dtype=torch.int32), row_w=torch.zeros(R),
                token_row=torch.zeros((T, K), dtype=torch.int32), R_cap=R)


def test_experts_on_another_device(calls):
    x, w = OnDevice(T, H), OnDevice(2, 2 * I, H)
    _, saved = train.experts_forward(x, w, w, perm())
    assert [c[0] for c in calls] == ["moe_grouped_mm", "moe_swiglu", "moe_grouped_mm", "moe_combine"]
    train.experts_backward(saved, OnDevice(T, H), w, w)
    assert len(calls) == 9 and all(c[1:] == (1, 101) for c in calls), calls
