"""A layer's calls run with x's device current, whichever device the caller has current (no GPU)."""
import pytest
import torch

import bit_quantized_moe_top_amd as mq
from bit_quantized_moe_top_amd import layer as layer_module


class OnDevice:
    """Stands for x: a tensor of device `index`."""
    def __init__(self, index, T=4, H=64):
        self.index, self.shape, self.dtype = index, (T, H), torch.bfloat16

    def get_device(self):
        return self.index


@pytest.fixture
def current(monkeypatch):
    """[the current device], and the devices that were current at each library call."""
    state, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, state[0] = state[0], self.index

        def __exit__(self, *_):
            state[0] = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state[0])

    def call(name):
        def fn(*args, **kw):
            seen.append((name, state[0]))
            return {"y": None}
        return fn

    for name in dir(layer_module):
        if name.startswith(("moe_", "quant_")) and name != "moe_plan_size":
            monkeypatch.setattr(layer_module, name, call(name))
    return state, seen


@pytest.mark.parametrize("now", [0, 1])
@pytest.mark.parametrize("index", [0, 1])
def test_calls_run_on_the_device_of_x(current, now, index):
    state, seen = current
    state[0] = now
    x, logits = OnDevice(index), object()
    mx = mq.MxMoELayer(64, 32, 4, 2, device="cpu")
    for fn in (mq.MoELayer(64, 32, 4, 2, device="cpu").forward, mx.forward, mx.forward_few):
        fn(x, logits)
        assert seen and {d for _, d in seen} == {index}, seen
        assert state[0] == now
        seen.clear()


def test_a_failing_call_gives_the_device_back(current, monkeypatch):
    state, _ = current

    def fail(*args, **kw):
        raise mq.MoeqError("call", 1)
    monkeypatch.setattr(layer_module, "moe_route_topk", fail)
    with pytest.raises(mq.MoeqError):
        mq.MxMoELayer(64, 32, 4, 2, device="cpu").forward(OnDevice(1), object())
    assert state[0] == 0
