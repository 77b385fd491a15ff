"""The layers' buffers follow the shared experts that are set (no GPU)."""
import pytest
import torch

import bit_quantized_moe_top_amd as mq
from bit_quantized_moe_top_amd import layer as layer_module

H, I, E, K, T, L, R = 64, 32, 4, 2, 5, 3, 8
BF = torch.bfloat16


def make(kind):
    if kind == "hybrid":
        return mq.HybridMoELayer(H, I, E, K, device="cpu")
    if kind == "mxfp4":
        return mq.MxMoELayer(H, I, E, K, device="cpu")
    return mq.MoELayer(H, I, E, K, kind, device="cpu")


def shared(S):
    return torch.zeros(2 * S, H, dtype=BF), torch.zeros(H, S, dtype=BF)


def adapters(S, n=L):
    return (torch.zeros(n, 2, R, H, dtype=BF), torch.zeros(n, 2 * S, R, dtype=BF),
            torch.zeros(n, 1, R, S, dtype=BF), torch.zeros(n, H, R, dtype=BF), torch.ones(n))


class Host(torch.Tensor):
    """x as a device tensor to the layer."""
    def get_device(self):
        return 0


@pytest.fixture
def calls(monkeypatch):
    """The library's calls, by name and output, and none of them made."""
    seen = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def call(name):
        def fn(*args, out=None, **kw):
            seen.append((name, args, dict(kw, out=out)))
            return {"y": None} if name == "moe_layer_mxfp4_few" else out
        return fn

    for name in dir(layer_module):
        if name.startswith(("moe_", "quant_")) and not name.endswith("_size"):
            monkeypatch.setattr(layer_module, name, call(name))
    return seen


@pytest.mark.parametrize("kind", ["w4a8", "fp8row", "hybrid", "mxfp4"])
def test_buffers_follow_the_shared_experts_width(kind):
    layer = make(kind)
    plain = layer.buffers(T)
    assert "sh_h" not in plain and layer.buffers(T) is plain
    held = {}
    for S in (32, 96, 32):
        layer.set_shared(*shared(S))
        b = layer.buffers(T)
        assert b["sh_h"].shape == (T, S) and b["shared"].shape == (T, H)
        assert held.setdefault(S, b) is b                # (a captured graph may hold them)
    layer.set_shared(None, None)
    assert layer.buffers(T) is plain


@pytest.mark.parametrize("kind", ["w4a8", "fp8row"])
def test_shared_experts_and_adapters_set_after_a_call(kind, calls):
    layer = make(kind)
    x, logits, plan = torch.zeros(T, H, dtype=BF).as_subclass(Host), torch.zeros(T, E), object()
    layer.forward(x, logits)
    for S in (32, 96):
        layer.set_shared(*shared(S))
        layer.set_shared_adapters(*adapters(S))
        for p in (None, plan):
            calls.clear()
            layer.forward(x, logits, adapter_plan=p)
            name = "moe_shared_gemm_bf16" if p is None else "moe_shared_gemm_lora_bf16"
            assert [c[2]["out"].shape for c in calls if c[0] == name] == [(T, S), (T, H)]


@pytest.mark.parametrize("kind", ["w4a8", "fp8row", "hybrid", "mxfp4"])
def test_every_layer_adds_its_shared_experts(kind, calls):
    layer = make(kind)
    x, logits, plan = torch.zeros(T, H, dtype=BF).as_subclass(Host), torch.zeros(T, E), object()
    layer.set_shared(*shared(96))
    with pytest.raises(ValueError, match="set_shared_adapters"):
        layer.forward(x, logits, adapter_plan=plan)
    layer.set_shared_adapters(*adapters(96))
    for p in (None, plan):
        calls.clear()
        layer.forward(x, logits, adapter_plan=p)
        down = [c for c in calls if c[0].startswith("moe_shared_gemm")][-1]
        combine = [c for c in calls if c[0] == "moe_combine"]
        assert len(combine) == 1 and combine[0][1][3] is down[2]["out"]
        assert down[0] == ("moe_shared_gemm_bf16" if p is None else "moe_shared_gemm_lora_bf16")
    layer.set_shared(None, None)
    calls.clear()
    layer.forward(x, logits)
    assert [c[1][3] for c in calls if c[0] == "moe_combine"] == [None]


def test_adapter_workspaces_by_what_they_hold():
    """Loading more adapters of the same shapes starts no further workspace; one batch size and one
    width each have their own."""
    layer = make("w4a8")
    layer.set_shared(*shared(96))
    layer.set_shared_adapters(*adapters(96))
    ws = layer._lora_ws(T)
    for n in (1, 7, 200):
        layer.set_shared_adapters(*adapters(96, n))
        assert layer._lora_ws(T) is ws
    assert layer._lora_ws(T + 1) is not ws
    layer.set_shared(*shared(416))
    layer.set_shared_adapters(*adapters(416))
    wide = layer._lora_ws(T)
    for w, a in ((layer.ws13, layer.adapters[0]), (layer.ws2, layer.adapters[2])):
        assert wide.numel() >= mq.moe_shared_gemm_lora_ws_size(T, *w.shape, *a.shape[:3])
    assert wide.numel() > ws.numel()
    layer.set_shared(*shared(96))
    layer.set_shared_adapters(*adapters(96))
    assert all(mq.moe_shared_gemm_lora_ws_size(m, 4096, 2048, n, 2, 16) ==
               mq.moe_shared_gemm_lora_ws_size(m, 4096, 2048, 1, 2, 16)
               for m in (1, 40, 64, 65, 300, 1000, 5000) for n in (2, 30, 1000))
    assert layer._lora_ws(T) is ws                       # (a captured graph may hold it)
