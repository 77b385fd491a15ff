"""The shared projection with adapters, without a GPU: the oracle's pins, symbols, and bad arguments
refused before a GPU is touched."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import bit_quantized_moe_top_amd as mq
from oracle import lora as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE, DEVICE = range(5)
N = None


def at(n):
    return ctypes.c_void_p(n)          # an address that is never dereferenced


A, W, LA, LB, SC, PL, OUT, WS = (at(1 << n) for n in range(24, 32))


# ---------------------------------------------------------------- the oracle
def test_oracle_by_hand():
    x = np.array([[1.0, 2.0], [1.0, 2.0], [1.0, 2.0]])
    w = np.array([[1.0, 0.0], [0.0, 1.0]])
    a = np.array([[[[1.0, 1.0]]], [[[1.0, -1.0]]]])          # two adapters of rank 1: u = 3, -1
    b = np.array([[[1.0], [0.0]], [[2.0], [5.0]]])
    v, mag = O.project(x, w, a, b, [2.0, 1.0], [1, -1, 0])
    np.testing.assert_array_equal(v, [[-1.0, -3.0], [1.0, 2.0], [7.0, 2.0]])
    np.testing.assert_array_equal(mag["shrink"], [[6.0, 15.0], [0, 0], [6.0, 0.0]])


def test_oracle_is_one_merged_weight_per_adapter():
    g = np.random.default_rng(1)
    x, w = g.standard_normal((7, 16)), g.standard_normal((32, 16))
    a, b = g.standard_normal((3, 2, 8, 16)), g.standard_normal((3, 32, 8))
    ids, scale = [2, 0, -1, 1, 3, 2, 0], [0.5, 2.0, -1.0]
    v, _ = O.project(x, w, a, b, scale, ids)
    for m, l in enumerate(ids):
        merged = w.copy()
        if 0 <= l < 3:
            merged[:16] += scale[l] * b[l, :16] @ a[l, 0]
            merged[16:] += scale[l] * b[l, 16:] @ a[l, 1]
        np.testing.assert_allclose(v[m], merged @ x[m], atol=1e-12)


def test_oracle_plan():
    p = O.adapter_plan([1, -1, 0, 7, 1, 2], 2)
    np.testing.assert_array_equal(p["sorted_rows"], [2, 0, 4, 1, 3, 5])
    np.testing.assert_array_equal(p["offsets"], [0, 1, 3, 6])


# ------------------------------------------------------------------- the ABI
def test_header_and_binding_agree():
    text = open(os.path.join(ROOT, "include", "moeq_lora.h")).read()
    body = re.sub(r"/\*.*?\*/", "", text[text.index('extern "C" {'):], flags=re.S)
    names = re.findall(r"^\s*[a-z_0-9]+\s+([a-z_0-9]+)\s*\(", body, flags=re.M)
    assert set(names) == set(mq.LORA_SYMBOLS) and len(names) == 3
    handle = ctypes.CDLL(mq.LIB_PATH)
    for n in names:
        assert hasattr(handle, n), n
    assert f"#define MOEQ_LORA_MAX_RANK {mq.LORA_MAX_RANK}" in text


def test_plan_refusals():
    f = mq.lib.moe_adapter_plan
    pb = mq.moe_plan_size(5, 100)
    assert f(A, 100, 4, PL, pb - 1, N) == WORKSPACE
    assert f(A, 100, 0, PL, pb, N) == INVALID
    assert f(A, -1, 4, PL, pb, N) == INVALID
    assert f(N, 100, 4, PL, pb, N) == INVALID
    assert f(A, 100, 4, N, pb, N) == INVALID
    assert f(at((1 << 24) + 2), 100, 4, PL, pb, N) == INVALID
    assert f(A, 100, 4, at((1 << 29) + 1), pb, N) == INVALID
    assert f(A, 100, 1024, PL, 1 << 40, N) == UNSUPPORTED
    assert f(A, 1 << 24, 4, PL, 1 << 40, N) == UNSUPPORTED


NAMES = ("a", "ld", "w", "M", "N", "K", "la", "lb", "scale", "L", "slices", "r", "plan", "pb", "epi",
         "out", "ws", "wb", "stream")


def call(**kw):
    args = [A, 64, W, 10, 96, 64, LA, LB, SC, 3, 1, 8, PL, mq.moe_plan_size(4, 10), 0, OUT, WS,
            mq.moe_shared_gemm_lora_ws_size(10, 96, 64, 3, 2, 8), N]
    for k, v in kw.items():
        args[NAMES.index(k)] = v
    return mq.lib.moe_shared_gemm_lora_bf16(*args)


def test_refusals():
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(L=0), dict(r=0), dict(slices=0),
                dict(slices=3), dict(epi=2), dict(ld=56), dict(a=N), dict(w=N), dict(la=N), dict(lb=N),
                dict(scale=N), dict(plan=N), dict(out=N), dict(ws=N), dict(a=at((1 << 24) + 8)),
                dict(w=at((1 << 25) + 2)), dict(la=at((1 << 26) + 4)), dict(lb=at((1 << 27) + 8)),
                dict(scale=at((1 << 28) + 2)), dict(out=at((1 << 30) + 8)), dict(ws=at((1 << 31) + 128)),
                dict(plan=at((1 << 29) + 2)),
                # outputs over inputs, and over each other
                dict(out=A), dict(out=at((1 << 25) + 96)), dict(out=LA), dict(out=LB), dict(out=SC),
                dict(out=PL), dict(ws=A), dict(ws=W), dict(ws=LA), dict(ws=LB), dict(ws=SC), dict(ws=PL),
                dict(out=WS)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(K=60, ld=64), dict(N=88), dict(N=48, epi=1), dict(N=48, slices=2), dict(r=12),
                dict(r=264), dict(L=1024), dict(M=1 << 24), dict(K=1 << 20, ld=1 << 20), dict(ld=68),
                dict(N=(1 << 20) + 32), dict(M=(1 << 24) - 1, N=1 << 20)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(pb=mq.moe_plan_size(4, 10) - 4) == WORKSPACE
    assert call(wb=mq.moe_shared_gemm_lora_ws_size(10, 96, 64, 3, 1, 8) - 1) == WORKSPACE
    assert call(M=0, a=N, out=N) == OK


def test_workspace_size():
    size = mq.moe_shared_gemm_lora_ws_size
    assert size(10, 96, 64, 3, 1, 8) > 0 and size(10, 96, 64, 3, 1, 8) % 256 == 0
    for bad in ((-1, 96, 64, 3, 1, 8), (10, 100, 64, 3, 1, 8), (10, 96, 60, 3, 1, 8),
                (10, 96, 64, 0, 1, 8), (10, 96, 64, 3, 4, 8), (10, 96, 64, 3, 1, 9)):
        assert size(*bad) == 0


def test_binding_refusals_without_a_gpu():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        mq.moe_shared_gemm_lora_bf16(x, w, x, x, x, x)
    with pytest.raises(TypeError, match="bfloat16"):
        mq.moe_shared_gemm_lora_bf16(x.float(), w, x, x, x, x)
    with pytest.raises(ValueError, match="device"):
        mq.moe_adapter_plan(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(TypeError, match="int32"):
        mq.moe_adapter_plan(torch.zeros(4, dtype=torch.int64), 2)


def test_sizes_past_32_bits_are_refused(monkeypatch):
    """Not cut down to their low 32 bits on the way into the library."""
    import bit_quantized_moe_top_amd.lora as lora
    size = mq.moe_shared_gemm_lora_ws_size
    good = [10, 96, 64, 3, 1, 8]
    assert size(*good) > 0
    for i in range(len(good)):
        for by in (2 ** 32, -2 ** 32):
            bad = list(good)
            bad[i] += by
            assert size(*bad) == 0, bad

    class OnDevice(torch.Tensor):
        def get_device(self):
            return 0

    calls = []
    monkeypatch.setattr(lora, "_launch", lambda *args: calls.append(args))
    monkeypatch.setattr(lora, "_output", lambda t, *args: torch.empty(0))
    none = torch.empty(0)                                        # (memory that nothing touches)
    bf = dict(dtype=torch.bfloat16)
    for L, S, r, n in ((1, 1, 2 ** 32 + 8, 0), (1, 2 ** 32 + 1, 8, 0), (2 ** 32 + 1, 1, 8, 0)):
        a, w = torch.empty(10, n, **bf), torch.empty(n, n, **bf)
        la, lb = torch.empty(L, S, r, n, **bf), torch.empty(L, n, r, **bf)
        sc, plan, ws = torch.empty(L), torch.empty(4, dtype=torch.int32), torch.empty(8, dtype=torch.uint8)
        args = [t.as_subclass(OnDevice) for t in (a, w, la, lb, sc, plan)]
        with pytest.raises(ValueError, match="past 32 bits"):
            mq.moe_shared_gemm_lora_bf16(*args, out=none, ws=ws.as_subclass(OnDevice))
    assert not calls
