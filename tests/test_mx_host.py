"""Host-side checks of the MXFP4 calls: symbols, and bad arguments refused before a GPU is touched."""
import ctypes
import os
import re

import pytest
import torch

import bit_quantized_moe_top_amd as mq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE, DEVICE = range(5)
N = None


def at(n):
    return ctypes.c_void_p(n)          # an address that is never dereferenced


A, B = at(1 << 20), at(1 << 30)


def test_header_and_binding_agree():
    text = open(os.path.join(ROOT, "include", "moeq_mx.h")).read()
    body = re.sub(r"/\*.*?\*/", "", text[text.index('extern "C" {'):], flags=re.S)
    names = re.findall(r"^\s*[a-z_0-9]+\s+([a-z_0-9]+)\s*\(", body, flags=re.M)
    assert set(names) == set(mq.MX_SYMBOLS) and len(names) == 6
    handle = ctypes.CDLL(mq.LIB_PATH)
    for n in names:
        assert hasattr(handle, n), n


def test_quant_and_dequant_refusals():
    f = mq.lib.quant_mxfp4
    assert f(A, 1, 4, 48, 48, B, B, N) == UNSUPPORTED            # K % 32
    assert f(A, 1, 4, 32, 36, B, B, N) == UNSUPPORTED            # ld % 8
    assert f(A, 1, 1 << 36, 32, 32, B, B, N) == UNSUPPORTED      # too many elements
    assert f(A, 1, 4, 32, 24, B, B, N) == INVALID                # ld < K
    assert f(A, 2, 4, 32, 32, B, B, N) == INVALID                # dtype
    assert f(A, 1, -1, 32, 32, B, B, N) == INVALID
    assert f(A, 1, 4, 0, 32, B, B, N) == INVALID
    assert f(N, 1, 4, 32, 32, B, B, N) == INVALID
    assert f(A, 1, 4, 32, 32, N, B, N) == INVALID
    assert f(A, 1, 4, 32, 32, B, N, N) == INVALID
    assert f(at((1 << 20) + 8), 1, 4, 32, 32, B, B, N) == INVALID
    assert f(A, 1, 4, 32, 32, at((1 << 30) + 4), B, N) == INVALID
    assert f(N, 1, 0, 32, 32, N, N, N) == OK
    g = mq.lib.dequant_mxfp4
    assert g(A, A, 4, 40, B, 1, N) == UNSUPPORTED
    assert g(A, A, 4, 32, B, 3, N) == INVALID
    assert g(N, A, 4, 32, B, 1, N) == INVALID
    assert g(A, A, 4, 32, at((1 << 30) + 8), 1, N) == INVALID
    assert g(N, N, 0, 32, N, 0, N) == OK


def test_tile_refusals():
    f = mq.lib.moe_tile_mxfp4_weights
    C, D = at(1 << 32), at(1 << 34)
    assert f(A, B, 24, 64, C, D, N) == UNSUPPORTED               # rows % 16
    assert f(A, B, 16, 48, C, D, N) == UNSUPPORTED               # K % 32
    assert f(A, B, 16, (1 << 20) + 32, C, D, N) == UNSUPPORTED   # K too long
    assert f(A, B, -16, 64, C, D, N) == INVALID
    assert f(N, B, 16, 64, C, D, N) == INVALID
    assert f(A, B, 16, 64, at((1 << 32) + 8), D, N) == INVALID
    assert f(A, B, 16, 64, at((1 << 20) + 256), D, N) == INVALID  # w over q
    assert f(A, B, 16, 64, C, at((1 << 32) + 2048), N) == INVALID  # ws over w
    assert f(A, B, 0, 64, C, D, N) == OK


def test_grouped_gemm_refusals():
    f = mq.lib.moe_grouped_gemm_mxfp4
    pb = mq.moe_plan_size(8, 32)
    ok = [A, A, 0, A, pb, 8, 32, A, A, 64, 96, 0, B, 1, N]

    def call(**kw):
        names = ("a_q", "a_s", "topk", "plan", "plan_bytes", "E", "R", "w", "ws", "N", "K", "epi",
                 "out", "dt", "stream")
        args = list(ok)
        for k, v in kw.items():
            args[names.index(k)] = v
        return f(*args)

    assert call(N=48) == UNSUPPORTED and call(K=40) == UNSUPPORTED
    assert call(K=(1 << 20) + 32) == UNSUPPORTED and call(E=1025) == UNSUPPORTED
    assert call(topk=9) == UNSUPPORTED
    assert call(topk=5) == INVALID                               # R % topk
    assert call(topk=-1) == INVALID and call(R=-1) == INVALID
    assert call(epi=2) == INVALID and call(dt=7) == INVALID
    assert call(epi=1, dt=0) == INVALID                          # the gated product is bf16
    for name in ("a_q", "a_s", "plan", "w", "ws", "out"):
        assert call(**{name: N}) == INVALID, name
    for name in ("a_q", "w", "ws", "out"):
        assert call(**{name: at((1 << 20) + 8)}) == INVALID, name
    assert call(a_s=at((1 << 20) + 2)) == INVALID and call(plan=at((1 << 20) + 2)) == INVALID
    assert call(plan_bytes=pb - 4) == WORKSPACE
    assert call(R=1 << 29, N=1 << 14, plan_bytes=1 << 40) == UNSUPPORTED   # too many workgroups
    assert call(R=0, a_q=N, w=N, out=N) == OK


def test_few_layer_refusals():
    size = mq.moe_layer_mxfp4_few_ws_size
    assert size(17, 2, 64, 64) == 0 and size(4, 9, 64, 64) == 0 and size(4, 2, 48, 64) == 0
    assert size(-1, 2, 64, 64) == 0 and size(4, 0, 64, 64) == 0 and size(4, 2, 64, 0) == 0
    need = size(4, 2, 64, 96)
    assert need >= 4 * 2 * (96 * 2 + 64 * 4)
    f = mq.lib.moe_layer_mxfp4_few
    names = ("logits", "bias", "T", "E", "k", "renorm", "x", "H", "w13", "ws13", "w2", "ws2", "I",
             "shared", "ids", "w", "y", "ws", "ws_bytes", "stream")
    ok = [A, N, 4, 8, 2, 1, A, 64, A, A, A, A, 96, N, B, B, B, B, need, N]

    def call(**kw):
        args = list(ok)
        for k, v in kw.items():
            args[names.index(k)] = v
        return f(*args)

    assert call(T=17) == UNSUPPORTED and call(k=9, E=16) == UNSUPPORTED
    assert call(H=80) == UNSUPPORTED and call(I=80) == UNSUPPORTED and call(E=2000) == UNSUPPORTED
    assert call(k=3, E=2) == INVALID and call(T=-1) == INVALID and call(E=0) == INVALID
    for name in ("logits", "x", "w13", "ws13", "w2", "ws2", "ids", "w", "y", "ws"):
        assert call(**{name: N}) == INVALID, name
    for name in ("x", "w13", "ws13", "w2", "ws2", "shared", "y", "ws"):
        assert call(**{name: at((1 << 20) + 8)}) == INVALID, name
    assert call(ws=at((1 << 20) + 128)) == INVALID               # 256-byte aligned
    assert call(ws_bytes=need - 1) == WORKSPACE
    assert call(T=0, logits=N, x=N, ws=N) == OK


@pytest.mark.parametrize("T,k,H,I", [(1, 1, 32, 32), (4, 2, 64, 96), (16, 8, 4096, 2048),
                                     (16, 8, 1 << 20, 1 << 20), (3, 5, 1440, 544)])
def test_few_layer_workspace_holds_every_part(T, k, H, I):
    """h as three bf16 values, o in fp32 and a counter per 32 columns, each part on 256 bytes."""
    R = T * k
    parts = (R * I * 6, R * H * 4, H // 32 * 4)
    assert mq.moe_layer_mxfp4_few_ws_size(T, k, H, I) == sum((n + 255) // 256 * 256 for n in parts)


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers")
def test_valid_calls_without_gpu_report_device_error():
    L = mq.lib
    assert L.quant_mxfp4(A, 1, 4, 32, 32, B, B, N) == DEVICE
    assert L.dequant_mxfp4(A, A, 4, 32, B, 1, N) == DEVICE
    assert L.moe_grouped_gemm_mxfp4(A, A, 0, A, mq.moe_plan_size(8, 32), 8, 32, A, A, 64, 96, 0, B,
                                    1, N) == DEVICE
    assert L.moe_layer_mxfp4_few(A, N, 4, 8, 2, 1, A, 64, A, A, A, A, 96, N, B, B, B, B,
                                 mq.moe_layer_mxfp4_few_ws_size(4, 2, 64, 96), N) == DEVICE


def test_python_binding_refusals():
    with pytest.raises(TypeError):
        mq.quant_mxfp4(torch.zeros(2, 32, dtype=torch.float16))
    with pytest.raises(ValueError):
        mq.quant_mxfp4(torch.zeros(2, 32))                        # host tensor
    u8 = torch.zeros(2, 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        mq.dequant_mxfp4(u8, torch.zeros(2, 1, dtype=torch.uint8))
    with pytest.raises(TypeError):
        mq.dequant_mxfp4(u8.int(), torch.zeros(2, 1, dtype=torch.uint8))
    with pytest.raises(ValueError):
        mq.tile_mxfp4_weights(u8, torch.zeros(2, 1, dtype=torch.uint8))
    with pytest.raises(TypeError):
        mq.moe_layer_mxfp4_few(torch.zeros(2, 8, dtype=torch.float64),
                               torch.zeros(2, 32, dtype=torch.bfloat16), u8, u8, u8, u8, 2)
