"""Binding of libmoeq's MXFP4 calls (include/moeq_mx.h): microscaled 4-bit floats.

E2M1 codes, two per byte with the low nibble first, and one E8M0 scale byte per 32
consecutive elements of a row; both are uint8 tensors here.  As in the rest of the
binding there is argument checking and allocation of missing outputs only; every
call runs on the current stream of its tensors' device.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

from . import (EPI_NONE, EPI_SILU_MUL, MAX_TOPK, MOEQ_BF16, MOEQ_F32, _check, _check_plan, _out,
               _ptr, _req, _stream, lib)

__all__ = ["MX_BLOCK", "FEW_TOKENS", "MX_SYMBOLS", "quant_mxfp4", "dequant_mxfp4",
           "tile_mxfp4_weights", "moe_grouped_gemm_mxfp4", "moe_layer_mxfp4_few",
           "moe_layer_mxfp4_few_ws_size"]

MX_BLOCK = 32                # elements per scale
FEW_TOKENS = 16              # MOEQ_FEW_TOKENS
_SUPER = 512                 # K of one super-group of the tiled order

_P, _I, _I64, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
# name -> (restype, argtypes); the exact list of entry points in include/moeq_mx.h
_SIGNATURES = {
    "quant_mxfp4": (_I, [_P, _I, _I64, _I, _I64, _P, _P, _P]),
    "dequant_mxfp4": (_I, [_P, _P, _I64, _I, _P, _I, _P]),
    "moe_tile_mxfp4_weights": (_I, [_P, _P, _I64, _I, _P, _P, _P]),
    "moe_grouped_gemm_mxfp4": (_I, [_P, _P, _I, _P, _SZ, _I, _I, _P, _P, _I, _I, _I, _P, _I, _P]),
    "moe_layer_mxfp4_few_ws_size": (_SZ, [_I, _I, _I, _I]),
    "moe_layer_mxfp4_few": (_I, [_P, _P, _I, _I, _I, _I, _P, _I, _P, _P, _P, _P, _I, _P, _P, _P,
                                 _P, _P, _SZ, _P]),
}
MX_SYMBOLS = tuple(_SIGNATURES)
for _name, (_res, _args) in _SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = _res, _args


def _on(device: torch.device):
    """Makes device the current one for the launch, if it is not."""
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _same_device(dev: torch.device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the call runs on {dev}")


def _float_dtype(dtype, name: str) -> int:
    if dtype == torch.bfloat16:
        return MOEQ_BF16
    if dtype == torch.float32:
        return MOEQ_F32
    raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")


def _checked_out(t: Optional[torch.Tensor], name: str, shape, dtype, dev) -> torch.Tensor:
    return _out({name: t}, name, tuple(shape), dtype, dev)


def _codes(q: torch.Tensor, scale: torch.Tensor, name: str) -> int:
    """K of MXFP4 rows: codes [..., K/2], scales [..., K/32]."""
    _req(q, name, torch.uint8)
    _req(scale, name + " scales", torch.uint8)
    if q.dim() < 1 or q.dim() != scale.dim() or q.shape[:-1] != scale.shape[:-1] or \
            q.shape[-1] != 16 * scale.shape[-1]:
        raise ValueError(f"{name}: codes [..., K/2] and scales [..., K/32] do not match: "
                         f"{tuple(q.shape)}, {tuple(scale.shape)}")
    _same_device(q.device, **{name + " scales": scale})
    return 2 * q.shape[-1]


def quant_mxfp4(x: torch.Tensor, q: Optional[torch.Tensor] = None,
                scale: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """x [..., K] fp32/bf16 -> (codes [..., K/2], scales [..., K/32]).  x is contiguous, or a
    2-D tensor whose rows are (columns of a wider matrix)."""
    dt = _float_dtype(x.dtype, "x")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    if x.dim() < 1:
        raise ValueError("x must have rows")
    K = x.shape[-1]
    if x.is_contiguous():
        ld = K
    elif x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= K:
        ld = x.stride(0)
    else:
        raise ValueError("x must be contiguous, or 2-D with contiguous rows")
    M = x.numel() // K if K else 0
    lead = tuple(x.shape[:-1])
    q = _checked_out(q, "q", lead + (K // 2,), torch.uint8, x.device)
    scale = _checked_out(scale, "scale", lead + (K // MX_BLOCK,), torch.uint8, x.device)
    with _on(x.device):
        _check("quant_mxfp4", lib.quant_mxfp4(_ptr(x), dt, M, K, ld, _ptr(q), _ptr(scale),
                                              _stream(x.device)))
    return q, scale


def dequant_mxfp4(q: torch.Tensor, scale: torch.Tensor, out: Optional[torch.Tensor] = None,
                  dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values [..., K] of MXFP4 rows, exact, in `dtype` (or out's)."""
    K = _codes(q, scale, "q")
    dtype = dtype if out is None else out.dtype
    dt = _float_dtype(dtype, "out")
    out = _checked_out(out, "out", tuple(q.shape[:-1]) + (K,), dtype, q.device)
    M = out.numel() // K if K else 0
    with _on(q.device):
        _check("dequant_mxfp4", lib.dequant_mxfp4(_ptr(q), _ptr(scale), M, K, _ptr(out), dt,
                                                  _stream(q.device)))
    return out


def tile_mxfp4_weights(q: torch.Tensor, scale: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Weights [E, N, K] in rows (codes [E, N, K/2], scales [E, N, K/32]) -> the products'
    tiled order (codes [E, N/16, G, 4, 64, 16], scales [E, N/16, G, 64, 4], G = ceil(K / 512))."""
    K = _codes(q, scale, "q")
    if q.dim() != 3 or q.shape[1] % 16 != 0 or K == 0:
        raise ValueError("weights are [E, N, K] with N a multiple of 16")
    E, N = q.shape[:2]
    G = (K + _SUPER - 1) // _SUPER
    w = torch.empty(E, N // 16, G, 4, 64, 16, dtype=torch.uint8, device=q.device)
    ws = torch.empty(E, N // 16, G, 64, 4, dtype=torch.uint8, device=q.device)
    with _on(q.device):
        _check("moe_tile_mxfp4_weights", lib.moe_tile_mxfp4_weights(
            _ptr(q), _ptr(scale), E * N, K, _ptr(w), _ptr(ws), _stream(q.device)))
    return w, ws


def _tiled(w: torch.Tensor, ws: torch.Tensor, K: int, name: str, dev) -> Tuple[int, int]:
    """(E, N) of tiled weights of K columns."""
    if not isinstance(w, torch.Tensor) or w.dim() != 6 or tuple(w.shape[3:]) != (4, 64, 16):
        raise ValueError(f"{name} must be in the tiled order [E, N/16, ceil(K/512), 4, 64, 16] "
                         "(tile_mxfp4_weights)")
    _req(w, name, torch.uint8)
    _req(ws, name + " scales", torch.uint8)
    E, nb, G = w.shape[:3]
    if G != (K + _SUPER - 1) // _SUPER or tuple(ws.shape) != (E, nb, G, 64, 4):
        raise ValueError(f"{name} does not hold weights of K = {K} with their scales: "
                         f"{tuple(w.shape)}, {tuple(ws.shape)}")
    _same_device(dev, **{name: w, name + " scales": ws})
    return E, 16 * nb


def moe_grouped_gemm_mxfp4(a_q: torch.Tensor, a_s: torch.Tensor, plan: torch.Tensor,
                           w: torch.Tensor, w_scale: torch.Tensor, epilogue: int = EPI_NONE,
                           topk: int = 0, out: Optional[torch.Tensor] = None,
                           out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Grouped GEMM with MXFP4 activations and (tiled) MXFP4 weights.  topk = 0: a holds the
    routed rows in plan order; topk = k: a holds the tokens and routed row r reads row r // k.
    Returns [R, N] (EPI_NONE) or [R, N/2] bf16 (EPI_SILU_MUL)."""
    K = _codes(a_q, a_s, "a_q")
    if a_q.dim() != 2:
        raise ValueError("a_q must have 2 dims")
    if not 0 <= topk <= MAX_TOPK:
        raise ValueError(f"topk must be 0 .. {MAX_TOPK}")
    dev = a_q.device
    E, N = _tiled(w, w_scale, K, "w", dev)
    R = a_q.shape[0] * max(topk, 1)
    _check_plan(plan, E, R)
    _same_device(dev, plan=plan)
    silu = epilogue == EPI_SILU_MUL
    dtype = out_dtype if out is None else out.dtype
    dt = _float_dtype(dtype, "out")
    out = _checked_out(out, "out", (R, N // 2 if silu else N), dtype, dev)
    with _on(dev):
        _check("moe_grouped_gemm_mxfp4", lib.moe_grouped_gemm_mxfp4(
            _ptr(a_q), _ptr(a_s), topk, _ptr(plan), plan.numel() * 4, E, R, _ptr(w),
            _ptr(w_scale), N, K, epilogue, _ptr(out), dt, _stream(dev)))
    return out


def moe_layer_mxfp4_few_ws_size(T: int, k: int, H: int, I: int) -> int:
    return lib.moe_layer_mxfp4_few_ws_size(T, k, H, I)


def moe_layer_mxfp4_few(logits: torch.Tensor, x: torch.Tensor, w13: torch.Tensor,
                        w13_scale: torch.Tensor, w2: torch.Tensor, w2_scale: torch.Tensor, k: int,
                        bias: Optional[torch.Tensor] = None, renormalize: bool = True,
                        shared: Optional[torch.Tensor] = None,
                        out: Optional[dict] = None) -> dict:
    """A whole layer for up to FEW_TOKENS tokens in two kernels: tiled MXFP4 weights, bf16
    activations.  Returns a dict with ids [T, k], w [T, k], y [T, H] and the workspace ws
    (reusing out's tensors; calls that may overlap need a ws of their own)."""
    _req(logits, "logits", torch.float32, 2)
    _req(x, "x", torch.bfloat16, 2)
    T, E = logits.shape
    H = x.shape[1]
    dev = x.device
    if x.shape[0] != T:
        raise ValueError(f"x has {x.shape[0]} rows, logits {T}")
    E13, N13 = _tiled(w13, w13_scale, H, "w13", dev)
    I = N13 // 2
    E2, N2 = _tiled(w2, w2_scale, I, "w2", dev)
    if E13 != E or E2 != E or N2 != H:
        raise ValueError("w13 [E, 2I, H] and w2 [E, H, I] do not fit logits [T, E] and x [T, H]")
    if bias is not None:
        _req(bias, "bias", torch.float32, 1)
        if bias.shape[0] != E:
            raise ValueError("bias must be [E]")
    if shared is not None:
        _req(shared, "shared", torch.bfloat16, 2)
        if tuple(shared.shape) != (T, H):
            raise ValueError("shared must be [T, H]")
    _same_device(dev, logits=logits, bias=bias, shared=shared)
    if T > FEW_TOKENS or not 1 <= k <= min(E, MAX_TOPK):
        raise ValueError(f"takes at most {FEW_TOKENS} tokens and 1 .. min(E, {MAX_TOPK}) experts "
                         f"per token, got T = {T}, k = {k}")
    nbytes = lib.moe_layer_mxfp4_few_ws_size(T, k, H, I)
    o = dict(out) if out is not None else {}
    _out(o, "ids", (T, k), torch.int32, dev)
    _out(o, "w", (T, k), torch.float32, dev)
    _out(o, "y", (T, H), torch.bfloat16, dev)
    ws = o.get("ws")
    if ws is None:
        ws = o["ws"] = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    else:
        _req(ws, "out['ws']", torch.uint8, 1)
        _same_device(dev, **{"out['ws']": ws})
    with _on(dev):
        _check("moe_layer_mxfp4_few", lib.moe_layer_mxfp4_few(
            _ptr(logits), _ptr(bias), T, E, k, 1 if renormalize else 0, _ptr(x), H, _ptr(w13),
            _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), I, _ptr(shared), _ptr(o["ids"]),
            _ptr(o["w"]), _ptr(o["y"]), _ptr(ws), ws.numel(), _stream(dev)))
    return o

