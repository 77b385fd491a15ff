"""Binding of libmoeq's MXFP4 calls (include/moeq_mx.h): microscaled 4-bit floats.

E2M1 codes, two per byte with the low nibble first, and one E8M0 scale byte per 32
consecutive elements of a row; both are uint8 tensors here.  As in the rest of the
binding there is argument checking and allocation of missing outputs only; every
call runs on the current stream of its tensors' device.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import EPI_NONE, EPI_SILU_MUL, MAX_TOPK, MOEQ_BF16, MOEQ_F32, _check, _plan_shape_ok, lib

__all__ = ["MX_BLOCK", "FEW_TOKENS", "MX_SYMBOLS", "quant_mxfp4", "dequant_mxfp4",
           "tile_mxfp4_weights", "moe_grouped_gemm_mxfp4", "moe_layer_mxfp4_few",
           "moe_layer_mxfp4_few_ws_size"]

MX_BLOCK = 32                # elements per scale
FEW_TOKENS = 16              # MOEQ_FEW_TOKENS
_SUPER = 512                 # K of one super-group of the tiled order
_INT_MAX = 0x7FFFFFFF

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
_CALL = {}
for _name, (_res, _args) in _SIGNATURES.items():
    _CALL[_name] = getattr(lib, _name)
    _CALL[_name].restype, _CALL[_name].argtypes = _res, _args


_F = {torch.bfloat16: MOEQ_BF16, torch.float32: MOEQ_F32}
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _launch(name: str, index: int, *args):
    """Calls lib.name(*args, stream) on device `index` and its current stream.  (A decode step's
    calls take a few microseconds of GPU time, so this path creates no stream or pointer objects.)"""
    if index == _current_device():
        status = _CALL[name](*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = _CALL[name](*args, _raw_stream(index))
    if status:
        _check(name, status)


def _float_dtype(dtype, name: str) -> int:
    dt = _F.get(dtype)
    if dt is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")
    return dt


def _tensor(t: torch.Tensor, name: str, dtype, ndim: int = 0, index: int = -1) -> int:
    """Checks a contiguous device tensor (of ndim dims, on device `index`, if given); returns its
    device's index."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    i = t.get_device()
    if t.dtype is dtype and (t.dim() == ndim or not ndim) and t.is_contiguous() and i >= 0 and \
            (i == index or index < 0):
        return i
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if i < 0:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on device {i}, the call runs on device {index}")


def _output(t: Optional[torch.Tensor], name: str, shape: tuple, dtype, index: int) -> torch.Tensor:
    """The caller's tensor, checked against what the call writes, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", index))
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"device {index}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t


def _codes(q: torch.Tensor, scale: torch.Tensor, name: str, ndim: int = 0) -> Tuple[int, int]:
    """K and the device of MXFP4 rows: codes [..., K/2], scales [..., K/32]."""
    index = _tensor(q, name, torch.uint8, ndim)
    _tensor(scale, name + " scales", torch.uint8, ndim, index)
    qs, ss = q.shape, scale.shape
    n = len(qs)
    if (qs[0] != ss[0] or len(ss) != 2 or qs[1] != 16 * ss[1]) if n == 2 else \
            (not n or qs[:-1] != ss[:-1] or qs[-1] != 16 * ss[-1]):
        raise ValueError(f"{name}: codes [..., K/2] and scales [..., K/32] do not match: "
                         f"{tuple(qs)}, {tuple(ss)}")
    half = qs[n - 1]
    if half > _INT_MAX // 2:
        raise ValueError(f"{name}: rows of {2 * half} elements are too long")
    return 2 * half, index


def quant_mxfp4(x: torch.Tensor, q: Optional[torch.Tensor] = None,
                scale: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """x [..., K] fp32/bf16 -> (codes [..., K/2], scales [..., K/32]).  x is contiguous, or a
    2-D tensor whose rows are (columns of a wider matrix)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a tensor")
    dt = _float_dtype(x.dtype, "x")
    dev = x.get_device()
    if dev < 0:
        raise ValueError("x must be a device tensor")
    shape = x.shape
    if not shape:
        raise ValueError("x must have rows")
    K = shape[-1]
    if K > _INT_MAX:
        raise ValueError(f"x: rows of {K} elements are too long")
    if x.is_contiguous():
        ld = K
    elif len(shape) == 2 and x.stride(1) == 1 and x.stride(0) >= K:
        ld = x.stride(0)
    else:
        raise ValueError("x must be contiguous, or 2-D with contiguous rows")
    M = x.numel() // K if K else 0
    q = _output(q, "q", shape[:-1] + (K // 2,), torch.uint8, dev)
    scale = _output(scale, "scale", shape[:-1] + (K // MX_BLOCK,), torch.uint8, dev)
    _launch("quant_mxfp4", dev, x.data_ptr(), dt, M, K, ld, q.data_ptr(), scale.data_ptr())
    return q, scale


def dequant_mxfp4(q: torch.Tensor, scale: torch.Tensor, out: Optional[torch.Tensor] = None,
                  dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values [..., K] of MXFP4 rows, exact, in `dtype` (or out's)."""
    K, dev = _codes(q, scale, "q")
    dtype = dtype if out is None else out.dtype
    dt = _float_dtype(dtype, "out")
    out = _output(out, "out", q.shape[:-1] + (K,), dtype, dev)
    M = out.numel() // K if K else 0
    _launch("dequant_mxfp4", dev, q.data_ptr(), scale.data_ptr(), M, K, out.data_ptr(), dt)
    return out


def tile_mxfp4_weights(q: torch.Tensor, scale: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Weights [E, N, K] in rows (codes [E, N, K/2], scales [E, N, K/32]) -> the products'
    tiled order (codes [E, N/16, G, 4, 64, 16], scales [E, N/16, G, 64, 4], G = ceil(K / 512)).
    The shapes tell K only to whole super-groups of 512.  The codes' tensor remembers K, and a call
    with another one is refused; a copy of it (.to, .clone, a loaded checkpoint) does not, and a
    call with another K of as many super-groups then reads zeros for the rest."""
    K, dev = _codes(q, scale, "q", 3)
    E, N = q.shape[:2]
    if N % 16 != 0 or K == 0:
        raise ValueError("weights are [E, N, K] with N a multiple of 16")
    G = (K + _SUPER - 1) // _SUPER
    w = torch.empty(E, N // 16, G, 4, 64, 16, dtype=torch.uint8, device=q.device)
    ws = torch.empty(E, N // 16, G, 64, 4, dtype=torch.uint8, device=q.device)
    _launch("moe_tile_mxfp4_weights", dev, q.data_ptr(), scale.data_ptr(), E * N, K,
            w.data_ptr(), ws.data_ptr())
    w._moeq_k = K              # the shape alone tells K only to whole super-groups
    return w, ws


def _tiled(w: torch.Tensor, ws: torch.Tensor, K: int, name: str, dev: int) -> Tuple[int, int]:
    """(E, N) of tiled weights of K columns."""
    if not isinstance(w, torch.Tensor) or w.dim() != 6:
        raise ValueError(f"{name} must be in the tiled order [E, N/16, ceil(K/512), 4, 64, 16] "
                         "(tile_mxfp4_weights)")
    _tensor(w, name, torch.uint8, 6, dev)
    _tensor(ws, name + " scales", torch.uint8, 5, dev)
    E, nb, G, steps, lanes, piece = w.shape
    if (steps, lanes, piece) != (4, 64, 16) or G != (K + _SUPER - 1) // _SUPER or \
            ws.shape != (E, nb, G, 64, 4):
        raise ValueError(f"{name} does not hold tiled weights of K = {K} with their scales: "
                         f"{tuple(w.shape)}, {tuple(ws.shape)}")
    if getattr(w, "_moeq_k", K) != K:
        raise ValueError(f"{name} holds weights of K = {w._moeq_k}, the call has {K}")
    return E, 16 * nb


def moe_grouped_gemm_mxfp4(a_q: torch.Tensor, a_s: torch.Tensor, plan: torch.Tensor,
                           w: torch.Tensor, w_scale: torch.Tensor, epilogue: int = EPI_NONE,
                           topk: int = 0, out: Optional[torch.Tensor] = None,
                           out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Grouped GEMM with MXFP4 activations and (tiled) MXFP4 weights.  topk = 0: a holds the
    routed rows in plan order; topk = k: a holds the tokens and routed row r reads row r // k.
    Returns [R, N] (EPI_NONE) or [R, N/2] bf16 (EPI_SILU_MUL)."""
    K, dev = _codes(a_q, a_s, "a_q", 2)
    if not 0 <= topk <= MAX_TOPK:
        raise ValueError(f"topk must be 0 .. {MAX_TOPK}")
    E, N = _tiled(w, w_scale, K, "w", dev)
    R = a_q.shape[0] * (topk or 1)
    if R > _INT_MAX:
        raise ValueError(f"{R} rows are too many")
    _tensor(plan, "plan", torch.int32, 1, dev)
    _plan_shape_ok(plan, E, R)
    dtype = out_dtype if out is None else out.dtype
    dt = _float_dtype(dtype, "out")
    out = _output(out, "out", (R, N // 2 if epilogue == EPI_SILU_MUL else N), dtype, dev)
    _launch("moe_grouped_gemm_mxfp4", dev, a_q.data_ptr(), a_s.data_ptr(), topk,
            plan.data_ptr(), plan.numel() * 4, E, R, w.data_ptr(), w_scale.data_ptr(), N, K,
            epilogue, out.data_ptr(), dt)
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
    dev = _tensor(logits, "logits", torch.float32, 2)
    _tensor(x, "x", torch.bfloat16, 2, dev)
    T, H = x.shape
    E = logits.shape[1]
    if logits.shape[0] != T:
        raise ValueError(f"x has {T} rows, logits {logits.shape[0]}")
    E13, N13 = _tiled(w13, w13_scale, H, "w13", dev)
    I = N13 // 2
    E2, N2 = _tiled(w2, w2_scale, I, "w2", dev)
    if E13 != E or E2 != E or N2 != H:
        raise ValueError("w13 [E, 2I, H] and w2 [E, H, I] do not fit logits [T, E] and x [T, H]")
    if bias is not None:
        _tensor(bias, "bias", torch.float32, 1, dev)
        if bias.shape[0] != E:
            raise ValueError("bias must be [E]")
    if shared is not None:
        _tensor(shared, "shared", torch.bfloat16, 2, dev)
        if shared.shape != (T, H):
            raise ValueError("shared must be [T, H]")
    if T > FEW_TOKENS or not 1 <= k <= min(E, MAX_TOPK):
        raise ValueError(f"takes at most {FEW_TOKENS} tokens and 1 .. min(E, {MAX_TOPK}) experts "
                         f"per token, got T = {T}, k = {k}")
    o = dict(out) if out is not None else {}
    ids = o["ids"] = _output(o.get("ids"), "out['ids']", (T, k), torch.int32, dev)
    w = o["w"] = _output(o.get("w"), "out['w']", (T, k), torch.float32, dev)
    y = o["y"] = _output(o.get("y"), "out['y']", (T, H), torch.bfloat16, dev)
    ws = o.get("ws")
    if ws is None:
        ws = o["ws"] = torch.empty(lib.moe_layer_mxfp4_few_ws_size(T, k, H, I), dtype=torch.uint8,
                                   device=x.device)
    else:
        _tensor(ws, "out['ws']", torch.uint8, 1, dev)
    _launch("moe_layer_mxfp4_few", dev, logits.data_ptr(),
            None if bias is None else bias.data_ptr(), T, E, k, 1 if renormalize else 0,
            x.data_ptr(), H, w13.data_ptr(), w13_scale.data_ptr(), w2.data_ptr(),
            w2_scale.data_ptr(), I, None if shared is None else shared.data_ptr(), ids.data_ptr(),
            w.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel())
    return o
