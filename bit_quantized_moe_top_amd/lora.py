"""Binding of libmoeq's shared projection with low-rank adapters (include/moeq_lora.h).

As in the rest of the binding there is argument checking and allocation of missing outputs only;
every call runs on the current stream of its tensors' device.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import EPI_NONE, EPI_SILU_MUL, MAX_EXPERTS, _mark_plan, _plan_shape_ok, lib, moe_plan_size
from .mx import _CALL, _INT_MAX, _launch, _output, _tensor

__all__ = ["LORA_MAX_RANK", "MAX_ADAPTERS", "LORA_SYMBOLS", "moe_adapter_plan",
           "moe_shared_gemm_lora_bf16", "moe_shared_gemm_lora_ws_size"]

LORA_MAX_RANK = 256                  # MOEQ_LORA_MAX_RANK
MAX_ADAPTERS = MAX_EXPERTS - 1       # MOEQ_MAX_ADAPTERS

_P, _I, _I64, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
# name -> (restype, argtypes); the exact list of entry points in include/moeq_lora.h
_SIGNATURES = {
    "moe_adapter_plan": (_I, [_P, _I, _I, _P, _SZ, _P]),
    "moe_shared_gemm_lora_ws_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "moe_shared_gemm_lora_bf16": (_I, [_P, _I64, _P, _I, _I, _I, _P, _P, _P, _I, _I, _I, _P, _SZ,
                                       _I, _P, _P, _SZ, _P]),
}
LORA_SYMBOLS = tuple(_SIGNATURES)
for _name, (_res, _args) in _SIGNATURES.items():
    _CALL[_name] = getattr(lib, _name)
    _CALL[_name].restype, _CALL[_name].argtypes = _res, _args


def moe_adapter_plan(ids: torch.Tensor, n_adapters: int,
                     plan: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The rows of a batch grouped by adapter: ids [M] int32, those outside [0, n_adapters) have
    none.  One plan serves every projection of every layer that the batch passes through."""
    dev = _tensor(ids, "ids", torch.int32, 1)
    M = ids.shape[0]
    if not 1 <= n_adapters <= MAX_ADAPTERS:
        raise ValueError(f"takes 1 .. {MAX_ADAPTERS} adapters, got {n_adapters}")
    if M > _INT_MAX:
        raise ValueError(f"{M} rows are too many")
    if plan is None:
        plan = torch.empty((moe_plan_size(n_adapters + 1, M) + 3) // 4, dtype=torch.int32,
                           device=ids.device)
    else:
        _tensor(plan, "plan", torch.int32, 1, dev)
    _launch("moe_adapter_plan", dev, ids.data_ptr(), M, n_adapters, plan.data_ptr(),
            plan.numel() * 4)
    _mark_plan(plan, n_adapters + 1, M)
    return plan


def moe_shared_gemm_lora_ws_size(M: int, N: int, K: int, L: int, slices: int, r: int) -> int:
    if not 0 <= min(M, N, K, L, slices, r) <= max(M, N, K, L, slices, r) <= _INT_MAX:
        return 0                         # refused, as by the call itself
    return lib.moe_shared_gemm_lora_ws_size(M, N, K, L, slices, r)


def moe_shared_gemm_lora_bf16(a: torch.Tensor, w: torch.Tensor, lora_a: torch.Tensor,
                              lora_b: torch.Tensor, scale: torch.Tensor, plan: torch.Tensor,
                              epilogue: int = EPI_NONE, out: Optional[torch.Tensor] = None,
                              ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_shared_gemm_bf16 with each row's low-rank adapter: a [M, K] bf16 (rows may be columns of
    a wider matrix), w [N, K] bf16, lora_a [L, slices, r, K] bf16 (slices 1, or 2 where gate and up
    have an adapter input each), lora_b [L, N, r] bf16, scale [L] fp32, plan from moe_adapter_plan.
    Returns [M, N], or [M, N/2] with EPI_SILU_MUL.  ws: moe_shared_gemm_lora_ws_size bytes, one per
    call that may overlap with another."""
    if not isinstance(a, torch.Tensor):
        raise TypeError("a must be a tensor")
    if a.dtype is not torch.bfloat16:
        raise TypeError(f"a must be bfloat16, got {a.dtype}")
    dev = a.get_device()
    if dev < 0:
        raise ValueError("a must be a device tensor")
    if a.dim() != 2:
        raise ValueError(f"a must be [M, K], got {tuple(a.shape)}")
    _tensor(w, "w", torch.bfloat16, 2, dev)
    _tensor(lora_a, "lora_a", torch.bfloat16, 4, dev)
    _tensor(lora_b, "lora_b", torch.bfloat16, 3, dev)
    _tensor(scale, "scale", torch.float32, 1, dev)
    _tensor(plan, "plan", torch.int32, 1, dev)
    M, K = a.shape
    N = w.shape[0]
    L, slices, r = lora_a.shape[:3]
    if w.shape[1] != K or lora_a.shape[3] != K:
        raise ValueError(f"K mismatch: a has {K}, w {w.shape[1]}, lora_a {lora_a.shape[3]}")
    if lora_b.shape != (L, N, r) or scale.shape[0] != L:
        raise ValueError(f"lora_a [L, slices, r, K], lora_b [L, N, r] and scale [L] do not match: "
                         f"{tuple(lora_a.shape)}, {tuple(lora_b.shape)}, {tuple(scale.shape)}")
    if max(M, N, K, L, slices, r) > _INT_MAX:
        raise ValueError("sizes past 32 bits")
    ld = a.stride(0) if M > 1 else (K + 7) // 8 * 8
    if (K > 1 and a.stride(1) != 1) or ld < K:
        raise ValueError("a must have contiguous rows that do not overlap")
    _plan_shape_ok(plan, L + 1, M)
    out = _output(out, "out", (M, N // 2 if epilogue == EPI_SILU_MUL else N), torch.bfloat16, dev)
    if ws is None:
        ws = torch.empty(lib.moe_shared_gemm_lora_ws_size(M, N, K, L, slices, r), dtype=torch.uint8,
                         device=a.device)
    else:
        _tensor(ws, "ws", torch.uint8, 1, dev)
    _launch("moe_shared_gemm_lora_bf16", dev, a.data_ptr(), ld, w.data_ptr(), M, N, K,
            lora_a.data_ptr(), lora_b.data_ptr(), scale.data_ptr(), L, slices, r, plan.data_ptr(),
            plan.numel() * 4, epilogue, out.data_ptr(), ws.data_ptr(), ws.numel())
    return out
