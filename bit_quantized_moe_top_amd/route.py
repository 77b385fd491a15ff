"""Binding of libmoeq's expert routing (include/moeq_route.h): softmax or sigmoid scores, a bias
that only the choice sees, groups of experts, renormalised weights.

As in the rest of the binding there is argument checking and allocation of missing outputs only;
every call runs on the current stream of its tensors' device.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import MAX_EXPERTS, MAX_TOPK, lib
from .mx import _CALL, _INT_MAX, _float_dtype, _launch, _output, _tensor

__all__ = ["SCORE_SOFTMAX", "SCORE_SIGMOID", "MAX_GROUPS", "ROUTE_SYMBOLS", "moe_route_experts"]

SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
MAX_GROUPS = 64                      # MOEQ_MAX_GROUPS

_P, _I, _I64, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
# name -> (restype, argtypes); the exact list of entry points in include/moeq_route.h
_SIGNATURES = {
    "moe_route_experts": (_I, [_P, _I, _I64, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P]),
}
ROUTE_SYMBOLS = tuple(_SIGNATURES)
for _name, (_res, _args) in _SIGNATURES.items():
    _CALL[_name] = getattr(lib, _name)
    _CALL[_name].restype, _CALL[_name].argtypes = _res, _args


def _check_options(E: int, k: int, scoring: int, n_group: int, topk_group: int, group_best: int,
                   scale: float) -> None:
    if scoring not in (SCORE_SOFTMAX, SCORE_SIGMOID):
        raise ValueError("scoring must be SCORE_SOFTMAX or SCORE_SIGMOID")
    if group_best not in (1, 2):
        raise ValueError("group_best must be 1 or 2")
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError(f"takes 1 .. {MAX_EXPERTS} experts, got {E}")
    if not 1 <= n_group <= MAX_GROUPS or E % n_group != 0 or not 1 <= topk_group <= n_group:
        raise ValueError(f"n_group (at most {MAX_GROUPS}) must divide the {E} experts and "
                         f"topk_group be 1 .. n_group, got {n_group}, {topk_group}")
    if not 1 <= k <= min(MAX_TOPK, topk_group * (E // n_group)):
        raise ValueError(f"k must be 1 .. {MAX_TOPK} and at most the experts of the groups that "
                         f"stay, got {k} of {topk_group * (E // n_group)}")
    if not math.isfinite(scale):
        raise ValueError("scale must be finite")


def moe_route_experts(logits: torch.Tensor, k: int, scoring: int = SCORE_SOFTMAX,
                      bias: Optional[torch.Tensor] = None, n_group: int = 1, topk_group: int = 1,
                      group_best: int = 1, renormalize: bool = True, scale: float = 1.0,
                      ids: Optional[torch.Tensor] = None,
                      weights: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """logits [T, E] fp32/bf16 (contiguous, or rows of a wider matrix), bias [E] fp32 ->
    (ids [T, k] int32, weights [T, k] fp32).  The k experts with the largest score + bias among the
    topk_group groups with the largest sum of their group_best best; weights are the scores, without
    the bias, over the chosen ones' sum if renormalize, times scale.  Logits of -inf mask experts."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a tensor")
    dt = _float_dtype(logits.dtype, "logits")
    dev = logits.get_device()
    if dev < 0:
        raise ValueError("logits must be a device tensor")
    if logits.dim() != 2:
        raise ValueError(f"logits must be [T, E], got {tuple(logits.shape)}")
    T, E = logits.shape
    if T > _INT_MAX:
        raise ValueError(f"{T} tokens are too many")
    ld = logits.stride(0) if T > 1 else E
    if (E > 1 and logits.stride(1) != 1) or ld < E:
        raise ValueError("logits must have contiguous rows that do not overlap")
    _check_options(E, k, scoring, n_group, topk_group, group_best, scale)
    if bias is not None:
        _tensor(bias, "bias", torch.float32, 1, dev)
        if bias.shape[0] != E:
            raise ValueError("bias must be [E]")
    ids = _output(ids, "ids", (T, k), torch.int32, dev)
    weights = _output(weights, "weights", (T, k), torch.float32, dev)
    _launch("moe_route_experts", dev, logits.data_ptr(), dt, ld,
            None if bias is None else bias.data_ptr(), T, E, k, scoring, n_group, topk_group,
            group_best, 1 if renormalize else 0, scale, ids.data_ptr(), weights.data_ptr())
    return ids, weights
