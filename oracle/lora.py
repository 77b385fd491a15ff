"""Float64 oracle of the shared projection with low-rank adapters."""
from __future__ import annotations

import numpy as np

from . import layer as L


def adapter_plan(ids, n):
    """permute_plan of the rows by adapter; ids outside [0, n) form the last group."""
    ids = np.asarray(ids).reshape(-1)
    return L.permute_plan(np.where((ids < 0) | (ids >= n), n, ids).reshape(-1, 1), n + 1)


def project(x, w, lora_a, lora_b, scale, ids):
    """(v [M, N], mag: a dict of the sums of magnitudes that error bounds need)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    lora_a, lora_b = np.asarray(lora_a, np.float64), np.asarray(lora_b, np.float64)
    M, N = x.shape[0], w.shape[0]
    n, S, r, _ = lora_a.shape
    v, base = x @ w.T, np.abs(x) @ np.abs(w).T
    u, um = np.zeros((M, S, r)), np.zeros((M, S, r))        # u, and |scale| |x| |A|
    d, dm, ds = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
    for m in range(M):
        l = int(ids[m])
        if not 0 <= l < n:
            continue
        f = float(scale[l])
        for s in range(S):
            cols = slice(s * (N // S), (s + 1) * (N // S))
            u[m, s] = f * (lora_a[l, s] @ x[m])
            um[m, s] = abs(f) * (np.abs(lora_a[l, s]) @ np.abs(x[m]))
            d[m, cols] = lora_b[l, cols] @ u[m, s]
            dm[m, cols] = np.abs(lora_b[l, cols]) @ np.abs(u[m, s])
            ds[m, cols] = np.abs(lora_b[l, cols]) @ um[m, s]
    return v + d, {"base": base, "v": np.abs(v), "delta": dm, "shrink": ds}


def silu_mul(v):
    half = v.shape[1] // 2
    return L.silu(v[:, :half]) * v[:, half:]
