"""MXFP4 in float64: quantization, values, the tiled weight order, the grouped
product and the few-token layer (OCP Microscaling Formats specification 1.0:
E2M1 elements, one E8M0 scale per block of 32).  Pinned by tests/test_oracle_mx.py.
"""
from __future__ import annotations

import numpy as np

from . import layer as L
from .formats import e2m1_decode, pack_fp4, unpack_fp4

BLOCK = 32
STEP_LANES = 64
_MAGS = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def e2m1_encode(y) -> np.ndarray:
    """Nearest E2M1 code of each value, ties to the even code, saturating, sign kept."""
    y = np.asarray(y, dtype=np.float64)
    d = np.abs(np.abs(y)[..., None] - _MAGS)
    tied = d == d.min(axis=-1, keepdims=True)
    lo = tied.argmax(axis=-1)                              # the lowest code at least distance
    hi = 7 - tied[..., ::-1].argmax(axis=-1)
    code = np.where(lo % 2 == 0, lo, hi)
    return (code + 8 * np.signbit(y)).astype(np.uint8)


def quant_mxfp4(x):
    """x [..., K] -> (packed codes [..., K/2], scale bytes [..., K/32])."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[:-1] + (-1, BLOCK))
    bad = ~np.isfinite(b).all(axis=-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(axis=-1)
    _, ex = np.frexp(amax)                                 # amax = m 2^ex, m in [1/2, 1)
    s = np.where(amax > 0, np.maximum(ex - 1 - 2, -127), -127)
    codes = e2m1_encode(np.ldexp(b, -s[..., None]))
    codes = np.where(bad[..., None], 0, codes).reshape(x.shape)
    return pack_fp4(codes), np.where(bad, 255, s + 127).astype(np.uint8)


def values(q, scale) -> np.ndarray:
    """The values [..., K] that packed codes and scale bytes stand for (NaN for scale 255)."""
    v = e2m1_decode(unpack_fp4(q))
    s = np.asarray(scale, dtype=np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return (v.reshape(v.shape[:-1] + (-1, BLOCK)) * f[..., None]).reshape(v.shape)


def tile(q, scale):
    """Weights [rows, K] in rows -> the tiled order of moe_tile_mxfp4_weights, byte by byte."""
    q, scale = np.asarray(q), np.asarray(scale)
    rows, KB = scale.shape
    G = (KB + 15) // 16
    w = np.zeros((rows // 16, G, 4, STEP_LANES, 16), dtype=np.uint8)
    ws = np.full((rows // 16, G, STEP_LANES, 4), 127, dtype=np.uint8)
    for c in range(KB):
        g, kb, j = c // 16, c % 16 // 4, c % 4
        for r in range(16):
            w[:, g, j, 16 * kb + r] = q[r::16, 16 * c:16 * c + 16]
            ws[:, g, 16 * kb + r, j] = scale[r::16, c]
    return w, ws


def grouped_rows(a, experts, w):
    """a [R, K] values, experts [R], w [E, N, K] values -> (out [R, N], sum of magnitudes)."""
    out = np.zeros((a.shape[0], w.shape[1]))
    mag = np.zeros_like(out)
    for e in np.unique(experts):
        m = experts == e
        out[m] = a[m] @ w[e].T
        mag[m] = np.abs(a[m]) @ np.abs(w[e]).T
    return out, mag


def few_layer(logits, x, w13, w2, k, bias=None, renormalize=True, shared=None):
    """The few-token layer on weight values w13 [E, 2I, H], w2 [E, H, I], in float64 throughout
    (h unrounded)."""
    ids, wt = L.route_topk(logits, k, bias, renormalize)
    T, I = x.shape[0], w2.shape[2]
    y = np.zeros((T, w2.shape[1]))
    for t in range(T):
        for j in range(k):
            gu = w13[ids[t, j]] @ x[t]
            h = L.silu(gu[:I]) * gu[I:]
            y[t] += wt[t, j] * (w2[ids[t, j]] @ h)
    if shared is not None:
        y = y + shared
    return {"ids": ids, "w": wt, "y": y}
