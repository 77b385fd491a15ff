"""Pins of the MXFP4 oracle: hand-derived codes, brute force, round trips."""
import numpy as np
import pytest

from oracle import formats as F
from oracle import mx as X


def test_e2m1_encode_ties_and_saturation():
    # midpoints between neighbouring codes go to the even code
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for v, c in ties.items():
        assert X.e2m1_encode(v) == c and X.e2m1_encode(-v) == c + 8
        assert X.e2m1_encode(np.nextafter(v, 0)) <= c
        assert X.e2m1_encode(np.nextafter(v, 9)) >= c
    assert X.e2m1_encode(7.99) == 7 and X.e2m1_encode(-100.0) == 15
    assert X.e2m1_encode(0.0) == 0 and X.e2m1_encode(-0.0) == 8


def test_e2m1_encode_inverts_decode():
    codes = np.arange(16)
    np.testing.assert_array_equal(X.e2m1_encode(F.e2m1_decode(codes)), codes)


@pytest.mark.parametrize("power", [-130, -126, -3, 0, 20, 125])
def test_quant_block_by_hand(power):
    # a block with amax = 6 * 2^power: scale 2^power exactly while it is representable
    x = np.zeros(32)
    x[:8] = np.ldexp([6, -4, 3, 2, 1.5, 1, 0.5, -0.25], power)
    q, s = X.quant_mxfp4(x[None])
    if power >= -127:
        assert s[0, 0] == power + 127
        assert F.unpack_fp4(q)[0, :8].tolist() == [7, 14, 5, 4, 3, 2, 1, 8]
    else:
        assert s[0, 0] == 0                       # the smallest scale
    step = np.ldexp(1.0, int(s[0, 0]) - 127)
    assert np.abs(X.values(q, s)[0] - x).max() <= step       # half of the widest gap, 2


def test_quant_error_bound_and_scale_rule():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 96)) * np.ldexp(1.0, rng.integers(-20, 20, (40, 1)))
    q, s = X.quant_mxfp4(x)
    b = x.reshape(40, 3, 32)
    scale = np.ldexp(1.0, s.astype(int) - 127)
    ratio = np.abs(b).max(-1) / scale
    assert (ratio >= 4).all() and (ratio < 8).all()
    v = X.values(q, s).reshape(b.shape)
    # nearest of the 15 values, and 6 for what lies above it
    y = np.clip(b / scale[..., None], -6, 6)
    grid = np.unique(F.E2M1_VALUES)
    best = np.abs(y[..., None] - grid).min(-1)
    np.testing.assert_array_equal(np.abs(y - v / scale[..., None]), best)


def test_quant_marks_nonfinite_blocks():
    x = np.ones((1, 96))
    x[0, 40] = np.inf
    x[0, 95] = np.nan
    q, s = X.quant_mxfp4(x)
    assert s[0].tolist() == [125, 255, 255]
    assert (q[0, 16:] == 0).all()
    v = X.values(q, s)[0]
    assert (v[:32] == 1).all() and np.isnan(v[32:]).all()


@pytest.mark.parametrize("rows,K", [(16, 32), (32, 512), (48, 544), (16, 1440)])
def test_tile_is_a_permutation_with_zero_padding(rows, K):
    rng = np.random.default_rng(rows + K)
    q = rng.integers(0, 256, (rows, K // 2), dtype=np.uint8)
    s = rng.integers(0, 255, (rows, K // 32), dtype=np.uint8)
    w, ws = X.tile(q, s)
    G = -(-K // 512)
    assert w.shape == (rows // 16, G, 4, 64, 16) and ws.shape == (rows // 16, G, 64, 4)
    back = np.zeros((rows, G * 16, 16), dtype=np.uint8)
    sback = np.zeros((rows, G * 16), dtype=np.uint8)
    for r in range(rows):
        for c in range(G * 16):
            lane = 16 * (c % 16 // 4) + r % 16
            back[r, c] = w[r // 16, c // 16, c % 4, lane]
            sback[r, c] = ws[r // 16, c // 16, lane, c % 4]
    np.testing.assert_array_equal(back[:, :K // 32].reshape(rows, -1), q)
    np.testing.assert_array_equal(sback[:, :K // 32], s)
    assert (back[:, K // 32:] == 0).all() and (sback[:, K // 32:] == 127).all()


def test_few_layer_is_the_dense_sum():
    rng = np.random.default_rng(3)
    T, E, k, H, I = 3, 5, 2, 32, 64
    x, w13, w2 = rng.standard_normal((T, H)), rng.standard_normal((E, 2 * I, H)), \
        rng.standard_normal((E, H, I))
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[1, :] = -np.inf
    logits[2, 1:] = -np.inf
    out = X.few_layer(logits, x, w13, w2, k)
    for t in range(T):
        p = np.exp(logits[t].astype(float)) if t != 1 else np.zeros(E)
        best = sorted(range(E), key=lambda e: (-logits[t, e], e))[:k]
        p = p[best] / (p[best].sum() or 1.0)
        ref = np.zeros(H)
        for e, pe in zip(best, p):
            g, u = np.split(w13[e] @ x[t], 2)
            ref += pe * (w2[e] @ (g / (1 + np.exp(-g)) * u))
        np.testing.assert_allclose(out["y"][t], ref, rtol=1e-12, atol=1e-12)
    assert out["ids"][1].tolist() == [0, 1] and (out["w"][1] == 0).all()
