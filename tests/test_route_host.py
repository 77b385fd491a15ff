"""Expert routing without a GPU: the oracle's pins, symbols, and bad arguments refused before a GPU
is touched."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import bit_quantized_moe_top_amd as mq
from oracle import layer as L
from oracle import route as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE, DEVICE = range(5)
N = None
INF = float("inf")


def at(n):
    return ctypes.c_void_p(n)          # an address that is never dereferenced


A, B, C = at(1 << 20), at(1 << 30), at(1 << 32)


# ---------------------------------------------------------------- the oracle
def test_oracle_plain_softmax_is_the_layer_routing():
    z = np.random.default_rng(0).standard_normal((20, 24)).astype(np.float32)
    for renorm in (True, False):
        ids, w = R.route_experts(z, 5, R.SOFTMAX, renormalize=renorm)
        ref_ids, ref_w = L.route_topk(z, 5, None, renorm)
        np.testing.assert_array_equal(ids, ref_ids)
        np.testing.assert_allclose(w, ref_w, rtol=1e-12)


def test_oracle_by_hand():
    z = np.log([[1.0, 3.0, 4.0, 8.0], [1.0, 1.0, 1.0, 1.0]])         # scores 1/2, 3/4, 4/5, 8/9
    ids, w = R.route_experts(z, 2, R.SIGMOID, renormalize=False, scale=2.0)
    np.testing.assert_array_equal(ids, [[3, 2], [0, 1]])
    np.testing.assert_allclose(w, [[16 / 9, 8 / 5], [1, 1]])
    # the bias moves the choice, not the weights
    ids, w = R.route_experts(z[:1], 2, R.SIGMOID, bias=[1.0, 0, 0, 0], renormalize=False)
    np.testing.assert_array_equal(ids, [[0, 3]])
    np.testing.assert_allclose(w, [[1 / 2, 8 / 9]])
    # groups (0, 1) and (2, 3): best of one 8/9, sums 5/4 against 76/45; with a bias on expert 0
    ids, _ = R.route_experts(z[:1], 2, R.SIGMOID, n_group=2, topk_group=1, group_best=2)
    np.testing.assert_array_equal(ids, [[3, 2]])
    ids, w = R.route_experts(z[:1], 2, R.SIGMOID, bias=[1.0, 0, 0, 0], n_group=2, topk_group=1,
                             group_best=2)
    np.testing.assert_array_equal(ids, [[0, 1]])
    np.testing.assert_allclose(w, [[2 / 5, 3 / 5]])


def test_oracle_masks():
    z = np.array([[0.0, -INF, 1.0, -INF], [-INF] * 4])
    ids, w = R.route_experts(z, 3, R.SOFTMAX)
    np.testing.assert_array_equal(ids, [[2, 0, 1], [0, 1, 2]])
    assert w[0, 2] == 0 and abs(w[0].sum() - 1) < 1e-15 and (w[1] == 0).all()
    # an empty group stays after every group that has an expert
    ids, w = R.route_experts(np.array([[-INF, -INF, -9.0, -INF]]), 2, R.SIGMOID, bias=[0, 0, -5.0, 0],
                             n_group=2, topk_group=1, group_best=2)
    np.testing.assert_array_equal(ids, [[2, 0]])
    assert w[0].tolist() == [1.0, 0.0]


# ------------------------------------------------------------------- the ABI
def test_header_and_binding_agree():
    text = open(os.path.join(ROOT, "include", "moeq_route.h")).read()
    body = re.sub(r"/\*.*?\*/", "", text[text.index('extern "C" {'):], flags=re.S)
    names = re.findall(r"^\s*[a-z_0-9]+\s+([a-z_0-9]+)\s*\(", body, flags=re.M)
    assert names == list(mq.ROUTE_SYMBOLS) == ["moe_route_experts"]
    assert hasattr(ctypes.CDLL(mq.LIB_PATH), "moe_route_experts")


def test_refusals():
    names = ("logits", "dt", "ld", "bias", "T", "E", "k", "scoring", "n_group", "topk_group", "best",
             "renorm", "scale", "ids", "w", "stream")
    ok = [A, 0, 64, N, 4, 64, 6, 1, 8, 4, 2, 1, 1.0, B, C, N]

    def call(**kw):
        args = list(ok)
        for k, v in kw.items():
            args[names.index(k)] = v
        return mq.lib.moe_route_experts(*args)

    for bad in (dict(logits=N), dict(ids=N), dict(w=N), dict(T=-1), dict(E=0), dict(k=0),
                dict(dt=2), dict(dt=-1), dict(scoring=2), dict(scoring=-1), dict(best=0),
                dict(best=3), dict(n_group=0), dict(topk_group=0), dict(topk_group=9),
                dict(n_group=7), dict(ld=63), dict(ld=-64), dict(scale=INF), dict(scale=float("nan")),
                dict(logits=at((1 << 20) + 2)), dict(logits=at((1 << 20) + 1), dt=1),
                dict(bias=at((1 << 20) + 2)), dict(ids=at((1 << 30) + 2)), dict(w=at((1 << 32) + 1)),
                dict(E=8, topk_group=4, k=5)):                     # four groups of one expert
        assert call(**bad) == INVALID, bad
    for bad in (dict(E=1025, ld=2000, n_group=1, topk_group=1), dict(k=9), dict(T=1 << 26), dict(T=(1 << 26) - 1), dict(T=(1 << 25) + 1),
                dict(E=130, ld=130, n_group=65, topk_group=4), dict(ld=1 << 41)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(T=0, logits=N, ids=N, w=N) == OK


def test_binding_refusals_without_a_gpu():
    z = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="device tensor"):
        mq.moe_route_experts(z, 2)
    with pytest.raises(TypeError, match="tensor"):
        mq.moe_route_experts([1.0], 2)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        mq.moe_route_experts(z.half(), 2)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        mq.moe_route_experts(z.double(), 2)


def test_more_tokens_than_32_bits_are_refused(monkeypatch):
    """Not cut down to their low 32 bits on the way into the library."""
    import bit_quantized_moe_top_amd.route as route

    class OnDevice(torch.Tensor):
        def get_device(self):
            return 0

    calls = []
    monkeypatch.setattr(route, "_launch", lambda *args: calls.append(args))
    monkeypatch.setattr(route, "_output", lambda t, *args: torch.empty(0))
    T = 2 ** 32 + 5
    z = torch.empty(T, 1, dtype=torch.bfloat16).as_subclass(OnDevice)        # (memory that nothing touches)
    with pytest.raises(ValueError, match="too many"):
        mq.moe_route_experts(z, 1)
    assert not calls
