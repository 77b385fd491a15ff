"""Expert routing on the GPU against the float64 oracle.

Ids are equal, whatever the scores.  Weights, with u = 2^-24: exp is within 2 ulp (4 u) of its
argument's, the argument l - max off by u of itself, which is u (max l - l) of the value; sum,
quotient and scale add a few u, the sum of at most 8 chosen 7 u.  Where the softmax denominator
counts (no renormalization): terms by the hardware's 2^x, (2.5 |x| + 2) u each with |x| <= 7 on
average for 1024 experts, and at most 38 rounded additions: 60 u.  So a relative
(80 + 2 (max l - min l)) u, and one smallest normal number where exp's result is flushed.
"""
import numpy as np
import pytest
import torch

import bit_quantized_moe_top_amd as mq
from oracle import route as R
from parity import to_np

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
INF = float("inf")
SOFT, SIGM = mq.SCORE_SOFTMAX, mq.SCORE_SIGMOID


def gen(seed):
    return torch.Generator().manual_seed(seed)


def check(logits, bias, k, **kw):
    """logits and bias on the host, in the type of the call."""
    ids, w = mq.moe_route_experts(logits.to(DEV), k, bias=None if bias is None else bias.to(DEV), **kw)
    z = to_np(logits).astype(np.float64)
    rid, rw = R.route_experts(z, k, bias=None if bias is None else bias.numpy(), **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    fin = np.where(np.isfinite(z), z, np.nan)
    with np.errstate(all="ignore"):
        spread = np.nan_to_num(np.nanmax(fin, 1) - np.nanmin(fin, 1))[:, None] if z.size else 0
    tol = (80 + 2 * spread) * U * np.abs(rw) + 2.0 ** -126 * max(1.0, abs(kw.get("scale", 1.0)))
    err = np.abs(w.cpu().numpy().astype(np.float64) - rw)
    assert (err <= tol).all(), (err / np.maximum(np.abs(rw), 1e-300)).max()
    return ids, w


# T, E, k, G, topk_group: one expert; one token; sizes off every power of two; groups of one
# expert; as many groups as there may be; groups that lie on 1 .. 32 lanes, with up to 31 experts a
# lane; every group stays; the most experts
SHAPES = [
    (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (3, 2, 2, 2, 2), (5, 7, 3, 7, 3), (4, 64, 8, 64, 8),
    (17, 65, 8, 1, 1), (6, 160, 6, 8, 3), (9, 150, 5, 5, 3), (33, 384, 8, 6, 2), (7, 1023, 8, 33, 4),
    (8, 1024, 8, 1, 1), (5, 1024, 8, 16, 5), (6, 999, 7, 3, 1), (5, 1022, 8, 2, 1), (64, 96, 4, 12, 4),
    (4, 992, 8, 32, 7), (130, 256, 8, 8, 4), (66, 40, 8, 10, 10), (5, 600, 1, 24, 1),
]


@pytest.mark.parametrize("T,E,k,G,tg", SHAPES)
@pytest.mark.parametrize("scoring", [SOFT, SIGM])
@pytest.mark.parametrize("biased,best", [(False, 1), (False, 2), (True, 1), (True, 2)])
def test_shapes(T, E, k, G, tg, scoring, biased, best):
    g = gen(T * E + k)
    logits = torch.randn(T, E, generator=g) * 1.5
    bias = torch.randn(E, generator=g) * (0.2 if scoring == SIGM else 2.0 / E) if biased else None
    for renorm, scale, dt in ((True, 1.0, torch.float32), (False, 2.5, torch.bfloat16),
                              (True, 0.5, torch.bfloat16)):
        check(logits.to(dt), bias, k, scoring=scoring, n_group=G, topk_group=tg, group_best=best,
              renormalize=renorm, scale=scale)


@pytest.mark.parametrize("E,G,tg", [(64, 1, 1), (256, 8, 4), (150, 5, 2), (1024, 32, 9)])
@pytest.mark.parametrize("scoring", [SOFT, SIGM])
def test_scores_too_close_for_fp32(E, G, tg, scoring):
    """Biases that bring every expert's s + b within a few 1e-8 of one number: fp32 sums tie or come
    out in the wrong order, the order of the real numbers decides."""
    g = gen(E + G)
    T = 24
    row = torch.randn(1, E, generator=g)
    s = R.scores(row.numpy(), scoring)[0]
    bias = torch.from_numpy((0.75 - s).astype(np.float32))
    logits = row.repeat(T, 1)
    c = s + bias.double().numpy()
    c32 = (torch.from_numpy(s).float() + bias).numpy()
    assert not np.array_equal(np.argsort(-c, kind="stable"), np.argsort(-c32, kind="stable"))
    logits[1::2] += torch.randn(T // 2, E, generator=g) * 1e-7       # rows of their own
    for k in (1, 6, 8):
        for best in (1, 2):
            check(logits, bias, k, scoring=scoring, n_group=G, topk_group=tg, group_best=best)


def test_groups_too_close_for_fp32():
    """Without a bias experts are ordered by logits, but sums of two scores decide the groups."""
    g = gen(5)
    E, G = 64, 8
    z = torch.full((16, E), -4.0)
    for t in range(16):
        for i in range(G):
            a = 0.5 + 0.03 * float(torch.rand((), generator=g))
            b = 1.25 - a                                             # scores a + b = 5/4, nearly
            z[t, 8 * i], z[t, 8 * i + 3] = np.log(a / (1 - a)), np.log(b / (1 - b))
    value = R.scores(z.numpy(), SIGM).reshape(16, G, 8)
    value = np.sort(value, axis=2)[:, :, -2:].sum(2)
    assert (np.ptp(value, axis=1) < 3e-7).all()
    for tg in (1, 3, 7):
        check(z, None, 2, scoring=SIGM, n_group=G, topk_group=tg, group_best=2)


@pytest.mark.parametrize("scoring", [SOFT, SIGM])
@pytest.mark.parametrize("biased", [False, True])
def test_ties_go_to_the_lower_index(scoring, biased):
    g = gen(7)
    logits = (torch.randn(40, 256, generator=g) * 2).round() / 2
    logits[0] = 1.0                                                  # all equal
    logits[1] = torch.finfo(torch.float32).min                       # the lowest value masks nothing
    bias = (torch.randn(256, generator=g) * 2).round() / 16 if biased else None
    for G, tg in ((1, 1), (8, 3)):
        for best in (1, 2):
            ids, _ = check(logits, bias, 8, scoring=scoring, n_group=G, topk_group=tg, group_best=best)
    if not biased:
        assert ids[0].tolist() == list(range(8))


@pytest.mark.parametrize("scoring", [SOFT, SIGM])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_experts_groups_and_tokens(scoring, biased, dtype):
    g = gen(9)
    E, k = 60, 6
    logits = torch.randn(12, E, generator=g)
    logits[0] = -INF                                                 # no expert left
    logits[1, 1:] = -INF                                             # one
    logits[2, :30] = -INF                                            # whole groups empty
    logits[3, torch.arange(E) % 10 != 7] = -INF                      # one expert in each group
    logits[4, 12:] = -INF
    logits[5:9][torch.rand(4, E, generator=g) < 0.8] = -INF
    bias = torch.randn(E, generator=g) - 3 if biased else None       # negative sums
    if biased:
        bias[4] = -INF                                               # the bias masks too
    for G, tg in ((1, 1), (6, 2), (6, 4), (30, 5)):
        for best in (1, 2):
            for renorm in (True, False):
                ids, w = check(logits.to(dtype), bias, k, scoring=scoring, n_group=G, topk_group=tg,
                               group_best=best, renormalize=renorm)
                assert ids[0].tolist() == list(range(k)) and (w[0] == 0).all()


def test_far_logits():
    """Scores that underflow, or are 1 in fp32: order and ratios are those of the logits."""
    z = torch.tensor([[-300.0, -301.0, -305.0, -400.0], [90.0, 95.0, 99.0, 80.0],
                      [-2.0, 300.0, 10.0, -1000.0]])
    ids, w = mq.moe_route_experts(z.to(DEV), 3, scoring=SIGM)
    assert ids.tolist() == [[0, 1, 2], [2, 1, 0], [1, 2, 0]]
    e = torch.exp(torch.tensor([0.0, -1.0, -5.0]))
    assert torch.allclose(w[0].cpu(), e / e.sum(), rtol=1e-6)
    assert torch.allclose(w[1].cpu(), torch.full((3,), 1 / 3), rtol=1e-6)
    check(z, None, 3, scoring=SOFT)
    check(z, torch.tensor([5.0, 0, 0, 9.0]), 2, scoring=SOFT)        # chosen though their scores are 0


@pytest.mark.parametrize("bits", [0x7FC00000, -1, 0x7F800000])       # NaNs of either sign, +inf
@pytest.mark.parametrize("biased", [False, True])
def test_nonfinite_scores_stay_inside_and_to_their_token(bits, biased):
    g = gen(11)
    logits = torch.randn(9, 48, generator=g)
    bias = (torch.randn(48, generator=g) * .1).to(DEV) if biased else None
    bad = torch.tensor(bits, dtype=torch.int32).view(torch.float32)
    for kw in (dict(), dict(n_group=6, topk_group=2, group_best=2), dict(n_group=6, topk_group=2)):
        for scoring in (SOFT, SIGM):
            clean = mq.moe_route_experts(logits.to(DEV), 5, scoring=scoring, bias=bias, **kw)
            z = logits.clone()
            z[2], z[5, 17] = bad, bad
            ids, w = mq.moe_route_experts(z.to(DEV), 5, scoring=scoring, bias=bias, **kw)
            assert ((ids >= 0) & (ids < 48)).all()
            assert all(len(set(r)) == 5 for r in ids.tolist())
            keep = [0, 1, 3, 4, 6, 7, 8]
            assert torch.equal(ids[keep], clean[0][keep]) and torch.equal(w[keep], clean[1][keep])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,pad", [(256, 1), (150, 10), (33, 3), (1024, 8)])
def test_rows_of_a_wider_matrix_and_caller_outputs(E, pad, dtype):
    T, k = 21, 7
    wide = torch.randn(T, E + pad, generator=gen(E)).to(dtype).to(DEV)
    wide[:, E:] = INF                                                # must not be read as scores
    ids = torch.full((T + 2, k), 77, dtype=torch.int32, device=DEV)
    w = torch.full((T + 2, k), 77.0, device=DEV)
    for kw in (dict(scoring=SIGM), dict(scoring=SOFT, renormalize=False)):
        got = mq.moe_route_experts(wide[:, :E], k, ids=ids[1:T + 1], weights=w[1:T + 1], **kw)
        ref = mq.moe_route_experts(wide[:, :E].contiguous(), k, **kw)
        assert got[0].data_ptr() == ids[1:].data_ptr()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        for t in (ids, w):
            assert (t[0] == 77).all() and (t[T + 1] == 77).all()


def test_plain_softmax_equals_the_layers_routing():
    logits = torch.randn(300, 256, generator=gen(3)).to(DEV)
    for renorm in (True, False):
        a = mq.moe_route_experts(logits, 6, renormalize=renorm)
        b = mq.moe_route_topk(logits, 6, renormalize=renorm)
        assert torch.equal(a[0], b[0])
        assert torch.allclose(a[1], b[1], rtol=128 * U, atol=0)


def test_no_tokens_and_refusals():
    z = torch.randn(4, 64, generator=gen(1)).to(DEV)
    ids, w = mq.moe_route_experts(z[:0], 3)
    assert ids.shape == w.shape == (0, 3)
    for kw in (dict(k=0), dict(k=9), dict(k=2, n_group=7), dict(k=2, n_group=8, topk_group=9),
               dict(k=5, n_group=16, topk_group=1), dict(k=2, group_best=3), dict(k=2, scoring=5),
               dict(k=2, scale=INF), dict(k=2, bias=torch.zeros(63, device=DEV)),
               dict(k=2, bias=torch.zeros(64)),
               dict(k=2, ids=torch.zeros(4, 3, dtype=torch.int32, device=DEV)),
               dict(k=2, weights=torch.zeros(4, 2, dtype=torch.bfloat16, device=DEV))):
        with pytest.raises(ValueError):
            mq.moe_route_experts(z, **kw)
    with pytest.raises(TypeError):
        mq.moe_route_experts(z, 2, bias=torch.zeros(64, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        mq.moe_route_experts(z.t(), 2)
    with pytest.raises(ValueError):
        mq.moe_route_experts(z[0].expand(4, 64), 2)                  # rows that overlap
    with pytest.raises(ValueError):
        mq.moe_route_experts(z[0], 2)


def test_captured_and_replayed_and_on_another_stream():
    g = gen(13)
    z = torch.randn(50, 256, generator=g).to(DEV)
    bias = (torch.randn(256, generator=g) * .1).to(DEV)
    kw = dict(scoring=SIGM, bias=bias, n_group=8, topk_group=4, group_best=2, scale=2.5)
    mq.moe_route_experts(z, 8, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, w = mq.moe_route_experts(z, 8, **kw)
    side = torch.cuda.Stream()
    for _ in range(4):
        z.copy_(torch.randn(50, 256, generator=g))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            ref = mq.moe_route_experts(z, 8, **kw)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, ref[0]) and torch.equal(w, ref[1])


def check_many(rows, bias, k, **kw):
    """The rows again and again up to a call of many tokens: each time what the oracle says of them,
    to the bit the same wherever in the call they stand."""
    n = rows.shape[0]
    T = 8195 + n                                                     # no multiple of a wave's tokens
    times = -(-T // n)
    logits = rows.repeat(times, 1)[:T]
    ids, w = mq.moe_route_experts(logits.to(DEV), k, bias=None if bias is None else bias.to(DEV), **kw)
    ids, w = ids.cpu(), w.cpu()
    again = torch.arange(T) % n
    assert torch.equal(ids, ids[:n][again]) and torch.equal(w, w[:n][again])
    small = check(rows, bias, k, **kw)                               # (both against the oracle)
    assert torch.equal(small[0].cpu(), ids[:n])
    z = to_np(rows).astype(np.float64)
    _, rw = R.route_experts(z, k, bias=None if bias is None else bias.numpy(), **kw)
    fin = np.where(np.isfinite(z), z, np.nan)
    with np.errstate(all="ignore"):
        spread = np.nan_to_num(np.nanmax(fin, 1) - np.nanmin(fin, 1))[:, None]
    tol = (80 + 2 * spread) * U * np.abs(rw) + 2.0 ** -126 * max(1.0, abs(kw.get("scale", 1.0)))
    assert (np.abs(w[:n].numpy().astype(np.float64) - rw) <= tol).all()


@pytest.mark.parametrize("E,k,G,tg", [(1, 1, 1, 1), (7, 3, 7, 3), (16, 8, 16, 9), (40, 8, 10, 10), (64, 8, 8, 3),
                                      (65, 8, 1, 1), (128, 8, 1, 1), (150, 5, 5, 3), (250, 8, 2, 1),
                                      (256, 8, 8, 4), (256, 8, 1, 1), (256, 6, 16, 5), (257, 4, 1, 1)])
@pytest.mark.parametrize("scoring", [SOFT, SIGM])
def test_many_tokens(E, k, G, tg, scoring):
    g = gen(E * k)
    rows = torch.randn(37, E, generator=g) * 1.5
    rows[3] = -INF                                                   # masked: all,
    rows[4, 1:] = -INF                                               # all but one,
    rows[5, :E // 2] = -INF                                          # half,
    rows[6:9][torch.rand(3, E, generator=g) < 0.8] = -INF            # most
    bias = torch.randn(E, generator=g) * (0.2 if scoring == SIGM else 2.0 / E)
    for best in (1, 2):
        kw = dict(scoring=scoring, n_group=G, topk_group=tg, group_best=best)
        check_many(rows, bias, k, **kw)
        check_many(rows.to(torch.bfloat16), None, k, renormalize=False, scale=2.5, **kw)


@pytest.mark.parametrize("E,G,tg", [(64, 1, 1), (256, 8, 4), (150, 5, 2), (256, 1, 1)])
@pytest.mark.parametrize("scoring", [SOFT, SIGM])
def test_many_tokens_too_close_for_fp32(E, G, tg, scoring):
    g = gen(E + G)
    row = torch.randn(1, E, generator=g)
    s = R.scores(row.numpy(), scoring)[0]
    bias = torch.from_numpy((0.75 - s).astype(np.float32))
    rows = row.repeat(29, 1)
    rows[1::2] += torch.randn(14, E, generator=g) * 1e-7
    rows[2::4] = torch.randn(7, E, generator=g)                      # some tokens of a wave are clear
    for k in (1, 8):
        for best in (1, 2):
            check_many(rows, bias, k, scoring=scoring, n_group=G, topk_group=tg, group_best=best)


@pytest.mark.parametrize("scoring", [SOFT, SIGM])
def test_many_tokens_ties_and_nonfinite(scoring):
    g = gen(17)
    rows = (torch.randn(31, 256, generator=g) * 2).round() / 2
    rows[0] = 1.0
    bias = (torch.randn(256, generator=g) * 2).round() / 16
    for G, tg in ((1, 1), (8, 3)):
        for b in (None, bias):
            check_many(rows, b, 8, scoring=scoring, n_group=G, topk_group=tg, group_best=2)
            z = rows.repeat(270, 1)
            kw = dict(scoring=scoring, n_group=G, topk_group=tg, bias=None if b is None else b.to(DEV))
            clean = mq.moe_route_experts(z.to(DEV), 8, **kw)
            bad = torch.arange(5, z.shape[0], 97)
            z[bad, 3] = float("nan")
            z[bad[1::3], 200] = INF
            z[bad[2::3]] = -float("nan")
            ids, w = mq.moe_route_experts(z.to(DEV), 8, **kw)
            ids, w = ids.cpu(), w.cpu()
            assert ((ids >= 0) & (ids < 256)).all()
            assert all(len(set(r)) == 8 for r in ids[bad].tolist())
            keep = torch.ones(z.shape[0], dtype=torch.bool)
            keep[bad] = False
            assert torch.equal(ids[keep], clean[0].cpu()[keep]) and torch.equal(w[keep], clean[1].cpu()[keep])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_past_32_bits(dtype):
    """Rows of a matrix wider than 2^31 elements."""
    ld, E = 2 ** 31 + 8, 96
    z = torch.empty(3 * ld, dtype=dtype, device=DEV).view(3, ld)[:, :E]
    rows = torch.randn(3, E, generator=gen(23)).to(dtype)
    z.copy_(rows)
    ids, w = mq.moe_route_experts(z, 5, scoring=SIGM)
    ref = mq.moe_route_experts(rows.to(DEV), 5, scoring=SIGM)
    assert torch.equal(ids, ref[0]) and torch.equal(w, ref[1])


@pytest.mark.parametrize("scoring", [SOFT, SIGM])
@pytest.mark.parametrize("many", [False, True])
def test_groups_whose_sums_pass_the_largest_fp32(scoring, many):
    """Biases of either end of fp32, as a mask of the lowest value or of an expert that is always
    taken: finite, while the sum of a group's best two is not in fp32."""
    g = gen(19)
    E, G, S, k = 64, 8, 8, 8
    low, high = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    rows = torch.randn(12, E, generator=g)
    rows[1:5, :3 * S][torch.rand(4, 3 * S, generator=g) < 0.9] = -INF
    rows[5:9][torch.rand(4, E, generator=g) < 0.7] = -INF
    rows[9] = -INF
    groups = [torch.full((E,), low), torch.full((E,), high), torch.randn(E, generator=g) * 0.1]
    groups[2][3 * S:] = low                                          # three groups without the lowest value
    groups.append(groups[2].roll(S))
    groups.append(torch.where(torch.arange(E) % S < 2, high, low))
    groups.append((torch.rand(E, generator=g) - 0.5) * 2 * high)
    groups.append(torch.where(torch.rand(E, generator=g) < 0.5, -0.75 * high, 0.1))
    fn = check_many if many else check
    for bias in groups:
        for tg in (1, 3, 4, 7):
            for best in (1, 2):
                fn(rows, bias, k, scoring=scoring, n_group=G, topk_group=tg, group_best=best)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E", [(2051, 64), (4097, 128), (8195, 256), (8198, 250), (5, 256), (130, 1024)])
def test_rows_and_bias_off_alignment_and_bytes_around(T, E, dtype):
    """Four tokens a wave (and one): row strides and starts off the wide loads' alignment, tokens that
    are no multiple of four, and nothing written past the last."""
    k = 8
    g = gen(E + T)
    data = torch.randn(T, E, generator=g).to(dtype).to(DEV)
    data[::5, ::3] = -INF
    shifted = torch.zeros(E + 1, device=DEV)
    shifted[1:] = (torch.randn(E, generator=g) * 0.1).to(DEV)
    ids = torch.full((T + 4, k), 77, dtype=torch.int32, device=DEV)
    w = torch.full((T + 4, k), 77.0, device=DEV)
    G = 8 if E % 8 == 0 else 5
    for kw in (dict(scoring=SIGM, bias=shifted[1:]), dict(scoring=SOFT, renormalize=False),
               dict(scoring=SIGM, bias=shifted[1:], n_group=G, topk_group=2, group_best=2)):
        aligned = dict(kw)
        if "bias" in kw:
            aligned["bias"] = kw["bias"].clone()
        ref = mq.moe_route_experts(data, k, **aligned)
        for first, pad in ((0, 1), (0, 2), (0, 4), (1, 3), (2, 2), (4, 4), (1, 1)):
            wide = torch.full((T, first + E + pad), INF, dtype=dtype, device=DEV)     # not to be read as scores
            wide[:, first:first + E] = data
            ids.fill_(77)
            w.fill_(77.0)
            got = mq.moe_route_experts(wide[:, first:first + E], k, ids=ids[1:T + 1], weights=w[1:T + 1], **kw)
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]), (first, pad)
            for t in (ids, w):
                assert (t[0] == 77).all() and (t[T + 1:] == 77).all()
    rows = data[:40].cpu()
    check(rows, shifted[1:].cpu(), k, scoring=SIGM, n_group=G, topk_group=2, group_best=2)
    assert torch.equal(ref[0][:40].cpu(), mq.moe_route_experts(rows.to(DEV), k, **aligned)[0].cpu())
