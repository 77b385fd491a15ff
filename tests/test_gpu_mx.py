"""The MXFP4 calls against the float64 oracle.

Quantization, its inverse and the tiled order are exact: every byte is compared.

Tolerances of the products, derived (u = 2^-24):
  fp32 sums    products of E2M1 values are exact; a product sum of K terms in any
               order and grouping is within K u' S of the exact one, S the sum of
               magnitudes, with u' = 2 u (truncating or rounding adders alike)
  rounding     bf16: half a step, 2^-8 of the value; fp32: 2^-24
  silu(g) u    |d silu| <= 1.1 |dg|, so 1.1 dg |u| + |silu(g)| du + dg du, plus 16 u of the
               value for exp, division and product
"""
import numpy as np
import pytest
import torch

import bit_quantized_moe_top_amd as mq
from oracle import layer as L
from oracle import mx as X
from parity import rel_l2, to_np

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def spread(rows, K, seed, lo=-12, hi=12):
    """Normal values, every block of 32 on a scale of its own."""
    g = gen(seed)
    x = torch.randn(rows, K // 32, 32, generator=g)
    return (x * torch.exp2(torch.randint(lo, hi, (rows, K // 32, 1), generator=g).float())).reshape(
        rows, K)


# ------------------------------------------------------------- quantization ----
@pytest.mark.parametrize("M,K", [(1, 32), (3, 64), (4, 4096), (37, 1440), (513, 96), (130, 2048),
                                 (1, 8192)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_every_byte(M, K, dtype):
    x = spread(M, K, M + K).to(dtype)
    q, s = mq.quant_mxfp4(x.to(DEV))
    rq, rs = X.quant_mxfp4(to_np(x))
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    ref = X.values(rq, rs)
    for dt in (torch.bfloat16, torch.float32):
        v = mq.dequant_mxfp4(q, s, dtype=dt)
        assert v.dtype == dt and torch.equal(v.double().cpu(), torch.from_numpy(ref))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_rounding_points_at_every_scale(dtype):
    """Every rounding midpoint, its neighbours one step away, saturation and signs, in blocks
    whose largest element puts the scale at every exponent of the type, subnormals included."""
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.0])
    rows = []
    for e in range(-149 if dtype == torch.float32 else -133, 126):
        m = (mids.double() * 2.0 ** e).to(dtype)
        bits = m.view(torch.int16 if dtype == torch.bfloat16 else torch.int32)
        near = torch.cat([m, (bits + 1).view(dtype), torch.clamp(bits - 1, min=0).view(dtype)])
        near = near * torch.tensor([1, -1] * 15, dtype=dtype)
        rows.append(torch.cat([near, torch.tensor([4.0 * 2.0 ** e, -0.0], dtype=torch.float64).to(dtype)]))
    x = torch.stack(rows)
    q, s = mq.quant_mxfp4(x.to(DEV))
    rq, rs = X.quant_mxfp4(to_np(x))
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    v = mq.dequant_mxfp4(q, s, dtype=torch.float32)
    assert torch.equal(v.double().cpu(), torch.from_numpy(X.values(rq, rs)))


def test_quant_zero_and_nonfinite_blocks():
    x = torch.ones(2, 128)
    x[0, :32] = 0
    x[0, 33], x[0, 70], x[1, 127] = float("inf"), float("nan"), float("-inf")
    for dt in (torch.bfloat16, torch.float32):
        q, s = mq.quant_mxfp4(x.to(dt).to(DEV))
        rq, rs = X.quant_mxfp4(x.numpy())
        assert s.cpu().tolist() == rs.tolist() == [[0, 255, 255, 125], [125, 125, 125, 255]]
        np.testing.assert_array_equal(q.cpu().numpy(), rq)
        v = mq.dequant_mxfp4(q, s, dtype=dt).float().cpu().numpy()
        np.testing.assert_array_equal(v, X.values(rq, rs))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,ld", [(1, 32, 40), (7, 96, 104), (129, 1440, 1536), (300, 32, 64)])
def test_quant_strided_rows_and_caller_outputs(M, K, ld, dtype):
    wide = spread(M, (ld + 31) // 32 * 32, 9 * M + K)[:, :ld].contiguous().to(dtype).to(DEV)
    q = torch.full((M + 1, K // 2), 0xAB, dtype=torch.uint8, device=DEV)
    s = torch.full((M + 1, K // 32), 0xCD, dtype=torch.uint8, device=DEV)
    mq.quant_mxfp4(wide[:, :K], q=q[:M], scale=s[:M])
    rq, rs = mq.quant_mxfp4(wide[:, :K].contiguous())
    assert torch.equal(q[:M], rq) and torch.equal(s[:M], rs)
    assert (q[M] == 0xAB).all() and (s[M] == 0xCD).all()


def test_quant_empty_and_shapes():
    q, s = mq.quant_mxfp4(torch.zeros(0, 64, device=DEV))
    assert q.shape == (0, 32) and s.shape == (0, 2)
    assert mq.dequant_mxfp4(q, s).shape == (0, 64)
    x = spread(6, 64, 2).reshape(2, 3, 64).to(DEV)
    q, s = mq.quant_mxfp4(x)
    assert q.shape == (2, 3, 32) and s.shape == (2, 3, 2)
    assert torch.equal(q.reshape(6, 32), mq.quant_mxfp4(x.reshape(6, 64))[0])


def test_rows_past_32_bits_are_refused():
    q = torch.empty(1 << 30, dtype=torch.uint8, device=DEV)
    s = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError, match="too long"):
        mq.dequant_mxfp4(q, s)
    with pytest.raises(ValueError, match="too many"):
        a_q, a_s = q.view(-1, 16)[:1 << 26], s[:1 << 26].view(-1, 1)
        w = torch.empty(1, 2, 1, 4, 64, 16, dtype=torch.uint8, device=DEV)
        ws = torch.empty(1, 2, 1, 64, 4, dtype=torch.uint8, device=DEV)
        plan = torch.empty(64, dtype=torch.int32, device=DEV)
        mq.moe_grouped_gemm_mxfp4(a_q.repeat(5, 1), a_s.repeat(5, 1), plan, w, ws, topk=8)


def test_quant_past_32_bits():
    """2^31 + 64 elements: the last block lies past 32-bit element offsets."""
    n = (1 << 31) + 64
    x = torch.zeros(n // 32, 32, dtype=torch.bfloat16, device=DEV)
    x[-1], x[-2], x[0] = 3.0, -0.5, 1.0
    q, s = mq.quant_mxfp4(x)
    assert s[-1].item() == 126 and s[-2].item() == 124 and s[0].item() == 125
    assert s[1:-2].max().item() == 0 and q[1:-2].max().item() == 0
    v = mq.dequant_mxfp4(q, s)
    assert torch.equal(v[-2:], x[-2:]) and torch.equal(v[:2], x[:2])
    assert int((v != 0).sum()) == 96


@pytest.mark.parametrize("E,N,K", [(1, 16, 32), (3, 32, 512), (2, 48, 544), (2, 64, 1440), (1, 16, 4096)])
def test_tile_every_byte(E, N, K):
    g = gen(E + N + K)
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    s = torch.randint(0, 256, (E, N, K // 32), generator=g, dtype=torch.uint8)
    w, ws = mq.tile_mxfp4_weights(q.to(DEV), s.to(DEV))
    rw, rws = X.tile(q.reshape(E * N, -1).numpy(), s.reshape(E * N, -1).numpy())
    np.testing.assert_array_equal(w.cpu().numpy().reshape(rw.shape), rw)
    np.testing.assert_array_equal(ws.cpu().numpy().reshape(rws.shape), rws)


# ---------------------------------------------------------- grouped product ----
def weights(E, N, K, seed, std=0.05):
    """Values [E, N, K] (float64) and the tiled tensors of random MXFP4 weights."""
    w = torch.randn(E, N, K, generator=gen(seed)) * std
    q, s = mq.quant_mxfp4(w.to(DEV))
    return X.values(q.cpu().numpy(), s.cpu().numpy()), mq.tile_mxfp4_weights(q, s)


def make_ids(T, k, E, seed, hot=None):
    g = gen(seed)
    score = torch.rand(T, E, generator=g)
    if hot is not None:
        score[:, hot] += 1.0                       # every token picks expert `hot`
    return score.topk(k, dim=1).indices.to(torch.int32)


def silu_bound(v, d):
    half = v.shape[1] // 2
    g, u, dg, du = v[:, :half], v[:, half:], d[:, :half], d[:, half:]
    h = L.silu(g) * u
    return h, 1.1 * dg * np.abs(u) + np.abs(L.silu(g)) * du + 1.1 * dg * du + 16 * U * np.abs(h)


GEMM_CASES = [
    # T, k, E, N, K, hot: one row; one block of K; a super-group and a bit; rows of scale bytes
    # that are no whole dwords; experts of 0, 1, 17, 64, 65 and 200+ rows
    (1, 1, 1, 32, 32, None), (4, 2, 8, 64, 96, None), (5, 3, 6, 96, 544, 2),
    (16, 2, 8, 256, 256, None), (17, 1, 2, 32, 1440, 0), (64, 1, 3, 32, 512, 1),
    (65, 2, 4, 160, 1024, 3), (100, 4, 5, 288, 2048, 0), (230, 3, 7, 96, 1056, 1),
    (300, 2, 40, 512, 640, None), (256, 1, 1, 544, 4096, 0), (700, 6, 16, 256, 512, 5),
    # enough row tiles and columns for the 256-row weight tiles, ragged in every direction
    (600, 4, 60, 2080, 160, 7), (900, 3, 24, 2336, 544, 5),
]


@pytest.mark.parametrize("T,k,E,N,K,hot", GEMM_CASES)
@pytest.mark.parametrize("tokens", [True, False])
def test_grouped_gemm(T, k, E, N, K, hot, tokens):
    wv, (w, ws) = weights(E, N, K, T + N)
    ids = make_ids(T, k, E, K, hot)
    plan, _, _ = mq.moe_permute(ids.to(DEV), E)
    pv = L.permute_plan(ids.numpy(), E)
    experts = ids.numpy().reshape(-1)[pv["sorted_rows"]]
    rows = T if tokens else T * k
    a_q, a_s = mq.quant_mxfp4(spread(rows, K, T * K + 1, -3, 3).to(DEV))
    av = X.values(a_q.cpu().numpy(), a_s.cpu().numpy())
    if tokens:
        av = av[pv["sorted_rows"] // k]
    v, mag = X.grouped_rows(av, experts, wv)
    d = K * 2 * U * mag
    topk = k if tokens else 0
    for dt in (torch.float32, torch.bfloat16):
        got = mq.moe_grouped_gemm_mxfp4(a_q, a_s, plan, w, ws, topk=topk, out_dtype=dt)
        assert got.dtype == dt and got.shape == v.shape
        err = np.abs(to_np(got).astype(np.float64) - v)
        assert (err <= d + HALF[dt] * (np.abs(v) + d)).all(), err.max()
    h, dh = silu_bound(v, d)
    got = mq.moe_grouped_gemm_mxfp4(a_q, a_s, plan, w, ws, epilogue=mq.EPI_SILU_MUL, topk=topk)
    err = np.abs(to_np(got).astype(np.float64) - h)
    assert (err <= dh + HALF[torch.bfloat16] * (np.abs(h) + dh)).all(), err.max()
    again = mq.moe_grouped_gemm_mxfp4(a_q, a_s, plan, w, ws, epilogue=mq.EPI_SILU_MUL, topk=topk)
    assert torch.equal(got, again)


@pytest.mark.parametrize("T,k,E,N,K", [(6, 2, 4, 64, 96), (90, 3, 5, 256, 1024)])
def test_grouped_gemm_integers_are_exact(T, k, E, N, K):
    """Codes with scale 1: every sum is a multiple of 1/4 below 2^22, exact in fp32."""
    g = gen(T)
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    s = torch.full((E, N, K // 32), 127, dtype=torch.uint8)
    a_q = torch.randint(0, 256, (T, K // 2), generator=g, dtype=torch.uint8)
    a_s = torch.full((T, K // 32), 127, dtype=torch.uint8)
    ids = make_ids(T, k, E, 3)
    plan, _, _ = mq.moe_permute(ids.to(DEV), E)
    pv = L.permute_plan(ids.numpy(), E)
    v, _ = X.grouped_rows(X.values(a_q.numpy(), a_s.numpy())[pv["sorted_rows"] // k],
                          ids.numpy().reshape(-1)[pv["sorted_rows"]], X.values(q.numpy(), s.numpy()))
    w, ws = mq.tile_mxfp4_weights(q.to(DEV), s.to(DEV))
    got = mq.moe_grouped_gemm_mxfp4(a_q.to(DEV), a_s.to(DEV), plan, w, ws, topk=k,
                                    out_dtype=torch.float32)
    np.testing.assert_array_equal(got.cpu().numpy().astype(np.float64), v)


@pytest.mark.parametrize("T,k,E,N,K", [(9, 2, 4, 64, 96), (150, 3, 6, 288, 544)])
def test_grouped_gemm_dropped_ids_and_nan_rows(T, k, E, N, K):
    """Rows of ids outside [0, E) are left as they were; a NaN row spoils only itself."""
    wv, (w, ws) = weights(E, N, K, 11)
    ids = make_ids(T, k, E, 12)
    ids[1, 0], ids[T - 1, k - 1] = -1, E
    plan, _, _ = mq.moe_permute(ids.to(DEV), E)
    moved = ids.clone()
    moved[(ids < 0) | (ids >= E)] = E
    pv = L.permute_plan(moved.numpy(), E + 1)
    kept = int(pv["offsets"][E])
    assert kept == T * k - 2
    x = spread(T, K, 13, -3, 3)
    x[2, 40 % K] = float("nan")
    a_q, a_s = mq.quant_mxfp4(x.to(DEV))
    out = torch.full((T * k, N), 77.0, device=DEV)
    mq.moe_grouped_gemm_mxfp4(a_q, a_s, plan, w, ws, topk=k, out=out)
    out = out.cpu().numpy().astype(np.float64)
    assert (out[kept:] == 77.0).all()
    tok = pv["sorted_rows"][:kept] // k
    v, mag = X.grouped_rows(np.nan_to_num(X.values(a_q.cpu().numpy(), a_s.cpu().numpy()))[tok],
                            moved.numpy().reshape(-1)[pv["sorted_rows"][:kept]], wv)
    bad = tok == 2
    assert np.isnan(out[:kept][bad]).all()
    err = np.abs(out[:kept] - v)[~bad]
    assert (err <= (K * 2 * U * mag + U * np.abs(v))[~bad]).all()


def test_grouped_gemm_no_rows_and_wrong_shapes():
    _, (w, ws) = weights(3, 32, 64, 1)
    plan, _, _ = mq.moe_permute(torch.zeros(0, 2, dtype=torch.int32, device=DEV), 3)
    a_q, a_s = mq.quant_mxfp4(torch.zeros(0, 64, device=DEV))
    assert mq.moe_grouped_gemm_mxfp4(a_q, a_s, plan, w, ws, topk=2).shape == (0, 32)
    a_q, a_s = mq.quant_mxfp4(torch.zeros(4, 64, device=DEV))
    with pytest.raises(ValueError, match="built for"):
        mq.moe_grouped_gemm_mxfp4(a_q, a_s, plan, w, ws, topk=2)
    plan, _, _ = mq.moe_permute(torch.zeros(2, 2, dtype=torch.int32, device=DEV), 3)
    with pytest.raises(ValueError, match="out"):
        mq.moe_grouped_gemm_mxfp4(a_q, a_s, plan, w, ws, out=torch.empty(4, 33, device=DEV))
    with pytest.raises(ValueError, match="K = 1056"):
        b_q, b_s = mq.quant_mxfp4(torch.zeros(4, 1056, device=DEV))
        mq.moe_grouped_gemm_mxfp4(b_q, b_s, plan, w, ws)
    with pytest.raises(ValueError, match="K = 64"):
        c_q, c_s = mq.quant_mxfp4(torch.zeros(4, 96, device=DEV))      # as many super-groups
        mq.moe_grouped_gemm_mxfp4(c_q, c_s, plan, w, ws)
    with pytest.raises(ValueError, match="tiled"):
        mq.moe_grouped_gemm_mxfp4(a_q, a_s, plan, a_q, a_s)
    with pytest.raises(mq.MoeqError):
        mq.moe_grouped_gemm_mxfp4(a_q, a_s, plan, w, ws, epilogue=mq.EPI_SILU_MUL,
                                  out_dtype=torch.float32)


# ---------------------------------------------------------- few-token layer ----
class Few:
    def __init__(self, T, k, E, H, I, seed, bias=False, shared=False):
        self.k = k
        self.w13v, self.w13 = weights(E, 2 * I, H, seed)
        self.w2v, self.w2 = weights(E, H, I, seed + 1)
        g = gen(seed + 2)
        self.x = torch.randn(T, H, generator=g).to(torch.bfloat16)
        self.logits = torch.randn(T, E, generator=g)
        self.bias = torch.randn(E, generator=g) if bias else None
        self.shared = torch.randn(T, H, generator=g).to(torch.bfloat16) if shared else None

    def run(self, renormalize=True, out=None):
        dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        return mq.moe_layer_mxfp4_few(dev(self.logits), dev(self.x), *self.w13, *self.w2, self.k,
                                      bias=dev(self.bias), renormalize=renormalize,
                                      shared=dev(self.shared), out=out)

    def check(self, got, renormalize=True):
        np_ = lambda t: None if t is None else to_np(t)  # noqa: E731
        x = to_np(self.x).astype(np.float64)
        ref = X.few_layer(self.logits.numpy(), x, self.w13v, self.w2v, self.k, np_(self.bias),
                          renormalize, np_(self.shared))
        np.testing.assert_array_equal(got["ids"].cpu().numpy(), ref["ids"])
        np.testing.assert_allclose(got["w"].cpu().numpy(), ref["w"], rtol=1e-6, atol=1e-30)
        # the bound: fp32 sums over H and I, h as two bf16 values (off by half a step of half a
        # step, 2^-16), the weighted sum, y rounded
        T, H = x.shape
        I = self.w2v.shape[2]
        d = np.zeros_like(ref["y"])
        for t in range(T):
            for j in range(self.k):
                e = ref["ids"][t, j]
                gu = self.w13v[e] @ x[t]
                h, dh = silu_bound(gu[None], (H * 2 * U * (np.abs(self.w13v[e]) @ np.abs(x[t])))[None])
                dh = dh[0] + 2.0 ** -16 * (np.abs(h[0]) + dh[0])
                w2 = np.abs(self.w2v[e])
                do = w2 @ dh + I * 2 * U * (w2 @ (np.abs(h[0]) + dh))
                d[t] += ref["w"][t, j] * (do + (1e-6 + 16 * U) * (w2 @ np.abs(h[0])))
        y = to_np(got["y"]).astype(np.float64)
        err = np.abs(y - ref["y"])
        assert (err <= d + 2.0 ** -8 * (np.abs(ref["y"]) + d)).all(), err.max()
        # one bf16 rounding: 2^-8 / sqrt(3) / 1.37 = 1.65e-3 relative rms (uniform over half
        # steps, root mean square of a uniform mantissa)
        if y.size >= 512:
            assert rel_l2(y, ref["y"]) <= 2e-3


FEW_CASES = [
    # T, k, E, H, I, bias, shared: one token; one expert; all experts; rows staged in LDS (<= 4
    # per expert) and read from memory; K of one block, of one super-group, of five; long rows
    (1, 1, 1, 32, 32, False, False), (1, 6, 256, 256, 96, False, False),
    (4, 2, 8, 512, 128, False, True), (5, 3, 10, 288, 96, True, True),
    (16, 8, 8, 96, 544, True, False), (16, 8, 1024, 64, 32, False, False),
    (16, 1, 2, 1440, 64, False, True), (7, 4, 40, 2080, 320, True, True),
    (3, 2, 4, 4096, 2048, False, False), (2, 2, 3, 8192, 64, False, False),
    (6, 2, 3, 64, 4640, False, True),
    # rows too long for LDS: one row staged, none (of x, of h)
    (5, 2, 3, 64, 4640, False, False), (3, 2, 3, 64, 4640, False, False),
    (2, 1, 2, 16896, 32, False, True),
]


@pytest.mark.parametrize("T,k,E,H,I,bias,shared", FEW_CASES)
@pytest.mark.parametrize("renormalize", [True, False])
def test_few_layer(T, k, E, H, I, bias, shared, renormalize):
    f = Few(T, k, E, H, I, T + H, bias, shared)
    got = f.run(renormalize)
    f.check(got, renormalize)
    y = got["y"].clone()
    # the same buffers again (a workspace with a finished call's contents): the same bits
    got["y"].fill_(float("nan"))
    again = f.run(renormalize, out=got)
    assert again["y"].data_ptr() == got["y"].data_ptr() and torch.equal(again["y"], y)


def test_few_layer_routing_equals_the_routing_call():
    f = Few(16, 6, 300, 64, 32, 5, bias=True)
    f.logits[3] = f.logits[3].round()              # ties
    got = f.run()
    ids, w = mq.moe_route_topk(f.logits.to(DEV), 6, f.bias.to(DEV))
    assert torch.equal(got["ids"], ids) and torch.equal(got["w"], w)


def test_few_layer_masked_experts():
    f = Few(6, 3, 12, 96, 64, 6, shared=True)
    f.logits[0, :] = float("-inf")                 # nothing left: the shared part alone
    f.logits[1, 1:] = float("-inf")                # one expert left
    f.logits[2, ::2] = float("-inf")
    f.logits[3, :] = torch.finfo(torch.float32).min
    got = f.run()
    f.check(got)
    assert torch.equal(got["y"][0].cpu(), f.shared[0]) and (got["w"][0] == 0).all()
    assert got["w"][1].tolist() == [1.0, 0.0, 0.0]


def test_few_layer_masked_experts_may_hold_anything():
    f = Few(5, 4, 8, 96, 64, 30)
    f.logits[:, 0] = float("-inf")
    f.logits[2, 2:] = float("-inf")                # one expert left: masked ones fill its slots
    clean = f.run()["y"].clone()
    f.w13[1][0].fill_(255)                         # expert 0: every block a NaN
    f.w2[1][0].fill_(255)
    got = f.run()
    assert (got["ids"][2] == 0).any() and torch.equal(got["y"], clean)
    f.w13v[0] = f.w2v[0] = 0.0
    f.check(got)


@pytest.mark.parametrize("bits", [0x7FC00000, -0x400000, -1])          # NaNs of either sign
def test_few_layer_nan_scores_stay_inside(bits):
    f = Few(4, 3, 6, 64, 32, 31)
    nan = torch.full((6,), bits, dtype=torch.int32).view(torch.float32)
    clean = f.run(out={"ws": torch.full((1 << 16,), 255, dtype=torch.uint8, device=DEV)})
    f.logits[1] = nan
    f.logits[3, 2] = nan[0]
    got = f.run(out={"ws": torch.full((1 << 16,), 255, dtype=torch.uint8, device=DEV)})
    assert ((got["ids"] >= 0) & (got["ids"] < 6)).all()
    for name in ("ids", "w", "y"):                  # the other tokens are as they were
        assert torch.equal(got[name][[0, 2]], clean[name][[0, 2]]), name


@pytest.mark.parametrize("bits", [0x7FC00000, -1])
def test_few_layer_nan_token_among_sixteen(bits):
    """A token without a candidate must not crowd the experts that the others share."""
    f = Few(16, 8, 9, 96, 64, 32)
    f.logits[:, 8] = 20.0                           # every token's first choice is the last expert
    clean = f.run(out={"ws": torch.full((1 << 18,), 255, dtype=torch.uint8, device=DEV)})
    f.logits[3] = torch.full((9,), bits, dtype=torch.int32).view(torch.float32)
    got = f.run(out={"ws": torch.full((1 << 18,), 255, dtype=torch.uint8, device=DEV)})
    assert sorted(set(got["ids"][3].tolist())) == sorted(got["ids"][3].tolist())
    others = [t for t in range(16) if t != 3]
    for name in ("ids", "w", "y"):
        assert torch.equal(got[name][others], clean[name][others]), name


def test_few_layer_every_token_on_one_expert():
    f = Few(16, 2, 6, 544, 96, 8)
    f.logits[:, 4] = 9.0
    f.logits[:, 0] = 8.0
    f.check(f.run())


def test_few_layer_empty_and_refusals():
    f = Few(4, 2, 6, 64, 32, 9)
    f.x, f.logits = f.x[:0], f.logits[:0]
    got = f.run()
    assert got["y"].shape == (0, 64) and got["ids"].shape == (0, 2)
    f = Few(17, 2, 6, 64, 32, 9)
    with pytest.raises(ValueError, match="at most 16"):
        f.run()
    f = Few(4, 2, 6, 64, 32, 9)
    with pytest.raises(mq.MoeqError, match="workspace"):
        f.run(out={"ws": torch.empty(256, dtype=torch.uint8, device=DEV)})
    with pytest.raises(ValueError, match="ids"):
        f.run(out={"ids": torch.empty(4, 3, dtype=torch.int32, device=DEV)})
    f.k = 7
    with pytest.raises(ValueError, match="experts"):
        f.run()


@pytest.mark.parametrize("T,k,E,H,I", [(1, 1, 1, 32, 32), (4, 2, 8, 512, 128), (16, 8, 9, 96, 544),
                                       (16, 8, 200, 1440, 352)])
def test_few_layer_stays_inside_its_workspace_and_outputs(T, k, E, H, I):
    """Every buffer is a slice of a larger one, exactly as long as the call asks for."""
    f = Few(T, k, E, H, I, T + E)
    sizes = {"ws": mq.moe_layer_mxfp4_few_ws_size(T, k, H, I), "ids": T * k * 4, "w": T * k * 4,
             "y": T * H * 2}
    dtypes = {"ws": torch.uint8, "ids": torch.int32, "w": torch.float32, "y": torch.bfloat16}
    bufs = {n: torch.full((256 + b + 256,), 0xA5, dtype=torch.uint8, device=DEV)
            for n, b in sizes.items()}
    out = {n: bufs[n][256:256 + b].view(dtypes[n]) for n, b in sizes.items()}
    out["ids"], out["w"], out["y"] = out["ids"].view(T, k), out["w"].view(T, k), out["y"].view(T, H)
    f.check(f.run(out=out))
    for n, b in sizes.items():
        assert (bufs[n][:256] == 0xA5).all() and (bufs[n][256 + b:] == 0xA5).all(), n


def test_few_layer_two_streams_with_their_own_workspaces():
    a, b = Few(8, 4, 20, 512, 256, 20), Few(16, 3, 20, 1024, 96, 21)
    ra, rb = a.run()["y"].clone(), b.run()["y"].clone()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(10):
        with torch.cuda.stream(sa):
            ya = a.run()["y"]
        with torch.cuda.stream(sb):
            yb = b.run()["y"]
        outs.append((ya, yb))
    torch.cuda.synchronize()
    for ya, yb in outs:
        assert torch.equal(ya, ra) and torch.equal(yb, rb)


@pytest.mark.parametrize("T,k,E,H,I", [
    # rows of an expert that do not fit in LDS: more than four; none, at most four of them and
    # more; a last super-group that ends inside; all sixteen tokens on one expert
    (7, 2, 2, 544, 1056), (16, 1, 1, 1056, 544), (3, 2, 3, 64, 6688), (9, 2, 2, 64, 6688),
    (2, 1, 2, 20512, 32), (5, 1, 1, 20512, 32), (16, 2, 2, 96, 8224)])
def test_few_layer_rows_from_memory(T, k, E, H, I):
    f = Few(T, k, E, H, I, T + I, shared=True)
    f.check(f.run())


# h between the two products: one expert per token (weight 1), so that y is W2 h alone.
def one_expert(T, H, I, w13, w2):
    """A Few whose only expert has the given weights (exact in MXFP4)."""
    f = Few(T, 1, 1, H, I, 40)
    f.w13v, f.w2v = w13[None], w2[None]
    for name, v in (("w13", f.w13v), ("w2", f.w2v)):
        q, s = X.quant_mxfp4(v)
        np.testing.assert_array_equal(X.values(q, s), v)
        setattr(f, name, mq.tile_mxfp4_weights(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)))
    return f


@pytest.mark.parametrize("T", [1, 2, 16])      # h staged in LDS, and read from memory
def test_few_layer_h_keeps_fp32(T):
    """y[c] = h[2c] - h[2c + 1], which differ by 2^-13 of themselves: a rounding of h to fewer bits
    than fp32's shows.  Per column: g is one exact product, the same for both; u is one product
    plus, for h[2c], a small one (2 u); h rounds once more (u each); the difference is a sum of the
    parts that h is split into, three at most each (6 terms, 2 u each of the magnitudes).  So
    |dy| <= 16 u |y| + (2 + 1 + 12) u (|h0| + |h1|), and y's own rounding."""
    H, I = 64, 128
    g = np.random.default_rng(50)
    w13, w2 = np.zeros((2 * I, H)), np.zeros((H, I))
    mags = np.array([1.0, 1.5, 2.0, 3.0])
    for c in range(H):
        a, b, d = g.integers(0, 32, 3)
        gate, up, low = g.choice(mags), g.choice(mags), g.choice(mags) * 2.0 ** -13
        for i in (2 * c, 2 * c + 1):
            w13[i, a], w13[I + i, b] = gate, up
        w13[I + 2 * c, 32 + d] = low
        w2[c, 2 * c], w2[c, 2 * c + 1] = 1.0, -1.0
    f = one_expert(T, H, I, w13, w2)
    f.x = (torch.rand(T, H, generator=gen(51)) + 0.5).to(torch.bfloat16)
    x = to_np(f.x).astype(np.float64)
    gu = x @ w13.T
    h = L.silu(gu[:, :I]) * gu[:, I:]
    ref = h @ w2.T
    d = 16 * U * np.abs(ref) + 15 * U * (np.abs(h) @ np.abs(w2).T)
    err = np.abs(to_np(f.run()["y"]).astype(np.float64) - ref)
    assert (err <= d + 2.0 ** -8 * (np.abs(ref) + d)).all(), (err / d).max()


@pytest.mark.parametrize("T", [1, 16])
def test_few_layer_h_up_to_the_largest_fp32(T):
    """h = 0.9995 * 2^128, finite in fp32 and past bf16's largest value, of either sign."""
    H, I = 64, 32
    w13, w2 = np.zeros((2 * I, H)), np.zeros((H, I))
    w13[:I, 0] = 1.0                               # g = 64: silu(g) = g in fp32
    w13[I:, 1], w13[I:, 32] = 2.0 ** 62, 2.0 ** 60
    w2[np.arange(H), np.arange(H) % I] = 2.0 ** -100
    f = one_expert(T, H, I, w13, w2)
    f.x = torch.zeros(T, H, dtype=torch.bfloat16)
    sign = 1 - 2 * (torch.arange(T) % 2)
    f.x[:, 0] = 64.0
    f.x[:, 1], f.x[:, 32] = sign * 1.9921875 * 2.0 ** 59, sign * 1.75 * 2.0 ** 53
    x = to_np(f.x).astype(np.float64)
    gu = x @ w13.T
    h = gu[:, :I] * gu[:, I:]
    assert 2.0 ** 128 * (1 - 2.0 ** -9) < np.abs(h).min() and np.abs(h).max() < np.finfo(np.float32).max
    ref = h @ w2.T
    y = to_np(f.run()["y"]).astype(np.float64)
    assert (np.abs(y - ref) <= (2.0 ** -8 + 32 * U) * np.abs(ref)).all()


# --------------------------------------------------------------- whole layer ----
def chain_reference(x, logits, bias, shared, w13v, w2v, k):
    """The layer as MxMoELayer.forward computes it, in float64 with its roundings: x and h in
    MXFP4, h and o in bf16."""
    from oracle import formats as F
    ids, wt = L.route_topk(logits, k, bias)
    xv = X.values(*X.quant_mxfp4(x))
    T, I = x.shape[0], w2v.shape[2]
    y = np.zeros((T, w2v.shape[1]))
    for t in range(T):
        for j in range(k):
            gu = w13v[ids[t, j]] @ xv[t]
            h = F.bf16_round(L.silu(gu[:I]) * gu[I:])
            y[t] += wt[t, j] * F.bf16_round(w2v[ids[t, j]] @ X.values(*X.quant_mxfp4(h)))
    return ids, y + (0 if shared is None else shared)


@pytest.mark.parametrize("T,k,E,H,I", [(3, 2, 6, 96, 64), (40, 3, 8, 544, 160), (150, 2, 5, 256, 96)])
def test_mx_layer(T, k, E, H, I):
    g = gen(T)
    w13, w2 = torch.randn(E, 2 * I, H, generator=g) * .1, torch.randn(E, H, I, generator=g) * .1
    layer = mq.MxMoELayer(H, I, E, k, device=DEV)
    layer.quantize_weights(w13.to(DEV), w2.to(DEV))
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    logits, bias = torch.randn(T, E, generator=g), torch.randn(E, generator=g)
    b = layer.forward(x.to(DEV), logits.to(DEV), bias.to(DEV), return_all=True)
    w13v = X.values(*X.quant_mxfp4(w13.numpy()))
    w2v = X.values(*X.quant_mxfp4(w2.numpy()))
    ids, ref = chain_reference(to_np(x).astype(np.float64), logits.numpy(), bias.numpy(), None,
                               w13v, w2v, k)
    np.testing.assert_array_equal(b["ids"].cpu().numpy(), ids)
    # rounding y, and of o in the combine's input: 1.7e-3 each.  h may round to the other bf16
    # neighbour where the fp32 sum lies within its error of a midpoint (K 2^-23 of the sum of
    # magnitudes against half steps of 2^-8: a few in 10^4 elements), and 1 in 64 bf16 values is
    # an E2M1 midpoint, so about one h code in 10^6 differs, by half of its value
    assert rel_l2(to_np(b["y"]), ref) <= 4e-3
    if T <= mq.FEW_TOKENS:
        few = layer.forward_few(x.to(DEV), logits.to(DEV), bias.to(DEV), return_all=True)
        exact = X.few_layer(logits.numpy(), to_np(x).astype(np.float64), w13v, w2v, k, bias.numpy())
        assert torch.equal(few["ids"], b["ids"])
        # one rounding, 1.65e-3 rms, of a small sample (288 values)
        assert rel_l2(to_np(few["y"]), exact["y"]) <= 2.5e-3


@pytest.mark.parametrize("T", [2, 16, 70])
def test_mx_layer_captured_and_replayed(T):
    k, E, H, I = 3, 12, 512, 256
    g = gen(T)
    layer = mq.MxMoELayer(H, I, E, k, device=DEV)
    layer.quantize_weights((torch.randn(E, 2 * I, H, generator=g) * .1).to(DEV),
                           (torch.randn(E, H, I, generator=g) * .1).to(DEV))
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    logits = torch.randn(T, E, generator=g).to(DEV)
    forms = [layer.forward] + ([layer.forward_few] if T <= mq.FEW_TOKENS else [])
    for fn in forms:
        fn(x, logits)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = fn(x, logits)
        for rep in range(4):
            x.copy_(torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV))
            logits.copy_(torch.randn(T, E, generator=g).to(DEV))
            expect = fn(x, logits).clone()          # the same buffers, eagerly
            torch.cuda.synchronize()
            y.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, expect), rep


@pytest.mark.parametrize("T", [2, 16, 70])
def test_mx_layer_replay_computes_every_step(T):
    """Between the eager call and the replay every intermediate is filled from other inputs, so a
    step missing from the graph shows."""
    k, E, H, I, S = 3, 12, 512, 256, 64
    g = gen(T + 1)
    layer = mq.MxMoELayer(H, I, E, k, device=DEV)
    layer.quantize_weights((torch.randn(E, 2 * I, H, generator=g) * .1).to(DEV),
                           (torch.randn(E, H, I, generator=g) * .1).to(DEV))
    layer.set_router((torch.randn(E, H, generator=g) / 16).to(DEV))
    layer.set_shared((torch.randn(2 * S, H, generator=g) * .1).to(torch.bfloat16).to(DEV),
                     (torch.randn(H, S, generator=g) * .1).to(torch.bfloat16).to(DEV))
    new = lambda: torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    x = new()
    for fn in [layer.forward] + ([layer.forward_few] if T <= mq.FEW_TOKENS else []):
        fn(x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b = fn(x, return_all=True)
        for rep in range(4):
            wanted = new()
            x.copy_(wanted)
            expect = {n: t.clone() for n, t in fn(x, return_all=True).items()}
            x.copy_(new())
            fn(x)                                       # other values in every buffer
            torch.cuda.synchronize()
            assert not any(torch.equal(b[n], expect[n]) for n in b if n != "logits"), rep
            b["y"].fill_(float("nan"))
            x.copy_(wanted)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for n in ("ids", "w", "y"):
                assert torch.equal(b[n], expect[n]), (rep, n)


def test_mx_layer_with_router_and_shared_experts():
    T, k, E, H, I, S = 6, 2, 8, 256, 96, 128
    g = gen(77)
    layer = mq.MxMoELayer(H, I, E, k, device=DEV)
    layer.quantize_weights((torch.randn(E, 2 * I, H, generator=g) * .1).to(DEV),
                           (torch.randn(E, H, I, generator=g) * .1).to(DEV))
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    with pytest.raises(ValueError, match="router"):
        layer.forward(x)
    with pytest.raises(ValueError, match="router"):
        layer.forward_few(x)
    layer.set_router((torch.randn(E, H, generator=g) / 16).to(DEV))
    layer.set_shared((torch.randn(2 * S, H, generator=g) * .1).to(torch.bfloat16).to(DEV),
                     (torch.randn(H, S, generator=g) * .1).to(torch.bfloat16).to(DEV))
    logits = mq.moe_router_logits(x, layer.w_router)
    shared = mq.moe_shared_gemm_bf16(mq.moe_shared_gemm_bf16(x, layer.ws13, mq.EPI_SILU_MUL), layer.ws2)
    events = []
    y = layer.forward(x, events=events).clone()
    assert torch.equal(layer.forward(x, logits), y)
    assert [e[0] for e in events] == ["router", "shared_gate_up", "shared_down", "route", "quant_x",
                                      "plan", "gemm_gate_up", "quant_h", "gemm_down", "combine"]
    few = layer.forward_few(x).clone()
    direct = mq.moe_layer_mxfp4_few(logits, x, layer.w13, layer.s13, layer.w2, layer.s2, k,
                                    shared=shared)
    assert torch.equal(few, direct["y"])
    plain = mq.moe_layer_mxfp4_few(logits, x, layer.w13, layer.s13, layer.w2, layer.s2, k)["y"]
    assert not torch.equal(few, plain)
    err = (few.double() - (plain.double() + shared.double())).abs()
    assert (err <= 2.0 ** -8 * (plain.double().abs() + few.double().abs()) * 1.01).all()
    with pytest.raises(ValueError):
        layer.set_weights_fnuz(None, None, None, None)
    with pytest.raises(TypeError):
        layer.forward(x.float())                       # shared experts take bf16


def test_mx_layer_shared_experts_of_another_width_after_a_call():
    T, k, E, H, I = 5, 2, 8, 256, 96
    g = gen(78)
    layer = mq.MxMoELayer(H, I, E, k, device=DEV)
    layer.quantize_weights((torch.randn(E, 2 * I, H, generator=g) * .1).to(DEV),
                           (torch.randn(E, H, I, generator=g) * .1).to(DEV))
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    logits = torch.randn(T, E, generator=g).to(DEV)
    first = layer.forward(x, logits)                   # buffers without shared experts
    alone = first.clone()
    for S in (64, 128):
        ws13 = (torch.randn(2 * S, H, generator=g) * .1).to(torch.bfloat16).to(DEV)
        ws2 = (torch.randn(H, S, generator=g) * .1).to(torch.bfloat16).to(DEV)
        layer.set_shared(ws13, ws2)
        b = layer.forward(x, logits, return_all=True)
        shared = mq.moe_shared_gemm_bf16(mq.moe_shared_gemm_bf16(x, ws13, mq.EPI_SILU_MUL), ws2)
        assert torch.equal(b["shared"], shared)
        assert torch.equal(b["y"], mq.moe_combine(b["o"], b["plan"], b["w"], shared, E=E))
    layer.set_shared(None, None)
    assert torch.equal(layer.forward(x, logits), alone)
    assert first.data_ptr() == layer.forward(x, logits).data_ptr()


def test_mx_layer_no_tokens_and_too_many():
    k, E, H, I = 2, 8, 256, 96
    g = gen(79)
    layer = mq.MxMoELayer(H, I, E, k, device=DEV)
    layer.quantize_weights((torch.randn(E, 2 * I, H, generator=g) * .1).to(DEV),
                           (torch.randn(E, H, I, generator=g) * .1).to(DEV))
    x = torch.randn(17, H, generator=g).to(torch.bfloat16).to(DEV)
    logits = torch.randn(17, E, generator=g).to(DEV)
    assert layer.forward_few(x[:0], logits[:0]).shape == (0, H)
    assert layer.forward(x[:0], logits[:0]).shape == (0, H)
    with pytest.raises(ValueError, match="16 tokens"):
        layer.forward_few(x, logits)
    assert torch.equal(layer.forward(x, logits)[:16], layer.forward(x[:16], logits[:16]))


@pytest.mark.parametrize("T", [6, 40])
@pytest.mark.parametrize("shared", [False, True])
def test_mx_layer_masked_experts_and_tokens(T, shared):
    """Both forms follow one rule: a token whose scores are all -inf gets weights 0 and keeps the
    shared experts' part; an expert of weight 0 adds nothing, whatever its weights hold."""
    k, E, H, I, S = 3, 8, 256, 96, 64
    g = gen(T)
    layer = mq.MxMoELayer(H, I, E, k, device=DEV)
    layer.quantize_weights((torch.randn(E, 2 * I, H, generator=g) * .1).to(DEV),
                           (torch.randn(E, H, I, generator=g) * .1).to(DEV))
    if shared:
        layer.set_shared((torch.randn(2 * S, H, generator=g) * .1).to(torch.bfloat16).to(DEV),
                         (torch.randn(H, S, generator=g) * .1).to(torch.bfloat16).to(DEV))
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    logits = torch.randn(T, E, generator=g)
    logits[:, 0] = float("-inf")                     # expert 0 is masked for every token
    logits[1, 2:] = float("-inf")                    # one expert left: masked ones fill the slots
    logits[T - 1, :] = float("-inf")                 # none left
    logits = logits.to(DEV)
    forms = [layer.forward] + ([layer.forward_few] if T <= mq.FEW_TOKENS else [])
    clean = [fn(x, logits).clone() for fn in forms]
    ids = [fn(x, logits, return_all=True)["ids"].clone() for fn in forms]
    assert (ids[0][1] == 0).any() and (ids[0][T - 1] == 0).any()
    layer.s13[0].fill_(255)                          # expert 0: every block a NaN
    layer.s2[0].fill_(255)
    own = torch.zeros(H, dtype=torch.bfloat16, device=DEV)
    if shared:
        own = mq.moe_shared_gemm_bf16(mq.moe_shared_gemm_bf16(x, layer.ws13, mq.EPI_SILU_MUL),
                                      layer.ws2)[T - 1]
    for fn, before, i in zip(forms, clean, ids):
        b = fn(x, logits, return_all=True)
        assert torch.equal(b["ids"], ids[0]) and torch.equal(i, ids[0])
        assert b["w"][1].tolist() == [1.0, 0.0, 0.0] and b["w"][T - 1].tolist() == [0.0] * k
        assert torch.isfinite(before).all() and torch.equal(b["y"], before)
        assert torch.equal(b["y"][T - 1], own)
