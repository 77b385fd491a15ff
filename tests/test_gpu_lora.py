"""The shared projection with low-rank adapters on the GPU against the float64 oracle.

Bounds, derived, with u = 2^-24 and 2 u per term of a sum (truncating or rounding adders alike, in
any order and grouping):
  base      K terms:  2 K u sum |x| |w|
  u         K terms, the scale, the sum of K parts:  2 (K + 4) u sum |x| |A| |scale|, and 2^-17 |u|
            for the two bf16 parts; both times |B|
  delta     2 r terms:  4 r u sum |u| |B|
  together  two more additions:  4 u (|v| + |delta|)
  rounding  bf16: half a step, 2^-8 of the value
  silu(g) h |d silu| <= 1.1 |dg|, so 1.1 dg |h| + |silu(g)| dh + 1.1 dg dh, plus 16 u of the value for
            exp, division and product
"""
import numpy as np
import pytest
import torch

import bit_quantized_moe_top_amd as mq
from oracle import layer as L
from oracle import lora as O
from parity import to_np

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
BF = torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def adapter_ids(M, n, how, seed):
    g = gen(seed)
    if how == "none":
        return torch.full((M,), -1, dtype=torch.int32)
    if how == "one":
        return torch.full((M,), n - 1, dtype=torch.int32)
    ids = torch.randint(-1, n + 1, (M,), generator=g)            # -1 and n: no adapter
    if how == "runs":
        ids = ids[torch.randint(0, max(1, M // 40), (M,), generator=g).sort().values]
    if how == "each":
        ids = torch.arange(M) % n
    return ids.to(torch.int32)


class Case:
    def __init__(self, M, N, K, n, S, r, how="mixed", seed=0, std=0.05):
        g = gen(seed + 7 * M + N + K + r)
        self.x = (torch.randn(M, K, generator=g)).to(BF)
        self.w = (torch.randn(N, K, generator=g) * std).to(BF)
        self.a = (torch.randn(n, S, r, K, generator=g) / max(1, K) ** 0.5).to(BF)
        self.b = (torch.randn(n, N, r, generator=g) * 0.2).to(BF)
        self.scale = torch.randn(n, generator=g)
        self.ids = adapter_ids(M, n, how, seed + M)
        self.n = n

    def run(self, epilogue=mq.EPI_NONE, **kw):
        d = lambda t: t.to(DEV)  # noqa: E731
        plan = kw.pop("plan", None)
        if plan is None:
            plan = mq.moe_adapter_plan(d(self.ids), self.n)
        x = kw.pop("x", None)
        return mq.moe_shared_gemm_lora_bf16(d(self.x) if x is None else x, d(self.w), d(self.a),
                                            d(self.b), d(self.scale), plan, epilogue=epilogue, **kw)

    def reference(self):
        """(v, the bound of its fp32 computation)"""
        K, r = self.x.shape[1], self.a.shape[2]
        v, m = O.project(to_np(self.x), to_np(self.w), to_np(self.a), to_np(self.b),
                         self.scale.double().numpy(), self.ids.numpy())
        d = 2 * K * U * m["base"] + 2 * (K + 4) * U * m["shrink"] + \
            (2.0 ** -17 + 4 * r * U) * m["delta"] + 4 * U * (m["v"] + m["delta"])
        return v, d

    def check(self, got, epilogue, rows=slice(None)):
        v, d = self.reference()
        if epilogue == mq.EPI_SILU_MUL:
            half = v.shape[1] // 2
            g, u, dg, du = v[:, :half], v[:, half:], d[:, :half], d[:, half:]
            v = O.silu_mul(v)
            d = 1.1 * dg * np.abs(u) + np.abs(L.silu(g)) * du + 1.1 * dg * du + 16 * U * np.abs(v)
        got = to_np(got).astype(np.float64)
        assert got.shape == v.shape
        err = np.abs(got - v)[rows]
        assert (err <= (d + 2.0 ** -8 * (np.abs(v) + d))[rows]).all(), err.max()


# M, N, K, adapters, slices, rank: one row; the smallest sizes; K below, at and past a step of 32 and
# 64, and odd multiples of 8; N off every tile; ranks below, at and past a step; rows of one tile, of
# two, of many; more adapters than rows
SHAPES = [
    (1, 16, 8, 1, 1, 8), (1, 32, 64, 4, 2, 16), (3, 192, 256, 2, 1, 8), (2, 64, 40, 3, 2, 32),
    (15, 96, 72, 5, 2, 24), (16, 256, 1024, 16, 2, 16), (17, 160, 104, 40, 1, 40),
    (40, 32, 4096, 3, 1, 64), (63, 2080, 320, 8, 2, 8), (64, 128, 512, 3, 1, 16),
    (65, 1504, 1448, 9, 1, 24), (128, 512, 2048, 6, 2, 16), (130, 96, 200, 7, 2, 64),
    (257, 544, 1032, 60, 2, 48), (300, 528, 136, 20, 1, 256), (600, 320, 448, 4, 1, 128),
    # enough tiles for the larger ones, ragged in every direction
    (260, 8544, 200, 5, 2, 16), (2500, 5408, 136, 4, 2, 24), (1300, 10272, 328, 70, 1, 64),
    (1500, 8736, 48, 3, 2, 8),
    # about as many tiles of 128 as there are CUs: K in halves, whole, odd, with a rest
    (300, 8736, 2248, 30, 2, 24), (513, 5920, 2176, 9, 1, 72), (1024, 4096, 2120, 5, 2, 16),
    (129, 13088, 2112, 40, 2, 136),
    # K past what one launch takes, and off its steps: few rows, and tiles of every size
    (1, 32, 520, 4, 2, 16), (2, 64, 552, 3, 2, 32), (15, 96, 584, 5, 2, 24), (17, 160, 616, 40, 1, 40),
    (63, 2080, 840, 8, 2, 8), (64, 128, 1016, 3, 1, 16), (130, 96, 712, 7, 2, 64), (300, 528, 648, 20, 1, 256),
    (260, 8544, 584, 5, 2, 16), (1500, 8736, 520, 3, 2, 8),
    # tiles of 256 rows and 128 columns: a step of K, none, many; ragged
    (1000, 7232, 200, 5, 2, 16), (770, 6720, 328, 70, 1, 64), (900, 8000, 40, 3, 1, 8), (1800, 3872, 1096, 6, 2, 40),
    # one launch: K at, below and above 32 and 256; an adapter in every row, and one; pieces of ranks
    # that two slices share; rows and columns off its blocks
    (16, 64, 256, 16, 1, 8), (33, 96, 248, 3, 2, 16), (5, 1040, 256, 5, 1, 16), (200, 336, 200, 8, 1, 8),
    (90, 64, 24, 1, 1, 128), (1, 16, 256, 70, 1, 128), (700, 160, 32, 2, 2, 24), (31, 48, 8, 8, 1, 16),
    (2, 4096, 128, 900, 2, 32), (16, 32, 264, 2, 2, 8),
]


@pytest.mark.parametrize("M,N,K,n,S,r", SHAPES)
@pytest.mark.parametrize("how", ["mixed", "runs", "none", "one", "each"])
def test_shapes(M, N, K, n, S, r, how):
    c = Case(M, N, K, n, S, r, how)
    for epilogue in (mq.EPI_NONE, mq.EPI_SILU_MUL) if N % 32 == 0 else (mq.EPI_NONE,):
        got = c.run(epilogue)
        c.check(got, epilogue)
        assert torch.equal(got, c.run(epilogue))                 # the same bits again


@pytest.mark.parametrize("M,K", [(70, 136), (70, 520), (20, 520)])
def test_integers_are_exact(M, K):
    """Small integers: every sum is exact in fp32, u in two bf16 parts, and the result in bf16."""
    g = gen(3)
    c = Case(M, 96, K, 5, 1, 16)
    c.x = torch.randint(-2, 3, c.x.shape, generator=g).to(BF)
    c.x[:, 128:K - 8] = 0
    c.w = torch.randint(-1, 2, c.w.shape, generator=g).to(BF)
    c.a = torch.randint(-1, 2, c.a.shape, generator=g).to(BF)
    c.b = (torch.rand(c.b.shape, generator=g) < 0.1).to(BF)
    c.scale = torch.tensor([1.0, -1.0, 2.0, 0.5, 0.0])
    v, _ = O.project(to_np(c.x), to_np(c.w), to_np(c.a), to_np(c.b), c.scale.numpy(), c.ids.numpy())
    assert np.abs(v).max() < 256 and (v * 2 == np.round(v * 2)).all()
    exact = np.abs(v) <= 128                                      # halves need 9 bits above that
    np.testing.assert_array_equal(to_np(c.run())[exact], v[exact])


@pytest.mark.parametrize("M,K", [(20, 64), (20, 584), (200, 584)])
def test_u_keeps_sixteen_bits(M, K):
    """Two ranks whose parts cancel but for 2^-12 of themselves: a u in one bf16 value (2^-9) would
    lose what is left."""
    N, r = 32, 8
    c = Case(M, N, K, 1, 1, r, how="one")
    g = gen(4)
    c.x = (torch.rand(M, K, generator=g) + 0.5).to(BF)
    c.x[:, 1] = c.x[:, 0] * 0 + 2.0 ** -12
    c.w.zero_()
    c.a.zero_()
    c.a[0, 0, 0, 0] = c.a[0, 0, 1, 0] = c.a[0, 0, 0, 1] = 1.0     # u0 = x0 + 2^-12, u1 = x0
    c.b.zero_()
    c.b[0, :, 0], c.b[0, :, 1] = 1.0, -1.0
    c.scale.fill_(1.0)
    got = to_np(c.run()).astype(np.float64)
    x0 = to_np(c.x)[:, :1].astype(np.float64)
    assert (np.abs(got - 2.0 ** -12) <= 2.0 ** -17 * (2 * x0 + 2.0 ** -12) + 2.0 ** -20).all()


@pytest.mark.parametrize("M,K", [(18, 16), (18, 520), (90, 520)])
def test_u_up_to_the_largest_fp32(M, K):
    """u = 1.9989 * 2^127, finite in fp32 and past bf16's largest value, of either sign."""
    N = 32
    c = Case(M, N, K, 1, 1, 8, how="one")
    c.x = torch.zeros(M, K, dtype=BF)
    c.x[:, 0] = 1 - 2 * (torch.arange(M) % 2)
    c.x[:, 1] = c.x[:, 0] * 2.0 ** -8
    c.w.zero_()
    c.a.zero_()
    c.a[0, 0, 0, 0], c.a[0, 0, 0, 1] = 1.9921875 * 2.0 ** 63, 1.75 * 2.0 ** 63
    c.b.zero_()
    c.b[0, :, 0] = 2.0 ** -100
    c.scale.fill_(2.0 ** 64)
    u = (1.9921875 + 1.75 / 256) * 2.0 ** 127
    assert u < np.finfo(np.float32).max
    ref = to_np(c.x)[:, :1].astype(np.float64) * u * 2.0 ** -100
    got = to_np(c.run()).astype(np.float64)
    assert (np.abs(got - ref) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(ref)).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("M,N,K,how", [(40, 96, 136, "mixed"), (200, 64, 64, "runs"), (12, 512, 1024, "each"),
                                         (40, 96, 520, "mixed"), (200, 64, 520, "runs"), (700, 2144, 520, "runs")])
def test_a_broken_adapter_or_row_spoils_only_its_own(M, N, K, how, bad):
    c = Case(M, N, K, 6, 1, 16, how)
    for epilogue in (mq.EPI_NONE, mq.EPI_SILU_MUL):
        clean = c.run(epilogue)
        for part in ("a", "b", "scale", "x"):
            k = Case(M, N, K, 6, 1, 16, how)
            own = k.ids == 2
            if part == "x":
                own = torch.zeros(M, dtype=torch.bool)
                own[3] = True
                k.x[3, 5] = bad
            elif part == "scale":
                k.scale[2] = bad
            else:
                getattr(k, part)[2] = bad
            got = k.run(epilogue)
            keep = ~own.to(DEV)
            assert torch.equal(got[keep], clean[keep]), part
            if own.any():
                assert not torch.isfinite(got[own.to(DEV)]).all(), part


@pytest.mark.parametrize("M,N,K,pad", [(1, 64, 72, 8), (5, 64, 72, 8), (100, 160, 1024, 56), (300, 96, 136, 24),
                                         (5, 64, 584, 8), (300, 96, 328, 24)])
def test_rows_of_a_wider_matrix_and_bytes_around(M, N, K, pad):
    c = Case(M, N, K, 4, 2, 8)
    wide = torch.full((M, K + pad), float("nan"), dtype=BF)
    wide[:, :K] = c.x
    need = mq.moe_shared_gemm_lora_ws_size(M, N, K, 4, 2, 8)
    for epilogue in (mq.EPI_NONE, mq.EPI_SILU_MUL):
        cols = N // 2 if epilogue else N
        bufs = {n: torch.full((512 + b + 512,), 0xA5, dtype=torch.uint8, device=DEV)
                for n, b in (("out", 2 * M * cols), ("ws", need))}
        out = bufs["out"][512:512 + 2 * M * cols].view(BF).view(M, cols)
        got = c.run(epilogue, x=wide.to(DEV)[:, :K], out=out, ws=bufs["ws"][512:512 + need])
        assert got.data_ptr() == out.data_ptr()
        assert torch.equal(got, c.run(epilogue))
        for n, t in bufs.items():
            assert (t[:512] == 0xA5).all() and (t[-512:] == 0xA5).all(), n


@pytest.mark.parametrize("M", [1, 64, 1000, 1024, 1025, 5000, 20000])
@pytest.mark.parametrize("n", [1, 5, 1023])
def test_plan(M, n):
    ids = adapter_ids(M, n, "mixed", M + n)
    ids[::7] = 2 ** 31 - 1
    ids[::11] = -2 ** 31
    plan = mq.moe_adapter_plan(ids.to(DEV), n)
    moved = torch.where((ids < 0) | (ids >= n), torch.tensor(n, dtype=torch.int32), ids)
    ref, _, _ = mq.moe_permute(moved.view(-1, 1).to(DEV), n + 1)
    f, g = mq.plan_fields(plan, n + 1, M), mq.plan_fields(ref, n + 1, M)
    nt, na = int(g["header"][3]), int(g["header"][2])
    for name in f:
        k = {"tile_expert": nt, "tile_row0": nt, "active": na, "scratch": 0}.get(name, len(f[name]))
        assert torch.equal(f[name][:k], g[name][:k]), name
    o = O.adapter_plan(ids.numpy(), n)
    np.testing.assert_array_equal(f["sorted_rows"].cpu().numpy(), o["sorted_rows"])


def test_no_rows_and_refusals():
    c = Case(6, 64, 64, 3, 1, 8)
    e = Case(6, 64, 64, 3, 1, 8)
    e.x, e.ids = e.x[:0], e.ids[:0]
    assert e.run().shape == (0, 64) and e.run(mq.EPI_SILU_MUL).shape == (0, 32)
    plan = mq.moe_adapter_plan(c.ids.to(DEV), 3)
    with pytest.raises(ValueError, match="built for"):
        c.run(plan=mq.moe_adapter_plan(c.ids.to(DEV), 4))
    with pytest.raises(ValueError, match="out"):
        c.run(plan=plan, out=torch.empty(6, 32, dtype=BF, device=DEV))
    with pytest.raises(mq.MoeqError, match="workspace"):
        c.run(plan=plan, ws=torch.empty(0, dtype=torch.uint8, device=DEV).new_empty(16))
    with pytest.raises(ValueError, match="contiguous rows"):
        c.run(plan=plan, x=c.x.to(DEV).t().contiguous().t())
    with pytest.raises(ValueError, match="contiguous rows"):
        c.run(plan=plan, x=c.x[0].to(DEV).expand(6, 64))
    with pytest.raises(mq.MoeqError):
        c.run(plan=plan, x=torch.zeros(6, 68, dtype=BF, device=DEV)[:, :64])      # row stride 68
    with pytest.raises(mq.MoeqError):
        c.run(plan=plan, epilogue=7)
    with pytest.raises(ValueError, match="adapters"):
        mq.moe_adapter_plan(c.ids.to(DEV), 0)
    with pytest.raises(mq.MoeqError, match="workspace"):
        mq.moe_adapter_plan(c.ids.to(DEV), 3, plan=torch.empty(4, dtype=torch.int32, device=DEV))
    for name, t in (("w", c.w[:, :56]), ("b", c.b[:2]), ("b", c.b[:, :32]), ("scale", c.scale[:2]),
                    ("a", c.a[..., :56])):
        k = Case(6, 64, 64, 3, 1, 8)
        setattr(k, name, t.contiguous())
        with pytest.raises(ValueError, match="match"):
            k.run(plan=plan)


@pytest.mark.parametrize("M", [4, 90, 700])
def test_captured_and_replayed(M):
    """Plan and projections in one graph; other rows and other adapters in every replay."""
    N, K, n = 256, 512, 9
    g = gen(M)
    c, d = Case(M, N, K, n, 2, 16), Case(M, K, N // 2, n, 1, 16)
    up = [t.to(DEV) for t in (c.w, c.a, c.b, c.scale)]
    down = [t.to(DEV) for t in (d.w, d.a, d.b, d.scale)]
    x, ids = c.x.to(DEV), c.ids.to(DEV)
    plan = mq.moe_adapter_plan(ids, n)
    bufs = {k: torch.empty(s, dtype=torch.uint8, device=DEV) for k, s in
            (("up", mq.moe_shared_gemm_lora_ws_size(M, N, K, n, 2, 16)),
             ("down", mq.moe_shared_gemm_lora_ws_size(M, K, N // 2, n, 1, 16)))}
    h = torch.empty(M, N // 2, dtype=BF, device=DEV)
    y = torch.empty(M, K, dtype=BF, device=DEV)

    def step():
        mq.moe_adapter_plan(ids, n, plan=plan)
        mq.moe_shared_gemm_lora_bf16(x, *up, plan, mq.EPI_SILU_MUL, out=h, ws=bufs["up"])
        return mq.moe_shared_gemm_lora_bf16(h, *down, plan, out=y, ws=bufs["down"])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(4):
        x.copy_(torch.randn(M, K, generator=g).to(BF))
        ids.copy_(adapter_ids(M, n, "mixed" if rep % 2 else "runs", rep))
        expect = step().clone()
        for t in (h, y, *bufs.values()):
            t.view(torch.uint8).fill_(0x7F)
        plan.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, expect), rep


def test_two_streams_with_their_own_workspaces():
    cases = [Case(30, 512, 1024, 8, 2, 16), Case(200, 256, 512, 5, 1, 32)]
    refs = [c.run() for c in cases]
    args = [[t.to(DEV) for t in (c.x, c.w, c.a, c.b, c.scale)] for c in cases]
    plans = [mq.moe_adapter_plan(c.ids.to(DEV), c.n) for c in cases]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(10):
        for s, a, p in zip(streams, args, plans):
            with torch.cuda.stream(s):
                outs.append(mq.moe_shared_gemm_lora_bf16(*a, p))
    torch.cuda.synchronize()
    for i, got in enumerate(outs):
        assert torch.equal(got, refs[i % 2])


def test_a_plan_of_zeros_stays_inside():
    """A plan that some other write cleared gives wrong values, no access outside the buffers."""
    c = Case(100, 96, 128, 4, 1, 8)
    plan = torch.zeros(mq.moe_plan_size(5, 100) // 4, dtype=torch.int32, device=DEV)
    got = c.run(plan=plan)
    assert got.shape == (100, 96)
    torch.cuda.synchronize()


@pytest.mark.parametrize("M", [3, 70])
def test_offsets_past_32_bits(M):
    """Adapters, and rows of a, that lie more than 2^32 bytes (and elements) from their tensor's start:
    as the same adapters and rows in small tensors."""
    n, N, K, r = 600, 16384, 16384, 256
    g = torch.Generator(device=DEV).manual_seed(M)
    rnd = lambda *s: (torch.randn(*s, generator=g, device=DEV) / 64).to(BF)  # noqa: E731
    used = [0, 417, n - 1]
    big_a = torch.empty(n, 1, r, K, dtype=BF, device=DEV)
    big_b = torch.empty(n, N, r, dtype=BF, device=DEV)
    assert big_a[-1].data_ptr() - big_a.data_ptr() > 2 ** 32 < big_b[-1].data_ptr() - big_b.data_ptr()
    for l in used:
        big_a[l], big_b[l] = rnd(1, r, K), rnd(N, r)
    w, scale = rnd(N, K), torch.rand(n, generator=g, device=DEV) + 0.5
    ld = 2 ** 33 // M // 8 * 8
    a = torch.empty(M * ld, dtype=BF, device=DEV).view(M, ld)[:, :K]
    a.copy_(rnd(M, K))
    which = torch.arange(M, device=DEV) % 4
    ids = torch.tensor(used + [-1], dtype=torch.int32, device=DEV)[which]
    got = mq.moe_shared_gemm_lora_bf16(a, w, big_a, big_b, scale, mq.moe_adapter_plan(ids, n))
    few = torch.tensor([0, 1, 2, -1], dtype=torch.int32, device=DEV)[which]
    ref = mq.moe_shared_gemm_lora_bf16(a.contiguous(), w, big_a[used], big_b[used], scale[used],
                                       mq.moe_adapter_plan(few, 3))
    assert got.abs().max() > 0
    assert torch.equal(got, ref)
