"""The shared projection with adapters on the paths that the shapes of test_gpu_lora.py do not take:
products and joins in parts, the largest tiles whole, u in few and in many parts.  Bounds as there."""
import pytest
import torch

import bit_quantized_moe_top_amd as mq
from test_gpu_lora import BF, DEV, Case, adapter_ids, gen

pytestmark = pytest.mark.gpu

# M, N, K, adapters, slices, rank; columns and K off the tiles, K with and without a rest of a slot
PATH_SHAPES = [
    # 128 x 128 tiles with K in four parts, joined by 64 x 64 tiles and by rows
    (130, 4384, 2120, 7, 2, 24), (200, 4384, 2072, 9, 1, 72), (130, 4128, 2120, 7, 2, 24),
    # in two
    (400, 4224, 2056, 30, 2, 16), (300, 5504, 2088, 5, 1, 40), (129, 8096, 2056, 6, 2, 16),
    # 64 x 64 tiles with K in two parts, joined by rows and by tiles, and in four, most of them empty
    (129, 2176, 520, 5, 1, 40), (1100, 832, 2056, 20, 2, 24), (90, 544, 72, 5, 2, 24),
    # whole tiles of 128 and of 64
    (1100, 6720, 136, 4, 1, 16), (1100, 6720, 72, 4, 2, 40), (1300, 704, 264, 4, 2, 40), (1300, 704, 264, 4, 2, 16),
    # one tile of 128 rows and very many columns, whole and by groups; one of 256
    (100, 33056, 72, 5, 2, 16), (72, 16672, 136, 4, 1, 24), (250, 16672, 72, 9, 1, 16),
    # u in one part for more than 4096 rows; few rows with several pieces of K in a part of u
    (4200, 96, 264, 5, 1, 16), (5, 64, 8712, 3, 2, 16), (40, 96, 16456, 50, 1, 40),
]


@pytest.mark.parametrize("M,N,K,n,S,r", PATH_SHAPES)
@pytest.mark.parametrize("how", ["mixed", "runs"])
def test_path_shapes(M, N, K, n, S, r, how):
    c = Case(M, N, K, n, S, r, how)
    for epilogue in (mq.EPI_NONE, mq.EPI_SILU_MUL):
        got = c.run(epilogue)
        c.check(got, epilogue)
        assert torch.equal(got, c.run(epilogue))                 # the same bits again


@pytest.mark.parametrize("M,N,K,n,S,r", [s for s in PATH_SHAPES if s[1] * s[2] < 2 ** 23])
def test_bytes_around_and_rows_of_a_wider_matrix(M, N, K, n, S, r):
    c = Case(M, N, K, n, S, r)
    wide = torch.full((M, K + 24), float("nan"), dtype=BF)
    wide[:, :K] = c.x
    need = mq.moe_shared_gemm_lora_ws_size(M, N, K, n, S, r)
    for epilogue in (mq.EPI_NONE, mq.EPI_SILU_MUL):
        cols = N // 2 if epilogue else N
        bufs = {k: torch.full((512 + b + 512,), 0xA5, dtype=torch.uint8, device=DEV)
                for k, b in (("out", 2 * M * cols), ("ws", need))}
        out = bufs["out"][512:512 + 2 * M * cols].view(BF).view(M, cols)
        got = c.run(epilogue, x=wide.to(DEV)[:, :K], out=out, ws=bufs["ws"][512:512 + need])
        assert torch.equal(got, c.run(epilogue))
        for k, t in bufs.items():
            assert (t[:512] == 0xA5).all() and (t[-512:] == 0xA5).all(), k


@pytest.mark.parametrize("M,N,K", [(130, 4384, 2120), (400, 4224, 2056), (129, 8096, 2056), (129, 2176, 520),
                                   (1100, 832, 2056), (1100, 6720, 136), (40, 96, 8712)])
def test_a_broken_adapter_spoils_only_its_own(M, N, K):
    for epilogue in (mq.EPI_NONE, mq.EPI_SILU_MUL):
        clean = Case(M, N, K, 6, 1, 16).run(epilogue)
        for part in ("a", "b", "scale"):
            k = Case(M, N, K, 6, 1, 16)
            getattr(k, part)[2] = float("nan")
            got, own = k.run(epilogue), (k.ids == 2).to(DEV)
            assert torch.equal(got[~own], clean[~own]), part
            assert not torch.isfinite(got[own]).any(), part


@pytest.mark.parametrize("M,N,K,n,S,r", [(10, 96, 520, 4, 1, 8), (40, 96, 8712, 4, 1, 40), (100, 96, 520, 4, 1, 8)] +
                         [s for s in PATH_SHAPES if s[0] > 64])
def test_a_plan_of_zeros_stays_inside_on_every_path(M, N, K, n, S, r):
    """A plan that some other write cleared gives wrong values, no access outside the buffers: no row
    but the first is written."""
    c = Case(M, N, K, n, S, r)
    plan = torch.zeros(mq.moe_plan_size(n + 1, M) // 4, dtype=torch.int32, device=DEV)
    for epilogue in (mq.EPI_NONE, mq.EPI_SILU_MUL):
        out = torch.full((M, N // 2 if epilogue else N), 7.0, dtype=BF, device=DEV)
        c.run(epilogue, plan=plan, out=out)
        assert (out[1:] == 7.0).all()
    torch.cuda.synchronize()


@pytest.mark.parametrize("M,N,K,n", [(130, 4384, 2120, 9), (400, 4224, 2056, 30), (129, 2176, 520, 5),
                                     (40, 96, 8712, 9)])
def test_captured_and_replayed_in_parts(M, N, K, n):
    """Rows, adapters and the workspace's contents new in every replay."""
    g = gen(M)
    c = Case(M, N, K, n, 1, 16)
    weights = [t.to(DEV) for t in (c.w, c.a, c.b, c.scale)]
    x, ids = c.x.to(DEV), c.ids.to(DEV)
    plan = mq.moe_adapter_plan(ids, n)
    ws = torch.empty(mq.moe_shared_gemm_lora_ws_size(M, N, K, n, 1, 16), dtype=torch.uint8, device=DEV)
    y = torch.empty(M, N, dtype=BF, device=DEV)

    def step():
        mq.moe_adapter_plan(ids, n, plan=plan)
        return mq.moe_shared_gemm_lora_bf16(x, *weights, plan, out=y, ws=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(3):
        x.copy_(torch.randn(M, K, generator=g).to(BF))
        ids.copy_(adapter_ids(M, n, "runs" if rep % 2 else "mixed", rep))
        expect = step().clone()
        ws.fill_(0x7F)
        y.fill_(float("nan"))
        plan.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, expect), rep
