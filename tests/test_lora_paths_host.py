"""Which kernels the shared projection with adapters takes for a shape (csrc/lora_paths.hpp, which is
host code), and that the GPU tests compare every one of them with the oracle (no GPU)."""
import itertools
import os
import random
import shutil
import subprocess

import pytest

import bit_quantized_moe_top_amd as mq
from test_gpu_lora import SHAPES
from test_gpu_lora_paths import PATH_SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which(os.environ.get("CXX", "g++"))
PROGRAM = r"""
#include <stdio.h>
#include "%s/bit_quantized_moe_top_amd/csrc/lora_paths.hpp"
int main() {
  moeq::LoraShape s = {};
  while (scanf("%%d %%d %%d %%d %%d %%d %%d", &s.M, &s.N, &s.K, &s.L, &s.slices, &s.r, &s.epilogue) == 7) {
    s.ld_a = s.K;
    const moeq::LoraPath p = moeq::lora_path(s);
    printf("%%d %%d %%d %%d %%d %%d %%d %%d %%d %%d %%zu %%zu %%zu\n", p.one_launch, p.few, p.bm, p.bn, p.groups,
           p.splits, p.slots, p.u_splits, p.u_pieces, p.join_rows, p.u_bytes, p.part_bytes, p.ws_bytes());
  }
}
"""


@pytest.fixture(scope="module")
def paths(tmp_path_factory):
    """[(M, N, K, L, slices, r, epilogue)] -> the fields of their LoraPath."""
    if CXX is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("paths")
    src, exe = d / "paths.cpp", d / "paths"
    src.write_text(PROGRAM % ROOT)
    subprocess.run([CXX, "-std=c++17", "-O1", "-Wall", "-Werror", str(src), "-o", str(exe)], check=True)
    names = ("one_launch", "few", "bm", "bn", "groups", "splits", "slots", "u_splits", "u_pieces",
             "join_rows", "u_bytes", "part_bytes", "ws_bytes")

    def ask(shapes):
        text = "\n".join(" ".join(str(v) for v in s) for s in shapes)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        got = [dict(zip(names, map(int, line.split()))) for line in out.splitlines()]
        assert len(got) == len(shapes)
        return got
    return ask


def labels(shape, p):
    """The kernels, by what their launch is compiled for, and the ways through them."""
    M, _, _, _, _, r, epilogue = shape
    rank = "r<=32" if r <= 32 else "r>32"
    if p["one_launch"]:
        return {("short", epilogue)}
    if p["few"]:
        rows = 1 if M <= 16 else 2 if M <= 32 else 4
        return {("few", rows), ("few u", "one piece" if p["u_pieces"] == 1 else "more"),
                ("few join", epilogue, rank)}
    tile = (p["bm"], p["bn"], p["groups"])
    found = {("shrink", p["u_splits"])}
    if p["splits"] == 1:
        return found | {("tile", tile, epilogue, rank)}
    join = ("join rows", epilogue, rank) if p["join_rows"] else ("join tiles", epilogue, rank)
    return found | {("parts", tile, p["splits"], p["join_rows"]), join}


def with_epilogues(shapes):
    return [s + (e,) for s in shapes for e in ((0, 1) if s[1] % 32 == 0 else (0,))]


def test_every_path_is_compared_with_the_oracle(paths):
    rng = random.Random(1)
    rows = list(range(1, 80)) + [96, 128, 129, 160, 200, 256, 257, 300, 400, 513, 640, 777, 1000, 1500, 2048,
                                 3000, 4096, 4097, 6000, 9000]
    columns = [32 * n for n in (1, 2, 3, 8, 17, 30, 32, 47, 64, 96, 128, 160, 200, 256, 300, 400, 512, 640, 1024)]
    depths = [8, 64, 256, 264, 1024, 1448, 2048, 2056, 4096, 8192, 8200, 9000, 16384]
    drawn = [(M, N, rng.choice(depths), rng.choice((1, 5, 60)), rng.choice((1, 2)), r, e)
             for M, N, r, e in itertools.product(rows, columns, (8, 32, 64, 256), (0, 1))]
    reached, tested = set(), set()
    for s, p in zip(drawn, paths(drawn)):
        reached |= labels(s, p)
    mine = with_epilogues(SHAPES + PATH_SHAPES)
    for s, p in zip(mine, paths(mine)):
        tested |= labels(s, p)
    assert len(reached) >= 30
    assert reached <= tested, sorted(map(str, reached - tested))


def test_workspace_holds_what_the_launches_write(paths):
    """u's parts, then the product's: as many as the launches are given, and the size that the library
    answers, which no epilogue changes."""
    rng = random.Random(2)
    shapes = [(rng.choice((1, 5, 16, 17, 33, 64, 65, 100, 128, 250, 300, 700, 1024, 2048, 5000)),
               32 * rng.randint(1, 400), 8 * rng.randint(1, 1200), rng.randint(1, 1023), rng.choice((1, 2)),
               8 * rng.randint(1, 32)) for _ in range(2000)]
    both = [paths([s + (e,) for s in shapes]) for e in (0, 1)]
    for s, p, q in zip(shapes, *both):
        M, N, K, L, S, r = s
        assert p["ws_bytes"] == q["ws_bytes"] == mq.moe_shared_gemm_lora_ws_size(*s)
        assert p["ws_bytes"] >= p["u_bytes"] + p["part_bytes"]
        assert p["u_bytes"] % 256 == 0 and p["u_bytes"] >= 4 * p["u_splits"] * M * S * r
        if p["few"]:
            assert M <= 64 and p["splits"] * p["slots"] >= K // 64 > 0 or K < 64
            assert p["u_splits"] * p["u_pieces"] * 512 >= K
        else:
            assert M > 64 and p["splits"] <= 4 and p["u_splits"] <= 4
        if p["few"] or p["splits"] > 1:
            assert p["part_bytes"] >= 4 * p["splits"] * (-(-M // 16) * 16) * N


def test_tiles_follow_the_rows_that_there_are(paths):
    """No tile of 256 rows for up to 128; no split of K past one go of whole tiles of 128; whole
    halves by groups, not splits, for rows of one tile."""
    for M, N, K in ((65, 20480, 4096), (100, 32768, 1024), (128, 40960, 4096), (128, 1 << 18, 520), (72, 1 << 20, 520)):
        assert paths([(M, N, K, 5, 1, 16, 0)])[0]["bm"] <= 128, (M, N, K)
    for M, N, K in ((256, 18432, 4096), (256, 16640, 4096), (512, 9216, 4096), (768, 6144, 4096), (100, 36864, 4096),
                    (300, 19456, 4096), (600, 12800, 1024)):
        p = paths([(M, N, K, 5, 1, 16, 0)])[0]
        assert p["splits"] == p["groups"] == 1 and (p["bm"], p["bn"]) in ((128, 128), (256, 128)), (M, N, K, p)
    for M, N, K in ((72, 20480, 4096), (128, 17408, 4096), (512, 7168, 1024), (512, 4224, 2048), (300, 9728, 4096)):
        assert paths([(M, N, K, 5, 1, 16, 0)])[0]["groups"] == 2, (M, N, K)
    for M, N, K, bm, bn, groups, splits in ((2048, 8192, 4096, 256, 256, 1, 1), (1024, 8192, 4096, 256, 128, 1, 1),
                                            (512, 8192, 4096, 128, 128, 2, 1), (256, 8192, 4096, 128, 128, 1, 2),
                                            (128, 8192, 4096, 128, 128, 1, 4), (777, 1504, 1448, 64, 64, 1, 1),
                                            (128, 2048, 4096, 64, 64, 1, 4)):
        p = paths([(M, N, K, 5, 1, 16, 0)])[0]
        assert (p["bm"], p["bn"], p["groups"], p["splits"]) == (bm, bn, groups, splits), (M, N, K, p)
