"""Which kernel variant a product grouped by expert takes, without a GPU: the rules of csrc/bsr_experts_internal.hpp, compiled for
the host. Every variant that the launchers hold is taken by some size, and by some size that a GPU test runs."""
import os
import random
import shutil
import subprocess

import pytest

from conftest import ROOT
from test_gpu_experts import LARGE, PRODUCTS, WIDE
from test_gpu_mx4 import MX_PRODUCTS

# (rows, columns) of the tiles that the launchers can start
FWD = {(16, 32), (32, 32), (64, 32), (128, 128), (256, 256)}
BWD_INPUT = {(16, 32), (16, 64), (32, 64), (64, 64), (128, 128), (256, 256)}
FWD_MX4 = {(16, 32), (16, 64), (32, 64), (128, 128)}

PROGRAM = r"""
#include <cstdio>
#include "bsr_experts_internal.hpp"
template <int n>
void ids(char kind, const bsr::TileKind (&kinds)[n]) {
    for (int i = 0; i < n; ++i) std::printf("%c %d\n", kind, kinds[i].id <= 4 ? 16 * kinds[i].id : kinds[i].id);
}
int main(int argc, char **) {
    if (argc > 1) {
        ids('f', bsr::kFwdTiles), ids('b', bsr::kBwdInputTiles), ids('m', bsr::kFwdMx4Tiles);
        return 0;
    }
    char kind;
    long R, E, N, K;
    while (std::scanf(" %c %ld %ld %ld %ld", &kind, &R, &E, &N, &K) == 5) {
        int id, rows, cols;
        if (kind == 'f') {
            id = bsr::best_tile(bsr::kFwdTiles, R, E, N, K);
            cols = id <= 4 ? 32 : id;
        } else if (kind == 'b') {
            id = bsr::best_tile(bsr::kBwdInputTiles, R, E, K, N);
            cols = id <= 4 ? bsr::few_cols_bwd_input(id, R, E, K) : id;
        } else {
            id = bsr::best_tile(bsr::kFwdMx4Tiles, R, E, N, K);
            cols = id <= 4 ? bsr::few_cols_mx4(id, R, E, N) : id;
        }
        rows = id <= 4 ? 16 * id : id;
        std::printf("%d %d\n", rows, cols);
    }
}
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("tiles")
    src, exe = d / "tiles.cpp", d / "tiles"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-O2", "-std=c++17", f"-I{os.path.join(ROOT, 'include')}",
                    f"-I{os.path.join(ROOT, 'sparse_gemm_amd', 'csrc')}", str(src), "-o", str(exe)], check=True)

    def ask(kind, sizes):
        text = "".join(f"{kind} {R} {E} {N} {K}\n" for R, E, N, K in sizes)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    ask.table = [line.split() for line in subprocess.run([str(exe), "table"], capture_output=True, text=True).stdout.splitlines()]
    return ask


def some_sizes(n, step):
    rng = random.Random(0)
    log = lambda top: int(round(2.0 ** rng.uniform(0.0, top)))   # noqa: E731
    return [(log(22), log(10), 8 * log(13), step * log(13)) for _ in range(n)]


@pytest.mark.parametrize("kind,step,variants", [("f", 8, FWD), ("b", 8, BWD_INPUT), ("m", 32, FWD_MX4)])
def test_every_variant_is_taken(tiles, kind, step, variants):
    """1 to 2^22 rows, 1 to 1024 experts, widths from one 16-byte piece to 65536."""
    assert set(tiles(kind, some_sizes(200000, step))) == variants
    assert {int(rows) for k, rows in tiles.table if k == kind} == {rows for rows, _ in variants}


def test_every_variant_runs_on_the_gpu(tiles):
    sizes = lambda cases: [(T * k, E, N, K) for _, T, k, E, N, K in cases]   # noqa: E731
    swapped = [(kind, T, k, E, K, N) for kind, T, k, E, N, K in WIDE]
    assert set(tiles("f", sizes(PRODUCTS + LARGE + WIDE))) == FWD
    assert set(tiles("b", sizes(PRODUCTS + LARGE + swapped))) == BWD_INPUT
    assert set(tiles("m", sizes(MX_PRODUCTS))) == FWD_MX4


def test_halved_tiles_are_tested(tiles):
    """The GPU test of halved tiles takes sizes whose products run in 256 x 256 tiles, in both directions."""
    from test_gpu_expert_halves import HALVES, ONE_EXPERT
    assert set(tiles("f", [(T * k, E, N, K) for _, T, k, E, N, K in HALVES + ONE_EXPERT])) == {(256, 256)}
    assert set(tiles("b", [(T * k, E, K, N) for _, T, k, E, N, K in HALVES])) == {(256, 256)}
