"""How many columns a tile of few rows on 8-bit weights takes (the rule of csrc/bsr_experts_internal.hpp, compiled for the host): 32 where
tiles of 64 leave CUs idle, where rows start in the same memory channels, and for a long contraction's half-empty last round; and every variant is run by some GPU test, by the rule
with the contraction's length."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT
from test_gpu_fp8_blocks import FP8_PRODUCTS
from test_gpu_fp8_sizes import STREAMED

PROGRAM = r"""
#include <cstdio>
#include "bsr_experts_internal.hpp"
int main() {
    long r, e, n, k;
    while (std::scanf("%ld %ld %ld %ld", &r, &e, &n, &k) == 4)
        std::printf("%d %d %d\n", bsr::best_tile(bsr::kFwdFp8Tiles, r, e, n, k), bsr::few_cols_fp8(1, r, e, n, k), bsr::stream_fp8(1, r, e, n, k));
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("columns")
    (d / "columns.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-O2", "-std=c++17", f"-I{os.path.join(ROOT, 'include')}", f"-I{os.path.join(ROOT, 'sparse_gemm_amd', 'csrc')}",
                    str(d / "columns.cpp"), "-o", str(d / "columns")], check=True)

    def ask(sizes):
        out = subprocess.run([str(d / "columns")], input="".join("%d %d %d %d\n" % s for s in sizes), capture_output=True, text=True,
                             check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return ask


# rows, experts, columns, contraction; the faster number of columns, measured
MEASURED = [(1, 1, 4096, 4096, 32), (1, 1, 8192, 4096, 32), (8, 8, 5120, 4096, 32), (8, 8, 8192, 4096, 32), (8, 8, 14336, 4096, 32),
            (8, 8, 8192, 8192, 32), (64, 64, 1024, 4096, 32), (1, 1, 32768, 4096, 64), (8, 8, 3584, 4096, 64), (64, 64, 512, 4096, 64),
            (8, 8, 14336, 1024, 64), (8, 8, 5120, 2048, 64), (8, 8, 8192, 2048, 64), (60, 60, 1008, 2064, 64), (64, 64, 768, 2048, 64),
            (64, 64, 1280, 2048, 64), (16, 16, 2304, 2560, 64), (8, 8, 14336, 3584, 64),
            (8, 8, 5120, 14336, 32), (8, 8, 5120, 6144, 32), (8, 8, 9728, 4608, 64)]


def test_the_measured_choice(rule):
    got = rule([s[:4] for s in MEASURED])
    assert [cols for _, cols, _ in got] == [s[4] for s in MEASURED]


def test_every_variant_runs_on_the_gpu(rule):
    sizes = [(T * k, E, N, K) for _, T, k, E, N, K in FP8_PRODUCTS] + list(STREAMED)
    assert {(cols, stream) for tile, cols, stream in rule(sizes) if tile == 1} == {(32, 0), (32, 1), (64, 0), (64, 1)}
