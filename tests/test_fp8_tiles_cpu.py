"""Which kernels the products on 8-bit weights and the whole layer for few tokens take, without a GPU: the rules of
csrc/bsr_experts_internal.hpp, compiled for the host. Every variant is taken by some size, and by some size that a GPU test runs."""
import os
import random
import shutil
import subprocess

import pytest

from conftest import ROOT
from test_gpu_expert_ffn import CASES, STEP, STREAMED, WIDE_CASES
from test_gpu_fp8_blocks import FP8_PRODUCTS
from test_gpu_fp8_sizes import STREAMED as LARGE_PRODUCTS

# rows and columns of a tile, weights streamed
BF16_ACT = {(16, 32, 0), (16, 32, 1), (16, 64, 0), (16, 64, 1), (32, 64, 0), (64, 64, 0), (128, 128, 0)}
FP8_ACT = {(128, 128, 0), (128, 128, 1), (256, 256, 0)}
VALUES = {"bf16": 64, "mx4": 256, "fp8": 128}   # of a line
# few, span, q, waves, wide, rs
LAYER = {(few, *v) for few in (0, 1) for v in ((128, 1, 16, 1, 2), (256, 1, 16, 0, 1), (256, 1, 16, 0, 2), (128, 2, 4, 0, 1),
                                               (128, 2, 8, 0, 1), (128, 2, 16, 0, 1))}
# the same by kernel: few, up product, streamed; few, rs, tiles shared, streamed
UP = {(few, up, stream) for few in (0, 1) for up in ("wide", "one", "two") for stream in (0, 1)}
DOWN = {(few, rs, split, stream) for few in (0, 1) for rs, split in ((2, 0), (1, 0), (1, 1)) for stream in (0, 1)}


def up_of(got):
    return {(few, "wide" if wide else "two" if q == 2 else "one", stream) for few, _, q, _, wide, _, _, stream, _ in got}


def down_of(got):
    return {(few, rs, split, stream) for few, _, _, _, _, rs, split, _, stream in got}


PROGRAM = r"""
#include <cstdio>
#include "bsr_experts_internal.hpp"
int main() {
    char kind;
    long a, b, c, d, e, f;
    while (std::scanf(" %c %ld %ld %ld %ld %ld %ld", &kind, &a, &b, &c, &d, &e, &f) == 7) {
        if (kind == 'b') {
            const int id = bsr::best_tile(bsr::kFwdFp8Tiles, a, b, c, d);
            std::printf("%d %d %d\n", id <= 4 ? 16 * id : id, id <= 4 ? bsr::few_cols_fp8(id, a, b, c) : id, id == 1 && bsr::stream_fp8(1, a, b, c, d));
        } else if (kind == 'f') {
            const int bm = bsr::wide_fp8(a, b, c, d) ? 256 : 128;
            std::printf("%d %d %d\n", bm, bm, bm == 128 && bsr::stream_fp8(4, a, b, c, d));
        } else {
            const bsr::FfnVariant v = bsr::ffn_variant(a, b, c, d, e, f);
            std::printf("%d %d %d %d %d %d %d %d %d\n", v.few, v.span, v.q, v.waves, v.wide, v.rs, v.splits > 1, v.stream_up, v.stream_down);
        }
    }
}
"""


@pytest.fixture(scope="module")
def variants(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("variants")
    src, exe = d / "variants.cpp", d / "variants"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-O2", "-std=c++17", f"-I{os.path.join(ROOT, 'include')}",
                    f"-I{os.path.join(ROOT, 'sparse_gemm_amd', 'csrc')}", str(src), "-o", str(exe)], check=True)

    def ask(kind, sizes):
        text = "".join(f"{kind} {' '.join(map(str, (*s, 0, 0)[:6]))}\n" for s in sizes)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return {tuple(map(int, line.split())) for line in out.splitlines()}

    return ask


def some(n, f):
    rng = random.Random(0)
    return [f(lambda top: int(round(2.0 ** rng.uniform(0.0, top)))) for _ in range(n)]


def test_every_variant_is_taken(variants):
    products = some(100000, lambda log: (log(22), log(10), 8 * log(13), 16 * log(13)))
    assert variants("b", products) == BF16_ACT
    assert variants("f", products) == FP8_ACT
    for values in VALUES.values():
        layers = some(100000, lambda log: (values, log(4), 32 * log(8), 32 * log(9), log(10), log(5)))   # noqa: B023
        got = variants("l", [s for s in layers if s[5] <= s[4]])
        assert {v[:6] for v in got} == LAYER and up_of(got) == UP and down_of(got) == DOWN


def test_every_variant_runs_on_the_gpu(variants):
    products = [(T * k, E, N, K) for _, T, k, E, N, K in FP8_PRODUCTS]
    assert variants("b", products + LARGE_PRODUCTS) == BF16_ACT
    assert variants("f", products + LARGE_PRODUCTS) == FP8_ACT
    for form, step in STEP.items():
        layers = [(T, dim * step, hidden * step, E, k) for T, dim, hidden, E, k, _, _ in CASES]
        got = variants("l", [(VALUES[form], *c) for c in layers + WIDE_CASES])
        assert {v[:6] for v in got} == LAYER
        large = variants("l", [(VALUES[form], *c) for f, *c in STREAMED if f == form])
        assert all(v[7] and v[8] for v in large)
        assert up_of(got) >= {v for v in UP if not v[2]} and down_of(got) >= {v for v in DOWN if not v[3]}
        if form == "bf16":
            assert up_of(large) == {v for v in UP if v[2]} and down_of(large) == {v for v in DOWN if v[3]}
