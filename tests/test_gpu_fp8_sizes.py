"""8-bit block operators and the whole layer for few tokens on operands past 2^31 and 2^32 bytes: quantisation bit for bit against that
of a slice, products against 64-bit ones on the device (tolerance: one rounding to bf16, 2^-8, plus 2^-23 of the sum of magnitudes for
each term of a 32-bit sum and, with both sides in 8 bits, 7 * 2^-13 of the largest product of each 8 columns), the layer against its
definition."""
import pytest
import torch

import fp8_ref
from expert_ref import f64
from gpu_util import dev, say
from sparse_gemm_amd import expert_layer, experts, fp8, mx4
from sparse_gemm_amd.fp8 import Fp8Blocks, Fp8Rows
from test_gpu_expert_sizes import a_plan, randn

pytestmark = pytest.mark.gpu

TOP = 0xF0000000     # the most bytes that one buffer resource of these kernels covers


def rows_of(q, a, b):
    return Fp8Rows(q.codes[a:b].contiguous(), q.scales[:, a:b].contiguous())


def near(got, x, w, eight):
    """got against x . w^T; x and w: the values in bf16."""
    x, w = x.double(), w.double()
    S = x.abs() @ w.abs().t()
    ref = x @ w.t()
    # the largest of 8 products is at most the sum of their magnitudes
    lost = 7 * 2.0 ** -13 * S if eight else torch.zeros_like(S)
    tol = 2.0 ** -8 * (ref.abs() + lost) + lost + (x.shape[1] + 4) * 2.0 ** -23 * S + 2.0 ** -133
    off = (got.double() - ref).abs()
    assert bool((off <= tol).all()), f"worst {float((off / tol).max()):.3f} of the tolerance"


def test_rows_past_4_gib():
    rows, K = (1 << 18) + 5, 16400
    say(f"case rows={rows} K={K}")
    X = randn(rows, K, seed=1)
    assert X.numel() > 1 << 32
    q = fp8.quantize_rows(X)
    back = fp8.dequantize(q)
    for at in (0, (1 << 31) // (2 * K) - 1, (1 << 31) // K - 1, (1 << 32) // K - 1, rows - 2):
        part = slice(at, min(at + 3, rows))
        one = fp8.quantize_rows(X[part].contiguous())
        assert torch.equal(q.codes[part], one.codes) and torch.equal(q.scales[:, part], one.scales)
        assert torch.equal(back[part], fp8.dequantize(one))


def test_large_blocks_and_their_expansion():
    """Matrices that are read, and expansions that are stored, as data not used again."""
    E, N, K = 4, 4112, 8192
    say(f"case large blocks E={E} N={N} K={K}")
    W = randn(E, N, K, seed=16)
    q, t = fp8.quantize_blocks(W, transposed=True)
    back, turned = fp8.dequantize(q), fp8.dequantize(t)
    for e in range(E):
        one, two = fp8.quantize_blocks(W[e, :2048].contiguous(), transposed=True)
        assert torch.equal(q.codes[e, :2048], one.codes) and torch.equal(q.scales[e, :16], one.scales)
        assert torch.equal(t.codes[e, :, :2048], two.codes) and torch.equal(t.scales[e, :, :16], two.scales)
        one = fp8.quantize_blocks(W[e, 2048:].contiguous())
        assert torch.equal(q.codes[e, 2048:], one.codes) and torch.equal(q.scales[e, 16:], one.scales)
        assert torch.equal(back[e, 2048:], fp8.dequantize(one)) and torch.equal(turned[e], back[e].t())


def test_many_rows_in_every_rest():
    """Four rows a wave, and what is left of them."""
    for rows in (8192, 8193, 8194, 8195):
        for K in (512, 1040):
            say(f"case rows={rows} K={K}")
            X = randn(rows, K, seed=17)
            q, values = fp8.quantize_rows(X, want_values=True)
            for a, b in ((0, 5), (4000, 4011), (rows - 9, rows)):
                one, v = fp8.quantize_rows(X[a:b].contiguous(), want_values=True)
                assert torch.equal(q.codes[a:b], one.codes) and torch.equal(q.scales[:, a:b], one.scales) and torch.equal(values[a:b], v)


def test_blocks_past_4_gib():
    E, N, K = 33, 8192, 16400
    say(f"case blocks E={E} N={N} K={K}")
    W = randn(E, N, K, seed=2)
    assert W.numel() > 1 << 32
    q, t = fp8.quantize_blocks(W, transposed=True)
    back = fp8.dequantize(t)
    for e in (0, 7, 8, 15, 16, 31, 32):
        one, turned = fp8.quantize_blocks(W[e:e + 1].contiguous(), transposed=True)
        for a, b in ((q, one), (t, turned)):
            assert torch.equal(a.codes[e], b.codes[0]) and torch.equal(a.scales[e], b.scales[0])
        assert torch.equal(back[e], fp8.dequantize(turned)[0])
    del back, t, W
    # products on the experts' weights at both ends of them
    for R in (40, 1500):
        say(f"case product R={R}")
        p, offsets, _ = a_plan(R, E, 3)
        x = randn(R, K, seed=3)
        for act in (x, fp8.quantize_rows(x)):
            eight = isinstance(act, Fp8Rows)
            value = fp8.dequantize(act) if eight else act
            y = fp8.expert_fwd(p, act, q, gather=False)
            for e in (0, 8, 15, 16, 31, 32):
                a, b = offsets[e], offsets[e + 1]
                near(y[a:b], value[a:b], fp8.dequantize(Fp8Blocks(q.codes[e:e + 1], q.scales[e:e + 1]))[0], eight)


STREAMED = [(8, 8, 8192, 4096), (7, 8, 14336, 4096), (64, 5, 4104, 13184)]   # R, E, N, K: weights read as not used again


@pytest.mark.parametrize("R,E,N,K", STREAMED)
def test_few_rows_of_large_weights(R, E, N, K):
    say(f"case few rows R={R} E={E} N={N} K={K}")
    p, offsets, token = a_plan(R, E, 2)
    x = randn(R, K, seed=14)
    q = fp8.quantize_blocks(randn(E, N, K, seed=15))
    for act in (x, fp8.quantize_rows(x)):
        eight = isinstance(act, Fp8Rows)
        value = fp8.dequantize(act) if eight else x
        y = fp8.expert_fwd(p, act, q)
        for e in range(E):
            a, b = offsets[e], offsets[e + 1]
            near(y[a:b], value[token[a:b]], fp8.dequantize(Fp8Blocks(q.codes[e:e + 1], q.scales[e:e + 1].clone()))[0], eight)
        assert not y[offsets[-1]:].any()


@pytest.mark.parametrize("R", [3, 200])
def test_one_expert_of_the_most_bytes(R):
    N, K = 245760, 16384
    assert N * K == TOP
    say(f"case one expert N={N} K={K} R={R}")
    p = experts.ExpertPlan.from_index(torch.zeros((R, 1), dtype=torch.int32, device=dev()), 1)
    W = randn(1, N, K, seed=4)
    q = fp8.quantize_blocks(W)
    del W
    x = randn(R, K, seed=5)
    for act in (x, fp8.quantize_rows(x)):
        eight = isinstance(act, Fp8Rows)
        value = fp8.dequantize(act) if eight else act
        y = fp8.expert_fwd(p, act, q)
        for n in (0, (1 << 17) - 128, N - 256):
            part = Fp8Blocks(q.codes[:, n:n + 256].contiguous(), q.scales[:, n // 128:n // 128 + 2].contiguous())
            near(y[:, n:n + 256], value, fp8.dequantize(part)[0], eight)


@pytest.mark.parametrize("eight", [False, True])
def test_rows_and_results_of_many_bytes(eight):
    """Rows of just so many bytes as are allowed, gathered; then results past 2^32 bytes."""
    K = 8192
    R, E = TOP // (K * (1 if eight else 2)), 3
    say(f"case rows R={R} K={K} eight={eight}")
    p, offsets, token = a_plan(R, E, 3)
    x = randn(R, K, seed=6)
    q = fp8.quantize_blocks(randn(E, 64, K, seed=7, std=0.1))
    act = fp8.quantize_rows(x) if eight else x
    y = fp8.expert_fwd(p, act, q)
    for e, ends in ((1, offsets[1:3]), (2, offsets[2:4])):
        for a in (ends[0], ends[1] - 300):
            t = token[a:a + 300]
            value = fp8.dequantize(Fp8Rows(act.codes[t], act.scales[:, t].contiguous())) if eight else x[t]
            near(y[a:a + 300], value, fp8.dequantize(q)[e], eight)
    assert not y[offsets[-1]:].any()
    del x, act, y
    R, N, K = (1 << 18) + 5, 8200, 64
    say(f"case results R={R} N={N} eight={eight}")
    p, offsets, token = a_plan(R, E, 3)
    x = randn(R, K, seed=8)
    q = fp8.quantize_blocks(randn(E, N, K, seed=9))
    act = fp8.quantize_rows(x) if eight else x
    y = fp8.expert_fwd(p, act, q, gather=False)
    value = fp8.dequantize(act) if eight else x
    for e in (1, 2):
        for a in (offsets[e], offsets[e + 1] - 300):
            near(y[a:a + 300], value[a:a + 300], fp8.dequantize(q)[e], eight)
    assert not y[offsets[-1]:].any()


@pytest.mark.parametrize("form,E", [("bf16", 80), ("fp8", 160), ("mx4", 270)])
def test_layer_past_4_gib(form, E):
    T, dim, hidden, k = 3, 4096, 4096, 2
    say(f"case layer {form} E={E}")
    hold = {"bf16": lambda W: W, "mx4": mx4.quantize, "fp8": fp8.quantize_blocks}[form]
    value = {"bf16": lambda W: W, "mx4": mx4.dequantize, "fp8": fp8.dequantize}[form]
    up, down = hold(randn(E, 2 * hidden, dim, seed=10, std=dim ** -0.5)), hold(randn(E, dim, hidden, seed=11, std=hidden ** -0.5))
    assert sum(getattr(up, n).numel() * getattr(up, n).element_size() for n in (("codes",) if form != "bf16" else ("data",))) > 1 << 32
    router, x = randn(E, dim, seed=12, std=dim ** -0.5), randn(T, dim, seed=13)
    router[E - 9:] *= 16   # one of the last experts is the largest for some token
    router[:3] *= 16
    pick = (lambda W, e: W[e]) if form == "bf16" else (lambda W, e: type(W)(W.codes[e], W.scales[e]))
    want, tol, index, gap = fp8_ref.layer(f64(x), f64(router), lambda e: f64(value(pick(up, e))), lambda e: f64(value(pick(down, e))), k, True)
    assert gap.min() > 1 and index.max() >= E - 9
    got = f64(expert_layer.expert_ffn(x, router, up, down, k))
    off = abs(got - want)
    assert (off <= tol).all(), f"worst {(off / tol).max():.3f} of the tolerance"
