"""Products grouped by expert on matrices past 2^31 and 2^32 bytes, every element against 64-bit products on the device (a piece at
a time). Tolerance: one rounding to bf16 (2^-8) plus 2^-23 of the sum of magnitudes for each term of a 32-bit sum."""
import pytest
import torch

from gpu_util import dev, say
from sparse_gemm_amd import experts, mx4
from sparse_gemm_amd.experts import ExpertPlan
from sparse_gemm_amd.mx4 import Mx4

pytestmark = pytest.mark.gpu

TOP = 0xF0000000     # the most bytes that one buffer resource of these kernels covers


def randn(*shape, seed=0, std=1.0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    out = torch.empty(shape, dtype=torch.bfloat16, device=dev())
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - at)
        flat[at:at + n] = torch.randn(n, generator=g, device=dev()) * std
    return out


def a_plan(R, E, dropped):
    """Sorted rows of E experts of different sizes (one of them empty), the last `dropped` of R without an expert; token t is
    the row's neighbour, so that rows are gathered out of order."""
    cut = torch.linspace(0, (R - dropped) ** 0.5, E).square().long()
    offsets = torch.cat([cut[:1], cut[:1], cut[1:]])[:E + 1]
    offsets[E] = R - dropped
    token = torch.arange(R) ^ 1
    token[R - dropped:] = -1
    p = ExpertPlan(offsets.int().to(dev()), token.int().to(dev()), torch.zeros((R, 1), dtype=torch.int32, device=dev()))
    return p, offsets.tolist(), token.to(dev())


def near(got, ref, S, terms):
    off = (got.double() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + (terms + 4) * 2.0 ** -23 * S + 2.0 ** -133
    assert bool((off <= tol).all()), f"worst {float((off / tol).max()):.3f} of the tolerance"


def check_rows(out, offsets, rows, weight, terms):
    """out[r] = rows(a, b) . weight(e)^T for the rows of each expert, 0 past them."""
    for e in range(len(offsets) - 1):
        w = weight(e).double() if offsets[e] < offsets[e + 1] else None
        for a in range(offsets[e], offsets[e + 1], 1 << 15):
            b = min(a + (1 << 15), offsets[e + 1])
            x = rows(a, b).double()
            near(out[a:b], x @ w.t(), x.abs() @ w.abs().t(), terms)
    assert not out[offsets[-1]:].any()


def test_input_gradient_past_4_gib():
    """dX, then dY of more bytes than a buffer resource covers."""
    R, E = (1 << 18) + 5, 5
    p, offsets, _ = a_plan(R, E, 3)
    for N, K in ((64, 8192), (8192, 64)):
        assert R * max(N, K) * 2 > 1 << 32
        say(f"case input gradient R={R} N={N} K={K}")
        dY, W = randn(R, N, seed=1), randn(E, N, K, seed=2, std=0.1)
        dX = experts.expert_bwd_input(p, dY, W)
        check_rows(dX, offsets, lambda a, b: dY[a:b], lambda e: W[e].t(), N)
        del dX, dY, W


def test_forward_of_sorted_rows_past_4_gib():
    """X, then Y of more bytes than a buffer resource covers."""
    R, E = (1 << 18) + 5, 5
    p, offsets, _ = a_plan(R, E, 3)
    for N, K in ((64, 8192), (8192, 64)):
        say(f"case forward of sorted rows R={R} N={N} K={K}")
        X, W = randn(R, K, seed=1), randn(E, N, K, seed=2, std=0.1)
        Y = experts.expert_fwd(p, X, W, gather=False)
        check_rows(Y, offsets, lambda a, b: X[a:b], lambda e: W[e], K)
        del X, Y, W


def test_gathered_tokens_up_to_the_limit():
    """X of exactly the most bytes, gathered by token: forward and weight gradient."""
    K, N, E = 4096, 64, 4
    R = TOP // (2 * K)
    p, offsets, token = a_plan(R, E, 2)
    X, W, dY = randn(R, K, seed=3), randn(E, N, K, seed=4, std=0.02), randn(R, N, seed=5)
    say(f"case gathered forward T=R={R} N={N} K={K}")
    check_rows(experts.expert_fwd(p, X, W), offsets, lambda a, b: X[token[a:b]], lambda e: W[e], K)
    say(f"case gathered weight gradient T=R={R} N={N} K={K}")
    check_weight(p, offsets, dY, X, token)


def check_weight(p, offsets, dY, X, token):
    dW, db = experts.expert_bwd_weight(p, dY, X, gather=token is not None, want_dbias=True)
    for e in range(p.E):
        w = torch.zeros(dW.shape[1:], dtype=torch.float64, device=dev())
        S, b, bS = torch.zeros_like(w), w.new_zeros(w.shape[0]), w.new_zeros(w.shape[0])
        for lo in range(offsets[e], offsets[e + 1], 1 << 15):
            hi = min(lo + (1 << 15), offsets[e + 1])
            d, x = dY[lo:hi].double(), (X[lo:hi] if token is None else X[token[lo:hi]]).double()
            w += d.t() @ x
            S += d.abs().t() @ x.abs()
            b += d.sum(0)
            bS += d.abs().sum(0)
        near(dW[e], w, S, offsets[e + 1] - offsets[e])
        near(db[e], b, bS, offsets[e + 1] - offsets[e])


@pytest.mark.parametrize("N,K", [(4096, 64), (64, 4096)])
def test_weight_gradient_of_sorted_rows_up_to_the_limit(N, K):
    """dY, then X of exactly the most bytes."""
    R = TOP // (2 * 4096)
    p, offsets, _ = a_plan(R, 3, 2)
    say(f"case weight gradient R={R} N={N} K={K}")
    check_weight(p, offsets, randn(R, N, seed=6), randn(R, K, seed=7), None)


@pytest.mark.parametrize("R", [40, 700])
def test_one_experts_weight_up_to_the_limit(R):
    """One weight of exactly the most bytes, the second expert's behind it: few rows and many."""
    K, E = 4096, 2
    N = TOP // (2 * K)
    W = randn(E, N, K, seed=8, std=0.02)
    index = torch.ones((R, 1), dtype=torch.int32, device=dev())
    index[:3] = 0
    p = ExpertPlan.from_index(index, E)
    X, dY = randn(R, K, seed=9), randn(R, N, seed=10)
    say(f"case forward R={R} N={N} K={K}")
    Y = experts.expert_fwd(p, X, W)
    for n in range(0, N, 1 << 16):
        m = min(n + (1 << 16), N)
        check_rows(Y[:, n:m], [0, 3, R], lambda a, b: X[a:b], lambda e: W[e, n:m], K)
    say(f"case input gradient R={R} N={N} K={K}")
    dX = experts.expert_bwd_input(p, dY, W)
    for k in range(0, K, 512):
        check_rows(dX[:, k:k + 512], [0, 3, R], lambda a, b: dY[a:b], lambda e: W[e, :, k:k + 512].t(), N)


@pytest.mark.parametrize("R", [64, 4000])
def test_layer_past_4_gib(R):
    """All experts' weights, and their gradients, of more than 2^32 bytes; in 4 bits too."""
    E, N, K = 100, 8192, 8192
    assert E * N * (K // 2) > 1 << 31 and E * N * K * 2 > 1 << 33
    index = (torch.arange(R, dtype=torch.int32, device=dev()) * 7 % E).view(R, 1)
    p = ExpertPlan.from_index(index, E)
    offsets, token = p.offsets.tolist(), p.row_token.long()
    W, X, dY = randn(E, N, K, seed=11, std=0.01), randn(R, K, seed=12), randn(R, N, seed=13)
    some = [e for e in range(E) if e % 9 == 0 or e > E - 3]

    def check(out, rows, weight, terms):
        for e in some:
            a, b = offsets[e], offsets[e + 1]
            if a < b:
                x, w = rows(a, b).double(), weight(e).double()
                near(out[a:b], x @ w.t(), x.abs() @ w.abs().t(), terms)

    say(f"case layer R={R} E={E} N={N} K={K}")
    check(experts.expert_fwd(p, X, W), lambda a, b: X[token[a:b]], lambda e: W[e], K)
    check(experts.expert_bwd_input(p, dY, W), lambda a, b: dY[a:b], lambda e: W[e].t(), N)
    dW, _ = experts.expert_bwd_weight(p, dY, X)
    for e in some:
        a, b = offsets[e], offsets[e + 1]
        d, x = dY[a:b].double(), X[token[a:b]].double()
        near(dW[e], d.t() @ x, d.abs().t() @ x.abs(), b - a)
    del dW
    say("    in 4 bits")
    q = mx4.quantize(W)
    values = lambda e: mx4.dequantize(Mx4(q.codes[e], q.scales[e]))   # noqa: E731
    check(mx4.expert_fwd(p, X, q), lambda a, b: X[token[a:b]], values, K)
    xq = mx4.quantize(X)
    xv = mx4.dequantize(xq)
    check(mx4.expert_fwd(p, xq, q), lambda a, b: xv[token[a:b]], values, K)


@pytest.mark.parametrize("gather", [True, False])
def test_4_bit_activations_up_to_the_limit(gather):
    """Codes of exactly the most bytes; their quantisation reads 16 GB."""
    K, N, E = 1024, 64, 3
    R = TOP * 2 // K
    p, offsets, token = a_plan(R, E, 2)
    say(f"case 4-bit activations R={R} N={N} K={K} gather={gather}")
    W = mx4.quantize(randn(E, N, K, seed=14, std=0.05))
    wv = mx4.dequantize(W)
    xq, xv = mx4.quantize(randn(R, K, seed=15), want_values=True)
    Y = mx4.expert_fwd(p, xq, W, gather=gather)
    check_rows(Y, offsets, lambda a, b: xv[token[a:b]] if gather else xv[a:b], lambda e: wv[e], K)


def test_combine_past_4_gib():
    """Rows of more than 2^32 bytes: the sum and its gradient, a token's rows far apart."""
    T, k, N = 150001, 3, 8192
    assert T * k * N * 2 > 1 << 32
    say(f"case combine T={T} k={k} N={N}")
    index = torch.arange(k, dtype=torch.int32, device=dev()).expand(T, k).contiguous()
    p = ExpertPlan.from_index(index, k)
    Y, dout = randn(p.R, N, seed=16), randn(T, N, seed=17)
    w = torch.rand(T, k, generator=torch.Generator(device=dev()).manual_seed(1), device=dev())
    out = experts.combine_fwd(p, Y, w)
    dY, dw = experts.combine_bwd(p, dout, Y, w)
    for a in range(0, T, 1 << 13):
        b = min(a + (1 << 13), T)
        t = [Y[j * T + a:j * T + b].double() * w[a:b, j, None].double() for j in range(k)]   # slot j's rows are expert j's
        near(out[a:b], sum(t), sum(x.abs() for x in t), k)
        d = dout[a:b].double()
        for j in range(k):
            ref = d * w[a:b, j, None].double()
            near(dY[j * T + a:j * T + b], ref, ref.abs(), 1)
            y = Y[j * T + a:j * T + b].double()
            near_f32(dw[a:b, j], (d * y).sum(1), (d * y).abs().sum(1), N)


def near_f32(got, ref, S, terms):
    assert bool(((got.double() - ref).abs() <= (terms + 4) * 2.0 ** -23 * S).all())


@pytest.mark.parametrize("gather", [True, False])
def test_4_bit_weights_with_activations_up_to_the_limit(gather):
    """bf16 activations of exactly the most bytes on 4-bit weights."""
    K, N, E = 4096, 64, 3
    R = TOP // (2 * K)
    p, offsets, token = a_plan(R, E, 2)
    say(f"case 4-bit weights R={R} N={N} K={K} gather={gather}")
    W = mx4.quantize(randn(E, N, K, seed=18, std=0.05))
    wv = mx4.dequantize(W)
    X = randn(R, K, seed=19)
    Y = mx4.expert_fwd(p, X, W, gather=gather)
    check_rows(Y, offsets, lambda a, b: X[token[a:b]] if gather else X[a:b], lambda e: wv[e], K)


def test_expansion_past_4_gib():
    """Codes of 4 GB, values of 16 GB: both passes write the same."""
    rows, K = TOP * 2 // 1024, 1024
    say(f"case expansion rows={rows} K={K}")
    q, values = mx4.quantize(randn(rows, K, seed=20), want_values=True)
    assert torch.equal(mx4.dequantize(q), values)
