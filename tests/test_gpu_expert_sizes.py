"""Products grouped by expert on matrices past 2^31 and 2^32 bytes, every element against 64-bit products on the device (a piece at
a time). Tolerance: one rounding to bf16 (2^-8) plus 2^-23 of the sum of magnitudes for each term of a 32-bit sum."""
import pytest
import torch

from gpu_util import dev, say
from sparse_gemm_amd import experts
from sparse_gemm_amd.experts import ExpertPlan

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
