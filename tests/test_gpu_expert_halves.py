"""Products in 256 x 256 tiles whose last round leaves half of the CUs idle: its tiles are halved. Forward and input gradient, with
and without whole tiles before them, gathered and sorted, with rows past the plan."""
import math

import pytest
import torch

from expert_ref import f64, grouped, near_bf16
from gpu_util import dev, say
from sparse_gemm_amd import experts
from test_gpu_experts import gen, product_inputs

pytestmark = pytest.mark.gpu

CUS = 256

# (plan, T, k, E, N, K) of the forward; the input gradient swaps N and K. Widths that end in a tile's second half, in its first half
# (whose second is empty) and at a tile's edge
HALVES = [("one", 2552, 1, 2, 8328, 72), ("dropped", 1710, 2, 3, 6144, 72), ("dropped", 2200, 2, 2, 7176, 136),
          ("ragged", 2130, 2, 4, 5336, 136)]
ONE_EXPERT = [("one", 2843, 1, 1, 7176, 72), ("one", 2746, 1, 1, 8200, 264)]   # forward: the input gradient takes smaller tiles


def halved(offsets, R, cols):
    """Tiles of the last round, if they are halved."""
    groups = [b - a for a, b in zip(offsets, offsets[1:])] + [R - offsets[-1]]
    rest = sum(-(-n // 256) for n in groups) * -(-cols // 256) % CUS
    return rest if rest <= CUS // 2 else 0


@pytest.mark.parametrize("kind,T,k,E,N,K", HALVES + ONE_EXPERT)
@pytest.mark.parametrize("gather", [True, False])
def test_forward(kind, T, k, E, N, K, gather):
    p, off, live, X, W, _, x = product_inputs(kind, T, k, E, N, K, gather)
    say(f"case halved forward {kind} T={T} k={k} E={E} N={N} K={K} gather={gather}: {halved(off.tolist(), p.R, N)} tiles")
    assert halved(off.tolist(), p.R, N) > 0
    b = torch.randn(E, N, generator=gen(9)).bfloat16()
    out = torch.full((p.R, N), math.nan, dtype=torch.bfloat16, device=dev())
    y = experts.expert_fwd(p, X.to(dev()), W.to(dev()), b.to(dev()), gather, out=out)
    Y, S = grouped(x, off, lambda e: f64(W[e]), f64(b))
    near_bf16(y, Y, S, K)
    assert (f64(y)[live:] == 0).all()


@pytest.mark.parametrize("kind,T,k,E,K,N", HALVES)
def test_input_gradient(kind, T, k, E, K, N):
    p, off, live, _, W, dY, _ = product_inputs(kind, T, k, E, N, K, False)
    say(f"case halved input gradient {kind} T={T} k={k} E={E} N={N} K={K}: {halved(off.tolist(), p.R, K)} tiles")
    assert halved(off.tolist(), p.R, K) > 0
    out = torch.full((p.R, K), math.nan, dtype=torch.bfloat16, device=dev())
    dX = experts.expert_bwd_input(p, dY.to(dev()), W.to(dev()), out=out)
    g = f64(dY)
    g[live:] = 0
    Y, S = grouped(g, off, lambda e: f64(W[e]).T)
    near_bf16(dX, Y, S, N)
