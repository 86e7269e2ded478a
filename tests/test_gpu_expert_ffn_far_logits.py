"""The whole layer for few tokens where a token's values are infinite: its logits are +-infinity, never NaN, wherever in the row the
infinity stands and whoever sums the logits (the up product's work-groups, a launch in pieces before it, the router's kernel)."""
import math

import pytest
import torch

from gpu_util import dev, say
from sparse_gemm_amd import expert_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [2, 12])
@pytest.mark.parametrize("E", [8, 20, 256, 300])
@pytest.mark.parametrize("dim", [1088, 2048, 4168])
def test_infinite_values_of_a_token(T, E, dim):
    """A token whose logits are all -infinity has no experts and a result of zeros; the others' results do not change."""
    say(f"case infinite values T={T} E={E} dim={dim}")
    g = torch.Generator().manual_seed(T + E + dim)
    bf = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).bfloat16().to(dev())   # noqa: E731
    router, x = bf(E, dim, std=dim ** -0.5), bf(T, dim)
    up, down = bf(E, 128, dim, std=dim ** -0.5), bf(E, dim, 64, std=0.125)
    columns = [c for c in (5, 500, 1030, 1087, 1540, 2047, 2600, 4167) if c < dim]
    router[:, columns] = -router[:, columns].abs().clamp_min(2.0 ** -10)
    clean = expert_layer.expert_ffn(x, router, up, down, 2)
    assert bool(clean.isfinite().all()) and bool(clean.any(1).all())
    for c in columns:
        far = x.clone()
        far[1, c] = math.inf
        got = expert_layer.expert_ffn(far, router, up, down, 2)
        assert not got[1].any(), f"column {c}"
        others = torch.arange(T) != 1
        assert torch.equal(got[others], clean[others]), f"column {c}"
