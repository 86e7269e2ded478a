"""Which path an ExpertFFN with decode_tokens takes where a gradient is wanted by a tensor that is not one of its parameters: a weight
computed from others (an adapter on a frozen layer) stands in the parameter's place."""
import pytest
import torch

from sparse_gemm_amd import expert_layer
from test_expert_calls_cpu import bf
from test_fp8_blocks_cpu import library  # noqa: F401


@pytest.mark.parametrize("name", ["router", "up", "down", "up_bias", "down_bias"])
def test_a_computed_weight_that_wants_a_gradient(library, name):  # noqa: F811
    m = expert_layer.ExpertFFN(64, 64, 4, 2, bias=True, device="cpu", decode_tokens=8).requires_grad_(False)
    base, adapter = getattr(m, name).detach(), torch.zeros(1, dtype=torch.bfloat16, requires_grad=True)
    delattr(m, name)
    setattr(m, name, base + adapter)
    called = lambda: any(n == "bsr_expert_ffn" for n, _ in library.calls)   # noqa: E731
    m(bf(3, 64)).sum().backward()
    assert adapter.grad is not None and not called()
    with torch.no_grad():
        m(bf(3, 64))
    assert called()
