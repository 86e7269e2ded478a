"""What expert_linear_fp8 keeps for its backward pass (a stand-in for the library; no GPU)."""
import weakref

import torch

from sparse_gemm_amd import expert_layer
from test_expert_calls_cpu import a_plan, bf
from test_fp8_blocks_cpu import library  # noqa: F401


def test_a_weight_may_change_between_forward_and_backward(library):  # noqa: F811
    """The input gradient takes the codes that the forward pass made, the weight gradient x: W itself is not read again and
    may be updated in place."""
    plan = a_plan()
    x, W, b = bf(4, 64).requires_grad_(), bf(3, 64, 64).requires_grad_(), bf(3, 64).requires_grad_()
    y = expert_layer.expert_linear_fp8(plan, x, W, b)
    with torch.no_grad():
        W.add_(1.0)
    y.backward(bf(8, 64))
    assert x.grad.shape == x.shape and W.grad.shape == W.shape and b.grad.shape == b.shape


def test_a_computed_weight_is_released_by_the_backward_pass(library):  # noqa: F811
    """A weight that is computed for the call (cast from another) does not stay alive with the result."""
    plan, leaf = a_plan(), bf(3, 64, 64).float().requires_grad_()
    W = leaf.to(torch.bfloat16)
    gone = weakref.ref(W)
    y = expert_layer.expert_linear_fp8(plan, bf(4, 64).requires_grad_(), W)
    del W
    assert gone() is not None
    y.backward(bf(8, 64))
    assert leaf.grad is not None and gone() is None
    W = bf(3, 64, 64)   # one that wants no gradient is not kept at all
    gone = weakref.ref(W)
    y = expert_layer.expert_linear_fp8(plan, bf(4, 64).requires_grad_(), W)
    del W
    assert gone() is None
    y.backward(bf(8, 64))
