"""The block-sparse layer refuses second derivatives, without a GPU: stand-ins for the library's calls compute on the CPU."""
import pytest
import torch

from sparse_gemm_amd import binding, linear


class Pattern:
    N = 16


@pytest.mark.parametrize("outer", ["sum", "square"])
def test_second_derivatives_are_refused(monkeypatch, outer):
    monkeypatch.setattr(binding, "linear_fwd", lambda p, x, v, b: x @ v.t())
    monkeypatch.setattr(binding, "linear_bwd_input", lambda p, dY, v: dY @ v)
    monkeypatch.setattr(binding, "linear_bwd_weight", lambda p, dY, x, want_dbias: (dY.t() @ x, dY.sum(0) if want_dbias else None))
    g = torch.Generator().manual_seed(0)
    x, s, v = (torch.randn(n, 8, generator=g).bfloat16().requires_grad_() for n in (5, 5, 16))
    out = linear.bsr_linear(x * s, Pattern, v)
    loss = out.sum() if outer == "sum" else (out * out).sum()
    plain = torch.autograd.grad(loss, [x, s, v], retain_graph=True)
    first = torch.autograd.grad(loss, [x, s, v], create_graph=True)
    for a, b in zip(plain, first):
        assert torch.equal(a, b)
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad(first[0].float().pow(2).sum(), s)
