"""Second derivatives are refused, without a GPU: stand-ins for the library's calls compute on the CPU. First gradients
under create_graph=True are those without it."""
import pytest
import torch

from sparse_gemm_amd import expert_layer, experts

T, K, N, E, k = 5, 8, 16, 4, 2


class Plan:
    """Rows in token order, all with one expert."""
    T, k, E, R = T, 1, 1, T


@pytest.fixture
def calls(monkeypatch):
    def router_fwd(logits, k, renormalize):
        weight, index = torch.softmax(logits, 1).topk(k, 1)
        return index.int(), weight

    def router_bwd(logits, index, weight, dweight, renormalize):
        p = torch.softmax(logits, 1)
        g = torch.zeros_like(p).scatter(1, index.long(), dweight)
        return p * (g - (g * p).sum(1, keepdim=True))

    monkeypatch.setattr(experts, "router_fwd", router_fwd)
    monkeypatch.setattr(experts, "router_bwd", router_bwd)
    monkeypatch.setattr(experts, "expert_fwd", lambda plan, x, W, bias, gather: x @ W[0].t() + (0 if bias is None else bias))
    monkeypatch.setattr(experts, "expert_bwd_input", lambda plan, dY, W: dY @ W[0])
    monkeypatch.setattr(experts, "expert_bwd_weight",
                        lambda plan, dY, x, gather, want, want_dW: ((dY.t() @ x)[None], dY.sum(0, keepdim=True) if want else None))
    monkeypatch.setattr(experts, "combine_fwd", lambda plan, Y, w=None: Y.clone() if w is None else (w * Y).to(Y.dtype))
    monkeypatch.setattr(experts, "combine_bwd", lambda plan, d, Y, w: ((w * d).to(Y.dtype), (d * Y).sum(1, keepdim=True).float()))


def leaf(*shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(sum(shape))).to(dtype).requires_grad_()


def route():
    x, r = leaf(T, K, dtype=torch.float32), leaf(E, K, dtype=torch.float32)
    return expert_layer.route(x @ r.t(), k)[1], [x, r]


def product():
    x, s, W = leaf(T, K), leaf(T, K), leaf(1, N, K)
    return expert_layer.expert_linear(Plan, x * s, W), [x, s, W]


def summed():
    y, s, w = leaf(T, N), leaf(T, N), leaf(T, 1, dtype=torch.float32)
    return expert_layer.combine(Plan, y * s, w), [y, s, w]


@pytest.mark.parametrize("make", [route, product, summed])
@pytest.mark.parametrize("outer", ["sum", "square"])
def test_second_derivatives_are_refused(calls, make, outer):
    """sum: the incoming gradient is a constant; square: it carries a graph of its own."""
    out, leaves = make()
    loss = out.sum() if outer == "sum" else (out * out).sum()
    plain = torch.autograd.grad(loss, leaves, retain_graph=True)
    first = torch.autograd.grad(loss, leaves, create_graph=True)
    for a, b in zip(plain, first):
        assert torch.equal(a, b)
    # the product with the other factor (x's with r, y's with s) gives the first gradient a graph
    assert first[0].requires_grad
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad(first[0].float().pow(2).sum(), leaves[1])
