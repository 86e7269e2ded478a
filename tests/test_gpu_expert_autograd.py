"""The autograd functions of the expert layers on slices, on frozen weights and under torch's transforms."""
import pytest
import torch

from gpu_util import dev
from sparse_gemm_amd import expert_layer, experts

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def test_slices_give_the_results_of_whole_tensors():
    """Logits, activations, rows and weights at an odd offset of a larger tensor, and gradients that are slices of a
    concatenation's: bit for bit what aligned copies give."""
    T, k, E, N, K = 5, 1, 3, 24, 40
    g = gen(0)

    def both(*shape, dtype=torch.bfloat16):
        whole = torch.randn(shape, generator=g).to(dtype).to(dev())
        flat = torch.empty(whole.numel() + 1, dtype=dtype, device=dev())
        flat[1:] = whole.flatten()
        part = flat[1:].view(shape)
        assert part.is_contiguous() and part.data_ptr() % 16
        return whole.requires_grad_(), part.requires_grad_()

    logits, x, y, w = both(T, E, dtype=torch.float32), both(T, K), both(T * k, N), both(T, k, dtype=torch.float32)
    W = torch.randn(E, N, K, generator=g).bfloat16().to(dev())
    lead = torch.ones(T, k, device=dev(), requires_grad=True)
    results = []
    for i in (0, 1):
        index, weight = expert_layer.route(logits[i], k, renormalize=False)
        plan = experts.ExpertPlan.from_index(index, E)
        rows = expert_layer.expert_linear(plan, x[i], W)
        out = expert_layer.combine(plan, y[i], w[i])
        # in a concatenation the gradient of `weight` is the last T * k of 2 T * k elements
        up = torch.arange(2 * T * k, dtype=torch.float32, device=dev()).view(2 * T, k)
        if i:
            (torch.cat([lead, weight]) * up).sum().backward()
        else:
            (weight * up[T:]).sum().backward()
        rows.float().square().sum().backward()
        out.float().square().sum().backward()
        results.append([index, weight, rows, out, logits[i].grad, x[i].grad, y[i].grad, w[i].grad])
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,E,N", [(70, 3, 136), (0, 2, 64)])
def test_the_bias_alone(T, E, N):
    """The bias gradient without the weight gradient is the one that comes with it."""
    K = 72
    g = gen(T)
    p = experts.ExpertPlan.from_index(torch.randint(-1, E, (T, 2), generator=g, dtype=torch.int32).to(dev()), E)
    dY, X = torch.randn(2 * T, N, generator=g).bfloat16().to(dev()), torch.randn(T, K, generator=g).bfloat16().to(dev())
    _, want = experts.expert_bwd_weight(p, dY, X, want_dbias=True)
    none, db = experts.expert_bwd_weight(p, dY, X, want_dbias=True, want_dW=False)
    assert none is None and torch.equal(db, want)
    with pytest.raises(ValueError):
        experts.expert_bwd_weight(p, dY, X, want_dW=False)
    with pytest.raises(ValueError):
        experts.expert_bwd_weight(p, dY, X, want_dbias=True, want_dW=False, out=torch.empty(E, N, K, dtype=torch.bfloat16, device=dev()))


@pytest.mark.filterwarnings("ignore")
def test_a_compiled_layer_is_the_eager_one():
    """torch.compile finds calls that it cannot trace and leaves them as they are: the same bits, forward and backward."""
    torch.manual_seed(0)
    m = expert_layer.ExpertFFN(64, 64, 4, 2, device=dev())
    x = torch.randn(24, 64, device=dev()).bfloat16()
    want = m(x)
    want.sum().backward()
    grads = [p.grad.clone() for p in m.parameters()]
    m.zero_grad()
    got = torch.compile(m, backend="eager")(x)
    got.sum().backward()
    assert torch.equal(got, want)
    for p, g in zip(m.parameters(), grads):
        assert torch.equal(p.grad, g)
