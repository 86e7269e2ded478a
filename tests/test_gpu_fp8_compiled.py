"""ExpertFFN with products in 8 bits and with decode_tokens under torch.compile: the results and gradients of the layer as it is; and a
weight that changes in place between forward and backward."""
import pytest
import torch

from gpu_util import dev
from sparse_gemm_amd import expert_layer, experts
from sparse_gemm_amd.expert_layer import ExpertFFN

pytestmark = pytest.mark.gpu


def layer(**kw):
    torch.manual_seed(11)
    return ExpertFFN(128, 96, 6, 2, bias=True, device=dev(), decode_tokens=8, **kw)


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("T", [3, 8, 40])
@pytest.mark.parametrize("form", ["bf16", "fp8 training", "mx4", "fp8"])
def test_a_compiled_layer(form, T):
    torch._dynamo.reset()
    m = layer(fp8=form == "fp8 training")
    if form in ("mx4", "fp8"):
        m.quantize_(form)
    compiled = torch.compile(m, backend="eager")
    x = torch.randn(T, 128, device=dev()).bfloat16()
    with torch.no_grad():
        want = m(x)
        for _ in range(2):
            assert torch.equal(compiled(x), want)
    if m.quantized:
        return
    a, b = x.clone().requires_grad_(True), x.clone().requires_grad_(True)
    dY = torch.randn(T, 128, device=dev()).bfloat16()
    got = torch.autograd.grad(compiled(a), [a, *m.parameters()], dY)
    for u, v in zip(got, torch.autograd.grad(m(b), [b, *m.parameters()], dY)):
        assert torch.equal(u, v)


def test_a_weight_changed_before_the_backward_pass():
    T, K, N, E = 60, 144, 80, 3
    p = experts.ExpertPlan.from_index(torch.randint(0, E, (T, 2), device=dev(), dtype=torch.int32), E)
    x, W = torch.randn(T, K, device=dev()).bfloat16().requires_grad_(True), torch.randn(E, N, K, device=dev()).bfloat16().requires_grad_(True)
    dY = torch.randn(2 * T, N, device=dev()).bfloat16()
    want = torch.autograd.grad(expert_layer.expert_linear_fp8(p, x, W), [x, W], dY)
    y = expert_layer.expert_linear_fp8(p, x, W)
    with torch.no_grad():
        W.mul_(3.0)
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(y, [x, W], dY), want))
