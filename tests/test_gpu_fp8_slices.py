"""8-bit weights of some of a layer's experts, as views of all: their scale bytes start anywhere."""
import pytest
import torch

from gpu_util import dev, say
from sparse_gemm_amd import expert_layer, experts, fp8
from sparse_gemm_amd.fp8 import Fp8Blocks

pytestmark = pytest.mark.gpu


def view(q, a, b):
    return Fp8Blocks(q.codes[a:b], q.scales[a:b])


def copied(q):
    return Fp8Blocks(q.codes.clone(), q.scales.clone())


@pytest.mark.parametrize("R", [3, 300, 3000])
def test_products_on_a_slice_of_experts(R):
    E, N, K = 5, 208, 304   # 6 scale bytes an expert
    say(f"case slices R={R}")
    g = torch.Generator(device=dev()).manual_seed(R)
    q = fp8.quantize_blocks(torch.randn(E, N, K, generator=g, device=dev()).bfloat16())
    x = torch.randn(R, K, generator=g, device=dev()).bfloat16()
    plan = experts.ExpertPlan.from_index(torch.randint(0, 2, (R, 1), generator=g, device=dev(), dtype=torch.int32), 2)
    for a in range(4):
        part = view(q, a, a + 2)
        assert a == 0 or part.scales.data_ptr() % 16
        assert torch.equal(fp8.dequantize(part), fp8.dequantize(copied(part)))
        for act in (x, fp8.quantize_rows(x)):
            assert torch.equal(fp8.expert_fwd(plan, act, part), fp8.expert_fwd(plan, act, copied(part)))


@pytest.mark.parametrize("T", [2, 12])
def test_the_whole_layer_on_a_slice_of_experts(T):
    E, dim, hidden = 6, 272, 144
    say(f"case slices of a layer T={T}")
    g = torch.Generator(device=dev()).manual_seed(T)
    bf = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=dev()) * std).bfloat16()   # noqa: E731
    up, down = fp8.quantize_blocks(bf(E, 2 * hidden, dim, std=dim ** -0.5)), fp8.quantize_blocks(bf(E, dim, hidden, std=hidden ** -0.5))
    x, router = bf(T, dim), bf(3, dim, std=dim ** -0.5)
    for a in range(4):
        parts = view(up, a, a + 3), view(down, a, a + 3)
        got = expert_layer.expert_ffn(x, router, *parts, 2)
        assert torch.equal(got, expert_layer.expert_ffn(x, router, *map(copied, parts), 2))
