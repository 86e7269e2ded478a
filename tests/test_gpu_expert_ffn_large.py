"""The whole layer for few tokens on 4-bit and 8-bit weights of 256 MB and more, which are read as data not used again, in the variants
that tests/test_gpu_expert_ffn.py runs on such weights in bf16 alone."""
import pytest

from gpu_util import say
from sparse_gemm_amd import expert_layer
from test_gpu_expert_ffn import Layer

pytestmark = pytest.mark.gpu

# form, T, dim, hidden, E, k
LARGE = [("fp8", 5, 4864, 9344, 2, 2), ("fp8", 5, 2560, 17536, 2, 2), ("fp8", 9, 2560, 17536, 2, 2), ("fp8", 9, 1024, 11008, 8, 4),
         ("fp8", 16, 2048, 1008, 64, 8), ("mx4", 4, 4096, 7168, 8, 2), ("mx4", 5, 2560, 35072, 2, 2), ("mx4", 6, 1024, 22016, 8, 4),
         ("mx4", 9, 4864, 18688, 2, 2), ("mx4", 9, 2560, 35072, 2, 2)]


@pytest.mark.parametrize("form,T,dim,hidden,E,k", LARGE)
def test_large_layer(form, T, dim, hidden, E, k):
    say(f"case expert_ffn {form} T={T} dim={dim} hidden={hidden} E={E} k={k}")
    m = Layer(form, T, dim, hidden, E, k, True, True)
    m.check(expert_layer.expert_ffn(**m.args()))
