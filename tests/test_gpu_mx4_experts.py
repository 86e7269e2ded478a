"""Weights of experts with odd numbers of rows in 4 bits: bit for bit like each expert's matrix."""
import pytest
import torch

from gpu_util import dev, say
from sparse_gemm_amd import mx4
from sparse_gemm_amd.mx4 import Mx4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,rows,K", [(3, 3, 32), (3, 5, 256), (4, 41, 32), (3, 7, 544), (2, 9, 288), (5, 1, 64), (1, 3, 32)])
def test_odd_rows(E, rows, K):
    say(f"case mx4 experts E={E} rows={rows} K={K}")
    W = torch.randn(E, rows, K, generator=torch.Generator().manual_seed(rows)).bfloat16().to(dev())
    q = mx4.quantize(W)
    values = mx4.dequantize(q)
    for e in range(E):
        one, want = mx4.quantize(W[e], want_values=True)
        assert torch.equal(q.codes[e], one.codes) and torch.equal(q.scales[e], one.scales)
        assert torch.equal(values[e], want) and torch.equal(mx4.dequantize(Mx4(one.codes, one.scales)), want)
