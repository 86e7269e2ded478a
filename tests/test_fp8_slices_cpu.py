"""Scale bytes of a slice of experts ([E, N/128, K/128] from some expert on) start at any byte: no call asks them to be aligned. (What the
C ABI checks, without a GPU: every call is refused for a later argument.)"""
import pytest

from sparse_gemm_amd import _lib
from test_fp8_blocks_cpu import INVALID, P, ffn, why


@pytest.mark.parametrize("at", [P + 1, P + 4, P + 15])
def test_block_scales_at_any_byte(at):
    L = _lib.load()
    assert "values is NULL" in why(L.bsr_fp8_dequantize_blocks(P, at, 2, 64, 64, None, None))
    assert "Y is NULL" in why(L.bsr_expert_fwd_fp8(P, 4, 4, 2, 64, 64, P, P, P, at, None, None, None))
    assert "Y is NULL" in why(L.bsr_expert_fwd_fp8_fp8(P, P, 4, 4, 2, 64, 64, P, P, P, at, None, None, None))
    assert "workspace is NULL" in why(ffn(form=2, up_scales=at, down_scales=at, workspace=None), INVALID)
