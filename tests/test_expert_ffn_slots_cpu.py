"""The numbers of slots and of experts that the Python calls pass on: never the low 32 bits of another number."""
import pytest
import torch

from sparse_gemm_amd import few_tokens
from sparse_gemm_amd.experts import ExpertPlan
from test_expert_calls_cpu import bf
from test_fp8_blocks_cpu import library  # noqa: F401


@pytest.mark.parametrize("k", [-(1 << 32) + 2, -1, 0, (1 << 32) + 2, 2])
def test_slots_are_passed_on_whole(library, k):  # noqa: F811
    few_tokens.expert_ffn(bf(4, 64), bf(3, 64), bf(3, 128, 64), bf(3, 64, 64), k)
    name, a = library.calls[-1]
    assert name == "bsr_expert_ffn" and -(1 << 31) <= a[5] < 1 << 31 and (a[5] == 2) == (k == 2) and (a[5] > 0) == (k > 0)


@pytest.mark.parametrize("E", [-(1 << 32) + 3, -1, 0, 3])
def test_experts_of_a_plan_are_passed_on_whole(library, E):  # noqa: F811
    ExpertPlan.from_index(torch.zeros((4, 2), dtype=torch.int32), E)
    name, a = library.calls[-1]
    assert name == "bsr_expert_plan" and -(1 << 31) <= a[3] < 1 << 31 and (a[3] == 3) == (E == 3) and (a[3] > 0) == (E > 0)
