"""Copies of a plan on the GPU: each works on its own memory."""
import copy
import pickle

import pytest
import torch

from gpu_util import dev
from sparse_gemm_amd import experts
from sparse_gemm_amd.experts import ExpertPlan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("copied", [copy.deepcopy, lambda p: pickle.loads(pickle.dumps(p))], ids=["deepcopy", "pickle"])
def test_a_copy_does_not_read_the_original(copied):
    T, k, E, N, K = 40, 2, 5, 64, 72
    g = torch.Generator().manual_seed(0)
    p = ExpertPlan.from_index(torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32).to(dev()), E)
    X, W = torch.randn(T, K, generator=g).bfloat16().to(dev()), torch.randn(E, N, K, generator=g).bfloat16().to(dev())
    dY, dout = torch.randn(p.R, N, generator=g).bfloat16().to(dev()), torch.randn(T, N, generator=g).bfloat16().to(dev())

    def results(plan):
        y = experts.expert_fwd(plan, X, W)
        return [y, experts.expert_bwd_input(plan, dY, W), *experts.expert_bwd_weight(plan, dY, X, want_dbias=True),
                experts.combine_fwd(plan, y), *experts.combine_bwd(plan, dout, y)]

    want = results(p)
    q = copied(p)
    for t in (p.offsets, p.row_token, p.slot_row):
        t.fill_(-1)
    for a, b in zip(results(q), want):
        assert torch.equal(a, b)
