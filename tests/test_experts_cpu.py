"""Expert layers and 4-bit values without a GPU: the C entry points refuse bad arguments before anything is
enqueued, the Python calls refuse tensors that are not on a GPU, and the scale layout is its own inverse."""
import pytest
import torch

from sparse_gemm_amd import _lib, experts, mx4

P = 4096     # an aligned address that no refused call reads
OK, INVALID, UNSUPPORTED, MISALIGNED, SMALL = 0, 1, 2, 3, 4


def fwd(L, X=P, T=4, R=8, E=2, N=64, K=64, offsets=P, token=P, W=P, bias=None, Y=P):
    return L.bsr_expert_fwd(X, T, R, E, N, K, offsets, token, W, bias, Y, None)


@pytest.mark.parametrize("change,status", [
    (dict(E=0), INVALID), (dict(E=1025), INVALID), (dict(N=0), INVALID), (dict(N=12), INVALID), (dict(K=4), INVALID),
    (dict(K=1 << 20), INVALID), (dict(R=-1), INVALID), (dict(R=(1 << 24) + 1), INVALID), (dict(T=-1), INVALID),
    (dict(T=1 << 24, K=1024), INVALID), (dict(N=1 << 18, K=1 << 18), INVALID), (dict(X=None), INVALID),
    (dict(W=None), INVALID), (dict(Y=None), INVALID), (dict(offsets=None), INVALID), (dict(X=P + 2), MISALIGNED),
    (dict(bias=P + 8), MISALIGNED), (dict(token=P + 4), MISALIGNED), (dict(R=0), OK),
    (dict(R=0, X=None, W=None, Y=None, offsets=None, token=None), OK)])
def test_expert_fwd_arguments(change, status):
    L = _lib.load()
    assert fwd(L, **change) == status
    if status:
        assert L.bsr_last_error()


def test_other_arguments():
    L = _lib.load()
    assert L.bsr_expert_bwd_input(P, 8, 2, 12, 64, P, P, P, None) == INVALID
    assert L.bsr_expert_bwd_input(P, 8, 2, 64, 64, P, P, P + 1, None) == MISALIGNED
    assert L.bsr_expert_bwd_input(None, 0, 2, 64, 64, None, None, None, None) == OK
    assert L.bsr_expert_bwd_weight(P, P, 4, 8, 2, 64, 64, P, P, None, None, None) == INVALID
    assert L.bsr_expert_bwd_weight(P, P, 4, 1 << 24, 2, 512, 8, P, P, P, None, None) == INVALID    # dY too large
    for k, E in ((0, 4), (5, 4), (33, 64), (1, 0), (1, 1025)):
        assert L.bsr_router_fwd(P, 0, 4, E, k, 1, P, P, None) == INVALID
        assert L.bsr_expert_plan(P, 4, k, E, P, P, P, None, 0, None) == INVALID
        assert L.bsr_expert_plan_workspace(4, k, E) == 0
    assert L.bsr_router_fwd(P, 2, 4, 8, 2, 1, P, P, None) == UNSUPPORTED
    assert L.bsr_router_fwd(P, 0, 4, 8, 2, 7, P, P, None) == INVALID
    assert L.bsr_router_fwd(P, 0, (1 << 24) + 1, 8, 1, 1, P, P, None) == INVALID
    assert L.bsr_router_bwd(P, 0, 4, 8, 2, 1, P, P, None, P, None) == INVALID
    assert L.bsr_expert_plan_workspace(experts.PLAN_SLOTS // 2, 2, 16) == 0
    assert L.bsr_expert_plan_workspace(experts.PLAN_SLOTS // 2 + 1, 2, 16) > 0
    need = L.bsr_expert_plan_workspace(5000, 2, 16)
    assert need > 0 and L.bsr_expert_plan_workspace(100, 2, 16) == 0
    assert L.bsr_expert_plan(P, 5000, 2, 16, P, P, P, P, need - 1, None) == SMALL
    assert L.bsr_expert_plan(P, 5000, 2, 16, P, P, P, None, need, None) == INVALID
    assert L.bsr_expert_combine_fwd(P, 4, 2, 12, P, P, P, None) == INVALID
    assert L.bsr_expert_combine_fwd(P, 4, 2, 64, P, P, P + 4, None) == MISALIGNED
    assert L.bsr_expert_combine_bwd(P, P, 4, 2, 8, 64, P, P, None, P, None, None) == INVALID
    assert L.bsr_expert_combine_fwd(P, 1 << 24, 1, 1 << 19, P, P, P, None) == INVALID    # more than one launch holds
    assert L.bsr_mx4_quantize(P, 4, 48, P, P, None, None) == INVALID
    assert L.bsr_mx4_quantize(P, -1, 64, P, P, None, None) == INVALID
    assert L.bsr_mx4_quantize(P, 4, 64, P, P + 8, None, None) == MISALIGNED
    assert L.bsr_mx4_quantize(None, 0, 64, None, None, None, None) == OK
    assert L.bsr_mx4_dequantize(P, P, 4, 64, None, None) == INVALID
    assert L.bsr_expert_fwd_mx4(P, 4, 8, 2, 64, 72, P, P, P, P, None, P, None) == INVALID       # K % 32
    assert L.bsr_expert_fwd_mx4(P, 4, 8, 2, 64, 64, P, P, P, None, None, P, None) == INVALID    # no scales
    assert L.bsr_expert_fwd_mx4_mx4(P, None, 4, 8, 2, 64, 64, P, P, P, P, None, P, None) == INVALID


def test_python_calls_refuse_cpu_tensors():
    with pytest.raises(ValueError):
        experts.router_fwd(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError):
        experts.ExpertPlan.from_index(torch.zeros((4, 2), dtype=torch.int32), 8)
    with pytest.raises(ValueError):
        experts.ExpertPlan(torch.zeros(9, dtype=torch.int32), torch.zeros(8, dtype=torch.int32),
                           torch.zeros((4, 2), dtype=torch.int32))
    with pytest.raises(ValueError):
        mx4.quantize(torch.zeros(4, 64, dtype=torch.bfloat16))


@pytest.mark.parametrize("lead,rows,groups", [((), 3, 1), ((), 5, 8), ((2,), 7, 9), ((3,), 4, 40)])
def test_scale_layout(lead, rows, groups):
    g = torch.Generator().manual_seed(rows)
    by_row = torch.randint(0, 256, (*lead, rows, groups), generator=g, dtype=torch.uint8)
    codes = torch.zeros((*lead, rows, 16 * groups), dtype=torch.uint8)
    q = mx4.Mx4.from_rows(codes, by_row)
    assert q.scales.shape == (*lead, -(-groups // 8), rows, 8)
    assert torch.equal(q.scale_rows(), by_row)
    for r in range(rows):
        for i in range(groups):
            assert torch.equal(q.scales[..., i // 8, r, i % 8], by_row[..., r, i])
    assert not q.scales.transpose(-3, -2).reshape(*lead, rows, -1)[..., groups:].any()
    with pytest.raises(ValueError):
        mx4.Mx4.from_rows(codes[..., :-1], by_row)
