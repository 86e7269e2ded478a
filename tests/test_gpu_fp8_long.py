"""Products on 8-bit weights over long contractions, on whole numbers: every product and sum is a whole number below 2^24, so that the
result is the exact sum rounded to bf16 once, and one lost or doubled column shows. (Codes of whole numbers to 8 with a scale of 1 are
themselves; of eight neighbouring products the largest is at most 64, and the matrix instruction drops nothing above 2^-13 of it.)"""
import pytest
import torch

from gpu_util import dev, say
from sparse_gemm_amd import experts, fp8
from sparse_gemm_amd.fp8 import Fp8Blocks, Fp8Rows

pytestmark = pytest.mark.gpu


def whole(g, *shape):
    return torch.randint(-8, 9, shape, generator=g, device=dev()).float()


def codes_of(v):
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def blocks(W):
    E, N, K = W.shape
    return Fp8Blocks(codes_of(W), torch.full((E, -(-N // 128), -(-K // 128)), 127, dtype=torch.uint8, device=dev()))


def rows(x):
    R, K = x.shape
    return Fp8Rows.from_rows(codes_of(x), torch.full((R, -(-K // 128)), 127, dtype=torch.uint8, device=dev()))


# rows, experts, columns: tiles of 16, 32, 64, 128 and 256 rows
@pytest.mark.parametrize("R,E,N", [(1, 1, 264), (5, 3, 264), (60, 3, 1032), (150, 3, 1032), (700, 2, 520), (3000, 2, 2056)])
@pytest.mark.parametrize("K", [8208, 16400, 32784])
@pytest.mark.parametrize("eight", [False, True])
def test_whole_numbers(eight, R, E, N, K):
    say(f"case whole numbers R={R} E={E} N={N} K={K} eight={eight}")
    g = torch.Generator(device=dev()).manual_seed(R + N + K)
    x, W = whole(g, R, K), whole(g, E, N, K)
    index = torch.randint(0, E, (R, 1), generator=g, device=dev(), dtype=torch.int32)
    plan = experts.ExpertPlan.from_index(index, E)
    y = fp8.expert_fwd(plan, rows(x) if eight else x.bfloat16(), blocks(W))
    off, tok = plan.offsets.tolist(), plan.row_token.long()
    for e in range(E):
        want = x[tok[off[e]:off[e + 1]]].double() @ W[e].double().t()
        assert torch.equal(y[off[e]:off[e + 1]].double(), want.bfloat16().double())


def test_every_column_counts():
    """One value of x at a time: the result is that column of W, at every place of a long row."""
    E, N, K = 1, 136, 16400
    g = torch.Generator(device=dev()).manual_seed(3)
    W = whole(g, E, N, K)
    W[W == 0] = 3
    at = torch.cat([torch.arange(0, 520), torch.arange(8100, 8300), torch.arange(16000, K)]).to(dev())
    x = torch.zeros(len(at), K, device=dev())
    x[torch.arange(len(at), device=dev()), at] = 1
    for R in (1, 9, 40, 120, len(at)):
        plan = experts.ExpertPlan.from_index(torch.zeros((R, 1), dtype=torch.int32, device=dev()), 1)
        for first in range(0, len(at) - R + 1, max(R, 97)):
            part = x[first:first + R]
            want = W[0, :, at[first:first + R]].t().contiguous()
            for act in (part.bfloat16(), rows(part)):
                assert torch.equal(fp8.expert_fwd(plan, act, blocks(W)).float(), want), (R, first)
