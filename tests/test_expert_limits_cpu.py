"""Sizes that the products grouped by expert take and refuse, without a GPU: a call whose sizes pass is refused for the
pointer that is missing, before anything is enqueued."""
import pytest

from sparse_gemm_amd import _lib

P = 4096     # an aligned address that no refused call reads
INVALID, MISALIGNED = 1, 3
TOP = 0xF0000000
BIG, WIDE = 1 << 18, 8192     # rows and columns of 4 GiB in bf16, past the limit of one buffer resource


def why(status):
    assert status == INVALID
    return _lib.load().bsr_last_error().decode()


def test_products_whose_rows_stand_alone_have_no_limit_on_them():
    """The input gradient and the forward of sorted rows read a tile's rows at a time and address what they write with
    64 bits: no matrix of R rows is limited in size."""
    L = _lib.load()
    assert BIG * WIDE * 2 > TOP
    # dX, then dY past the limit
    assert "dY is NULL" in why(L.bsr_expert_bwd_input(None, BIG, 8, 64, WIDE, P, P, P, None))
    assert "dY is NULL" in why(L.bsr_expert_bwd_input(None, BIG, 8, WIDE, 64, P, P, P, None))
    # X, then Y past the limit
    assert "X is NULL" in why(L.bsr_expert_fwd(None, 0, BIG, 8, 64, WIDE, P, None, P, None, P, None))
    assert "X is NULL" in why(L.bsr_expert_fwd(None, 0, BIG, 8, WIDE, 64, P, None, P, None, P, None))


def test_limits_that_stay():
    L = _lib.load()
    assert TOP // (2 * WIDE) * 2 * WIDE == TOP
    top = TOP // (2 * WIDE)       # rows of exactly the limit
    for rows, ok in ((top, True), (top + 8, False)):
        want = "is NULL" if ok else "more than 0xF0000000 bytes"
        # X gathered by token; X and dY of the weight gradient
        assert want in why(L.bsr_expert_fwd(None, rows, 8, 8, 64, WIDE, P, P, P, None, P, None))
        assert want in why(L.bsr_expert_bwd_weight(P, None, rows, 8, 8, 64, WIDE, P, P, P, None, None))
        assert want in why(L.bsr_expert_bwd_weight(P, None, 0, rows, 8, 64, WIDE, P, None, P, None, None))
        assert want in why(L.bsr_expert_bwd_weight(None, P, 4, rows, 8, WIDE, 64, P, P, P, None, None))
        # one expert's weight
        assert want in why(L.bsr_expert_bwd_input(None, 8, 8, rows, WIDE, P, P, P, None))
        assert want in why(L.bsr_expert_fwd(None, 8, 8, 8, rows, WIDE, P, P, P, None, P, None))
        # activations of the 4-bit products, gathered or sorted
        for token, T, R in ((P, rows, 8), (None, 0, rows)):
            assert want in why(L.bsr_expert_fwd_mx4(None, T, R, 8, 64, WIDE, P, token, P, P, None, P, None))
    top = TOP * 2 // WIDE
    for rows, ok in ((top, True), (top + 8, False)):
        want = "is NULL" if ok else "more than 0xF0000000 bytes"
        for token, T, R in ((P, rows, 8), (None, 0, rows)):
            assert want in why(L.bsr_expert_fwd_mx4_mx4(None, P, T, R, 8, 64, WIDE, P, token, P, P, None, P, None))


@pytest.mark.parametrize("R", [-1, (1 << 24) + 1])
def test_rows_out_of_range(R):
    L = _lib.load()
    assert "R must" in why(L.bsr_expert_bwd_input(P, R, 8, 64, 64, P, P, P, None))
    assert "R must" in why(L.bsr_expert_fwd(P, 0, R, 8, 64, 64, P, None, P, None, P, None))


def test_the_weight_gradient_may_be_the_bias_alone():
    L = _lib.load()
    # every pointer in its place but the last, which is refused for its alignment
    assert L.bsr_expert_bwd_weight(P, P, 4, 8, 2, 64, 64, P, P, None, P + 4, None) == MISALIGNED
    assert "dbias" in L.bsr_last_error().decode()
    assert "dW is NULL" in why(L.bsr_expert_bwd_weight(P, P, 4, 8, 2, 64, 64, P, P, None, None, None))
