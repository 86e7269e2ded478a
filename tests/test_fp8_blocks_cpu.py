"""8-bit block operators and the whole layer for few tokens without a GPU: what the C ABI refuses before anything is enqueued, what
the Python calls pass, and the formats' helpers."""
import numpy as np
import pytest
import torch

import fp8_ref
import test_expert_calls_cpu as calls_cpu
from sparse_gemm_amd import _lib, expert_layer, experts, few_tokens, fp8, mx4
from test_expert_calls_cpu import a_plan, bf, off_by_one
from test_second_derivatives_cpu import E, K, N, Plan, T, leaf

P = 4096     # an aligned address that no refused call reads
OK, INVALID, UNSUPPORTED, MISALIGNED, SMALL = 0, 1, 2, 3, 4
TOP = 0xF0000000


@pytest.fixture
def library(monkeypatch):
    rec = calls_cpu.Recorder()
    rec.bsr_expert_ffn_workspace = lambda *a: 64
    for module in (experts, mx4, fp8, few_tokens):
        monkeypatch.setattr(module, "C", rec)
        monkeypatch.setattr(module, "current_device", lambda: 0)
        monkeypatch.setattr(module, "raw_stream", lambda d: None)
    for module in (experts, mx4, few_tokens):
        monkeypatch.setattr(module, "empty_strided", lambda shape, strides, dtype: torch.empty_strided(shape, strides, dtype=dtype))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    return rec


def why(status, code=INVALID):
    assert status == code
    return _lib.load().bsr_last_error().decode()


def test_the_definition_itself():
    """The table against the format's formula, and rounding against the nearest of all codes."""
    for c in range(256):
        s, e, m = c >> 7, c >> 3 & 15, c & 7
        want = float("nan") if e == 15 and m == 7 else (-1) ** s * (m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        got = fp8_ref.value(np.array(c))
        assert got == want or (np.isnan(got) and np.isnan(want))
    u = np.concatenate([fp8_ref.TABLE, fp8_ref.MIDDLE, np.linspace(0, 448, 4001)])
    codes = fp8_ref.encode(u, 127)
    d = np.abs(fp8_ref.TABLE[None] - u[:, None])
    assert (np.abs(fp8_ref.value(codes) - u) == d.min(1)).all()
    tied = (d == d.min(1, keepdims=True)).sum(1) == 2
    assert tied.sum() >= 126 and (codes[tied] % 2 == 0).all()
    assert [fp8_ref.scale_byte(np.array([a])) for a in (0.0, 448.0, 448.5, 224.0, 225.0, 2.0 ** -133, 2.0 ** -118, np.nan)] == [
        0, 127, 128, 126, 127, 0, 1, 0]   # 448 * 2^-127 is 1.75 * 2^-119, below 2^-118


def test_refused_sizes():
    L = _lib.load()
    for K in (0, 8, 24, -16, 1 << 20):
        assert "K must" in why(L.bsr_fp8_quantize_rows(P, 4, K, P, P, None, None))
        assert "K must" in why(L.bsr_fp8_dequantize_rows(P, P, 4, K, P, None))
        assert "K must" in why(L.bsr_fp8_quantize_blocks(P, 1, 64, K, P, P, None, None, None))
        assert "K must" in why(L.bsr_expert_fwd_fp8(P, 4, 4, 2, 64, K, P, P, P, P, None, P, None))
        assert "K must" in why(L.bsr_expert_fwd_fp8_fp8(P, P, 4, 4, 2, 64, K, P, P, P, P, None, P, None))
    assert "rows" in why(L.bsr_fp8_quantize_rows(P, -1, 64, P, P, None, None))
    for N in (0, 12, 1 << 20):
        assert "N must" in why(L.bsr_fp8_quantize_blocks(P, 1, N, 64, P, P, None, None, None))
        assert "N must" in why(L.bsr_expert_fwd_fp8(P, 4, 4, 2, N, 64, P, P, P, P, None, P, None))
    assert "multiple of 16" in why(L.bsr_fp8_quantize_blocks(P, 1, 24, 64, P, P, P, P, None))
    assert "scales_t is NULL" in why(L.bsr_fp8_quantize_blocks(P, 1, 32, 64, P, P, P, None, None))
    assert "codes_t is NULL" in why(L.bsr_fp8_quantize_blocks(P, 1, 32, 64, P, P, None, P, None))
    for E in (0, 1025):
        assert "E must" in why(L.bsr_fp8_quantize_blocks(P, E, 64, 64, P, P, None, None, None))
        assert "E must" in why(L.bsr_expert_fwd_fp8(P, 4, 4, E, 64, 64, P, P, P, P, None, P, None))
    assert "scales" in why(L.bsr_fp8_quantize_rows(P, 4, 64, P, P + 4, None, None), MISALIGNED)
    # no rows: nothing to do, and nothing to point at
    assert L.bsr_fp8_quantize_rows(None, 0, 64, None, None, None, None) == OK
    assert L.bsr_expert_fwd_fp8(None, 0, 0, 2, 64, 64, None, None, None, None, None, None, None) == OK
    assert L.bsr_expert_fwd_fp8_fp8(None, None, 0, 0, 2, 64, 64, None, None, None, None, None, None, None) == OK


def test_the_largest_operands():
    L = _lib.load()
    wide = 8192
    for bits, call in ((16, lambda T, R, N, tok: L.bsr_expert_fwd_fp8(None, T, R, 8, N, wide, P, tok, P, P, None, P, None)),
                       (8, lambda T, R, N, tok: L.bsr_expert_fwd_fp8_fp8(None, P, T, R, 8, N, wide, P, tok, P, P, None, P, None))):
        top = TOP * 8 // (bits * wide)
        for rows, want in ((top, "is NULL"), (top + 8, "more than 0xF0000000 bytes")):
            assert want in why(call(rows, 8, 64, P)) and want in why(call(0, rows, 64, None))
        top = TOP // wide
        for N, want in ((top, "is NULL"), (top + 8, "more than 0xF0000000 bytes")):
            assert want in why(call(8, 8, N, P))


def ffn(T=2, dim=64, hidden=64, E=4, k=2, renorm=1, form=0, ws=1 << 20, **over):
    a = dict(x=P, router=P, up=P, up_scales=P, down=P, down_scales=P, up_bias=None, down_bias=None, out=P, workspace=P)
    a.update(over)
    return _lib.load().bsr_expert_ffn(a["x"], T, dim, hidden, E, k, renorm, a["router"], form, a["up"], a["up_scales"], a["down"],
                                      a["down_scales"], a["up_bias"], a["down_bias"], a["out"], a["workspace"], ws, None)


def test_refused_layers():
    for T in (17, -1):
        assert "T" in why(ffn(T=T))
    for dim in (0, 12, 1 << 20):
        assert "dim must" in why(ffn(dim=dim))
    for hidden in (0, 4, 1 << 19):
        assert "hidden must" in why(ffn(hidden=hidden))
    assert "E must" in why(ffn(E=1025))
    for k in (0, 5, 33):
        assert "k must" in why(ffn(E=4 if k < 6 else 64, k=k))
    assert "renormalize" in why(ffn(renorm=2))
    assert "weights must" in why(ffn(form=3), UNSUPPORTED)
    assert "multiples of 16" in why(ffn(form=2, dim=72)) and "multiples of 32" in why(ffn(form=1, hidden=48))
    assert "more than 0xF0000000 bytes" in why(ffn(dim=65536, hidden=32768))
    for name in ("x", "router", "up", "down", "out", "workspace"):
        assert f"{name} is NULL" in why(ffn(**{name: None}))
        assert name in why(ffn(**{name: P + 8}), MISALIGNED)
    for name in ("up_scales", "down_scales"):
        assert f"{name} is NULL" in why(ffn(form=1, **{name: None})) and f"{name} is NULL" in why(ffn(form=2, **{name: None}))
    need = _lib.load().bsr_expert_ffn_workspace(2, 64, 64, 4, 2)
    assert need > 0 and "workspace" in why(ffn(ws=need - 1), SMALL)
    assert ffn(T=0, ws=0, x=None, out=None, router=None, up=None, down=None, workspace=None) == OK
    assert _lib.load().bsr_expert_ffn_workspace(17, 64, 64, 4, 2) == 0


def test_scale_rows_are_laid_out():
    rows, K = 5, 1040      # 9 groups, 3 chunks of 4
    scale_rows = torch.arange(rows * 9, dtype=torch.uint8).reshape(rows, 9)
    q = fp8.Fp8Rows.from_rows(torch.zeros(rows, K, dtype=torch.uint8), scale_rows)
    assert q.scales.shape == (3, rows, 4) and q.shape == (rows, K)
    for r in range(rows):
        for g in range(12):
            assert q.scales[g // 4, r, g % 4] == (scale_rows[r, g] if g < 9 else 0)
    assert torch.equal(q.scale_rows(), scale_rows)
    with pytest.raises(ValueError):
        fp8.Fp8Rows.from_rows(torch.zeros(rows, K, dtype=torch.uint8), scale_rows[:, :8])


def test_arguments_reach_the_library(library):
    plan, W = a_plan(), bf(3, 64, 64)
    q, qt = fp8.quantize_blocks(W, transposed=True)
    y = fp8.expert_fwd(plan, bf(4, 64), q)
    z = fp8.expert_fwd(plan, fp8.quantize_rows(y), qt, gather=False)
    (n0, a0), (n1, a1), (n2, a2), (n3, a3) = library.calls
    assert (n0, n1, n2, n3) == ("bsr_fp8_quantize_blocks", "bsr_expert_fwd_fp8", "bsr_fp8_quantize_rows", "bsr_expert_fwd_fp8_fp8")
    assert a0[:9] == (W.data_ptr(), 3, 64, 64, q.codes.data_ptr(), q.scales.data_ptr(), qt.codes.data_ptr(), qt.scales.data_ptr(), None)
    assert a1[1:6] == (4, 8, 3, 64, 64) and a1[6] == plan.offsets.data_ptr() and a1[7] == plan.row_token.data_ptr()
    assert a3[8] is None and z.shape == (8, 64)
    up, down = bf(3, 128, 64), bf(3, 64, 64)
    out = few_tokens.expert_ffn(bf(4, 64), bf(3, 64), up, down, 2, renormalize=False)
    name, a = library.calls[-1]
    assert name == "bsr_expert_ffn" and out.shape == (4, 64)
    assert a[1:7] == (4, 64, 64, 3, 2, False) and a[8:13] == (0, up.data_ptr(), None, down.data_ptr(), None)


def test_what_a_gradient_needs(library):
    """No transposed weights where the input wants no gradient, no weight gradient where none is wanted."""
    plan = a_plan()
    for want_x in (False, True):
        for want_w in (False, True):
            x, W = bf(4, 64).requires_grad_(want_x), bf(3, 64, 64).requires_grad_(want_w)
            library.calls.clear()
            y = expert_layer.expert_linear_fp8(plan, x, W)
            (name, args), = [c for c in library.calls if c[0] == "bsr_fp8_quantize_blocks"]
            assert (args[6] is not None) == want_x
            if want_x or want_w:
                library.calls.clear()
                y.backward(bf(8, 64))
                names = [n for n, _ in library.calls]
                assert ("bsr_expert_fwd_fp8_fp8" in names) == want_x and ("bsr_expert_bwd_weight" in names) == want_w
    with torch.no_grad():
        library.calls.clear()
        expert_layer.expert_linear_fp8(plan, bf(4, 64).requires_grad_(), bf(3, 64, 64))
        assert library.calls[0][1][6] is None


def test_slices_are_copied(library, monkeypatch):
    def aligned(rec, name):
        def call(*args):
            assert not [a for a in args if isinstance(a, int) and a > 1 << 20 and a % 16], name
            return 0
        return call

    monkeypatch.setattr(calls_cpu.Recorder, "__getattr__", aligned)
    plan = a_plan(3, 1, 3)
    x = off_by_one(bf(3, 64)).requires_grad_()
    expert_layer.expert_linear_fp8(plan, x, bf(3, 64, 64).requires_grad_(), bf(3, 64).requires_grad_()).backward(off_by_one(bf(3, 64)))
    expert_layer.expert_ffn(off_by_one(bf(3, 64)), bf(3, 64), bf(3, 128, 64), bf(3, 64, 64), 1)


def test_sizes_past_32_bits_are_refused(library):
    big = (1 << 32) + 64
    meta = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="meta")   # noqa: E731
    plan, u8 = a_plan(1, 1, 1), torch.uint8
    for call in (lambda: fp8.quantize_rows(meta(1, big)), lambda: fp8.quantize_blocks(meta(big, 64)), lambda: fp8.quantize_blocks(meta(1, 64, big)),
                 lambda: fp8.dequantize(fp8.Fp8Rows(meta(1, big, dtype=u8), meta(big // 512 + 1, 1, 4, dtype=u8))),
                 lambda: fp8.dequantize(fp8.Fp8Blocks(meta(big, 64, dtype=u8), meta(big // 128 + 1, 1, dtype=u8))),
                 lambda: fp8.expert_fwd(plan, meta(1, 64), fp8.Fp8Blocks(meta(1, big, 64, dtype=u8), meta(1, big // 128 + 1, 1, dtype=u8))),
                 lambda: few_tokens.expert_ffn(meta(1, big), meta(1, big), meta(1, 64, big), meta(1, big, 32), 1),
                 lambda: few_tokens.expert_ffn(meta(1, 64), meta(1, 64), meta(1, big, 64), meta(1, 64, big // 2), 1)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
        assert not library.calls


def test_a_layer_without_a_gpu():
    W, q = bf(3, 128, 64), fp8.Fp8Blocks(torch.zeros(3, 64, 64, dtype=torch.uint8), torch.zeros(3, 1, 1, dtype=torch.uint8))
    for call in (lambda: fp8.quantize_rows(bf(4, 64)), lambda: fp8.quantize_blocks(W), lambda: fp8.dequantize(q),
                 lambda: few_tokens.expert_ffn(bf(4, 64), bf(3, 64), W, bf(3, 64, 64), 2)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_the_layer_modules_choice(library):
    """Few tokens that want no gradient take one call; all others take the single calls."""
    m = expert_layer.ExpertFFN(64, 64, 4, 2, device="cpu", decode_tokens=8)
    ffn_called = lambda: any(n == "bsr_expert_ffn" for n, _ in library.calls)   # noqa: E731
    for tokens, grad, want in ((8, False, True), (9, False, False), (8, True, False), (0, False, False)):
        library.calls.clear()
        with torch.set_grad_enabled(grad):
            assert m(bf(tokens, 64)).shape == (tokens, 64)
        assert ffn_called() == want
    m.requires_grad_(False)
    library.calls.clear()
    m(bf(1, 64))
    assert ffn_called()
    library.calls.clear()
    m(bf(1, 64).requires_grad_())
    assert not ffn_called()
    with pytest.raises(RuntimeError, match="no backward"):
        expert_layer.expert_ffn(bf(1, 64).requires_grad_(), m.router, m.up, m.down, 2)
    for bad in (dict(decode_tokens=17), dict(decode_tokens=-1)):
        with pytest.raises(ValueError):
            expert_layer.ExpertFFN(64, 64, 4, 2, device="cpu", **bad)
    with pytest.raises(ValueError):
        expert_layer.ExpertFFN(72, 64, 4, 2, device="cpu", fp8=True)
    t = expert_layer.ExpertFFN(64, 64, 4, 2, device="cpu", fp8=True)
    library.calls.clear()
    t(bf(5, 64)).sum().backward()
    names = [n for n, _ in library.calls]
    assert names.count("bsr_expert_fwd_fp8_fp8") == 3 and "bsr_expert_fwd" not in names   # x of the layer wants no gradient
    q = expert_layer.ExpertFFN(64, 64, 4, 2, device="cpu").quantize_("fp8")
    for tokens, name in ((64, "bsr_expert_fwd_fp8"), (65, "bsr_expert_fwd_fp8_fp8")):
        library.calls.clear()
        assert q(bf(tokens, 64)).shape == (tokens, 64)
        assert [n for n, _ in library.calls].count(name) == 2
    del t.__dict__["fp8"], t.__dict__["decode_tokens"]   # a layer that was stored before it had them
    t(bf(5, 64))


@pytest.mark.parametrize("outer", ["sum", "square"])
def test_second_derivatives_are_refused(monkeypatch, outer):
    """Stand-ins compute on the CPU, without rounding."""
    class Held:
        def __init__(self, codes, scales):
            self.codes, self.scales = codes, scales

    one = torch.ones(1)
    monkeypatch.setattr(fp8, "Fp8Blocks", Held)
    monkeypatch.setattr(fp8, "quantize_rows", lambda x: x)
    monkeypatch.setattr(fp8, "quantize_blocks", lambda W, transposed=False: (
        (Held(W, one), Held(W.transpose(1, 2).contiguous(), one)) if transposed else Held(W, one)))
    monkeypatch.setattr(fp8, "expert_fwd", lambda plan, x, W, bias=None, gather=True: x @ W.codes[0].t())
    monkeypatch.setattr(experts, "expert_bwd_weight", lambda plan, dY, x, gather, want, want_dW: ((dY.t() @ x)[None], None))
    monkeypatch.setattr(experts, "combine_fwd", lambda plan, Y, w=None: Y.clone())
    x, s, W = leaf(T, K), leaf(T, K), leaf(1, N, K)
    out = expert_layer.expert_linear_fp8(Plan, x * s, W)
    loss = out.sum() if outer == "sum" else (out * out).sum()
    plain = torch.autograd.grad(loss, [x, s, W], retain_graph=True)
    first = torch.autograd.grad(loss, [x, s, W], create_graph=True)
    for a, b in zip(plain, first):
        assert torch.equal(a, b)
    for leafs in ([s], [W]):
        with pytest.raises(RuntimeError, match="second derivatives"):
            torch.autograd.grad(first[0].float().pow(2).sum(), leafs, retain_graph=True)
