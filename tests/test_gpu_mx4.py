"""Microscaled 4-bit values on the GPU: quantisation and expansion bit for bit against the format's
definition, the grouped products on them against 64 bits."""
import math

import numpy as np
import pytest
import torch

import expert_ref as ref
from expert_ref import f64, near_bf16
from gpu_util import dev, say
from sparse_gemm_amd import _lib, expert_layer, experts, mx4
from sparse_gemm_amd.mx4 import Mx4
from test_gpu_experts import a_plan, gen, PRODUCTS

pytestmark = pytest.mark.gpu


def unpack(q: Mx4):
    c = q.codes.cpu().numpy().astype(np.int64)
    codes = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)
    return codes, q.scale_rows().cpu().numpy().astype(np.int64)


def hard_rows(rows, K, seed):
    """Normal values of very different sizes, with ties, zeros, subnormals, the largest finite values, NaN
    and infinities in some groups."""
    g = gen(seed)
    x = torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g).float())
    x = x.bfloat16()
    flat = x.reshape(-1, 32)
    n = flat.shape[0]
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 0.0, -0.0, 6.0, 4.0, 7.96875, 0.249, 0.251, 5.03125]).bfloat16()
    for i, f in enumerate([1.0, 2.0 ** -100, 2.0 ** 100, 2.0 ** -126, 2.0 ** 125]):
        if i < n:
            flat[i] = torch.cat([ties, -ties]) * f
    special = [(5, 0.0), (6, 2.0 ** -133), (7, 3 * 2.0 ** -130), (8, float(torch.finfo(torch.bfloat16).max)), (9, math.nan),
               (10, math.inf), (11, -math.inf), (12, -0.0), (13, 2.0 ** -126), (14, 2.0 ** -125), (15, 2.0 ** -124)]
    for i, v in special:
        if i < n:
            flat[i, (i * 5) % 32] = v
            if v == 0.0 or abs(v) < 2.0 ** -120:
                flat[i, torch.arange(32) != (i * 5) % 32] = 0.0
    return x


@pytest.mark.parametrize("rows,K", [(1, 32), (16, 32), (3, 64), (5, 256), (7, 288), (33, 512), (9, 1056), (2, 4096)])
def test_quantize_bit_exact(rows, K):
    say(f"case mx4 quantize rows={rows} K={K}")
    x = hard_rows(rows, K, rows + K)
    q, values = mx4.quantize(x.to(dev()), want_values=True)
    plain = mx4.quantize(x.to(dev()))
    assert torch.equal(plain.codes, q.codes) and torch.equal(plain.scales, q.scales)
    codes, bytes_ = unpack(q)
    rc, rb = ref.mx4_quantize(f64(x))
    assert np.array_equal(bytes_, rb)
    assert np.array_equal(codes, rc)
    pad = q.scales.cpu().numpy().transpose(1, 0, 2).reshape(rows, -1)[:, K // 32:]
    assert not pad.any()
    want = ref.mx4_values(rc, rb)
    for got in (values, mx4.dequantize(q)):
        assert np.array_equal(f64(got), want, equal_nan=True)
        assert np.array_equal(np.signbit(f64(got))[~np.isnan(want)], np.signbit(want)[~np.isnan(want)])


def test_every_code_and_scale_expands_exactly():
    codes = torch.arange(256, dtype=torch.uint8).reshape(1, 16, 16).expand(256, 16, 16).reshape(256, 256).contiguous()
    scale_rows = torch.arange(256, dtype=torch.uint8).reshape(256, 1).expand(256, 16).contiguous()
    q = Mx4.from_rows(codes.to(dev()), scale_rows.to(dev()))
    assert torch.equal(q.scale_rows().cpu(), scale_rows)
    want = ref.mx4_values(*unpack(q))
    most = float(torch.finfo(torch.bfloat16).max)
    want = np.where(np.abs(want) > most, np.copysign(math.inf, want), want)   # 4 * 2^126 and above: past bf16's range
    assert np.array_equal(f64(mx4.dequantize(q)), want, equal_nan=True)


def test_experts_weights_quantize_like_matrices():
    W = torch.randn(3, 40, 320, generator=gen(1)).bfloat16().to(dev())
    q = mx4.quantize(W)
    for e in range(3):
        one = mx4.quantize(W[e])
        assert torch.equal(one.codes, q.codes[e]) and torch.equal(one.scales, q.scales[e])
    assert torch.equal(mx4.dequantize(q)[1], mx4.dequantize(Mx4(q.codes[1], q.scales[1])))
    assert q.shape == (3, 40, 320)


MX_PRODUCTS = [(kind, T, k, E, N, max(32, K // 32 * 32)) for kind, T, k, E, N, K in PRODUCTS] + [
    ("ragged", 3, 2, 4, 1024, 2048), ("one", 20, 1, 2, 72, 1056), ("one", 270, 1, 1, 304, 800), ("ragged", 70, 4, 8, 256, 768),
    ("ragged", 10000, 2, 70, 1032, 544), ("ragged", 150, 4, 4, 200, 352),
    ("one", 530, 1, 1, 16392, 96), ("ragged", 400, 2, 2, 12296, 288), ("dropped", 700, 2, 3, 16400, 544)]


@pytest.mark.parametrize("kind,T,k,E,N,K", MX_PRODUCTS)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("act", ["bf16", "mx4"])
def test_product(kind, T, k, E, N, K, gather, act):
    say(f"case mx4 product {act} {kind} T={T} k={k} E={E} N={N} K={K} gather={gather}")
    index, p, (off, tok, row) = a_plan(kind, T, k, E, T)
    live = int(off[-1])
    g = gen(3)
    X = torch.randn(T if gather else p.R, K, generator=g).bfloat16()
    if gather:
        X[[t for t in range(T) if t not in set(tok[:live].tolist())]] = math.nan
    else:
        X[live:] = math.nan
    W = (torch.randn(E, N, K, generator=g) * K ** -0.5).bfloat16()
    W[np.diff(off) == 0] = math.nan
    Wq = mx4.quantize(W.to(dev()))
    Wv = f64(mx4.dequantize(Wq))
    Xq = mx4.quantize(X.to(dev()))
    xv = f64(X) if act == "bf16" else f64(mx4.dequantize(Xq))
    x = np.zeros((p.R, K))
    x[:live] = xv[tok[:live]] if gather else xv[:live]
    for bias in (None, torch.randn(E, N, generator=gen(9)).bfloat16()):
        out = torch.full((p.R, N), math.nan, dtype=torch.bfloat16, device=dev())
        y = mx4.expert_fwd(p, X.to(dev()) if act == "bf16" else Xq, Wq, None if bias is None else bias.to(dev()), gather, out=out)
        Y, S = ref.grouped(x, off, lambda e: Wv[e], None if bias is None else f64(bias))
        near_bf16(y, Y, S, K)
        assert (f64(y)[live:] == 0).all()


@pytest.mark.parametrize("act", ["bf16", "mx4"])
def test_product_with_scales_of_all_sizes(act):
    """Scale bytes far apart within a row, down to 2^-127 on one side: products stay exact, NaN groups
    reach exactly their rows and columns."""
    T, N, K = 5, 24, 544
    g = gen(4)
    e = torch.randint(-40, 40, (T, K // 32, 1), generator=g).float()
    X = (torch.randn(T, K // 32, 32, generator=g) * torch.exp2(e)).reshape(T, K).bfloat16()
    e = torch.randint(-40, 40, (N, K // 32, 1), generator=g).float()
    W = (torch.randn(N, K // 32, 32, generator=g) * torch.exp2(e)).reshape(1, N, K).bfloat16()
    W[0, 5] = W[0, 5] * 2.0 ** -126 if act == "bf16" else W[0, 5]
    W[0, 7, 100] = math.nan
    p = experts.ExpertPlan.from_index(torch.zeros((T, 1), dtype=torch.int32, device=dev()), 1)
    Wq, Xq = mx4.quantize(W.to(dev())), mx4.quantize(X.to(dev()))
    y = f64(mx4.expert_fwd(p, X.to(dev()) if act == "bf16" else Xq, Wq))
    xv = f64(X) if act == "bf16" else f64(mx4.dequantize(Xq))
    wv = f64(mx4.dequantize(Wq))[0]
    want, S = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    assert np.isnan(y[:, 7]).all()
    keep = np.arange(N) != 7
    tol = 2.0 ** -8 * np.abs(want) + (K + 4) * 2.0 ** -23 * S + 2.0 ** -126
    assert (np.abs(y - want) <= tol)[:, keep].all()


@pytest.mark.parametrize("T", [3, 100])
def test_layer_in_4_bits(T):
    """The quantised layer equals the layer whose bf16 weights are the values of the codes: on bf16 activations
    up to the roundings (the weights' values are bf16 numbers), beyond prompt_tokens up to the activations' own
    4-bit rounding (a quarter of a value at most, 2^-3 of it in the mean square)."""
    torch.manual_seed(2)
    m = expert_layer.ExpertFFN(128, 256, 4, 2, bias=True, device=dev())
    x = torch.randn(T, 128, device=dev()).bfloat16()
    with torch.no_grad():
        for q in (m.up, m.down):
            q.copy_(mx4.dequantize(mx4.quantize(q.data)))
        want = m(x).double()
        m.quantize_()
        got = m(x).double()
    rel = float((got - want).norm() / want.norm())
    say(f"    relative difference {rel:.2e}")
    assert rel < (4 * 2.0 ** -8 if T <= m.prompt_tokens else 0.3)
    with pytest.raises(RuntimeError):
        m(x.requires_grad_())


def test_refusals():
    d = dev()
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=d)  # noqa: E731
    with pytest.raises(_lib.BsrError, match="multiple of 32"):
        mx4.quantize(bf(4, 48))
    with pytest.raises(TypeError):
        mx4.quantize(bf(4, 64).float())
    with pytest.raises(ValueError):
        mx4.quantize(bf(64, 4).t())
    with pytest.raises(ValueError):
        mx4.quantize(torch.zeros(4, 64, dtype=torch.bfloat16))
    p = experts.ExpertPlan.from_index(torch.zeros((4, 1), dtype=torch.int32, device=d), 2)
    W = mx4.quantize(bf(2, 64, 64))
    with pytest.raises(ValueError):
        mx4.expert_fwd(p, bf(4, 96), W)
    with pytest.raises(ValueError):
        mx4.expert_fwd(p, bf(4, 64), Mx4(W.codes, W.scales[:, :, :32].contiguous()))
    with pytest.raises(TypeError):
        mx4.expert_fwd(p, bf(4, 64), Mx4(W.codes.int(), W.scales))
    with pytest.raises(_lib.BsrError, match="multiple of 8"):
        mx4.expert_fwd(p, bf(4, 64), mx4.quantize(bf(2, 12, 64)))
    with pytest.raises(ValueError):
        Mx4.from_rows(W.codes[0], torch.zeros((64, 3), dtype=torch.uint8, device=d))


def test_layer_in_4_bits_keeps_its_weights_in_the_state():
    """A quantised layer's state loads into another quantised layer, and moves with it."""
    torch.manual_seed(3)
    a = expert_layer.ExpertFFN(64, 64, 4, 2, device=dev()).quantize_()
    b = expert_layer.ExpertFFN(64, 64, 4, 2, device=dev()).quantize_()
    assert a.quantize_() is a
    x = torch.randn(9, 64, device=dev()).bfloat16()
    with torch.no_grad():
        assert not torch.equal(a(x), b(x))
        b.load_state_dict(a.state_dict())
        assert torch.equal(a(x), b(x))
        assert a(x[:0]).shape == (0, 64)
