"""8-bit floating point with a scale for each block of 128 on the GPU: quantisation and expansion bit for bit against the
definition, the grouped products and their gradients against 64 bits."""
import math

import numpy as np
import pytest
import torch

import expert_ref as ref
import fp8_ref
from expert_ref import f64, near_bf16
from gpu_util import dev, say
from sparse_gemm_amd import _lib, expert_layer, experts, fp8
from sparse_gemm_amd.fp8 import Fp8Blocks, Fp8Rows
from test_gpu_experts import a_plan, gen, PRODUCTS

pytestmark = pytest.mark.gpu


def in_bf16(want):
    """Values as bf16 holds them: (2 - 2^-7) 2^127 is its largest, and rounds to the code of 256 * 2^120 = 2^128, past its range."""
    return np.where(np.abs(want) >= 2.0 ** 128, np.copysign(math.inf, want), want)


def whole(t):
    return t.cpu().numpy().astype(np.int64)


def hard(rows, K, seed):
    """Normal values of very different sizes, with ties, zeros, subnormals, the largest finite values, NaN and infinities."""
    g = gen(seed)
    x = (torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g).float())).bfloat16()
    top = float(torch.finfo(torch.bfloat16).max)
    ties = torch.tensor([448.0, 432.0, 208.0, 17.0, 19.0, 2.0 ** -7, 3 * 2.0 ** -10, 2.0 ** -10, -(2.0 ** -10), 5 * 2.0 ** -10, -0.0,
                         0.0, 15.5, -14.5, 300.0, 464.0]).bfloat16()
    for i in range(rows):
        f = [1.0, 2.0 ** -100, 2.0 ** 100, 2.0 ** -126, 2.0 ** 119][i % 5]
        n = min(16, K)
        if i % 3 == 0:
            x[i, :n] = ties[:n] * f
        if i % 3 == 1 and i > 1:
            v = [0.0, 2.0 ** -133, 3 * 2.0 ** -130, top, math.nan, math.inf, -math.inf, -math.nan, 449.0, 450.0][i // 3 % 10]
            if v == 0.0 or abs(v) < 2.0 ** -100:
                x[i] = 0.0
            x[i, (7 * i) % K] = v
            if i % 2:
                x[i, (7 * i + 1) % K] = -v
    if rows > 8:
        x[8] = math.nan      # nothing finite
    return x


@pytest.mark.parametrize("rows,K", [(1, 16), (16, 32), (3, 128), (31, 144), (64, 512), (33, 528), (9, 1040), (2, 4096), (70, 2064)])
def test_quantize_rows_bit_exact(rows, K):
    say(f"case fp8 rows rows={rows} K={K}")
    x = hard(rows, K, rows + K)
    q, values = fp8.quantize_rows(x.to(dev()), want_values=True)
    plain = fp8.quantize_rows(x.to(dev()))
    assert torch.equal(plain.codes, q.codes) and torch.equal(plain.scales, q.scales)
    rc, rb = fp8_ref.quantize_rows(f64(x))
    assert np.array_equal(whole(q.scale_rows()), rb)
    assert np.array_equal(whole(q.codes), rc)
    pad = whole(q.scales).transpose(1, 0, 2).reshape(rows, -1)[:, rb.shape[1]:]
    assert not pad.any()
    want = in_bf16(fp8_ref.row_values(rc, rb))
    for got in (values, fp8.dequantize(q)):
        assert np.array_equal(f64(got), want, equal_nan=True)
        assert np.array_equal(np.signbit(f64(got))[~np.isnan(want)], np.signbit(want)[~np.isnan(want)])
    back = Fp8Rows.from_rows(q.codes, q.scale_rows())
    assert torch.equal(back.scales, q.scales)


@pytest.mark.parametrize("lead,N,K", [((), 8, 16), ((), 128, 128), ((2,), 136, 144), ((3,), 264, 400), ((1,), 24, 1040), ((), 392, 16)])
@pytest.mark.parametrize("transposed", [False, True])
def test_quantize_blocks_bit_exact(lead, N, K, transposed):
    if transposed and N % 16:
        N += 8
    say(f"case fp8 blocks {lead} N={N} K={K} transposed={transposed}")
    E = lead[0] if lead else 1
    W = torch.stack([hard(N, K, 7 * N + K + e) for e in range(E)]).reshape(*lead, N, K)
    got = fp8.quantize_blocks(W.to(dev()), transposed=transposed)
    q, qt = got if transposed else (got, None)
    assert q.shape == (*lead, N, K) and q.scales.shape == (*lead, -(-N // 128), -(-K // 128))
    values = f64(fp8.dequantize(q)).reshape(E, N, K)
    for e in range(E):
        rc, rb = fp8_ref.quantize_blocks(f64(W).reshape(E, N, K)[e])
        assert np.array_equal(whole(q.scales).reshape(E, *rb.shape)[e], rb)
        assert np.array_equal(whole(q.codes).reshape(E, N, K)[e], rc)
        assert np.array_equal(values[e], in_bf16(fp8_ref.block_values(rc, rb)), equal_nan=True)
    if transposed:
        assert torch.equal(qt.codes, q.codes.transpose(-1, -2)) and torch.equal(qt.scales, q.scales.transpose(-1, -2))


def test_every_value_is_rounded_like_the_definition():
    """All 65536 bf16 values, in groups whose scale another value sets (scales from the smallest to the largest)."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    tops = torch.tensor([0.0, 2.0 ** -120, 2.0 ** -60, 2.0 ** -7, 1.0, 448.0, 449.0, 2.0 ** 60, 2.0 ** 120]).bfloat16()
    x = torch.zeros(tops.numel(), 65536 // 112, 128, dtype=torch.bfloat16)
    n = 65536 // 112 * 112
    x[:, :, :112] = bits[:n].reshape(1, -1, 112)
    x = x[:, torch.randperm(65536 // 112, generator=gen(0))[:256]]
    x[:, :, 120] = tops[:, None]
    x = torch.cat([x.reshape(-1, 128), torch.nn.functional.pad(bits[n:], (0, 128 - (65536 - n)))[None]])
    q = fp8.quantize_rows(x.to(dev()))
    rc, rb = fp8_ref.quantize_rows(f64(x))
    assert np.array_equal(whole(q.scale_rows()), rb) and np.array_equal(whole(q.codes), rc)


def test_every_code_and_scale_expands_exactly():
    codes = torch.arange(256, dtype=torch.uint8).reshape(1, 256).expand(256, 256).contiguous()
    byte = torch.arange(256, dtype=torch.uint8).reshape(256, 1).expand(256, 2).contiguous()
    q = Fp8Rows.from_rows(codes.to(dev()), byte.to(dev()))
    want = fp8_ref.row_values(whole(codes), whole(byte))
    want = torch.from_numpy(want).to(torch.float32).bfloat16()   # values below 2^-133 or past bf16's range; 64 bits to 32 is exact here
    assert np.array_equal(f64(fp8.dequantize(q)), f64(want), equal_nan=True)
    b = Fp8Blocks(codes[:, :128].contiguous().to(dev()), torch.tensor([[3], [255]], dtype=torch.uint8, device=dev()))
    v = f64(fp8.dequantize(b))
    assert np.isnan(v[128:]).all()
    assert np.array_equal(v[:128], f64(torch.from_numpy(fp8_ref.value(whole(codes[:128, :128])) * 2.0 ** -124).float().bfloat16()), equal_nan=True)


def cut(x, w):
    """By how much products of codes may differ from exact ones: the matrix instruction adds the products of 8 neighbouring columns
    aligned to the largest of their exponents e_x + e_w, and drops what lies below 2^-13 of that power of two (found with one
    large and one small product at all positions: 2^-13 of it is kept, 2^-14 dropped, in the same eight only). The largest itself has 6
    fraction bits and is whole; each of the 7 others loses less than 2^-13 * 2^(e_x + e_w) <= 2^-13 of the largest product."""
    x, w = (torch.from_numpy(np.abs(v)).to(dev()).float() for v in (x, w))
    out = torch.zeros(x.shape[0], w.shape[0], device=dev())
    for k0 in range(0, x.shape[1], 8):
        top = torch.zeros_like(out)
        for k in range(k0, min(k0 + 8, x.shape[1])):
            top = torch.maximum(top, x[:, k, None] * w[None, :, k])
        out += top
    return f64(out) * 7 * 2.0 ** -13 * (1 + 2.0 ** -10)   # sums of up to 2^13 / 8 groups in 32 bits


def cut_grouped(x, off, W, N):
    """cut of the rows of each expert."""
    out = np.zeros((x.shape[0], N))
    for e in range(len(off) - 1):
        r = slice(int(off[e]), int(off[e + 1]))
        if r.start < r.stop:
            out[r] = cut(x[r], W(e))
    return out


def near(got, want, S, terms, lost=0.0):
    """near_bf16 with what the instruction drops."""
    g = f64(got)
    assert g.shape == want.shape and np.isfinite(g).all()
    tol = 2.0 ** -8 * (np.abs(want) + lost) + lost + (terms + 4) * 2.0 ** -23 * S + 2.0 ** -133
    off = np.abs(g - want)
    assert (off <= tol).all(), f"worst {np.max(off / tol):.3f} of the tolerance at {np.unravel_index(np.argmax(off / tol), want.shape)}"


FP8_PRODUCTS = [(kind, T, k, E, N, max(16, K // 16 * 16)) for kind, T, k, E, N, K in PRODUCTS] + [
    ("ragged", 3, 2, 4, 1024, 2048), ("one", 20, 1, 2, 72, 1040), ("one", 270, 1, 1, 304, 784), ("ragged", 70, 4, 8, 256, 768),
    ("ragged", 10000, 2, 70, 1032, 528), ("ragged", 150, 4, 4, 200, 352),
    ("one", 530, 1, 1, 16392, 96), ("ragged", 400, 2, 2, 12296, 288), ("dropped", 700, 2, 3, 16400, 528), ("ragged", 128, 2, 4, 2056, 784)]


@pytest.mark.parametrize("kind,T,k,E,N,K", FP8_PRODUCTS)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("act", ["bf16", "fp8"])
def test_product(kind, T, k, E, N, K, gather, act):
    say(f"case fp8 product {act} {kind} T={T} k={k} E={E} N={N} K={K} gather={gather}")
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
    Wq = fp8.quantize_blocks(W.to(dev()))
    Wv = f64(fp8.dequantize(Wq))
    Xq = fp8.quantize_rows(X.to(dev()))
    xv = f64(X) if act == "bf16" else f64(fp8.dequantize(Xq))
    x = np.zeros((p.R, K))
    x[:live] = xv[tok[:live]] if gather else xv[:live]
    lost = cut_grouped(x, off, lambda e: Wv[e], N) if act == "fp8" else 0.0
    for bias in (None, torch.randn(E, N, generator=gen(9)).bfloat16()):
        out = torch.full((p.R + 2, N), math.nan, dtype=torch.bfloat16, device=dev())
        y = fp8.expert_fwd(p, X.to(dev()) if act == "bf16" else Xq, Wq, None if bias is None else bias.to(dev()), gather, out=out[:p.R])
        Y, S = ref.grouped(x, off, lambda e: Wv[e], None if bias is None else f64(bias))
        near(y, Y, S, K, lost)
        assert (f64(y)[live:] == 0).all()
        assert torch.isnan(out[p.R:]).all()


@pytest.mark.parametrize("kind,T,k,E,N,K", FP8_PRODUCTS)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("act", ["bf16", "fp8"])
def test_product_of_whole_numbers(kind, T, k, E, N, K, gather, act):
    """Whole numbers up to 15: products are whole and below 2^8, nothing is dropped, sums below 2^24 are exact in any order."""
    say(f"case fp8 whole numbers {act} {kind} T={T} k={k} E={E} N={N} K={K} gather={gather}")
    index, p, (off, tok, row) = a_plan(kind, T, k, E, T)
    live = int(off[-1])
    g = gen(T + K)
    X = torch.randint(-15, 16, (T if gather else p.R, K), generator=g).bfloat16()
    W = torch.randint(-15, 16, (E, N, K), generator=g).bfloat16()
    Wq, Xq = fp8.quantize_blocks(W.to(dev())), fp8.quantize_rows(X.to(dev()))
    y = fp8.expert_fwd(p, X.to(dev()) if act == "bf16" else Xq, Wq, gather=gather)
    want = torch.zeros(p.R, N, device=dev())
    x = (X[tok[:live]] if gather else X[:live]).to(dev()).float()
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        want[a:b] = x[a:b] @ W[e].to(dev()).float().t()
    assert torch.equal(y, want.bfloat16())


@pytest.mark.parametrize("act", ["bf16", "fp8"])
@pytest.mark.parametrize("T", [5, 700])
def test_product_with_scales_of_all_sizes(act, T):
    """Scale bytes far apart within a row and between blocks: products stay exact. NaN and infinite values reach exactly their
    rows and columns."""
    N, K = 264, 656
    g = gen(4)
    spread = lambda n: torch.exp2(torch.randint(-40, 40, (n, -(-K // 128), 1), generator=g).float())   # noqa: E731
    X = (torch.randn(T, -(-K // 128), 128, generator=g) * spread(T)).reshape(T, -1)[:, :K].bfloat16()
    W = (torch.randn(N, -(-K // 128), 128, generator=g) * spread(3).repeat_interleave(128, 0)[:N]).reshape(1, N, -1)[:, :, :K].bfloat16()
    W, X = W.contiguous(), X.contiguous()
    W[0, 7, 100], W[0, 200, 655] = math.nan, math.inf
    X[3, 200] = -math.inf
    p = experts.ExpertPlan.from_index(torch.zeros((T, 1), dtype=torch.int32, device=dev()), 1)
    Wq, Xq = fp8.quantize_blocks(W.to(dev())), fp8.quantize_rows(X.to(dev()))
    y = f64(fp8.expert_fwd(p, X.to(dev()) if act == "bf16" else Xq, Wq))
    xv = f64(X) if act == "bf16" else f64(fp8.dequantize(Xq))
    wv = f64(fp8.dequantize(Wq))[0]
    assert not np.isfinite(y[3]).any() and not np.isfinite(y[:, [7, 200]]).any()
    rows, cols = np.arange(T) != 3, (np.arange(N) != 7) & (np.arange(N) != 200)
    xv, wv, y = xv[rows], wv[cols], y[rows][:, cols]
    want, S = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    lost = cut(xv, wv) if act == "fp8" else 0.0
    tol = 2.0 ** -8 * (np.abs(want) + lost) + lost + (K + 4) * 2.0 ** -23 * S + 2.0 ** -126
    assert (np.abs(y - want) <= tol).all()


LINEARS = [(5, 2, 3, 48, 64, True), (70, 2, 4, 272, 144, False), (300, 1, 1, 128, 528, True), (1, 1, 2, 16, 16, True),
           (600, 4, 8, 256, 256, False), (0, 2, 3, 32, 32, True)]


@pytest.mark.parametrize("T,k,E,N,K,bias", LINEARS)
@pytest.mark.parametrize("gather", [False, True])
def test_linear_gradients(T, k, E, N, K, bias, gather):
    """Against the formula in 64 bits: input gradient of the quantised gradient and weights, weight gradient of x and dY."""
    say(f"case expert_linear_fp8 T={T} k={k} E={E} N={N} K={K} gather={gather}")
    g = gen(T + N)
    index = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32)
    p = experts.ExpertPlan.from_index(index.to(dev()), E)
    off, tok, row = ref.plan(index.numpy(), E)
    R, live = T * k, int(off[-1])
    x = torch.randn(T if gather else R, K, generator=g).bfloat16()
    W = (torch.randn(E, N, K, generator=g) * K ** -0.5).bfloat16()
    b = torch.randn(E, N, generator=g).bfloat16() if bias else None
    dY = torch.randn(R, N, generator=g).bfloat16()
    leaves = [t.to(dev()).requires_grad_() for t in (x, W, b) if t is not None]
    Y = expert_layer.expert_linear_fp8(p, *leaves, *([] if bias else [None]), gather=gather)
    grads = torch.autograd.grad(Y, leaves, dY.to(dev()))
    xq, dq = fp8_ref.row_values(*fp8_ref.quantize_rows(f64(x))), fp8_ref.row_values(*fp8_ref.quantize_rows(f64(dY)))
    Wq = [fp8_ref.block_values(*fp8_ref.quantize_blocks(f64(W[e]))) for e in range(E)]
    rows = lambda v: np.concatenate([v[tok[:live]] if gather else v[:live], np.zeros((R - live, K))])   # noqa: E731
    want, S = ref.grouped(rows(xq), off, lambda e: Wq[e], None if b is None else f64(b))
    near(Y, want, S, K, cut_grouped(rows(xq), off, lambda e: Wq[e], N))
    dX, SX = ref.grouped(dq, off, lambda e: Wq[e].T)
    lost = cut_grouped(dq, off, lambda e: Wq[e].T, K)
    if gather:   # a token's rows, each rounded, then their sum
        token = lambda v: np.stack([v[row[t][row[t] >= 0]].sum(0) for t in range(T)]) if T else np.zeros((0, K))   # noqa: E731
        mags = token(np.abs(dX) + lost)
        dX, SX, lost = token(dX), token(SX), token(lost)
        tol = 2.0 ** -8 * (np.abs(dX) + lost + mags * (1 + 2.0 ** -8)) + lost + (N + k + 4) * 2.0 ** -23 * SX + 2.0 ** -133
        assert (np.abs(f64(grads[0]) - dX) <= tol).all()
    else:
        near(grads[0], dX, SX, N, lost)
    xr, d = rows(f64(x)), f64(dY)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        near_bf16(grads[1][e], d[r].T @ xr[r], np.abs(d[r]).T @ np.abs(xr[r]), R)
        if bias:
            near_bf16(grads[2][e], d[r].sum(0), np.abs(d[r]).sum(0), R)


def test_linear_gradients_against_differences():
    """Small whole numbers: codes, products and results are exact, the function is linear, so differences are the gradients."""
    T, k, E, N, K = 4, 2, 3, 16, 32
    g = gen(5)
    ints = lambda *s: torch.randint(-1, 2, s, generator=g).bfloat16()   # noqa: E731
    index = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    p = experts.ExpertPlan.from_index(index.to(dev()), E)
    x, W, dY = ints(T, K), ints(E, N, K), ints(T * k, N)

    def f(x, W):
        with torch.no_grad():
            return float((f64(expert_layer.expert_linear_fp8(p, x.to(dev()), W.to(dev()))) * f64(dY)).sum())

    leaves = [x.to(dev()).requires_grad_(), W.to(dev()).requires_grad_()]
    dX, dW = torch.autograd.grad(expert_layer.expert_linear_fp8(p, *leaves), leaves, dY.to(dev()))
    for t, c in [(0, 0), (1, 5), (3, 31), (2, 16)]:
        up, dn = x.clone(), x.clone()
        up[t, c] += 1
        dn[t, c] -= 1
        assert (f(up, W) - f(dn, W)) / 2 == float(dX[t, c])
    for e, n, c in [(0, 0, 0), (1, 15, 31), (2, 7, 16)]:
        up, dn = W.clone(), W.clone()
        up[e, n, c] += 1
        dn[e, n, c] -= 1
        assert (f(x, up) - f(x, dn)) / 2 == float(dW[e, n, c])


def test_calls_are_captured_and_replayed():
    """A graph of quantisation, product and expansion follows its inputs, with eager work between the replays."""
    T, k, E, N, K = 40, 2, 4, 272, 400
    g = gen(6)
    p = experts.ExpertPlan.from_index(torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).to(dev()), E)
    x, W = torch.randn(T, K, generator=g).bfloat16().to(dev()), torch.randn(E, N, K, generator=g).bfloat16().to(dev())

    def run():
        q, qt = fp8.quantize_blocks(W, transposed=True)
        y = fp8.expert_fwd(p, fp8.quantize_rows(x), q)
        return y, fp8.expert_fwd(p, x, q), fp8.expert_fwd(p, fp8.quantize_rows(y), qt, gather=False), fp8.dequantize(qt)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(3):
        x.copy_(torch.randn(T, K, generator=g))
        W.copy_(torch.randn(E, N, K, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, run()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [3, 100])
def test_layer_in_8_bits(T):
    """The quantised layer equals the layer whose bf16 weights are the values of the codes: on bf16 activations up to the
    roundings, beyond prompt_tokens up to the activations' rounding to E4M3 (2^-4 of a value at most)."""
    torch.manual_seed(2)
    m = expert_layer.ExpertFFN(128, 256, 4, 2, bias=True, device=dev())
    x = torch.randn(T, 128, device=dev()).bfloat16()
    with torch.no_grad():
        for q in (m.up, m.down):
            q.copy_(fp8.dequantize(fp8.quantize_blocks(q.data)))
        want = m(x).double()
        assert m.form == "bf16" and m.quantize_("fp8") is m and m.form == "fp8" and m.quantize_("fp8") is m
        got = m(x).double()
    rel = float((got - want).norm() / want.norm())
    say(f"    relative difference {rel:.2e}")
    # x, silu(gate) * up: 2^-4 each at most; silu and the product pass on their factors' 2^-4 at most twice
    assert rel < (4 * 2.0 ** -8 if T <= m.prompt_tokens else 4 * 2.0 ** -4)
    with pytest.raises(RuntimeError):
        m(x.requires_grad_())
    with pytest.raises(RuntimeError):
        m.quantize_("mx4")
    with pytest.raises(ValueError):
        m.quantize_("fp4")
    b = expert_layer.ExpertFFN(128, 256, 4, 2, bias=True, device=dev()).quantize_("fp8")
    b.load_state_dict(m.state_dict())
    with torch.no_grad():
        assert torch.equal(b(x), m(x))


def test_refusals():
    d = dev()
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=d)  # noqa: E731
    with pytest.raises(_lib.BsrError, match="multiple of 16"):
        fp8.quantize_rows(bf(4, 24))
    with pytest.raises(TypeError):
        fp8.quantize_rows(bf(4, 64).float())
    with pytest.raises(ValueError):
        fp8.quantize_rows(bf(64, 4).t())
    with pytest.raises(ValueError):
        fp8.quantize_rows(torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(_lib.BsrError, match="multiple of 8"):
        fp8.quantize_blocks(bf(2, 12, 64))
    with pytest.raises(_lib.BsrError, match="multiple of 16"):
        fp8.quantize_blocks(bf(2, 24, 64), transposed=True)
    p = experts.ExpertPlan.from_index(torch.zeros((4, 1), dtype=torch.int32, device=d), 2)
    W = fp8.quantize_blocks(bf(2, 64, 64))
    with pytest.raises(ValueError):
        fp8.expert_fwd(p, bf(4, 96), W)
    with pytest.raises(ValueError):
        fp8.expert_fwd(p, bf(4, 64), Fp8Blocks(W.codes, torch.cat([W.scales, W.scales], 1)))
    with pytest.raises(TypeError):
        fp8.expert_fwd(p, bf(4, 64), Fp8Blocks(W.codes.int(), W.scales))
    with pytest.raises(ValueError):
        fp8.expert_fwd(p, Fp8Rows(torch.zeros((4, 64), dtype=torch.uint8, device=d), torch.zeros((1, 5, 4), dtype=torch.uint8, device=d)), W)
    with pytest.raises(ValueError):
        Fp8Rows.from_rows(W.codes[0], torch.zeros((64, 3), dtype=torch.uint8, device=d))
