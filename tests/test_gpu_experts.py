"""Expert layers on the GPU against the 64-bit definitions: router and its gradient, the plan, the products
grouped by expert in each direction, the sum and its gradient, the whole layer with autograd."""
import math

import numpy as np
import pytest
import torch
from torch.nn import functional as F

import expert_ref as ref
from expert_ref import f64, near_bf16
from gpu_util import dev, say
from sparse_gemm_amd import _lib, expert_layer, experts
from sparse_gemm_amd.experts import ExpertPlan

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def some_logits(T, E, dtype, seed):
    """Normal logits in steps of 1/8 (many ties), some -inf, some of the type's lowest value, some rows all
    -inf, all of the lowest value or all equal."""
    g = gen(seed)
    x = (torch.randn(T, E, generator=g) * 8).round() / 8
    x[torch.rand(T, E, generator=g) < 0.1] = -math.inf
    x[torch.rand(T, E, generator=g) < 0.05] = torch.finfo(dtype).min
    if T > 4:
        x[1], x[2], x[3] = -math.inf, torch.finfo(dtype).min, 0.0
        x[4] = -math.inf
        x[4, E // 2] = -3.0
    return x.to(dtype)


ROUTES = [(1, 1, 1), (1, 8, 2), (5, 2, 2), (64, 8, 2), (37, 60, 6), (130, 64, 8), (33, 65, 4), (20, 128, 8), (9, 255, 8),
          (7, 256, 1), (6, 1000, 32), (8, 1024, 16), (19, 64, 17),
          (21, 200, 32), (100, 120, 16)]


@pytest.mark.parametrize("T,E,k", ROUTES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
def test_router(T, E, k, dtype, renorm):
    say(f"case router T={T} E={E} k={k} {dtype} renorm={renorm}")
    x = some_logits(T, E, dtype, T + E)
    index, weight = experts.router_fwd(x.to(dev()), k, renorm)
    ri, rw, _ = ref.router(f64(x), k, renorm)
    assert np.array_equal(index.cpu().numpy(), ri)
    assert index.dtype == torch.int32 and weight.dtype == torch.float32
    # exp of a difference of up to 88 and a sum of E terms in 32 bits
    assert np.allclose(f64(weight), rw, rtol=(E + 100) * 2.0 ** -24, atol=1e-37)
    dw = torch.randn(T, k, generator=gen(3))
    d = experts.router_bwd(x.to(dev()), index, weight, dw.to(dev()), renorm)
    assert d.dtype == dtype
    rd = ref.router_grad(f64(x), k, renorm, f64(dw))
    big = np.abs(f64(dw)).max() * k
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert (np.abs(f64(d) - rd) <= u * np.abs(rd) + (2 * E + 200) * 2.0 ** -24 * big * np.maximum(np.abs(rd), rw.max(1, keepdims=True))
            + 1e-37).all()


@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_against_differences(renorm):
    T, E, k = 6, 12, 3
    x = torch.randn(T, E, generator=gen(1)) * 2
    dw = torch.randn(T, k, generator=gen(2))
    index, weight = experts.router_fwd(x.to(dev()), k, renorm)
    d = f64(experts.router_bwd(x.to(dev()), index, weight, dw.to(dev()), renorm))
    h = 1e-6
    for t in range(T):
        for e in range(E):
            up, dn = f64(x), f64(x)
            up[t, e] += h
            dn[t, e] -= h
            diff = ((ref.router(up, k, renorm)[1] - ref.router(dn, k, renorm)[1])[t] * f64(dw)[t]).sum() / (2 * h)
            assert abs(diff - d[t, e]) < 1e-5, (t, e)   # 64-bit differences: h^2 and 1e-16 / h; 32-bit gradient: 1e-6


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_not_finite(dtype, renorm):
    """NaN is chosen first and makes the weights NaN, as +inf does; indexes stay those of the order."""
    x = torch.randn(6, 70, generator=gen(5)).to(dtype)
    x[0, 66] = math.nan
    x[1, 3] = math.inf
    x[2, 5], x[2, 68] = math.inf, math.nan
    x[3] = math.nan
    x[4, 1] = -math.nan
    index, weight = experts.router_fwd(x.to(dev()), 3, renorm)
    ri, _, _ = ref.router(f64(x), 3, renorm)
    assert np.array_equal(index.cpu().numpy(), ri)
    bad = torch.isnan(weight).all(1).cpu().tolist()
    assert bad == [True, True, True, True, True, False]
    d = experts.router_bwd(x.to(dev()), index, weight, torch.ones_like(weight), renorm)
    assert torch.isfinite(d[5]).all() and torch.isnan(d[:5]).any(1).all()


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 8, 64), (3, 2, 5), (64, 2, 8), (128, 8, 64), (129, 8, 64), (1024, 1, 3),
                                   (1025, 1, 1024), (700, 6, 60), (4099, 4, 16), (2500, 32, 1000), (33000, 8, 9), (300000, 2, 300)])
def test_plan(T, k, E):
    say(f"case plan T={T} k={k} E={E}")
    index = torch.randint(-1, E, (T, k), generator=gen(T + k), dtype=torch.int32)
    if T > 10:
        index[3] = E + 7           # out of range: dropped
        index[4] = -2147483648
        index[5:8] = E - 1
    p = ExpertPlan.from_index(index.to(dev()), E)
    clean = index.numpy().astype(np.int64)
    clean[(clean < 0) | (clean >= E)] = -1
    off, tok, row = ref.plan(clean, E)
    assert np.array_equal(p.offsets.cpu().numpy(), off)
    assert np.array_equal(p.row_token.cpu().numpy(), tok)
    assert np.array_equal(p.slot_row.cpu().numpy(), row)


def a_plan(kind, T, k, E, seed):
    """Routings that go wrong easily: ragged, one expert takes all, most experts empty, dropped tokens."""
    g = gen(seed)
    if kind == "ragged":
        index = (torch.randn(T, E, generator=g) + torch.randn(E, generator=g)).topk(min(k, E), 1).indices.int()
    elif kind == "one":
        index = torch.full((T, k), E // 2, dtype=torch.int32)
    elif kind == "dropped":
        index = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32)
        index[torch.rand(T, generator=g) < 0.3] = -1
    else:
        assert kind == "none"
        index = torch.full((T, k), -1, dtype=torch.int32)
    return index, ExpertPlan.from_index(index.to(dev()), E), ref.plan(index.numpy().astype(np.int64), E)


# (T, k, E, N, K): one row; widths of one 16-byte piece; widths that end inside a tile; groups below, at and above tile heights
PRODUCTS = [("ragged", 1, 1, 1, 8, 8), ("ragged", 1, 2, 4, 136, 72), ("ragged", 5, 2, 8, 64, 64), ("ragged", 40, 2, 4, 264, 200),
            ("one", 129, 1, 3, 136, 264), ("ragged", 300, 2, 5, 520, 392), ("dropped", 77, 3, 6, 128, 136), ("none", 9, 2, 3, 40, 24),
            ("one", 600, 1, 1, 264, 520), ("dropped", 257, 4, 70, 72, 96), ("ragged", 33, 4, 64, 1000, 256),
            ("one", 16, 1, 2, 1032, 1000), ("one", 17, 1, 2, 16, 4104), ("ragged", 1100, 2, 2, 776, 328),
            ("dropped", 2050, 2, 3, 512, 512)]


# more than 64 experts, rows and columns for 256 x 256 tiles in every direction
LARGE = [("ragged", 11000, 3, 130, 520, 1032), ("dropped", 10000, 2, 70, 1032, 520), ("dropped", 9000, 1, 2, 712, 2056)]

# enough rows and columns for 256 x 256 tiles: (T, k, E, N, K) of the forward; the input gradient swaps N and K
WIDE = [("one", 530, 1, 1, 16392, 72), ("ragged", 400, 2, 2, 12296, 200), ("dropped", 700, 2, 3, 16400, 264)]


def product_inputs(kind, T, k, E, N, K, gather, seed=0):
    index, p, (off, tok, row) = a_plan(kind, T, k, E, seed + T)
    g = gen(seed + 7)
    R, live = p.R, int(off[-1])
    X = torch.randn(T if gather else R, K, generator=g).bfloat16()
    W = (torch.randn(E, N, K, generator=g) * K ** -0.5).bfloat16()
    dY = torch.randn(R, N, generator=g).bfloat16()
    # what no result may depend on: tokens without a row, rows past the plan, experts without rows
    if gather:
        X[[t for t in range(T) if t not in set(tok[:live].tolist())]] = math.nan
    else:
        X[live:] = math.nan
    dY[live:] = math.inf
    W[np.diff(off) == 0] = math.nan
    x = np.zeros((R, K))
    x[:live] = f64(X)[tok[:live]] if gather else f64(X)[:live]
    return p, off, live, X, W, dY, x


@pytest.mark.parametrize("kind,T,k,E,N,K", PRODUCTS + LARGE + WIDE)
@pytest.mark.parametrize("gather", [False, True])
def test_expert_fwd(kind, T, k, E, N, K, gather):
    say(f"case expert_fwd {kind} T={T} k={k} E={E} N={N} K={K} gather={gather}")
    p, off, live, X, W, _, x = product_inputs(kind, T, k, E, N, K, gather)
    for bias in (None, torch.randn(E, N, generator=gen(9)).bfloat16()):
        out = torch.full((p.R, N), math.nan, dtype=torch.bfloat16, device=dev())
        y = experts.expert_fwd(p, X.to(dev()), W.to(dev()), None if bias is None else bias.to(dev()), gather, out=out)
        assert y is out
        Y, S = ref.grouped(x, off, lambda e: f64(W[e]), None if bias is None else f64(bias))
        near_bf16(y, Y, S, K)
        assert (f64(y)[live:] == 0).all()


@pytest.mark.parametrize("kind,T,k,E,N,K", PRODUCTS + LARGE + [(kind, T, k, E, K, N) for kind, T, k, E, N, K in WIDE])
def test_expert_bwd_input(kind, T, k, E, N, K):
    say(f"case expert_bwd_input {kind} T={T} k={k} E={E} N={N} K={K}")
    p, off, live, _, W, dY, _ = product_inputs(kind, T, k, E, N, K, False)
    out = torch.full((p.R, K), math.nan, dtype=torch.bfloat16, device=dev())
    dX = experts.expert_bwd_input(p, dY.to(dev()), W.to(dev()), out=out)
    g = f64(dY)
    g[live:] = 0
    Y, S = ref.grouped(g, off, lambda e: f64(W[e]).T)
    near_bf16(dX, Y, S, N)


@pytest.mark.parametrize("kind,T,k,E,N,K", PRODUCTS + LARGE + [("ragged", 130, 2, 3, 2056, 2056), ("dropped", 300, 1, 25, 776, 520),
                                                         ("ragged", 500, 2, 7, 1032, 1544), ("one", 2200, 1, 25, 776, 520),
                                                         ("one", 1600, 1, 2, 136, 200), ("dropped", 2300, 2, 2, 264, 72)])
@pytest.mark.parametrize("gather", [False, True])
def test_expert_bwd_weight(kind, T, k, E, N, K, gather):
    say(f"case expert_bwd_weight {kind} T={T} k={k} E={E} N={N} K={K} gather={gather}")
    p, off, live, X, W, dY, x = product_inputs(kind, T, k, E, N, K, gather)
    out = torch.full((E, N, K), math.nan, dtype=torch.bfloat16, device=dev())
    dW, db = experts.expert_bwd_weight(p, dY.to(dev()), X.to(dev()), gather, True, out=out)
    again, none = experts.expert_bwd_weight(p, dY.to(dev()), X.to(dev()), gather)
    assert none is None and torch.equal(dW, again)
    g = f64(dY)
    rw, rs = np.zeros((E, N, K)), np.zeros((E, N, K))
    rb, bs = np.zeros((E, N)), np.zeros((E, N))
    for e in range(E):
        r = slice(off[e], off[e + 1])
        rw[e], rs[e] = g[r].T @ x[r], np.abs(g[r]).T @ np.abs(x[r])
        rb[e], bs[e] = g[r].sum(0), np.abs(g[r]).sum(0)
    near_bf16(dW, rw, rs, live)
    near_bf16(db, rb, bs, live)


def test_products_without_tokens():
    p = ExpertPlan.from_index(torch.empty((0, 2), dtype=torch.int32, device=dev()), 3)
    X = torch.empty((0, 64), dtype=torch.bfloat16, device=dev())
    W = torch.randn(3, 40, 64, device=dev()).bfloat16()
    assert experts.expert_fwd(p, X, W).shape == (0, 40)
    dY = torch.empty((0, 40), dtype=torch.bfloat16, device=dev())
    assert experts.expert_bwd_input(p, dY, W).shape == (0, 64)
    dW, db = experts.expert_bwd_weight(p, dY, X, want_dbias=True)
    assert not dW.any() and not db.any()
    assert experts.combine_fwd(p, dY, torch.empty((0, 2), device=dev())).shape == (0, 40)


@pytest.mark.parametrize("kind,T,k,E,N", [("ragged", 1, 1, 2, 8), ("ragged", 7, 2, 4, 72), ("dropped", 50, 3, 6, 520),
                                          ("none", 4, 2, 3, 16), ("ragged", 33, 8, 64, 4104), ("dropped", 130, 32, 40, 264),
                                          ("one", 300, 1, 2, 2048), ("dropped", 40000, 2, 8, 16)])
def test_combine(kind, T, k, E, N):
    say(f"case combine {kind} T={T} k={k} E={E} N={N}")
    index, p, (off, tok, row) = a_plan(kind, T, k, E, T)
    live = int(off[-1])
    g = gen(11)
    Y = torch.randn(p.R, N, generator=g).bfloat16()
    Y[live:] = math.nan
    w = torch.rand(T, k, generator=g)
    w[torch.from_numpy(row < 0)] = math.nan
    dout = torch.randn(T, N, generator=g).bfloat16()
    y, d, ww = f64(Y), f64(dout), f64(w)
    for weighted in (True, False):
        a = ww if weighted else np.ones_like(ww)
        ro, so = np.zeros((T, N)), np.zeros((T, N))
        rd, rw, sw = np.zeros((p.R, N)), np.zeros((T, k)), np.zeros((T, k))
        for t in range(T):
            for j in range(k):
                if row[t, j] >= 0:
                    ro[t] += a[t, j] * y[row[t, j]]
                    so[t] += np.abs(a[t, j] * y[row[t, j]])
                    rd[row[t, j]] = a[t, j] * d[t]
                    rw[t, j], sw[t, j] = (d[t] * y[row[t, j]]).sum(), np.abs(d[t] * y[row[t, j]]).sum()
        wd = w.to(dev()) if weighted else None
        near_bf16(experts.combine_fwd(p, Y.to(dev()), wd), ro, so, k)
        dY, dw = experts.combine_bwd(p, dout.to(dev()), Y.to(dev()), wd)
        near_bf16(dY, rd, np.abs(rd), 1)
        assert (np.abs(f64(dw) - rw) <= (N + 4) * 2.0 ** -23 * sw).all()


def test_a_plan_that_does_not_fit_stays_in_bounds():
    """offsets, row_token and slot_row beyond the arrays give no access out of bounds: results of the rows
    that do fit are right, the outputs' neighbours keep their contents."""
    E, N, K, T = 2, 64, 64, 4
    X, W = torch.randn(T, K).bfloat16().to(dev()), torch.randn(E, N, K).bfloat16().to(dev())
    p = ExpertPlan(torch.tensor([-5, 2, 1000], dtype=torch.int32, device=dev()),
                   torch.tensor([0, 9, -7, 3], dtype=torch.int32, device=dev()),
                   torch.tensor([[0], [77], [-3], [3]], dtype=torch.int32, device=dev()))
    guarded = torch.full((3, p.R, N), 7.0, dtype=torch.bfloat16, device=dev())
    y = experts.expert_fwd(p, X, W, out=guarded[1])
    assert (guarded[0] == 7).all() and (guarded[2] == 7).all()
    near_bf16(y[0], f64(X[0]) @ f64(W[0]).T, np.abs(f64(X[0])) @ np.abs(f64(W[0])).T, K)
    near_bf16(y[3], f64(X[3]) @ f64(W[1]).T, np.abs(f64(X[3])) @ np.abs(f64(W[1])).T, K)
    out = experts.combine_fwd(p, y)
    assert torch.equal(out[0], y[0]) and torch.equal(out[3], y[3]) and not out[1:3].any()
    experts.expert_bwd_weight(p, y, X)
    torch.cuda.synchronize()


def ffn_reference(m, x, dout):
    """The layer in 64 bits on the CPU with autograd; the router's choice is taken from the 64-bit logits."""
    P = {n: q.detach().cpu().double().requires_grad_() for n, q in m.named_parameters()}
    x = x.detach().cpu().double().requires_grad_()
    logits = (x @ P["router"].t()).detach().to(torch.bfloat16).double() + (x @ P["router"].t() - (x @ P["router"].t()).detach())
    index = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :m.k]
    w = torch.softmax(torch.gather(logits, 1, index), 1) if m.renormalize else torch.gather(torch.softmax(logits, 1), 1, index)
    rows = []
    for t in range(x.shape[0]):
        acc = 0
        for j in range(m.k):
            e = int(index[t, j])
            h = P["up"][e] @ x[t] + (P["up_bias"][e] if "up_bias" in P else 0)
            h = F.silu(h[:m.hidden]) * h[m.hidden:]
            acc = acc + w[t, j] * (P["down"][e] @ h + (P["down_bias"][e] if "down_bias" in P else 0))
        rows.append(acc)
    y = torch.stack(rows)
    y.backward(dout.cpu().double())
    return y.detach(), x.grad, {n: q.grad for n, q in P.items()}


@pytest.mark.parametrize("T,k,E,N,K", [(30, 2, 4, 72, 40), (700, 2, 3, 264, 136)])
def test_product_and_sum_gradients_against_differences(T, k, E, N, K):
    """L = <dout, combine(x W^T + b, w)> in 64 bits, moved by +-h along a random direction of each input, against the
    gradients' product with that direction. A gradient's elements are off by a few roundings to bf16 (the sum's
    gradient, the product's, the sum over a token's rows), each at most 2^-8 of what it rounds."""
    index, p, (off, tok, row) = a_plan("dropped", T, k, E, T)
    live = int(off[-1])
    g = gen(5)
    X, W = torch.randn(T, K, generator=g).bfloat16(), (torch.randn(E, N, K, generator=g) * K ** -0.5).bfloat16()
    b, w = torch.randn(E, N, generator=g).bfloat16(), torch.rand(T, k, generator=g)
    dout = torch.randn(T, N, generator=g).bfloat16()

    def loss(X, W, b, w):
        y, total = np.zeros((T * k, N)), 0.0
        for e in range(E):
            r = slice(off[e], off[e + 1])
            y[r] = X[tok[r]] @ W[e].T + b[e]
        for j in range(k):
            t = np.nonzero(row[:, j] >= 0)[0]
            total += (f64(dout)[t] * w[t, j, None] * y[row[t, j]]).sum()
        return total

    leaves = [q.to(dev()).requires_grad_() for q in (X, W, b, w)]
    y = expert_layer.expert_linear(p, leaves[0], leaves[1], leaves[2])
    expert_layer.combine(p, y, leaves[3]).backward(dout.to(dev()))
    at = [f64(q) for q in (X, W, b, w)]
    rng = np.random.default_rng(2)
    for i, name in enumerate("XWbw"):
        v, h = rng.standard_normal(at[i].shape), 1e-4
        up, dn = list(at), list(at)
        up[i], dn[i] = at[i] + h * v, at[i] - h * v
        diff = (loss(*up) - loss(*dn)) / (2 * h)
        grad = f64(leaves[i].grad)
        say(f"    {name}: difference {diff:.6f}, gradient {(grad * v).sum():.6f}")
        # 4 roundings of every term of the gradient's product with the direction
        assert abs((grad * v).sum() - diff) <= 4 * 2.0 ** -8 * np.abs(grad * v).sum() + 1e-6 * abs(diff) + 1e-6


@pytest.mark.parametrize("renorm,bias", [(True, False), (False, True)])
def test_layer_forward_and_gradients(renorm, bias):
    """Each step rounds to bf16 (2^-8): up, silu * up, down, sum, and as many on the way back. The 2-norm of the
    difference stays within 8 of them."""
    torch.manual_seed(0)
    m = expert_layer.ExpertFFN(64, 96, 6, 2, renormalize=renorm, bias=bias, device=dev())
    x = torch.randn(50, 64, device=dev()).bfloat16().requires_grad_()
    dout = torch.randn(50, 64, device=dev()).bfloat16()
    y = m(x.reshape(5, 10, 64)).reshape(50, 64)
    y.backward(dout)
    ry, rx, rp = ffn_reference(m, x, dout)
    for name, got, want in [("y", y, ry), ("x", x.grad, rx)] + [(n, q.grad, rp[n]) for n, q in m.named_parameters()]:
        rel = float((got.detach().cpu().double() - want).norm() / want.norm())
        say(f"    {name}: relative difference {rel:.2e}")
        assert rel < 8 * 2.0 ** -8, name


def test_layer_replays_in_a_graph():
    """Router, plan, products and sum hold no host state: a captured layer, replayed with other tokens between
    eager work, equals the eager result each time."""
    torch.manual_seed(1)
    m = expert_layer.ExpertFFN(128, 128, 8, 2, device=dev()).eval()
    x = torch.zeros(24, 128, device=dev(), dtype=torch.bfloat16)
    with torch.no_grad():
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            m(x)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = m(x)
        for i in range(4):
            x.copy_(torch.randn(24, 128, generator=gen(i)).bfloat16())
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, m(x))


def test_another_stream():
    p, off, live, X, W, _, x = product_inputs("ragged", 200, 2, 4, 256, 256, True)
    Xd, Wd = X.to(dev()), W.to(dev())
    want = experts.expert_fwd(p, Xd, Wd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = experts.expert_fwd(p, Xd, Wd)
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    d = dev()
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=d)  # noqa: E731
    p = ExpertPlan.from_index(torch.zeros((4, 2), dtype=torch.int32, device=d), 3)
    with pytest.raises(TypeError):
        experts.router_fwd(torch.zeros(4, 3, device=d, dtype=torch.float16), 2)
    with pytest.raises(ValueError):
        experts.router_fwd(torch.zeros(3, 4, device=d).t(), 2)
    with pytest.raises(ValueError):
        experts.router_fwd(torch.zeros(3, 4), 2)
    for k in (0, 4, 33):
        with pytest.raises(_lib.BsrError):
            experts.router_fwd(torch.zeros(4, 3, device=d), k)
    with pytest.raises(_lib.BsrError):
        ExpertPlan.from_index(torch.zeros((4, 2), dtype=torch.int32, device=d), 1025)
    with pytest.raises(TypeError):
        ExpertPlan.from_index(torch.zeros((4, 2), dtype=torch.int64, device=d), 3)
    with pytest.raises(ValueError):
        experts.expert_fwd(p, bf(5, 64), bf(3, 64, 64))
    with pytest.raises(ValueError):
        experts.expert_fwd(p, bf(4, 64), bf(2, 64, 64))
    with pytest.raises(ValueError):
        experts.expert_fwd(p, bf(4, 64), bf(3, 64, 128).transpose(1, 2)[:, :, :64])
    with pytest.raises(TypeError):
        experts.expert_fwd(p, bf(4, 64).float(), bf(3, 64, 64))
    with pytest.raises(_lib.BsrError, match="multiple of 8"):
        experts.expert_fwd(p, bf(4, 12), bf(3, 64, 12))
    with pytest.raises(_lib.BsrError, match="multiple of 8"):
        experts.expert_bwd_input(p, bf(8, 12), bf(3, 12, 64))
    with pytest.raises(_lib.BsrError, match="MISALIGNED"):
        experts.expert_fwd(p, bf(4 * 64 + 1)[1:].reshape(4, 64), bf(3, 64, 64))
    with pytest.raises(ValueError):
        experts.combine_fwd(p, bf(7, 64))
    with pytest.raises(ValueError):
        experts.expert_fwd(p, bf(4, 64), bf(3, 64, 64), out=bf(8, 32))


def test_layer_without_tokens():
    m = expert_layer.ExpertFFN(64, 64, 4, 2, device=dev())
    x = torch.zeros(0, 64, device=dev(), dtype=torch.bfloat16, requires_grad=True)
    y = m(x)
    assert y.shape == (0, 64)
    y.sum().backward()
    assert x.grad.shape == (0, 64)
    for name in ("router", "up", "down"):
        assert not getattr(m, name).grad.any(), name
