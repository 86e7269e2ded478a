"""Measured cases of the 8-bit operators with a scale for each block of 128, and of a whole expert layer for a few tokens.

Four kinds of case:
  quantize  bf16 values to 8-bit floating point (E4M3) with power-of-two scales: groups of 128 along a row (`form` "rows": activations), or
            128 x 128 blocks of weights with their transposed codes (`form` "blocks")
  product   the product grouped by expert on 8-bit weights: activations in bf16 (`act` "bf16": single tokens, small batches) or
            quantised by row within the call (`act` "fp8": prompts); E = 1 is a plain linear layer
  train     the same product in a training step: weights and activations quantised within the step, input gradient in 8 bits,
            weight and bias gradient in bf16
  ffn       a whole layer of experts for a few tokens: router, top k, gate and up product, silu(gate) * up, down product, weighted sum;
            weights in bf16, in microscaled 4 bits or in 8 bits (`form`)

Plain forms are elementary torch operations in 32 bits, with a loop over the experts that have rows.

Scale bytes b stand for 2^(b - 127). Rows: [ceil(K / 512), rows, 4], one byte for each 128 columns. Blocks: [E, ceil(N / 128), ceil(K / 128)].
"""
import math

import torch

own = False

_DEV = "cuda"
_G = 128       # values that share a scale
_TOP = 448.0   # largest E4M3 value


# ------------------------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # activations of a small batch before an 8-bit product
        dict(name="quantize_rows", kind="quantize", form="rows", E=1, N=37, K=4096, std=1.0),
        # a layer's weights when it is loaded for training, both orientations
        dict(name="quantize_blocks", kind="quantize", form="blocks", E=8, N=4096, K=4096, std=0.02),
        # one token, two experts: the smallest product
        dict(name="product_token", kind="product", act="bf16", T=1, E=8, k=2, K=2048, N=1024, bias=False, skew=0.0),
        # decode: a few tokens on wide experts
        dict(name="product_decode", kind="product", act="bf16", T=4, E=8, k=2, K=4096, N=14336, bias=True, skew=0.0),
        # a middling batch whose activations stay in bf16, ragged groups, odd widths
        dict(name="product_batch", kind="product", act="bf16", T=301, E=60, k=4, K=2064, N=1008, bias=True, skew=1.0),
        # a long prompt, both sides in 8 bits
        dict(name="product_prompt", kind="product", act="fp8", T=16384, E=8, k=2, K=4096, N=11008, bias=False, skew=0.5),
        # training step of many narrow experts, ragged groups, odd widths
        dict(name="train_narrow", kind="train", T=4099, E=64, k=4, K=2048, N=1008, bias=True, skew=1.0),
        # training step of few wide experts
        dict(name="train_wide", kind="train", T=8192, E=8, k=2, K=4096, N=4096, bias=False, skew=0.5),
        # one token through a small layer: latency alone
        dict(name="ffn_token", kind="ffn", form="bf16", T=1, E=8, k=2, K=2048, N=1024, bias=False, renorm=True),
        # decode step of a small batch on 4-bit weights
        dict(name="ffn_mx4", kind="ffn", form="mx4", T=4, E=8, k=2, K=4096, N=7168, bias=True, renorm=True),
        # decode step of sixteen sequences, many narrow experts in 8 bits
        dict(name="ffn_fp8", kind="ffn", form="fp8", T=16, E=64, k=8, K=2048, N=1008, bias=False, renorm=False),
        # decode step of an odd batch on wide bf16 experts
        dict(name="ffn_bf16", kind="ffn", form="bf16", T=7, E=8, k=2, K=4096, N=11008, bias=False, renorm=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_any(rng):
    kind = rng.choice(["quantize", "product", "product", "train", "ffn", "ffn"])
    if kind == "quantize":
        form = rng.choice(["rows", "blocks"])
        if form == "rows":
            return dict(kind=kind, form=form, E=1, N=_log(rng, 1, 16384), K=16 * _log(rng, 8, 688), std=rng.choice([0.02, 1.0, 8.0]))
        return dict(kind=kind, form=form, E=rng.choice([1, 4, 8]), N=16 * _log(rng, 8, 256), K=16 * _log(rng, 8, 256), std=rng.choice([0.02, 1.0]))
    if kind == "product":
        act = rng.choice(["bf16", "fp8"])
        return dict(kind=kind, act=act, T=_log(rng, 1, 301 if act == "bf16" else 16384), E=rng.choice([1, 4, 8, 60]), k=rng.choice([1, 2, 4]),
                    K=16 * _log(rng, 8, 256), N=8 * _log(rng, 16, 1792), bias=rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.0]))
    if kind == "train":
        return dict(kind=kind, T=_log(rng, 1, 8192), E=rng.choice([1, 4, 8, 64]), k=rng.choice([1, 2, 4]), K=16 * _log(rng, 16, 256),
                    N=16 * _log(rng, 16, 256), bias=rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.0]))
    return dict(kind=kind, form=rng.choice(["bf16", "mx4", "fp8"]), T=_log(rng, 1, 16), E=rng.choice([4, 8, 60, 64, 128]),
                k=rng.choice([1, 2, 4, 8]), K=32 * _log(rng, 8, 128), N=32 * _log(rng, 8, 344), bias=rng.random() < 0.5,
                renorm=rng.random() < 0.5)


def draw(rng):
    """A case of the listed ones' ranges that costs no more than the largest of them, in work or in memory."""
    most = lambda f: max(f(c) for c in listed())   # noqa: E731
    flops, size, held = most(lambda c: work(c)["flops"]), most(lambda c: work(c)["bytes"]), most(_held)
    while True:
        c = _draw_any(rng)
        if c.get("k", 1) > c["E"]:
            continue
        w = work(c)
        if w["flops"] <= flops and w["bytes"] <= size and _held(c) <= held:
            return c


def _held(c):
    """Weights of all experts, used or not."""
    return c["E"] * c["N"] * c["K"] * (3 if c["kind"] == "ffn" else 1)


def _active(c):
    """Experts that have rows, at least: at most one expert a slot, at most E."""
    return min(c["E"], c["T"] * c["k"])


def work(c):
    kind, E, N, K = c["kind"], c["E"], c["N"], c["K"]
    if kind == "quantize":
        n = E * N * K
        if c["form"] == "rows":     # read, codes, values
            return {"bytes": 5 * n + n // _G, "flops": 3 * n}
        return {"bytes": 8 * n, "flops": 3 * n}   # read, codes and values in both orientations
    T, R, A = c["T"], c["T"] * c["k"], _active(c)
    if kind == "product":
        return {"bytes": 2 * T * K + A * N * K + 2 * R * N, "flops": 2 * R * N * K}
    if kind == "train":   # x, W, dY; Y, dX, dW
        return {"bytes": 2 * (2 * T * K + 2 * R * N + (A + E) * N * K), "flops": 6 * R * N * K}
    size = {"bf16": 2.0, "fp8": 1.0, "mx4": 17 / 32}[c["form"]]
    return {"bytes": int(A * 3 * N * K * size) + 2 * E * K + 4 * T * K, "flops": 6 * R * N * K + 2 * T * E * K}


# ------------------------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 31))
    return g


def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=_DEV) * std).to(dtype)


def _weights(g, E, N, K, std):
    W = torch.empty(E, N, K, dtype=torch.bfloat16, device=_DEV)
    for e in range(E):
        W[e] = _randn(g, N, K, std=std)
    return W


def _sorted_slots(idx, E):
    """offsets [E+1], row_token [T k], slot_row [T, k] of a stable sort of the slots by expert."""
    T, k = idx.shape
    order = torch.sort(idx.reshape(-1), stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=idx.device)
    offsets[1:] = torch.bincount(idx.reshape(-1), minlength=E).cumsum(0)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    return offsets.int(), (order // k).int(), place.reshape(T, k).int()


def _mx4_random(g, E, N, K, std):
    """Codes and scale bytes [E, ceil(K / 256), N, 8] of normal weights: every group of 32 has a value near its scale's top."""
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device=_DEV, dtype=torch.uint8)
    byte = torch.randint(0, 2, (E, -(-K // 256), N, 8), generator=g, device=_DEV) + 127 + round(math.log2(std / 2.5))
    byte = torch.where((torch.arange(-(-K // 256) * 8, device=_DEV) < K // 32).reshape(1, -1, 1, 8), byte, 0)
    return codes, byte.to(torch.uint8)


def _layer_weights(g, form, E, N, K, std):
    if form == "mx4":
        return _mx4_random(g, E, N, K, std)
    W = _weights(g, E, N, K, std)
    return (W,) if form == "bf16" else _blocks(W)


def _tokens(g, T, router, k):
    """Tokens whose k-th logit stands off from the next by more than 32-bit sums can differ: others are drawn anew."""
    E, K = router.shape
    x = _randn(g, T, K)
    for _ in range(8):
        top = (x.double() @ router.double().t()).topk(min(k + 1, E), dim=1).values
        near = (top[:, k - 1] - top[:, -1] < 1e-4) & (E > k)
        x = torch.where(near[:, None], _randn(g, T, K), x)
    return x


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(c)
    E, N, K = c["E"], c["N"], c["K"]
    if c["kind"] == "quantize":
        if c["form"] == "rows":
            row = torch.exp(0.5 * torch.randn(N, 1, generator=g, device=_DEV))   # rows of different size
            s["X"] = (torch.randn(N, K, generator=g, device=_DEV) * row * c["std"]).bfloat16()
        else:
            s["W"] = _weights(g, E, N, K, c["std"])
        return s
    T, k = c["T"], c["k"]
    if c["kind"] == "ffn":
        s["router"] = _randn(g, E, K, std=K ** -0.5)
        s["x"] = _tokens(g, T, s["router"], k)
        s["up"] = _layer_weights(g, c["form"], E, 2 * N, K, K ** -0.5)
        s["down"] = _layer_weights(g, c["form"], E, K, N, N ** -0.5)
        s["up_bias"] = _randn(g, E, 2 * N, std=0.1) if c["bias"] else None
        s["down_bias"] = _randn(g, E, K, std=0.1) if c["bias"] else None
        return s
    lg = torch.randn(T, E, generator=g, device=_DEV) + c["skew"] * torch.randn(E, generator=g, device=_DEV)
    s["offsets"], s["row_token"], s["slot_row"] = _sorted_slots(lg.topk(k, dim=1).indices, E)
    s["counts"] = torch.diff(s["offsets"]).tolist()   # the plain forms' loop lengths
    s["X"] = _randn(g, T, K)
    s["bias"] = _randn(g, E, N, std=0.1) if c["bias"] else None
    W = _weights(g, E, N, K, 0.02)
    if c["kind"] == "train":
        s["W"], s["dY"] = W, _randn(g, T * k, N, std=0.1)
    else:
        s["codes"], s["scales"] = _blocks(W)
    return s


# ------------------------------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------------------------------

def _scale_of(a):
    """The smallest exponent s >= -127 with a <= 448 * 2^s, for magnitudes a (32 bits)."""
    m, e = torch.frexp(a)
    return torch.where(a == 0, -127, (e - 9 + (m > 0.875)).clamp_min(-127))


def _e4m3(v, s):
    """Codes of v with scale 2^s."""
    code = torch.ldexp(v, -s).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.where(v.isfinite(), code, torch.where(v.signbit(), 0xFF, 0x7F).to(torch.uint8))


def _values(codes, s):
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), s)


def _padded(x, *multiples):
    """x with zeros up to multiples of its last dimensions."""
    pad = []
    for n, m in zip(reversed(x.shape), reversed(multiples)):
        pad += [0, -n % m]
    return torch.nn.functional.pad(x, pad)


def _rows(X):
    """Codes [rows, K] and exponents [rows, ceil(K / 128)] of X [rows, K]."""
    rows, K = X.shape
    v = _padded(X.float(), _G).reshape(rows, -1, _G)
    s = _scale_of(torch.where(v.isfinite(), v.abs(), 0.0).amax(2))
    return _e4m3(v, s[..., None]).reshape(rows, -1)[:, :K].contiguous(), s


def _row_values(codes, s):
    return _values(codes, s.repeat_interleave(_G, 1)[:, :codes.shape[1]])


def _row_bytes(s):
    """Scale bytes [ceil(K / 512), rows, 4] of exponents [rows, ceil(K / 128)]."""
    b = _padded((s + 127).to(torch.uint8), 4)
    return b.reshape(b.shape[0], -1, 4).transpose(0, 1).contiguous()


def _block_exponents(bytes_, N, K):
    """Exponents of every value of [N, K], from scale bytes [ceil(N / 128), ceil(K / 128)]."""
    return (bytes_.int() - 127).repeat_interleave(_G, 0)[:N].repeat_interleave(_G, 1)[:, :K]


def _blocks(W):
    """Codes [E, N, K] and scale bytes [E, ceil(N / 128), ceil(K / 128)] of W [E, N, K]."""
    E, N, K = W.shape
    codes = torch.empty(E, N, K, dtype=torch.uint8, device=W.device)
    scales = torch.empty(E, -(-N // _G), -(-K // _G), dtype=torch.uint8, device=W.device)
    for e in range(E):
        v = W[e].float()
        big = _padded(torch.where(v.isfinite(), v.abs(), 0.0), _G, _G)
        big = big.reshape(scales.shape[1], _G, scales.shape[2], _G).amax((1, 3))
        scales[e] = (_scale_of(big) + 127).to(torch.uint8)
        codes[e] = _e4m3(v, _block_exponents(scales[e], N, K))
    return codes, scales


def _block_values(codes, scales):
    return _values(codes, _block_exponents(scales, *codes.shape))


def _quantize(s):
    if s["form"] == "rows":
        codes, e = _rows(s["X"])
        return [_row_bytes(e), _row_values(codes, e).bfloat16()]
    codes, scales = _blocks(s["W"])
    E, N, K = codes.shape
    values = torch.empty(E, N, K, dtype=torch.bfloat16, device=codes.device)
    for e in range(E):
        values[e] = _block_values(codes[e], scales[e])
    return [values, values.transpose(1, 2).contiguous()]


def _grouped(s, rows, weight):
    """rows [R, K] (32 bits) times each group's weight(e) [N, K], transposed, plus bias, rounded once."""
    Y = torch.empty(rows.shape[0], s["N"], dtype=torch.bfloat16, device=rows.device)
    at = 0
    for e, n in enumerate(s["counts"]):
        if n:
            y = rows[at:at + n] @ weight(e).t()
            Y[at:at + n] = y if s["bias"] is None else y + s["bias"][e].float()
            at += n
    return Y


def _product(s):
    x = s["X"].float() if s["act"] == "bf16" else _row_values(*_rows(s["X"]))
    return _grouped(s, x[s["row_token"].long()], lambda e: _block_values(s["codes"][e], s["scales"][e]))


def _train(s):
    W, tok = s["W"], s["row_token"].long()
    codes, scales = _blocks(W)
    weight = lambda e: _block_values(codes[e], scales[e])   # noqa: E731
    Y = _grouped(s, _row_values(*_rows(s["X"]))[tok], weight)
    d, dq, x = s["dY"].float(), _row_values(*_rows(s["dY"])), s["X"].float()[tok]
    dX = torch.empty_like(x)
    dW = torch.empty_like(W)
    db = torch.empty(s["E"], s["N"], dtype=torch.bfloat16, device=W.device)
    at = 0
    for e, n in enumerate(s["counts"]):
        r = slice(at, at + n)
        dX[r] = dq[r] @ weight(e)
        dW[e] = d[r].t() @ x[r]
        db[e] = d[r].sum(0)
        at += n
    dX = dX[s["slot_row"].long()].sum(1).bfloat16()   # a token's rows
    return [Y, dX, dW, db] if s["bias"] is not None else [Y, dX, dW]


_MX4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _layer_values(form, held, e):
    """32-bit values of expert e's weight."""
    if form == "bf16":
        return held[0][e].float()
    if form == "fp8":
        return _block_values(held[0][e], held[1][e])
    codes, scales = held[0][e], held[1][e]
    rows, half = codes.shape
    table = torch.tensor(_MX4 + tuple(-m for m in _MX4), device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], 2).reshape(rows, half // 16, 32)
    byte = scales.transpose(0, 1).reshape(rows, -1)[:, :half // 16].int()
    return torch.ldexp(table[c.int()], (byte - 127)[..., None]).reshape(rows, 2 * half)


def _ffn(s):
    x, k, N = s["x"].float(), s["k"], s["N"]
    logits = s["x"].double() @ s["router"].double().t()   # neighbouring logits decide the experts
    top = torch.sort(logits, dim=1, descending=True, stable=True)
    val, idx = top.values[:, :k].float(), top.indices[:, :k]
    ex = torch.exp(val - val[:, :1])
    w = ex / (ex if s["renorm"] else torch.exp(logits.float() - val[:, :1])).sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for e in idx.unique().tolist():
        t, j = torch.nonzero(idx == e, as_tuple=True)
        h = x[t] @ _layer_values(s["form"], s["up"], e).t()
        if s["up_bias"] is not None:
            h = h + s["up_bias"][e].float()
        gate, up = h[:, :N], h[:, N:]
        y = (gate / (1.0 + torch.exp(-gate)) * up) @ _layer_values(s["form"], s["down"], e).t()
        if s["down_bias"] is not None:
            y = y + s["down_bias"][e].float()
        out[t] += w[t, j, None] * y
    return out.bfloat16()


# ------------------------------------------------------------------------------------------------------------------
# the framework's calls
# ------------------------------------------------------------------------------------------------------------------

def _own(s):
    from sparse_gemm_amd import experts, expert_layer, fp8, mx4
    if s["kind"] == "quantize":
        if s["form"] == "rows":
            q, values = fp8.quantize_rows(s["X"], want_values=True)
            return [q.scales, values]
        return [fp8.dequantize(q) for q in fp8.quantize_blocks(s["W"], transposed=True)]
    if s["kind"] == "ffn":
        form = {"bf16": lambda W: W, "mx4": mx4.Mx4, "fp8": fp8.Fp8Blocks}[s["form"]]
        return expert_layer.expert_ffn(s["x"], s["router"], form(*s["up"]), form(*s["down"]), s["k"], renormalize=s["renorm"],
                                       up_bias=s["up_bias"], down_bias=s["down_bias"])
    plan = experts.ExpertPlan(s["offsets"], s["row_token"], s["slot_row"])
    if s["kind"] == "product":
        X = s["X"] if s["act"] == "bf16" else fp8.quantize_rows(s["X"])
        return fp8.expert_fwd(plan, X, fp8.Fp8Blocks(s["codes"], s["scales"]), s["bias"])
    leaves = [t.detach().requires_grad_() for t in (s["X"], s["W"], s["bias"]) if t is not None]
    Y = expert_layer.expert_linear_fp8(plan, *leaves)
    return [Y.detach(), *torch.autograd.grad(Y, leaves, s["dY"])]


def run(state):
    if own:
        return _own(state)
    return dict(quantize=_quantize, product=_product, train=_train, ffn=_ffn)[state["kind"]](state)


# ------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------------------------

def _pow2(e):
    """2^e in 64 bits, from its bits (-1022 <= e <= 1023)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest(v, big):
    """Finite v (64 bits) rounded to E4M3 numbers times the scale that the largest magnitude `big` asks for."""
    s = torch.ceil(torch.log2((big / _TOP).clamp_min(2.0 ** -140))).clamp_min(-127)
    s = torch.where(big <= _TOP * _pow2(s - 1), s - 1, s)          # log2 may land on either side of a whole number
    s = torch.where(big > _TOP * _pow2(s), s + 1, s).clamp_min(-127)
    u = v / _pow2(s)
    mag = u.abs()
    exponent = torch.frexp(torch.where(mag < 2.0 ** -6, torch.full_like(mag, 2.0 ** -6), mag)).exponent - 1
    step = _pow2(exponent - 3)                                       # 4 significant bits, 2^-9 below 2^-6
    return torch.round(u / step) * step * _pow2(s)                   # torch.round: ties to even


def _exact_rows(X):
    rows, K = X.shape
    out = torch.empty(rows, K, dtype=torch.float64, device=X.device)
    for k0 in range(0, K, _G):
        v = X[:, k0:k0 + _G].double()
        out[:, k0:k0 + _G] = _nearest(v, v.abs().amax(1, keepdim=True))
    return out


def _exact_blocks(W):
    N, K = W.shape
    v = W.double()
    big = torch.nn.functional.max_pool2d(v.abs()[None, None], _G, ceil_mode=True)[0, 0]
    for n0 in range(0, N, _G):
        piece = v[n0:n0 + _G]
        piece.copy_(_nearest(piece, big[n0 // _G].repeat_interleave(_G)[:K]))
    return v


def _exact_held(codes, scales):
    """Values of held 8-bit weights, from the bits of their codes."""
    c = codes.long()
    e, m = (c >> 3) & 15, c & 7
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * _pow2(e - 10)) * (1 - 2 * (c >> 7))
    n, k = torch.arange(c.shape[0], device=c.device) // _G, torch.arange(c.shape[1], device=c.device) // _G
    return v * _pow2(scales.long()[n][:, k] - 127)


def _exact_layer(form, held, e):
    if form == "bf16":
        return held[0][e].double()
    if form == "fp8":
        return _exact_held(held[0][e], held[1][e])
    b, by = held[0][e].long(), held[1][e].long()
    half = torch.tensor(_MX4, dtype=torch.float64, device=b.device)
    nib = torch.stack([b % 16, b // 16], -1).reshape(b.shape[0], -1)
    cols = torch.arange(nib.shape[1], device=b.device)
    return half[nib % 8] * (1 - 2 * (nib // 8)) * _pow2(by.permute(1, 0, 2).reshape(b.shape[0], -1)[:, cols // 32] - 127)


def exact(case, seed):
    s = prepare(case, seed)
    kind, E = s["kind"], s["E"]
    if kind == "quantize":
        if s["form"] == "rows":
            return [None, _exact_rows(s["X"])]
        v = torch.stack([_exact_blocks(s["W"][e]) for e in range(E)])
        return [v, v.transpose(1, 2)]
    if kind == "ffn":
        T, N, k = s["T"], s["N"], s["k"]
        x = s["x"].double()
        logits = torch.matmul(x, s["router"].double().t())
        p = torch.softmax(logits, 1)
        idx = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k]
        w = p.gather(1, idx)
        if s["renorm"]:
            w = w / w.sum(1, keepdim=True)
        full = torch.zeros_like(p).scatter_(1, idx, w)
        out = torch.zeros(T, s["K"], dtype=torch.float64, device=_DEV)
        for e in range(E):
            rows = full[:, e].nonzero().reshape(-1)
            if rows.numel() == 0:
                continue
            h = torch.matmul(x[rows], _exact_layer(s["form"], s["up"], e).t())
            if s["up_bias"] is not None:
                h += s["up_bias"][e].double()
            h = h[:, :N] * torch.sigmoid(h[:, :N]) * h[:, N:]
            y = torch.matmul(h, _exact_layer(s["form"], s["down"], e).t())
            if s["down_bias"] is not None:
                y += s["down_bias"][e].double()
            out.index_add_(0, rows, full[rows, e, None] * y)
        return out
    off, tok = s["offsets"].tolist(), s["row_token"].long()
    R = tok.numel()
    quantised = kind == "train" or s["act"] == "fp8"
    X = _exact_rows(s["X"]) if quantised else s["X"].double()
    dq = _exact_rows(s["dY"]) if kind == "train" else None
    Y = torch.zeros(R, s["N"], dtype=torch.float64, device=_DEV)
    dX = torch.zeros(s["T"], s["K"], dtype=torch.float64, device=_DEV)
    dW = torch.zeros(E, s["N"], s["K"], dtype=torch.float64, device=_DEV) if kind == "train" else None
    db = torch.zeros(E, s["N"], dtype=torch.float64, device=_DEV)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if r.start == r.stop:
            continue
        W = _exact_blocks(s["W"][e]) if kind == "train" else _exact_held(s["codes"][e], s["scales"][e])
        y = torch.matmul(X[tok[r]], W.t())
        Y[r] = y if s["bias"] is None else y + s["bias"][e].double()
        if kind == "train":
            d = s["dY"][r].double()
            dX.index_add_(0, tok[r], torch.matmul(dq[r], W))
            dW[e] = torch.matmul(d.t(), s["X"].double()[tok[r]])
            db[e] = d.sum(0)
    if kind == "product":
        return Y
    return [Y, dX, dW, db] if s["bias"] is not None else [Y, dX, dW]
