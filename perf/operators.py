"""Measured cases of the expert-layer and microscaled 4-bit operators.

Five operators, each a `kind` of case:
  route     softmax router over E logits, top k, and the plan that sorts the token slots by expert (with its gradient
            where `grad` is set)
  experts   products grouped by expert with ragged sizes: `dir` "fwd" (Y = X W_e^T + b_e, rows gathered by token) or
            "bwd" (input gradient, weight gradient, bias gradient)
  combine   weighted sum of a token's expert rows (with its gradient where `grad` is set)
  quantize  bf16 rows to microscaled 4-bit values: 32 E2M1 codes share a power-of-two scale byte
  mx4       the grouped product on microscaled weights: activations in bf16 (`act` "bf16", single tokens and small
            batches) or quantised to the same 4-bit form within the call (`act` "mx4", prompts); E = 1 is a plain linear layer

Plain forms are elementary torch operations in 32 bits. A loop over the experts stands in the grouped products: padding the
groups to one length for a batched product would give the plain form more work than the layer has.

Scale bytes are laid out [K / 256, rows, 8]: the 8 scales of a row's 256 columns side by side (the last 256 may be partial).
"""
import math

import torch

own = False

_DEV = "cuda"
_CHUNK = 256   # columns whose scale bytes lie side by side


# ------------------------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a small batch: latency alone
        dict(name="route_decode", kind="route", T=8, E=64, k=8, renorm=True, f32=True, grad=False, pad=0),
        # a training step's tokens, some of them padding (rows without any expert), with the gradient
        dict(name="route_train", kind="route", T=16390, E=128, k=8, renorm=False, f32=False, grad=True, pad=500),
        # one token, two experts: the smallest product
        dict(name="experts_fwd_token", kind="experts", dir="fwd", T=1, E=8, k=2, K=2048, N=1024, bias=False, skew=0.0),
        # a long prompt through wide experts
        dict(name="experts_fwd_prompt", kind="experts", dir="fwd", T=16384, E=8, k=2, K=4096, N=11008, bias=False, skew=0.5),
        # fine-tuning step: many narrow experts, ragged groups, odd widths
        dict(name="experts_bwd_narrow", kind="experts", dir="bwd", T=4099, E=64, k=4, K=2048, N=1000, bias=True, skew=1.0),
        # training step: few wide experts
        dict(name="experts_bwd_wide", kind="experts", dir="bwd", T=8192, E=8, k=2, K=4096, N=4096, bias=False, skew=0.5),
        # decode step's sum over 8 experts
        dict(name="combine_decode", kind="combine", T=8, k=8, N=4096, E=64, grad=False, pad=0),
        # training step's sum and its gradient
        dict(name="combine_train", kind="combine", T=8191, k=8, N=2048, E=64, grad=True, pad=100),
        # activations of a small batch before a 4-bit product
        dict(name="quantize_rows", kind="quantize", T=37, K=4096, std=1.0),
        # weights of a layer when it is loaded
        dict(name="quantize_weights", kind="quantize", T=57344, K=4096, std=0.02),
        # decode: a few tokens on 4-bit experts
        dict(name="mx4_decode", kind="mx4", act="bf16", T=4, E=8, k=2, K=4096, N=14336, bias=True, skew=0.0),
        # prompt: both sides in 4 bits
        dict(name="mx4_prompt", kind="mx4", act="mx4", T=8192, E=8, k=2, K=4096, N=4096, bias=False, skew=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_any(rng):
    kind = rng.choice(["route", "experts", "experts", "combine", "quantize", "mx4", "mx4"])
    if kind == "route":
        T, E = _log(rng, 1, 16390), rng.choice([8, 16, 60, 64, 128, 255, 256])
        return dict(kind=kind, T=T, E=E, k=rng.choice([1, 2, 4, 6, 8]), renorm=rng.random() < 0.5, f32=rng.random() < 0.5,
                    grad=rng.random() < 0.5, pad=rng.choice([0, T // 32]))
    if kind == "experts":
        return dict(kind=kind, dir=rng.choice(["fwd", "bwd"]), T=_log(rng, 1, 16384), E=rng.choice([1, 4, 8, 16, 60, 64]),
                    k=rng.choice([1, 2, 4, 8]), K=8 * _log(rng, 32, 512), N=8 * _log(rng, 32, 1376),
                    bias=rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.0]))
    if kind == "combine":
        T = _log(rng, 1, 8191)
        return dict(kind=kind, T=T, k=rng.choice([1, 2, 4, 8]), N=8 * _log(rng, 32, 512), E=rng.choice([8, 64]),
                    grad=rng.random() < 0.5, pad=rng.choice([0, T // 32]))
    if kind == "quantize":
        return dict(kind=kind, T=_log(rng, 1, 57344), K=32 * _log(rng, 8, 344), std=rng.choice([0.02, 1.0, 8.0]))
    act = rng.choice(["bf16", "mx4"])
    return dict(kind=kind, act=act, T=_log(rng, 1, 64 if act == "bf16" else 8192), E=rng.choice([1, 4, 8, 32]), k=rng.choice([1, 2, 4]),
                K=32 * _log(rng, 8, 128), N=8 * _log(rng, 32, 1792), bias=rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.0]))


def draw(rng):
    """A case of the listed ones' ranges that costs no more than the largest of them."""
    top = max((work(c) for c in listed()), key=lambda w: w["flops"])
    while True:
        c = _draw_any(rng)
        if c.get("k", 1) > c.get("E", 256):
            continue
        w = work(c)
        if w["flops"] <= top["flops"] and w["bytes"] <= top["bytes"]:
            return c


def _active(c):
    """Experts that have rows, at least: at most one expert a slot, at most E."""
    return min(c["E"], c["T"] * c["k"])


def work(c):
    kind, T = c["kind"], c["T"]
    if kind == "route":
        es = 4 if c["f32"] else 2
        S = T * c["k"]
        b = T * c["E"] * es + S * 8 + S * 8 + (c["E"] + 1) * 4
        f = 3 * T * c["E"]
        if c["grad"]:
            b += S * 4 + T * c["E"] * es   # the logits are read once for both directions
            f += 4 * T * c["E"]
        return {"bytes": b, "flops": f}
    if kind == "experts":
        R, K, N, A = T * c["k"], c["K"], c["N"], _active(c)
        if c["dir"] == "fwd":
            return {"bytes": 2 * (T * K + A * N * K + R * N), "flops": 2 * R * N * K}
        return {"bytes": 2 * (R * N + T * K + A * N * K + R * K + c["E"] * N * K + c["E"] * N), "flops": 4 * R * N * K + R * N}
    if kind == "combine":
        R, N = T * c["k"], c["N"]
        b, f = 2 * (R * N + T * N) + 8 * R, 2 * R * N
        if c["grad"]:
            b += 2 * (T * N + R * N) + 4 * R
            f += 3 * R * N
        return {"bytes": b, "flops": f}
    if kind == "quantize":
        n = T * c["K"]
        return {"bytes": 2 * n + n // 2 + n // 32 + 2 * n, "flops": 4 * n}
    R, K, N, A = T * c["k"], c["K"], c["N"], _active(c)
    return {"bytes": 2 * T * K + A * N * (K // 2 + K // 32) + 2 * R * N, "flops": 2 * R * N * K}


# ------------------------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 31))
    return g


def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=_DEV) * std).to(dtype)


def _routed(g, T, E, k, skew, pad=0):
    """Expert of every slot [T, k] (int64, -1 in padding tokens), popular experts the more so the larger skew is."""
    lg = torch.randn(T, E, generator=g, device=_DEV) + skew * torch.randn(E, generator=g, device=_DEV)
    idx = lg.topk(k, dim=1).indices
    if pad:
        idx[torch.randperm(T, generator=g, device=_DEV)[:pad]] = -1
    return idx


def _sorted_slots(idx, E):
    """offsets [E+1], row_token [T k], slot_row [T, k] of a stable sort of the slots by expert."""
    T, k = idx.shape
    flat = torch.where(idx < 0, E, idx).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=idx.device)
    offsets[1:] = counts.cumsum(0)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    slot_row = torch.where(idx.reshape(-1) < 0, -1, place).reshape(T, k)
    row_token = torch.where(torch.arange(T * k, device=idx.device) < offsets[E], order // k, -1)
    return offsets.int(), row_token.int(), slot_row.int()


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(c)
    T = c["T"]
    if c["kind"] == "route":
        lg = torch.randn(T, c["E"], generator=g, device=_DEV) * 1.5 + torch.randn(c["E"], generator=g, device=_DEV) * 0.5
        lg = torch.where(torch.rand(T, c["E"], generator=g, device=_DEV) < 0.02, -math.inf, lg)   # experts out of a token's reach
        if c["pad"]:
            lg[torch.randperm(T, generator=g, device=_DEV)[:c["pad"]]] = -math.inf                # padding tokens
        s["logits"] = lg.to(torch.float32 if c["f32"] else torch.bfloat16).contiguous()
        s["dw"] = torch.randn(T, c["k"], generator=g, device=_DEV)
        return s
    if c["kind"] == "quantize":
        row = torch.exp(0.5 * torch.randn(T, 1, generator=g, device=_DEV))   # rows of different size
        s["X"] = (torch.randn(T, c["K"], generator=g, device=_DEV) * row * c["std"]).bfloat16()
        return s
    E, k = c["E"], c["k"]
    idx = _routed(g, T, E, k, c.get("skew", 0.5), c.get("pad", 0))
    s["offsets"], s["row_token"], s["slot_row"] = _sorted_slots(idx, E)
    s["counts"] = torch.diff(s["offsets"]).tolist()   # the plain forms' loop lengths
    R = T * k
    if c["kind"] == "combine":
        s["Y"] = _randn(g, R, c["N"])
        s["w"] = torch.rand(T, k, generator=g, device=_DEV).masked_fill(s["slot_row"] < 0, 0.0)
        s["dout"] = _randn(g, T, c["N"])
        return s
    K, N = c["K"], c["N"]
    s["X"] = _randn(g, T, K)
    s["bias"] = _randn(g, E, N, std=0.1) if c["bias"] else None
    if c["kind"] == "experts":
        s["W"] = torch.empty(E, N, K, dtype=torch.bfloat16, device=_DEV)
        for e in range(E):
            s["W"][e] = _randn(g, N, K, std=0.02)
        if c["dir"] == "bwd":
            s["dY"] = _randn(g, R, N, std=0.1)
        return s
    s["codes"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device=_DEV)
    s["scales"] = torch.zeros(E, -(-K // _CHUNK), N, _CHUNK // 32, dtype=torch.uint8, device=_DEV)
    for e in range(E):
        s["codes"][e], s["scales"][e] = _mx4(_randn(g, N, K, std=0.02))
    return s


# ------------------------------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------------------------------

def _route(s):
    x = s["logits"].float()
    T, E = x.shape
    k = s["k"]
    top = torch.sort(x, dim=1, descending=True, stable=True)
    val, idx = top.values[:, :k], top.indices[:, :k]
    gone = val == -math.inf
    m = val[:, :1].clamp_min(torch.finfo(torch.float32).min)
    ex, exk = torch.exp(x - m), torch.exp(val - m)
    den = (exk if s["renorm"] else ex).sum(1, keepdim=True)
    w = torch.where(gone, 0.0, exk / den)
    idx = torch.where(gone, -1, idx)
    offsets, row_token, slot_row = _sorted_slots(idx, E)
    out = [idx.int(), w, offsets, row_token, slot_row]
    if s["grad"]:
        dw = torch.where(gone, 0.0, s["dw"])
        inner = (w * dw).sum(1, keepdim=True)
        if s["renorm"]:
            d = torch.zeros_like(x)
            d.scatter_add_(1, idx.clamp_min(0).long(), torch.where(gone, 0.0, w * (dw - inner)))
        else:
            p = torch.where(x == -math.inf, 0.0, ex / den)
            d = -p * inner
            d.scatter_add_(1, idx.clamp_min(0).long(), torch.where(gone, 0.0, w * dw))
        out.append(d.to(s["logits"].dtype))
    return out


def _mx4(x):
    """Codes [rows, K / 2] (low half first) and scale bytes [K / 256, rows, 8] of x [rows, K]."""
    rows, K = x.shape
    v = x.float().reshape(rows, K // 32, 32)
    bits = v.view(torch.int32)
    top = (bits & 0x7FFFFFFF).amax(2) >> 23                       # exponent field of the group's largest magnitude
    byte = torch.where(top == 255, 255, (top - 2).clamp_min(0))
    a = (v * ((254 - byte.clamp_max(253)) << 23).int().view(torch.float32)[..., None]).abs()
    code = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)   # ties to the even code
    code = torch.where((byte == 255)[..., None], 0, code + torch.where(bits < 0, 8, 0)).reshape(rows, K // 2, 2)
    codes = (code[..., 0] + 16 * code[..., 1]).to(torch.uint8)
    scales = torch.zeros(rows, -(-K // _CHUNK) * (_CHUNK // 32), dtype=torch.uint8, device=x.device)
    scales[:, :K // 32] = byte.to(torch.uint8)
    return codes, scales.reshape(rows, -1, _CHUNK // 32).transpose(0, 1).contiguous()


def _mx4_values(codes, scales):
    """32-bit values of codes [rows, K / 2] and scale bytes [K / 256, rows, 8]."""
    rows, half = codes.shape
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], 2).reshape(rows, half // 16, 32)
    byte = scales.transpose(0, 1).reshape(rows, -1)[:, :half // 16].int()
    scale = torch.where(byte == 0, 0x00400000, byte << 23).view(torch.float32)
    scale = torch.where(byte == 255, math.nan, scale)
    return (table[c.int()] * scale[..., None]).reshape(rows, 2 * half)


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


def _experts(s):
    if s["dir"] == "fwd":
        return _grouped(s, s["X"].float()[s["row_token"].long()], lambda e: s["W"][e].float())
    W = s["W"]
    dY, X = s["dY"].float(), s["X"].float()[s["row_token"].long()]
    dX = torch.empty(dY.shape[0], s["K"], dtype=torch.bfloat16, device=W.device)
    dW = torch.empty_like(W)
    db = torch.empty(s["E"], s["N"], dtype=torch.bfloat16, device=W.device)
    at = 0
    for e, n in enumerate(s["counts"]):
        d, x = dY[at:at + n], X[at:at + n]
        dX[at:at + n] = d @ W[e].float()
        dW[e] = d.t() @ x
        db[e] = d.sum(0)
        at += n
    return [dX, dW, db] if s["bias"] is not None else [dX, dW]


def _combine(s):
    row, w = s["slot_row"].long(), s["w"]
    kept = (row >= 0)[..., None]
    y = torch.where(kept, s["Y"].float()[row.clamp_min(0)], 0.0)        # [T, k, N]
    out = [(w[..., None] * y).sum(1).bfloat16()]
    if s["grad"]:
        d = s["dout"].float()[:, None, :]
        dY = torch.zeros_like(s["Y"])
        live = row >= 0
        dY[row[live]] = (w[..., None] * d)[live].bfloat16()
        out += [dY, (d * y).sum(2)]
    return out


def _quantize(s):
    codes, scales = _mx4(s["X"])
    return [codes, scales, _mx4_values(codes, scales).bfloat16()]


def _mx4_product(s):
    x = s["X"].float() if s["act"] == "bf16" else _mx4_values(*_mx4(s["X"]))
    return _grouped(s, x[s["row_token"].long()], lambda e: _mx4_values(s["codes"][e], s["scales"][e]))


# ------------------------------------------------------------------------------------------------------------------
# the framework's calls
# ------------------------------------------------------------------------------------------------------------------

def _own(s):
    from sparse_gemm_amd import experts, mx4
    if s["kind"] == "route":
        idx, w = experts.router_fwd(s["logits"], s["k"], renormalize=s["renorm"])
        plan = experts.ExpertPlan.from_index(idx, s["E"])
        out = [idx, w, plan.offsets, plan.row_token, plan.slot_row]
        if s["grad"]:
            out.append(experts.router_bwd(s["logits"], idx, w, s["dw"], renormalize=s["renorm"]))
        return out
    if s["kind"] == "quantize":
        q, values = mx4.quantize(s["X"], want_values=True)
        return [q.codes, q.scales, values]
    plan = experts.ExpertPlan(s["offsets"], s["row_token"], s["slot_row"])
    if s["kind"] == "combine":
        out = [experts.combine_fwd(plan, s["Y"], s["w"])]
        if s["grad"]:
            out += experts.combine_bwd(plan, s["dout"], s["Y"], s["w"])
        return out
    if s["kind"] == "mx4":
        W = mx4.Mx4(s["codes"], s["scales"])
        X = s["X"] if s["act"] == "bf16" else mx4.quantize(s["X"])
        return mx4.expert_fwd(plan, X, W, s["bias"])
    if s["dir"] == "fwd":
        return experts.expert_fwd(plan, s["X"], s["W"], s["bias"])
    dX = experts.expert_bwd_input(plan, s["dY"], s["W"])
    dW, db = experts.expert_bwd_weight(plan, s["dY"], s["X"], want_dbias=s["bias"] is not None)
    return [dX, dW, db] if s["bias"] is not None else [dX, dW]


def run(state):
    if own:
        return _own(state)
    return dict(route=_route, experts=_experts, combine=_combine, quantize=_quantize, mx4=_mx4_product)[state["kind"]](state)


# ------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------------------------

_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_mx4(x):
    """x [rows, K] in 64 bits -> the values nearest to it in the microscaled form."""
    g = x.double().reshape(x.shape[0], -1, 32)
    big = g.abs().amax(2, keepdim=True)
    e = (torch.frexp(big).exponent - 1 - 2).clamp_min(-127)
    e = torch.where(big == 0, torch.full_like(e, -127), e)
    step = ((e.long() + 1023) << 52).view(torch.float64)           # 2^e, from its bits
    mag = torch.tensor(_MAGNITUDES, dtype=torch.float64, device=x.device)
    u = g.abs() / step
    hi = torch.searchsorted(mag, u.contiguous()).clamp(1, 7)       # mag[hi - 1] < u <= mag[hi]
    lo = hi - 1
    below, above = u - mag[lo], mag[hi] - u
    pick = torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)
    return (torch.copysign(mag[pick], g) * step).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "route":
        x = s["logits"].double()
        order = torch.sort(-x, dim=1, stable=True).indices[:, :s["k"]]
        val = torch.gather(x, 1, order)
        dead = torch.isneginf(val)
        p = torch.softmax(x, 1).nan_to_num(0.0)                    # a row without experts has no probabilities
        w = torch.gather(p, 1, order)
        tot = w.sum(1, keepdim=True)
        dl = None
        wn = torch.where(tot > 0, w / tot, 0.0) if s["renorm"] else w
        if s["grad"]:
            dw = s["dw"].double().masked_fill(dead, 0.0)
            # d w_j / d logit_e of the plain softmax, chained through the division by the chosen ones' sum
            dp = torch.zeros_like(p)
            gw = torch.where(tot > 0, (dw - (wn * dw).sum(1, keepdim=True)) / tot, 0.0) if s["renorm"] else dw
            dp.scatter_(1, order, gw)
            dl = p * (dp - (dp * p).sum(1, keepdim=True))
        return [None, wn.masked_fill(dead, 0.0), None, None, None] + ([dl] if s["grad"] else [])
    if kind == "quantize":
        return [None, None, _exact_mx4(s["X"])]
    slot_row = s["slot_row"].long()
    if kind == "combine":
        T, k = slot_row.shape
        Y, w, d = s["Y"].double(), s["w"].double(), s["dout"].double()
        out = torch.zeros(T, s["N"], dtype=torch.float64, device=_DEV)
        dY, dw = torch.zeros_like(Y), torch.zeros_like(w)
        for j in range(k):
            t = torch.nonzero(slot_row[:, j] >= 0).reshape(-1)
            r = slot_row[t, j]
            out[t] += w[t, j, None] * Y[r]
            dY[r] = w[t, j, None] * d[t]
            dw[t, j] = (d[t] * Y[r]).sum(1)
        return [out, dY, dw] if s["grad"] else [out]
    E, N, K = s["E"], s["N"], s["K"]
    off, tok = s["offsets"].tolist(), s["row_token"].long()
    X = s["X"].double()
    if kind == "mx4" and s["act"] == "mx4":
        X = _exact_mx4(s["X"])
    groups = [(e, slice(off[e], off[e + 1])) for e in range(E)]
    if kind == "experts" and s["dir"] == "bwd":
        dX = torch.zeros(tok.numel(), K, dtype=torch.float64, device=_DEV)
        dW = torch.zeros(E, N, K, dtype=torch.float64, device=_DEV)
        db = torch.zeros(E, N, dtype=torch.float64, device=_DEV)
        for e, r in groups:
            d = s["dY"][r].double()
            dX[r] = torch.matmul(d, s["W"][e].double())
            dW[e] = torch.matmul(d.t(), X[tok[r]])
            db[e] = d.sum(0)
        return [dX, dW, db] if s["bias"] is not None else [dX, dW]
    Y = torch.zeros(tok.numel(), N, dtype=torch.float64, device=_DEV)
    if kind == "mx4":
        half = torch.tensor(_MAGNITUDES, dtype=torch.float64, device=_DEV)
    for e, r in groups:
        if r.start == r.stop:
            continue
        if kind == "experts":
            W = s["W"][e].double()
        else:
            b = s["codes"][e]
            nib = torch.stack([b % 16, b // 16], -1).reshape(N, K // 32, 32).long()
            by = s["scales"][e].permute(1, 0, 2).reshape(N, -1)[:, :K // 32].long()
            W = half[nib % 8] * (1 - 2 * (nib // 8)) * torch.pow(2.0, (by - 127).double())[..., None]
            W = W.reshape(N, K)
        y = torch.matmul(X[tok[r]], W.t())
        Y[r] = y if s["bias"] is None else y + s["bias"][e].double()
    return Y
