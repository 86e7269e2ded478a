"""Plain 64-bit definitions of the expert-layer and microscaled 4-bit operators (numpy, CPU), and the
tolerance of a bf16 result: one rounding to bf16 (unit roundoff 2^-8) plus `terms` roundings of 32-bit
sums, each at most 2^-23 of the sum S of the terms' magnitudes."""
from __future__ import annotations

import math

import numpy as np
import torch

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def near_bf16(got: torch.Tensor, ref: np.ndarray, S: np.ndarray, terms: int, roundings: int = 1) -> None:
    g = f64(got)
    assert g.shape == ref.shape
    assert np.isfinite(g).all()
    tol = roundings * 2.0 ** -8 * np.abs(ref) + (terms + 4) * 2.0 ** -23 * S + 2.0 ** -133
    off = np.abs(g - ref)
    assert (off <= tol).all(), f"worst {np.max(off / tol):.3f} of the tolerance at {np.unravel_index(np.argmax(off / tol), ref.shape)}"


def router(logits: np.ndarray, k: int, renorm: bool):
    """(index, weight, p) with ties to the lowest expert; -inf is never chosen, NaN is the largest."""
    T, E = logits.shape
    index, weight, P = np.full((T, k), -1, np.int64), np.zeros((T, k)), np.zeros((T, E))
    for t in range(T):
        x = logits[t].astype(np.float64)
        order = sorted(range(E), key=lambda e: (0, 0.0, e) if math.isnan(x[e]) else (1, -x[e], e))
        chosen = [e for e in order[:k] if x[e] != -math.inf]
        if not chosen:
            continue
        m = x[chosen[0]]
        with np.errstate(invalid="ignore"):
            ex = np.exp(x - m) if not math.isnan(m) else np.full(E, math.nan)
        P[t] = ex / ex.sum()
        den = ex[chosen].sum() if renorm else ex.sum()
        index[t, :len(chosen)] = chosen
        weight[t, :len(chosen)] = ex[chosen] / den
    return index, weight, P


def router_grad(logits: np.ndarray, k: int, renorm: bool, dweight: np.ndarray) -> np.ndarray:
    index, weight, P = router(logits, k, renorm)
    d = np.zeros(logits.shape)
    for t in range(logits.shape[0]):
        live = index[t] >= 0
        g, w, e = dweight[t][live], weight[t][live], index[t][live]
        inner = float((g * w).sum())
        if renorm:
            d[t, e] = w * (g - inner)
        else:
            d[t] = -P[t] * inner
            d[t, e] += P[t, e] * g
    return d


def plan(index: np.ndarray, E: int):
    T, k = index.shape
    flat = index.reshape(-1)
    rows = [s for e in range(E) for s in np.nonzero(flat == e)[0]]
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    row_token, slot_row = np.full(T * k, -1), np.full(T * k, -1)
    for r, s in enumerate(rows):
        row_token[r], slot_row[s] = s // k, r
    return offsets, row_token, slot_row.reshape(T, k)


def grouped(x: np.ndarray, offsets, W, bias=None):
    """(Y, S) of rows x [R, K]; rows past offsets[E] are 0. W: function of e giving [N, K]."""
    N = W(0).shape[0]
    Y, S = np.zeros((x.shape[0], N)), np.zeros((x.shape[0], N))
    for e in range(len(offsets) - 1):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        if r.start == r.stop:
            continue
        Y[r], S[r] = x[r] @ W(e).T, np.abs(x[r]) @ np.abs(W(e)).T
        if bias is not None:
            Y[r] += bias[e]
            S[r] += np.abs(bias[e])
    return Y, S


def mx4_quantize(x: np.ndarray):
    """(codes [rows, K], bytes [rows, K/32]) as whole numbers, from the format's definition."""
    rows, K = x.shape
    codes, bytes_ = np.zeros((rows, K), np.int64), np.zeros((rows, K // 32), np.int64)
    for r in range(rows):
        for g in range(K // 32):
            v = x[r, 32 * g:32 * g + 32].astype(np.float64)
            if not np.isfinite(v).all():
                bytes_[r, g] = 255
                continue
            a = np.abs(v).max()
            b = 0 if a == 0 else max(0, 127 + (math.frexp(a)[1] - 1) - 2)
            bytes_[r, g] = b
            u = np.abs(v) / 2.0 ** (b - 127)
            for i in range(32):
                d = np.abs(MAGNITUDES - u[i])
                best = np.nonzero(d == d.min())[0]
                c = int(best[0]) if len(best) == 1 or best[0] % 2 == 0 else int(best[1])
                codes[r, 32 * g + i] = c + (8 if np.signbit(v[i]) else 0)
    return codes, bytes_


def mx4_values(codes: np.ndarray, bytes_: np.ndarray) -> np.ndarray:
    scale = np.where(bytes_ == 255, np.nan, 2.0 ** (bytes_.astype(np.float64) - 127))
    v = MAGNITUDES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return v * np.repeat(scale, 32, axis=-1)
