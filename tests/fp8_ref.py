"""Plain 64-bit definitions of 8-bit floating point with a scale for each block of 128, and of a whole expert layer (numpy, CPU)."""
from __future__ import annotations

import numpy as np

import expert_ref

CODES = np.arange(127)                        # finite magnitudes 0x00 .. 0x7E
TABLE = np.where(CODES >> 3 == 0, (CODES & 7) * 2.0 ** -9, (8 + (CODES & 7)) * 2.0 ** ((CODES >> 3) - 10.0))
MIDDLE = (TABLE[1:] + TABLE[:-1]) / 2         # exact


def value(codes: np.ndarray) -> np.ndarray:
    """Values of codes 0 .. 255."""
    mag = np.append(TABLE, np.nan)[codes & 0x7F]
    return np.where(codes & 0x80, -mag, mag)


def scale_byte(group: np.ndarray) -> int:
    """The byte of a group: the smallest s >= -127 with the largest finite magnitude <= 448 * 2^s, plus 127."""
    finite = np.abs(group[np.isfinite(group)])
    a = finite.max() if finite.size else 0.0
    s = -127
    if a > 0:
        s = max(-127, int(np.frexp(a)[1]) - 10)
        while a > 448.0 * 2.0 ** s:
            s += 1
    return s + 127


def encode(v: np.ndarray, byte) -> np.ndarray:
    u = np.abs(v) / 2.0 ** (np.asarray(byte, np.float64) - 127)
    u = np.where(np.isfinite(v), u, 0.0)
    lo = np.searchsorted(MIDDLE, u, side="left")      # first code whose upper middle is >= u: below the middle, or on it
    tie = (lo < 126) & (u == MIDDLE[np.minimum(lo, 125)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo)
    code = np.where(np.isfinite(v), code, 0x7F)
    return code + np.where(np.signbit(v), 0x80, 0)


def quantize_rows(x: np.ndarray):
    """(codes [rows, K], bytes [rows, ceil(K/128)])."""
    rows, K = x.shape
    codes, bytes_ = np.zeros((rows, K), np.int64), np.zeros((rows, -(-K // 128)), np.int64)
    for r in range(rows):
        for g in range(bytes_.shape[1]):
            v = x[r, 128 * g:128 * g + 128]
            bytes_[r, g] = scale_byte(v)
            codes[r, 128 * g:128 * g + 128] = encode(v, bytes_[r, g])
    return codes, bytes_


def row_values(codes, bytes_):
    return value(codes) * scales(np.repeat(bytes_, 128, 1)[:, :codes.shape[1]])


def scales(bytes_):
    return np.where(bytes_ == 255, np.nan, 2.0 ** (bytes_.astype(np.float64) - 127))


def quantize_blocks(w: np.ndarray):
    """(codes [N, K], bytes [ceil(N/128), ceil(K/128)])."""
    N, K = w.shape
    codes, bytes_ = np.zeros((N, K), np.int64), np.zeros((-(-N // 128), -(-K // 128)), np.int64)
    for i in range(bytes_.shape[0]):
        for j in range(bytes_.shape[1]):
            at = (slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
            bytes_[i, j] = scale_byte(w[at])
            codes[at] = encode(w[at], bytes_[i, j])
    return codes, bytes_


def block_values(codes, bytes_):
    N, K = codes.shape
    return value(codes) * scales(np.repeat(np.repeat(bytes_, 128, 0)[:N], 128, 1)[:, :K])


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def layer(x, router, up, down, k, renorm, up_bias=None, down_bias=None, terms=0):
    """(out, tolerance, index, gap) of a whole layer; up(e) and down(e) give [2 hidden, dim] and [dim, hidden].

    The tolerance, u = 2^-23 a 32-bit operation (a sum of n terms is off by n u of the sum of their magnitudes):
      gate, up    (dim + 4) u S each
      h           1.1 |u| dg + |silu| du (the slope of silu is at most 1.1) + (|g| + 8) 2u |h| for exp and the quotient
                  + 2^-8 |h| for its rounding to bf16
      weight      2 dl + (E + 100) u / 2 relative, dl the error of a logit
      out         the sums of all these, (k hidden + k + 8) u of the magnitudes, 2^-8 |out| for its rounding
    gap: by how much the k-th logit of a token stands off from the next, in units of their possible error."""
    T, dim = x.shape
    u = 2.0 ** -23
    logits, Sl = x @ router.T, np.abs(x) @ np.abs(router).T
    dl = (dim + 4) * u * Sl
    index, weight, _ = expert_ref.router(logits, k, renorm)
    E = router.shape[0]
    gap = np.full(T, np.inf)
    if k < E:
        order = np.argsort(-logits, axis=1, kind="stable")
        a, b = order[:, k - 1], order[:, k]
        t = np.arange(T)
        gap = (logits[t, a] - logits[t, b]) / (dl[t, a] + dl[t, b])
    out, tol, mag = np.zeros((T, dim)), np.zeros((T, dim)), np.zeros((T, dim))
    for e in range(E):
        t, j = np.nonzero(index == e)
        if t.size == 0:
            continue
        U, D = up(e), down(e)
        hidden = U.shape[0] // 2
        z, S = x[t] @ U.T, np.abs(x[t]) @ np.abs(U).T
        if up_bias is not None:
            z, S = z + up_bias[e], S + np.abs(up_bias[e])
        dz = (dim + 4) * u * S
        g, v = z[:, :hidden], z[:, hidden:]
        h = silu(g) * v
        dh = 1.1 * np.abs(v) * dz[:, :hidden] + np.abs(silu(g)) * dz[:, hidden:] + ((np.abs(g) + 8) * 2 * u + 2.0 ** -8) * np.abs(h)
        y, Sy, dy = h @ D.T, np.abs(h) @ np.abs(D).T, dh @ np.abs(D).T
        if down_bias is not None:
            y, Sy = y + down_bias[e], Sy + np.abs(down_bias[e])
        w = weight[t, j][:, None]
        dw = 2 * dl[t].max(1, keepdims=True) + (E + 100) * u / 2
        np.add.at(out, t, w * y)
        np.add.at(mag, t, w * Sy)
        np.add.at(tol, t, w * (dy + dw * np.abs(y)))
    tol += ((k * (up(0).shape[0] // 2) + k + 8) * u) * mag + 2.0 ** -8 * np.abs(out) + 2.0 ** -126
    return out, tol, index, gap
