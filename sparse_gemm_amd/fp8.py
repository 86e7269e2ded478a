"""Python face of include/bsr_fp8_blocks.h: 8-bit floating point (E4M3) with a power-of-two scale for each block of 128 (128 columns
of a row for activations, 128 x 128 for weights) and the product grouped by expert on 8-bit weights.

A plain linear layer on 8-bit weights W [1, N, K] is one expert that takes every row, its plan made once for a number of rows T:
    plan = ExpertPlan.from_index(torch.zeros((T, 1), dtype=torch.int32, device=x.device), 1)
    y = fp8.expert_fwd(plan, fp8.quantize_rows(x), W)"""
from __future__ import annotations

from typing import Optional, Union

import torch

from . import _lib
from .experts import C, ExpertPlan, current_device, elsewhere, narrow, new2, new3, pointer, raw_stream, sizes

_BF16, _U8 = torch.bfloat16, torch.uint8
GROUP = 128     # columns of a row, or rows and columns of a matrix, that share a scale
CHUNK = 512     # columns whose 4 scale bytes lie side by side (rows)


def _up(n: int, m: int) -> int:
    return -(-n // m)


class Fp8Rows:
    """Activations [rows, K] in 8 bits: codes uint8 [rows, K] (E4M3) and scales uint8 [ceil(K/512), rows, 4], one byte b
    (2^(b - 127)) for each 128 columns of a row."""

    __slots__ = ("codes", "scales")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        self.codes, self.scales = codes, scales

    @property
    def shape(self):
        return tuple(self.codes.shape)

    @classmethod
    def from_rows(cls, codes: torch.Tensor, scale_rows: torch.Tensor) -> "Fp8Rows":
        """From scale bytes stored row by row ([rows, ceil(K/128)]): lays them out once."""
        rows, K = codes.shape
        groups = _up(K, GROUP)
        if tuple(scale_rows.shape) != (rows, groups):
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scale_rows.shape)} do not fit")
        c = _up(K, CHUNK)
        padded = torch.zeros((rows, 4 * c), dtype=_U8, device=scale_rows.device)
        padded[:, :groups] = scale_rows
        return cls(codes.contiguous(), padded.reshape(rows, c, 4).transpose(0, 1).contiguous())

    def scale_rows(self) -> torch.Tensor:
        """The scale bytes row by row, [rows, ceil(K/128)]."""
        rows, K = self.codes.shape
        return self.scales.transpose(0, 1).reshape(rows, 4 * _up(K, CHUNK))[:, :_up(K, GROUP)].contiguous()


class Fp8Blocks:
    """A weight [N, K] or those of E experts [E, N, K] in 8 bits: codes uint8 [..., N, K] (E4M3) and scales uint8
    [..., ceil(N/128), ceil(K/128)], one byte b (2^(b - 127)) for each block of 128 x 128."""

    __slots__ = ("codes", "scales")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        self.codes, self.scales = codes, scales

    @property
    def shape(self):
        return tuple(self.codes.shape)


def quantize_rows(X: torch.Tensor, want_values: bool = False):
    """Fp8Rows of X [rows, K] (bf16, K a multiple of 16) via bsr_fp8_quantize_rows. want_values: also the bf16 values that the
    codes stand for, as (Fp8Rows, values)."""
    d = X.get_device()
    if d < 0 or d != current_device():
        return elsewhere(quantize_rows, d, X, want_values)
    rows, K = sizes(X, "X", 2)
    xp = pointer(X, "X", (rows, K), _BF16, d)
    codes, scales = new2(rows, K, _U8), new3(_up(K, CHUNK), rows, 4, _U8)
    values = new2(rows, K, _BF16) if want_values else None
    status = C.bsr_fp8_quantize_rows(xp, rows, K, codes.data_ptr(), scales.data_ptr(),
                                     None if values is None else values.data_ptr(), raw_stream(d))
    if status:
        _lib.check(status, "bsr_fp8_quantize_rows")
    q = Fp8Rows(codes, scales)
    return (q, values) if want_values else q


def quantize_blocks(W: torch.Tensor, transposed: bool = False):
    """Fp8Blocks of W [N, K] or [E, N, K] (bf16, K a multiple of 16, N of 8) via bsr_fp8_quantize_blocks. transposed (N a
    multiple of 16): also those of the transposed matrices [..., K, N], in the same pass, as (Fp8Blocks, Fp8Blocks)."""
    d = W.get_device()
    if d < 0 or d != current_device():
        return elsewhere(quantize_blocks, d, W, transposed)
    if W.dim() not in (2, 3):
        raise ValueError(f"W must have 2 or 3 dimensions, got {W.dim()}")
    N, K = W.shape[-2:]
    E = W.shape[0] if W.dim() == 3 else 1
    for n in (E, N, K):
        narrow(n, "W")
    wp = pointer(W, "W", W.shape, _BF16, d)
    nb, kb = _up(N, GROUP), _up(K, GROUP)
    codes, scales = new3(E, N, K, _U8), new3(E, nb, kb, _U8)
    ct, st = (new3(E, K, N, _U8), new3(E, kb, nb, _U8)) if transposed else (None, None)
    status = C.bsr_fp8_quantize_blocks(wp, E, N, K, codes.data_ptr(), scales.data_ptr(), ct.data_ptr() if transposed else None,
                                       st.data_ptr() if transposed else None, raw_stream(d))
    if status:
        _lib.check(status, "bsr_fp8_quantize_blocks")
    lay = (lambda t: t) if W.dim() == 3 else (lambda t: t[0])
    q = Fp8Blocks(lay(codes), lay(scales))
    return (q, Fp8Blocks(lay(ct), lay(st))) if transposed else q


def dequantize(q: Union[Fp8Rows, Fp8Blocks]) -> torch.Tensor:
    """The bf16 values of q via bsr_fp8_dequantize_rows or bsr_fp8_dequantize_blocks."""
    d = q.codes.get_device()
    if d < 0 or d != current_device():
        return elsewhere(dequantize, d, q)
    if isinstance(q, Fp8Rows):
        rows, K = sizes(q.codes, "codes", 2)
        cp = pointer(q.codes, "codes", (rows, K), _U8, d)
        sp = pointer(q.scales, "scales", (_up(K, CHUNK), rows, 4), _U8, d)
        out = new2(rows, K, _BF16)
        what, status = "bsr_fp8_dequantize_rows", C.bsr_fp8_dequantize_rows(cp, sp, rows, K, out.data_ptr(), raw_stream(d))
    else:
        if q.codes.dim() not in (2, 3):
            raise ValueError(f"codes must have 2 or 3 dimensions, got {q.codes.dim()}")
        *lead, N, K = q.codes.shape
        E = lead[0] if lead else 1
        for n in (E, N, K):
            narrow(n, "codes")
        cp = pointer(q.codes, "codes", (*lead, N, K), _U8, d)
        sp = pointer(q.scales, "scales", (*lead, _up(N, GROUP), _up(K, GROUP)), _U8, d)
        out = new3(E, N, K, _BF16)
        what, status = "bsr_fp8_dequantize_blocks", C.bsr_fp8_dequantize_blocks(cp, sp, E, N, K, out.data_ptr(), raw_stream(d))
        out = out if lead else out[0]
    if status:
        _lib.check(status, what)
    return out


def expert_fwd(plan: ExpertPlan, X: Union[torch.Tensor, Fp8Rows], W: Fp8Blocks, bias: Optional[torch.Tensor] = None,
               gather: bool = True, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """experts.expert_fwd with W [E, N, K] in 8 bits: activations in bf16 (bsr_expert_fwd_fp8) or in 8 bits
    (bsr_expert_fwd_fp8_fp8)."""
    T, R, E, d = plan.T, plan.R, plan.E, plan.device
    if d != current_device():
        return elsewhere(expert_fwd, d, plan, X, W, bias, gather, out)
    _, N, K = sizes(W.codes, "W.codes", 3)
    rows = T if gather else R
    cp = pointer(W.codes, "W.codes", (E, N, K), _U8, d)
    sp = pointer(W.scales, "W.scales", (E, _up(N, GROUP), _up(K, GROUP)), _U8, d)
    bp = None if bias is None else pointer(bias, "bias", (E, N), _BF16, d)
    if out is None:
        out = new2(R, N, _BF16)
        op = out.data_ptr()
    else:
        op = pointer(out, "out", (R, N), _BF16, d)
    token = plan._token.data_ptr() if gather else None
    if isinstance(X, Fp8Rows):
        xc = pointer(X.codes, "X.codes", (rows, K), _U8, d)
        xs = pointer(X.scales, "X.scales", (_up(K, CHUNK), rows, 4), _U8, d)
        status = C.bsr_expert_fwd_fp8_fp8(xc, xs, T, R, E, N, K, plan._offsets.data_ptr(), token, cp, sp, bp, op, raw_stream(d))
        what = "bsr_expert_fwd_fp8_fp8"
    else:
        xp = pointer(X, "X", (rows, K), _BF16, d)
        status = C.bsr_expert_fwd_fp8(xp, T, R, E, N, K, plan._offsets.data_ptr(), token, cp, sp, bp, op, raw_stream(d))
        what = "bsr_expert_fwd_fp8"
    if status:
        _lib.check(status, what)
    return out
