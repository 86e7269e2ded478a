"""Python face of include/bsr_mx4.h: microscaled 4-bit values (32 E2M1 codes share one power-of-two scale
byte) and the grouped product on 4-bit weights.

A plain linear layer on 4-bit weights W [1, N, K] is one expert that takes every row, its plan made once for a number of rows T:
    plan = ExpertPlan.from_index(torch.zeros((T, 1), dtype=torch.int32, device=x.device), 1)
    y = mx4.expert_fwd(plan, x, W)"""
from __future__ import annotations

from typing import Optional, Union

import torch

from . import _lib
from .experts import C, ExpertPlan, current_device, elsewhere, empty_strided, narrow, new2, new3, pointer, raw_stream, sizes

_BF16, _U8 = torch.bfloat16, torch.uint8
GROUP = 32      # elements that share a scale
CHUNK = 256     # columns whose 8 scale bytes lie side by side


def chunks(K: int) -> int:
    return -(-K // CHUNK)


class Mx4:
    """A matrix [rows, K] or the weights of E experts [E, rows, K] in microscaled 4-bit form:
    codes uint8 [..., rows, K/2] and scales uint8 [..., ceil(K/256), rows, 8]."""

    __slots__ = ("codes", "scales")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        self.codes, self.scales = codes, scales

    @property
    def shape(self):
        return (*self.codes.shape[:-1], 2 * self.codes.shape[-1])

    @classmethod
    def from_rows(cls, codes: torch.Tensor, scale_rows: torch.Tensor) -> "Mx4":
        """From scale bytes stored row by row ([..., rows, K/32]): lays them out once."""
        *lead, rows, groups = scale_rows.shape
        if 2 * codes.shape[-1] != GROUP * groups or tuple(codes.shape[:-1]) != (*lead, rows):
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scale_rows.shape)} do not fit")
        c = chunks(GROUP * groups)
        padded = torch.zeros((*lead, rows, c * 8), dtype=torch.uint8, device=scale_rows.device)
        padded[..., :groups] = scale_rows
        return cls(codes.contiguous(), padded.reshape(*lead, rows, c, 8).transpose(-3, -2).contiguous())

    def scale_rows(self) -> torch.Tensor:
        """The scale bytes row by row, [..., rows, K/32]."""
        s = self.scales.transpose(-3, -2)
        return s.reshape(*s.shape[:-2], -1)[..., :self.shape[-1] // GROUP].contiguous()


def _quantize(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, values: Optional[torch.Tensor], d: int) -> None:
    rows, K = X.shape
    status = C.bsr_mx4_quantize(X.data_ptr(), rows, K, codes.data_ptr(), scales.data_ptr(),
                                None if values is None else values.data_ptr(), raw_stream(d))
    if status:
        _lib.check(status, "bsr_mx4_quantize")


def _own_piece(c: int, rows: int) -> Optional[torch.Tensor]:
    """Where one expert's scales [c, rows, 8] stand during a call, if they do not lie on whole 16 bytes among all experts'
    (c * rows odd): the library takes 16-byte aligned arrays."""
    return new3(c, rows, 8, _U8) if c * rows % 2 else None


def quantize(X: torch.Tensor, want_values: bool = False):
    """Mx4 of X [rows, K] or [E, rows, K] (bf16, K a multiple of 32) via bsr_mx4_quantize. want_values: also the
    bf16 values that the codes stand for (X [rows, K] only), as (Mx4, values)."""
    d = X.get_device()
    if d < 0 or d != current_device():
        return elsewhere(quantize, d, X, want_values)
    if X.dim() == 3:
        if want_values:
            raise ValueError("want_values needs X of 2 dimensions")
        E, rows, K = X.shape
        narrow(K, "X")
        pointer(X, "X", (E, rows, K), _BF16, d)
        c = chunks(K)
        codes = new3(E, rows, K // 2, _U8)
        scales = empty_strided((E, c, rows, 8), (c * rows * 8, rows * 8, 8, 1), _U8)
        own = _own_piece(c, rows)
        for e in range(E):
            _quantize(X[e], codes[e], scales[e] if own is None else own, None, d)
            if own is not None:
                scales[e].copy_(own)
        return Mx4(codes, scales)
    rows, K = sizes(X, "X", 2)
    pointer(X, "X", (rows, K), _BF16, d)
    codes, scales = new2(rows, K // 2, _U8), new3(chunks(K), rows, 8, _U8)
    values = new2(rows, K, _BF16) if want_values else None
    _quantize(X, codes, scales, values, d)
    return (Mx4(codes, scales), values) if want_values else Mx4(codes, scales)


def dequantize(q: Mx4) -> torch.Tensor:
    """The bf16 values of q [rows, K] or [E, rows, K] via bsr_mx4_dequantize."""
    d = q.codes.get_device()
    if d < 0 or d != current_device():
        return elsewhere(dequantize, d, q)
    *lead, rows, half = q.codes.shape
    K = 2 * half
    narrow(K, "the matrix")
    if len(lead) > 1:
        raise ValueError("codes must have 2 or 3 dimensions")
    cp = pointer(q.codes, "codes", (*lead, rows, half), _U8, d)
    sp = pointer(q.scales, "scales", (*lead, chunks(K), rows, 8), _U8, d)
    out = torch.empty((*lead, rows, K), dtype=_BF16, device=q.codes.device)
    own = _own_piece(chunks(K), rows) if lead else None
    for e in range(lead[0] if lead else 1):
        if own is not None:
            own.copy_(q.scales[e])
        status = C.bsr_mx4_dequantize(cp + e * rows * half, sp + e * chunks(K) * rows * 8 if own is None else own.data_ptr(),
                                      rows, K, out.data_ptr() + e * rows * K * 2, raw_stream(d))
        if status:
            _lib.check(status, "bsr_mx4_dequantize")
    return out


def expert_fwd(plan: ExpertPlan, X: Union[torch.Tensor, Mx4], W: Mx4, bias: Optional[torch.Tensor] = None,
               gather: bool = True, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """experts.expert_fwd with W [E, N, K] in 4 bits: activations in bf16 (bsr_expert_fwd_mx4) or in 4 bits
    (bsr_expert_fwd_mx4_mx4)."""
    T, R, E, d = plan.T, plan.R, plan.E, plan.device
    if d != current_device():
        return elsewhere(expert_fwd, d, plan, X, W, bias, gather, out)
    _, N, half = sizes(W.codes, "W.codes", 3)
    K, rows = 2 * half, T if gather else R
    cp = pointer(W.codes, "W.codes", (E, N, half), _U8, d)
    sp = pointer(W.scales, "W.scales", (E, chunks(K), N, 8), _U8, d)
    bp = None if bias is None else pointer(bias, "bias", (E, N), _BF16, d)
    if out is None:
        out = new2(R, N, _BF16)
        op = out.data_ptr()
    else:
        op = pointer(out, "out", (R, N), _BF16, d)
    token = plan._token.data_ptr() if gather else None
    if isinstance(X, Mx4):
        xc = pointer(X.codes, "X.codes", (rows, half), _U8, d)
        xs = pointer(X.scales, "X.scales", (chunks(K), rows, 8), _U8, d)
        status = C.bsr_expert_fwd_mx4_mx4(xc, xs, T, R, E, N, K, plan._offsets.data_ptr(), token, cp, sp, bp, op, raw_stream(d))
        what = "bsr_expert_fwd_mx4_mx4"
    else:
        xp = pointer(X, "X", (rows, K), _BF16, d)
        status = C.bsr_expert_fwd_mx4(xp, T, R, E, N, K, plan._offsets.data_ptr(), token, cp, sp, bp, op, raw_stream(d))
        what = "bsr_expert_fwd_mx4"
    if status:
        _lib.check(status, what)
    return out
