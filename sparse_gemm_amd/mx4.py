"""Python face of include/bsr_mx4.h: microscaled 4-bit values (32 E2M1 codes share one power-of-two scale
byte) and the grouped product on 4-bit weights."""
from __future__ import annotations

from typing import Optional, Union

import torch

from .experts import C, ExpertPlan, _sizes, call, device_of, output, pointer

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


def quantize(X: torch.Tensor, want_values: bool = False):
    """Mx4 of X [rows, K] or [E, rows, K] (bf16, K a multiple of 32) via bsr_mx4_quantize. want_values: also the
    bf16 values that the codes stand for (X [rows, K] only), as (Mx4, values)."""
    d = device_of(X, "X")
    if X.dim() == 3:
        if want_values:
            raise ValueError("want_values needs X of 2 dimensions")
        E, rows, K = X.shape
        xp = pointer(X, "X", (E, rows, K), _BF16, d)
        codes = output(None, "codes", (E, rows, K // 2), _U8, d)
        scales = output(None, "scales", (E, chunks(K), rows, 8), _U8, d)
        cp, sp = codes.data_ptr(), scales.data_ptr()
        for e in range(E):
            call(C.bsr_mx4_quantize, "bsr_mx4_quantize", d, xp + e * rows * K * 2, rows, K, cp + e * rows * (K // 2),
                 sp + e * chunks(K) * rows * 8, None)
        return Mx4(codes, scales)
    rows, K = _sizes(X, "X", 2)
    xp = pointer(X, "X", (rows, K), _BF16, d)
    codes = output(None, "codes", (rows, K // 2), _U8, d)
    scales = output(None, "scales", (chunks(K), rows, 8), _U8, d)
    values = output(None, "values", (rows, K), _BF16, d) if want_values else None
    call(C.bsr_mx4_quantize, "bsr_mx4_quantize", d, xp, rows, K, codes.data_ptr(), scales.data_ptr(),
         values.data_ptr() if want_values else None)
    return (Mx4(codes, scales), values) if want_values else Mx4(codes, scales)


def dequantize(q: Mx4) -> torch.Tensor:
    """The bf16 values of q [rows, K] or [E, rows, K] via bsr_mx4_dequantize."""
    d = device_of(q.codes, "codes")
    *lead, rows, half = q.codes.shape
    K = 2 * half
    if len(lead) > 1:
        raise ValueError("codes must have 2 or 3 dimensions")
    cp = pointer(q.codes, "codes", (*lead, rows, half), _U8, d)
    sp = pointer(q.scales, "scales", (*lead, chunks(K), rows, 8), _U8, d)
    out = output(None, "values", (*lead, rows, K), _BF16, d)
    for e in range(lead[0] if lead else 1):
        call(C.bsr_mx4_dequantize, "bsr_mx4_dequantize", d, cp + e * rows * half, sp + e * chunks(K) * rows * 8, rows, K,
             out.data_ptr() + e * rows * K * 2)
    return out


def expert_fwd(plan: ExpertPlan, X: Union[torch.Tensor, Mx4], W: Mx4, bias: Optional[torch.Tensor] = None,
               gather: bool = True, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """experts.expert_fwd with W [E, N, K] in 4 bits: activations in bf16 (bsr_expert_fwd_mx4) or in 4 bits
    (bsr_expert_fwd_mx4_mx4)."""
    _, N, half = _sizes(W.codes, "W.codes", 3)
    K, T, R, E, d = 2 * half, plan.T, plan.R, plan.E, plan.device
    rows = T if gather else R
    cp = pointer(W.codes, "W.codes", (E, N, half), _U8, d)
    sp = pointer(W.scales, "W.scales", (E, chunks(K), N, 8), _U8, d)
    bp = None if bias is None else pointer(bias, "bias", (E, N), _BF16, d)
    out = output(out, "out", (R, N), _BF16, d)
    token = plan._token if gather else None
    if isinstance(X, Mx4):
        xc = pointer(X.codes, "X.codes", (rows, half), _U8, d)
        xs = pointer(X.scales, "X.scales", (chunks(K), rows, 8), _U8, d)
        call(C.bsr_expert_fwd_mx4_mx4, "bsr_expert_fwd_mx4_mx4", d, xc, xs, T, R, E, N, K, plan._offsets, token, cp, sp, bp,
             out.data_ptr())
    else:
        xp = pointer(X, "X", (rows, K), _BF16, d)
        call(C.bsr_expert_fwd_mx4, "bsr_expert_fwd_mx4", d, xp, T, R, E, N, K, plan._offsets, token, cp, sp, bp,
             out.data_ptr())
    return out
