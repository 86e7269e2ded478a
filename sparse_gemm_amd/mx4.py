"""Python face of include/bsr_mx4.h: microscaled 4-bit values (32 E2M1 codes share one power-of-two scale
byte) and the grouped product on 4-bit weights."""
from __future__ import annotations

from typing import Optional, Union

import torch

from .binding import lib
from .experts import ExpertPlan, _out, _sizes, call, check, device_of, rows_of

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
        codes = torch.empty((E, rows, K // 2), dtype=torch.uint8, device=d)
        scales = torch.empty((E, chunks(K), rows, 8), dtype=torch.uint8, device=d)
        xp = check(X, "X", (E, rows, K), torch.bfloat16, d)
        for e in range(E):
            call(lib().bsr_mx4_quantize, "bsr_mx4_quantize", d, xp + e * rows * K * 2, rows, K, codes[e].data_ptr(),
                 scales[e].data_ptr(), None)
        return Mx4(codes, scales)
    rows, K = _sizes(X, "X", 2)
    xp = check(X, "X", (rows, K), torch.bfloat16, d)
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=d)
    scales = torch.empty((chunks(K), rows, 8), dtype=torch.uint8, device=d)
    values = torch.empty((rows, K), dtype=torch.bfloat16, device=d) if want_values else None
    call(lib().bsr_mx4_quantize, "bsr_mx4_quantize", d, xp, rows, K, codes.data_ptr(), scales.data_ptr(),
         values.data_ptr() if want_values else None)
    return (Mx4(codes, scales), values) if want_values else Mx4(codes, scales)


def dequantize(q: Mx4) -> torch.Tensor:
    """The bf16 values of q [rows, K] or [E, rows, K] via bsr_mx4_dequantize."""
    d = device_of(q.codes, "codes")
    *lead, rows, half = q.codes.shape
    K = 2 * half
    if len(lead) > 1:
        raise ValueError("codes must have 2 or 3 dimensions")
    cp = check(q.codes, "codes", (*lead, rows, half), torch.uint8, d)
    sp = check(q.scales, "scales", (*lead, chunks(K), rows, 8), torch.uint8, d)
    out = torch.empty((*lead, rows, K), dtype=torch.bfloat16, device=d)
    for e in range(lead[0] if lead else 1):
        call(lib().bsr_mx4_dequantize, "bsr_mx4_dequantize", d, cp + e * rows * half, sp + e * chunks(K) * rows * 8, rows, K,
             out.data_ptr() + e * rows * K * 2)
    return out


def expert_fwd(plan: ExpertPlan, X: Union[torch.Tensor, Mx4], W: Mx4, bias: Optional[torch.Tensor] = None,
               gather: bool = True, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """experts.expert_fwd with W [E, N, K] in 4 bits: activations in bf16 (bsr_expert_fwd_mx4) or in 4 bits
    (bsr_expert_fwd_mx4_mx4)."""
    E, N, half = _sizes(W.codes, "W.codes", 3)
    K, d = 2 * half, plan.device
    rows = rows_of(plan, gather)
    cp = check(W.codes, "W.codes", (plan.E, N, half), torch.uint8, d)
    sp = check(W.scales, "W.scales", (plan.E, chunks(K), N, 8), torch.uint8, d)
    bp = None if bias is None else check(bias, "bias", (E, N), torch.bfloat16, d)
    out, op = _out(out, "out", (plan.R, N), torch.bfloat16, d)
    tail = (plan.T, plan.R, E, N, K, plan.offsets.data_ptr(), plan.row_token.data_ptr() if gather else None, cp, sp, bp, op)
    if isinstance(X, Mx4):
        xc = check(X.codes, "X.codes", (rows, half), torch.uint8, d)
        xs = check(X.scales, "X.scales", (chunks(K), rows, 8), torch.uint8, d)
        call(lib().bsr_expert_fwd_mx4_mx4, "bsr_expert_fwd_mx4_mx4", d, xc, xs, *tail)
    else:
        xp = check(X, "X", (rows, K), torch.bfloat16, d)
        call(lib().bsr_expert_fwd_mx4, "bsr_expert_fwd_mx4", d, xp, *tail)
    return out
