"""Python face of include/bsr_expert_ffn.h: a whole layer of experts for a few tokens in one call."""
from __future__ import annotations

from typing import Optional, Union

import torch

from . import _lib
from .experts import C, MOST, current_device, elsewhere, empty_strided, narrow, new2, pointer, raw_stream, sizes
from .fp8 import GROUP, Fp8Blocks
from .mx4 import Mx4, chunks

_BF16, _U8 = torch.bfloat16, torch.uint8
TOKENS = 16     # BSR_EXPERT_FFN_TOKENS
Weight = Union[torch.Tensor, Mx4, Fp8Blocks]


def _weight(W: Weight, name: str, E: int, rows: int, cols: int, d: int):
    """(form, address of the weights, of their scales or None) of W [E, rows, cols]."""
    if isinstance(W, Mx4):
        return (1, pointer(W.codes, f"{name}.codes", (E, rows, cols // 2), _U8, d),
                pointer(W.scales, f"{name}.scales", (E, chunks(cols), rows, 8), _U8, d))
    if isinstance(W, Fp8Blocks):
        return (2, pointer(W.codes, f"{name}.codes", (E, rows, cols), _U8, d),
                pointer(W.scales, f"{name}.scales", (E, -(-rows // GROUP), -(-cols // GROUP)), _U8, d))
    return 0, pointer(W, name, (E, rows, cols), _BF16, d), None


def expert_ffn(x: torch.Tensor, router: torch.Tensor, up: Weight, down: Weight, k: int, renormalize: bool = True,
               up_bias: Optional[torch.Tensor] = None, down_bias: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [T, dim] of up to 16 tokens x [T, dim] (bf16) through the k experts that router [E, dim] chooses for each, via
    bsr_expert_ffn: sum over them of weight * (down_e(silu(gate_e x) * up_e x)). up [E, 2 * hidden, dim] holds the gate rows before
    the up rows, down is [E, dim, hidden]; both in bf16, both Mx4 or both Fp8Blocks. Biases [E, 2 * hidden] and [E, dim]. Forward only."""
    d = x.get_device()
    if d < 0 or d != current_device():
        return elsewhere(expert_ffn, d, x, router, up, down, k, renormalize, up_bias, down_bias, out)
    T, dim = sizes(x, "x", 2)
    E = sizes(router, "router", 2)[0]
    if type(up) is not type(down) and (isinstance(up, (Mx4, Fp8Blocks)) or isinstance(down, (Mx4, Fp8Blocks))):
        raise TypeError("up and down must be held in the same form")
    rows = sizes(up if isinstance(up, torch.Tensor) else up.codes, "up", 3)[1]
    if T > TOKENS:
        raise ValueError(f"x has {T} rows, expected at most {TOKENS}")
    if rows % 2:
        raise ValueError(f"up has {rows} rows an expert, expected gate and up rows")
    narrow(E, "router")
    hidden = rows // 2
    xp, rp = pointer(x, "x", (T, dim), _BF16, d), pointer(router, "router", (E, dim), _BF16, d)
    form, wp, wsp = _weight(up, "up", E, rows, dim, d)
    _, vp, vsp = _weight(down, "down", E, dim, hidden, d)
    bp = None if up_bias is None else pointer(up_bias, "up_bias", (E, rows), _BF16, d)
    cp = None if down_bias is None else pointer(down_bias, "down_bias", (E, dim), _BF16, d)
    if out is None:
        out = new2(T, dim, _BF16)
        op = out.data_ptr()
    else:
        op = pointer(out, "out", (T, dim), _BF16, d)
    k = max(min(k, MOST), -1)   # ctypes would pass the low 32 bits
    need = C.bsr_expert_ffn_workspace(T, dim, hidden, E, k)
    ws = empty_strided((need,), (1,), _U8)
    status = C.bsr_expert_ffn(xp, T, dim, hidden, E, k, renormalize, rp, form, wp, wsp, vp, vsp, bp, cp, op, ws.data_ptr(), need,
                              raw_stream(d))
    if status:
        _lib.check(status, "bsr_expert_ffn")
    return out
