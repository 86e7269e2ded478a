"""Python face of include/bsr_experts.h: the router, the plan, the grouped products and the sum of an
expert layer, on torch tensors and the current stream.

T tokens, k slots a token, E experts, R = T * k rows sorted by expert. Every call checks its arguments and
only enqueues work; nothing is copied to the host."""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _lib
from .binding import lib

_LOGITS = {torch.float32: 0, torch.bfloat16: 1}


def check(t: torch.Tensor, name: str, shape, dtype, device: torch.device) -> int:
    """Data pointer of a contiguous tensor of that shape and type on that device; raises otherwise."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def device_of(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    return t.device


_raw_stream = torch._C._cuda_getCurrentRawStream   # the stream's handle alone: current_stream() builds an object


def call(f, what: str, device: torch.device, *args) -> None:
    """f(*args, current stream of device), with that device current; raises BsrError on a status."""
    index = device.index
    if index == torch._C._cuda_getDevice():
        status = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = f(*args, _raw_stream(index))
    if status:
        _lib.check(status, what)


def _sizes(t: torch.Tensor, name: str, dims: int) -> torch.Size:
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    return t.shape


def _out(out: Optional[torch.Tensor], name: str, shape, dtype, device) -> Tuple[torch.Tensor, int]:
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
        return out, out.data_ptr()
    return out, check(out, name, shape, dtype, device)


def router_fwd(logits: torch.Tensor, k: int, renormalize: bool = True, out=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(index int32 [T, k], weight f32 [T, k]): the k largest of logits [T, E] (f32 or bf16), ties to the
    lowest expert, and their softmax weights, over all experts or over the chosen ones, via bsr_router_fwd.
    Experts at -infinity are never chosen: index -1, weight 0."""
    T, E = _sizes(logits, "logits", 2)
    if logits.dtype not in _LOGITS:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    d = device_of(logits, "logits")
    lp = check(logits, "logits", (T, E), logits.dtype, d)
    index, ip = _out(out[0] if out else None, "index", (T, k), torch.int32, d)
    weight, wp = _out(out[1] if out else None, "weight", (T, k), torch.float32, d)
    call(lib().bsr_router_fwd, "bsr_router_fwd", d, lp, _LOGITS[logits.dtype], T, E, k, int(renormalize), ip, wp)
    return index, weight


def router_bwd(logits: torch.Tensor, index: torch.Tensor, weight: torch.Tensor, dweight: torch.Tensor,
               renormalize: bool = True, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dlogits [T, E] (the logits' type) of router_fwd's weights, via bsr_router_bwd."""
    T, E = _sizes(logits, "logits", 2)
    k = _sizes(index, "index", 2)[1]
    if logits.dtype not in _LOGITS:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    d = device_of(logits, "logits")
    lp = check(logits, "logits", (T, E), logits.dtype, d)
    ip = check(index, "index", (T, k), torch.int32, d)
    wp = check(weight, "weight", (T, k), torch.float32, d)
    gp = check(dweight, "dweight", (T, k), torch.float32, d)
    out, op = _out(out, "out", (T, E), logits.dtype, d)
    call(lib().bsr_router_bwd, "bsr_router_bwd", d, lp, _LOGITS[logits.dtype], T, E, k, int(renormalize), ip, wp, gp, op)
    return out


class ExpertPlan:
    """Which rows belong to which expert, on the device: offsets [E+1], row_token [T*k], slot_row [T, k] (int32)."""

    __slots__ = ("offsets", "row_token", "slot_row", "T", "k", "E", "R", "device")

    def __init__(self, offsets: torch.Tensor, row_token: torch.Tensor, slot_row: torch.Tensor):
        self.T, self.k = _sizes(slot_row, "slot_row", 2)
        self.R = self.T * self.k
        self.E = _sizes(offsets, "offsets", 1)[0] - 1
        self.device = device_of(offsets, "offsets")
        check(offsets, "offsets", (self.E + 1,), torch.int32, self.device)
        check(row_token, "row_token", (self.R,), torch.int32, self.device)
        check(slot_row, "slot_row", (self.T, self.k), torch.int32, self.device)
        self.offsets, self.row_token, self.slot_row = offsets, row_token, slot_row

    @classmethod
    def from_index(cls, index: torch.Tensor, E: int) -> "ExpertPlan":
        """The plan of index [T, k] int32 (entries outside [0, E) are dropped), via bsr_expert_plan."""
        T, k = _sizes(index, "index", 2)
        d = device_of(index, "index")
        ip = check(index, "index", (T, k), torch.int32, d)
        self = cls.__new__(cls)
        self.T, self.k, self.R, self.E, self.device = T, k, T * k, E, d
        self.offsets = torch.empty((max(E, 0) + 1,), dtype=torch.int32, device=d)
        self.row_token = torch.empty((self.R,), dtype=torch.int32, device=d)
        self.slot_row = torch.empty((T, k), dtype=torch.int32, device=d)
        need = lib().bsr_expert_plan_workspace(T, k, E)
        ws = torch.empty((need,), dtype=torch.uint8, device=d) if need else None
        call(lib().bsr_expert_plan, "bsr_expert_plan", d, ip, T, k, E, self.offsets.data_ptr(),
             self.row_token.data_ptr(), self.slot_row.data_ptr(), ws.data_ptr() if need else None, need)
        return self


def rows_of(plan: ExpertPlan, gather: bool) -> int:
    return plan.T if gather else plan.R


def expert_fwd(plan: ExpertPlan, X: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None,
               gather: bool = True, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y [R, N] bf16: row r of expert e is x(r) . W[e]^T + bias[e]; W [E, N, K], bias [E, N] or None, via
    bsr_expert_fwd. gather: X is [T, K] by token; otherwise [R, K], sorted like Y."""
    E, N, K = _sizes(W, "W", 3)
    d = plan.device
    xp = check(X, "X", (rows_of(plan, gather), K), torch.bfloat16, d)
    wp = check(W, "W", (plan.E, N, K), torch.bfloat16, d)
    bp = None if bias is None else check(bias, "bias", (E, N), torch.bfloat16, d)
    out, op = _out(out, "out", (plan.R, N), torch.bfloat16, d)
    call(lib().bsr_expert_fwd, "bsr_expert_fwd", d, xp, plan.T, plan.R, E, N, K, plan.offsets.data_ptr(),
         plan.row_token.data_ptr() if gather else None, wp, bp, op)
    return out


def expert_bwd_input(plan: ExpertPlan, dY: torch.Tensor, W: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dX [R, K] = dY . W[e] by rows sorted like dY [R, N], via bsr_expert_bwd_input. For a gathered X sum a
    token's rows: combine_fwd(plan, dX, None)."""
    E, N, K = _sizes(W, "W", 3)
    d = plan.device
    gp = check(dY, "dY", (plan.R, N), torch.bfloat16, d)
    wp = check(W, "W", (plan.E, N, K), torch.bfloat16, d)
    out, op = _out(out, "out", (plan.R, K), torch.bfloat16, d)
    call(lib().bsr_expert_bwd_input, "bsr_expert_bwd_input", d, gp, plan.R, E, N, K, plan.offsets.data_ptr(), wp, op)
    return out


def expert_bwd_weight(plan: ExpertPlan, dY: torch.Tensor, X: torch.Tensor, gather: bool = True, want_dbias: bool = False,
                      out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(dW [E, N, K], dbias [E, N] or None) via bsr_expert_bwd_weight; X and gather as for expert_fwd."""
    N, K = _sizes(dY, "dY", 2)[1], _sizes(X, "X", 2)[1]
    d = plan.device
    gp = check(dY, "dY", (plan.R, N), torch.bfloat16, d)
    xp = check(X, "X", (rows_of(plan, gather), K), torch.bfloat16, d)
    dW, op = _out(out, "out", (plan.E, N, K), torch.bfloat16, d)
    db = torch.empty((plan.E, N), dtype=torch.bfloat16, device=d) if want_dbias else None
    call(lib().bsr_expert_bwd_weight, "bsr_expert_bwd_weight", d, gp, xp, plan.T, plan.R, plan.E, N, K,
         plan.offsets.data_ptr(), plan.row_token.data_ptr() if gather else None, op, db.data_ptr() if want_dbias else None)
    return dW, db


def combine_fwd(plan: ExpertPlan, Y: torch.Tensor, weight: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [T, N] = sum over a token's slots of weight [T, k] (f32; None: 1) times its rows of Y [R, N], via
    bsr_expert_combine_fwd."""
    N = _sizes(Y, "Y", 2)[1]
    d = plan.device
    yp = check(Y, "Y", (plan.R, N), torch.bfloat16, d)
    wp = None if weight is None else check(weight, "weight", (plan.T, plan.k), torch.float32, d)
    out, op = _out(out, "out", (plan.T, N), torch.bfloat16, d)
    call(lib().bsr_expert_combine_fwd, "bsr_expert_combine_fwd", d, yp, plan.T, plan.k, N, plan.slot_row.data_ptr(), wp, op)
    return out


def combine_bwd(plan: ExpertPlan, dout: torch.Tensor, Y: torch.Tensor,
                weight: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dY [R, N] bf16, dweight [T, k] f32) of combine_fwd, via bsr_expert_combine_bwd."""
    N = _sizes(Y, "Y", 2)[1]
    d = plan.device
    gp = check(dout, "dout", (plan.T, N), torch.bfloat16, d)
    yp = check(Y, "Y", (plan.R, N), torch.bfloat16, d)
    wp = None if weight is None else check(weight, "weight", (plan.T, plan.k), torch.float32, d)
    dY = torch.empty((plan.R, N), dtype=torch.bfloat16, device=d)
    dw = torch.empty((plan.T, plan.k), dtype=torch.float32, device=d)
    call(lib().bsr_expert_combine_bwd, "bsr_expert_combine_bwd", d, gp, yp, plan.T, plan.k, plan.E, N,
         plan.offsets.data_ptr(), plan.slot_row.data_ptr(), wp, dY.data_ptr(), dw.data_ptr())
    return dY, dw
