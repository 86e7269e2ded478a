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
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


class _Calls:
    """The library's functions, each looked up once (the library is loaded on first use)."""

    def __getattr__(self, name):
        f = getattr(lib(), name)
        setattr(self, name, f)
        return f


C = _Calls()

# What a call of a few microseconds spends on the host is most of its time. The current stream's handle and the
# current device come without building objects for them, and outputs from the allocation call that torch's
# compiled graphs use (on the current device, shape and strides as tuples). These names are private to torch: where it lacks
# one, the public call stands in.
raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda device: torch.cuda.current_stream(device).cuda_stream)
current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
try:
    from torch._C._dynamo.guards import _empty_strided_cuda as empty_strided
except ImportError:
    def empty_strided(shape, strides, dtype):
        return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")


def pointer(t: torch.Tensor, name: str, shape, dtype, device: int) -> int:
    """Data pointer of a contiguous tensor of that shape and type on GPU `device`; raises otherwise."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def new2(rows: int, cols: int, dtype) -> torch.Tensor:
    return empty_strided((rows, cols), (cols, 1), dtype)


def new3(n: int, rows: int, cols: int, dtype) -> torch.Tensor:
    return empty_strided((n, rows, cols), (rows * cols, cols, 1), dtype)


def elsewhere(f, device: int, *args):
    """f(*args) with GPU `device` current (every call here starts by asking for that); raises if there is none."""
    if device < 0:
        raise ValueError("tensors must be on a GPU")
    with torch.cuda.device(device):
        return f(*args)


MOST = (1 << 31) - 1   # what the library takes as a 32-bit number; beyond that ctypes would pass the low bits


def narrow(n: int, name: str) -> None:
    if n > MOST:
        raise ValueError(f"{name} has a dimension of 2^31 or more")


def sizes(t: torch.Tensor, name: str, dims: int) -> torch.Size:
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {len(shape)}")
    if t.numel() > MOST:
        narrow(max(shape[1:] or shape), name)   # rows are taken as 64-bit numbers
    return shape


def router_fwd(logits: torch.Tensor, k: int, renormalize: bool = True, out=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(index int32 [T, k], weight f32 [T, k]): the k largest of logits [T, E] (f32 or bf16), ties to the
    lowest expert, and their softmax weights, over all experts or over the chosen ones, via bsr_router_fwd.
    Experts at -infinity are never chosen: index -1, weight 0."""
    d = logits.get_device()
    if d < 0 or d != current_device():
        return elsewhere(router_fwd, d, logits, k, renormalize, out)
    T, E = sizes(logits, "logits", 2)
    kind = _LOGITS.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    lp = pointer(logits, "logits", (T, E), logits.dtype, d)
    if out is None:
        index, weight = new2(T, k, _I32), new2(T, k, _F32)
        ip, wp = index.data_ptr(), weight.data_ptr()
    else:
        index, weight = out
        ip, wp = pointer(index, "index", (T, k), _I32, d), pointer(weight, "weight", (T, k), _F32, d)
    status = C.bsr_router_fwd(lp, kind, T, E, min(k, MOST), renormalize, ip, wp, raw_stream(d))
    if status:
        _lib.check(status, "bsr_router_fwd")
    return index, weight


def router_bwd(logits: torch.Tensor, index: torch.Tensor, weight: torch.Tensor, dweight: torch.Tensor,
               renormalize: bool = True, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dlogits [T, E] (the logits' type) of router_fwd's weights, via bsr_router_bwd."""
    d = logits.get_device()
    if d < 0 or d != current_device():
        return elsewhere(router_bwd, d, logits, index, weight, dweight, renormalize, out)
    T, E = sizes(logits, "logits", 2)
    k = sizes(index, "index", 2)[1]
    kind = _LOGITS.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    lp = pointer(logits, "logits", (T, E), logits.dtype, d)
    ip = pointer(index, "index", (T, k), _I32, d)
    wp = pointer(weight, "weight", (T, k), _F32, d)
    gp = pointer(dweight, "dweight", (T, k), _F32, d)
    if out is None:
        out = new2(T, E, logits.dtype)
        op = out.data_ptr()
    else:
        op = pointer(out, "out", (T, E), logits.dtype, d)
    status = C.bsr_router_bwd(lp, kind, T, E, k, renormalize, ip, wp, gp, op, raw_stream(d))
    if status:
        _lib.check(status, "bsr_router_bwd")
    return out


PLAN_SLOTS = 1024   # BSR_EXPERT_PLAN_SLOTS: up to here a plan needs no workspace


class ExpertPlan:
    """Which rows belong to which expert, on the device: offsets [E+1], row_token [T*k], slot_row [T, k] (int32).
    The plan keeps the three tensors and every call asks them for their addresses, so that a copy (copy, deepcopy, pickle)
    works on its own memory; copies are checked like plans from tensors."""

    __slots__ = ("_offsets", "_token", "_row", "T", "k", "E", "R", "device")
    offsets = property(lambda self: self._offsets)
    row_token = property(lambda self: self._token)
    slot_row = property(lambda self: self._row)

    def __init__(self, offsets: torch.Tensor, row_token: torch.Tensor, slot_row: torch.Tensor):
        d = offsets.get_device()
        if d < 0:
            raise ValueError(f"offsets must be on a GPU, got {offsets.device}")
        T, k = sizes(slot_row, "slot_row", 2)
        E = sizes(offsets, "offsets", 1)[0] - 1
        self.T, self.k, self.R, self.E, self.device = T, k, T * k, E, d
        pointer(offsets, "offsets", (E + 1,), _I32, d)
        pointer(row_token, "row_token", (T * k,), _I32, d)
        pointer(slot_row, "slot_row", (T, k), _I32, d)
        self._offsets, self._token, self._row = offsets, row_token, slot_row

    def __reduce__(self):
        return type(self), (self._offsets, self._token, self._row)

    @classmethod
    def from_index(cls, index: torch.Tensor, E: int) -> "ExpertPlan":
        """The plan of index [T, k] int32 (entries outside [0, E) are dropped), via bsr_expert_plan."""
        d = index.get_device()
        if d < 0 or d != current_device():
            return elsewhere(cls.from_index, d, index, E)
        T, k = sizes(index, "index", 2)
        R = T * k
        ip = pointer(index, "index", (T, k), _I32, d)
        self = cls.__new__(cls)
        self.T, self.k, self.R, self.E, self.device = T, k, R, E, d
        self._offsets = o = empty_strided((max(E, 0) + 1,), (1,), _I32)
        self._token = t = empty_strided((R,), (1,), _I32)
        self._row = s = new2(T, k, _I32)
        E, need, ws = max(min(E, MOST), -1), 0, None
        if R > PLAN_SLOTS:
            need = C.bsr_expert_plan_workspace(T, k, E)
            ws = empty_strided((need,), (1,), torch.uint8)
        status = C.bsr_expert_plan(ip, T, k, E, o.data_ptr(), t.data_ptr(), s.data_ptr(),
                                   None if ws is None else ws.data_ptr(), need, raw_stream(d))
        if status:
            _lib.check(status, "bsr_expert_plan")
        return self


def expert_fwd(plan: ExpertPlan, X: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None,
               gather: bool = True, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y [R, N] bf16: row r of expert e is x(r) . W[e]^T + bias[e]; W [E, N, K], bias [E, N] or None, via
    bsr_expert_fwd. gather: X is [T, K] by token; otherwise [R, K], sorted like Y."""
    T, R, E, d = plan.T, plan.R, plan.E, plan.device
    if d != current_device():
        return elsewhere(expert_fwd, d, plan, X, W, bias, gather, out)
    _, N, K = sizes(W, "W", 3)
    xp = pointer(X, "X", (T if gather else R, K), _BF16, d)
    wp = pointer(W, "W", (E, N, K), _BF16, d)
    bp = None if bias is None else pointer(bias, "bias", (E, N), _BF16, d)
    if out is None:
        out = new2(R, N, _BF16)
        op = out.data_ptr()
    else:
        op = pointer(out, "out", (R, N), _BF16, d)
    status = C.bsr_expert_fwd(xp, T, R, E, N, K, plan._offsets.data_ptr(), plan._token.data_ptr() if gather else None,
                              wp, bp, op, raw_stream(d))
    if status:
        _lib.check(status, "bsr_expert_fwd")
    return out


def expert_bwd_input(plan: ExpertPlan, dY: torch.Tensor, W: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dX [R, K] = dY . W[e] by rows sorted like dY [R, N], via bsr_expert_bwd_input. For a gathered X sum a
    token's rows: combine_fwd(plan, dX, None)."""
    R, E, d = plan.R, plan.E, plan.device
    if d != current_device():
        return elsewhere(expert_bwd_input, d, plan, dY, W, out)
    _, N, K = sizes(W, "W", 3)
    gp = pointer(dY, "dY", (R, N), _BF16, d)
    wp = pointer(W, "W", (E, N, K), _BF16, d)
    if out is None:
        out = new2(R, K, _BF16)
        op = out.data_ptr()
    else:
        op = pointer(out, "out", (R, K), _BF16, d)
    status = C.bsr_expert_bwd_input(gp, R, E, N, K, plan._offsets.data_ptr(), wp, op, raw_stream(d))
    if status:
        _lib.check(status, "bsr_expert_bwd_input")
    return out


def expert_bwd_weight(plan: ExpertPlan, dY: torch.Tensor, X: torch.Tensor, gather: bool = True, want_dbias: bool = False,
                      out: Optional[torch.Tensor] = None,
                      want_dW: bool = True) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(dW [E, N, K] or None, dbias [E, N] or None) via bsr_expert_bwd_weight; X and gather as for expert_fwd."""
    T, R, E, d = plan.T, plan.R, plan.E, plan.device
    if d != current_device():
        return elsewhere(expert_bwd_weight, d, plan, dY, X, gather, want_dbias, out, want_dW)
    N, K = sizes(dY, "dY", 2)[1], sizes(X, "X", 2)[1]
    gp = pointer(dY, "dY", (R, N), _BF16, d)
    xp = pointer(X, "X", (T if gather else R, K), _BF16, d)
    dW = op = None
    if want_dW:
        dW = new3(E, N, K, _BF16) if out is None else out
        op = pointer(dW, "out", (E, N, K), _BF16, d)
    elif out is not None or not want_dbias:
        raise ValueError("without dW there is no out, and dbias must be wanted")
    db = new2(E, N, _BF16) if want_dbias else None
    status = C.bsr_expert_bwd_weight(gp, xp, T, R, E, N, K, plan._offsets.data_ptr(), plan._token.data_ptr() if gather else None,
                                     op, db.data_ptr() if want_dbias else None, raw_stream(d))
    if status:
        _lib.check(status, "bsr_expert_bwd_weight")
    return dW, db


def combine_fwd(plan: ExpertPlan, Y: torch.Tensor, weight: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [T, N] = sum over a token's slots of weight [T, k] (f32; None: 1) times its rows of Y [R, N], via
    bsr_expert_combine_fwd."""
    T, k, d = plan.T, plan.k, plan.device
    if d != current_device():
        return elsewhere(combine_fwd, d, plan, Y, weight, out)
    N = sizes(Y, "Y", 2)[1]
    yp = pointer(Y, "Y", (plan.R, N), _BF16, d)
    wp = None if weight is None else pointer(weight, "weight", (T, k), _F32, d)
    if out is None:
        out = new2(T, N, _BF16)
        op = out.data_ptr()
    else:
        op = pointer(out, "out", (T, N), _BF16, d)
    status = C.bsr_expert_combine_fwd(yp, T, k, N, plan._row.data_ptr(), wp, op, raw_stream(d))
    if status:
        _lib.check(status, "bsr_expert_combine_fwd")
    return out


def combine_bwd(plan: ExpertPlan, dout: torch.Tensor, Y: torch.Tensor,
                weight: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dY [R, N] bf16, dweight [T, k] f32) of combine_fwd, via bsr_expert_combine_bwd."""
    T, k, R, d = plan.T, plan.k, plan.R, plan.device
    if d != current_device():
        return elsewhere(combine_bwd, d, plan, dout, Y, weight)
    N = sizes(Y, "Y", 2)[1]
    gp = pointer(dout, "dout", (T, N), _BF16, d)
    yp = pointer(Y, "Y", (R, N), _BF16, d)
    wp = None if weight is None else pointer(weight, "weight", (T, k), _F32, d)
    dY, dw = new2(R, N, _BF16), new2(T, k, _F32)
    status = C.bsr_expert_combine_bwd(gp, yp, T, k, plan.E, N, plan._offsets.data_ptr(), plan._row.data_ptr(), wp,
                                      dY.data_ptr(), dw.data_ptr(), raw_stream(d))
    if status:
        _lib.check(status, "bsr_expert_combine_bwd")
    return dY, dw
