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
# compiled graphs use, where this torch has it.
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
try:
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    _empty_strided_cuda = None


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


def device_of(t: torch.Tensor, name: str) -> int:
    """Index of the GPU that t is on; raises if it is on none."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    return t.get_device()


def output(out: Optional[torch.Tensor], name: str, shape, dtype, device: int) -> torch.Tensor:
    """`out`, checked, or a new tensor of that shape (1 to 4 dimensions) and type."""
    if out is not None:
        pointer(out, name, shape, dtype, device)
        return out
    if _empty_strided_cuda is None or device != _current_device():
        return torch.empty(shape, dtype=dtype, device=f"cuda:{device}")
    strides = (1,)
    for n in shape[:0:-1]:
        strides = (n * strides[0], *strides)
    return _empty_strided_cuda(shape, strides, dtype)


def call(f, what: str, device: int, *args) -> None:
    """f(*args, current stream of GPU `device`), with that device current; raises BsrError on a status."""
    if device == _current_device():
        status = f(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            status = f(*args, _raw_stream(device))
    if status:
        _lib.check(status, what)


def _sizes(t: torch.Tensor, name: str, dims: int) -> torch.Size:
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {len(shape)}")
    return shape


def router_fwd(logits: torch.Tensor, k: int, renormalize: bool = True, out=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(index int32 [T, k], weight f32 [T, k]): the k largest of logits [T, E] (f32 or bf16), ties to the
    lowest expert, and their softmax weights, over all experts or over the chosen ones, via bsr_router_fwd.
    Experts at -infinity are never chosen: index -1, weight 0."""
    T, E = _sizes(logits, "logits", 2)
    kind = _LOGITS.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    d = device_of(logits, "logits")
    lp = pointer(logits, "logits", (T, E), logits.dtype, d)
    index, weight = out if out else (None, None)
    index = output(index, "index", (T, k), _I32, d)
    weight = output(weight, "weight", (T, k), _F32, d)
    call(C.bsr_router_fwd, "bsr_router_fwd", d, lp, kind, T, E, k, int(renormalize), index.data_ptr(), weight.data_ptr())
    return index, weight


def router_bwd(logits: torch.Tensor, index: torch.Tensor, weight: torch.Tensor, dweight: torch.Tensor,
               renormalize: bool = True, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dlogits [T, E] (the logits' type) of router_fwd's weights, via bsr_router_bwd."""
    T, E = _sizes(logits, "logits", 2)
    k = _sizes(index, "index", 2)[1]
    kind = _LOGITS.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    d = device_of(logits, "logits")
    lp = pointer(logits, "logits", (T, E), logits.dtype, d)
    ip = pointer(index, "index", (T, k), _I32, d)
    wp = pointer(weight, "weight", (T, k), _F32, d)
    gp = pointer(dweight, "dweight", (T, k), _F32, d)
    out = output(out, "out", (T, E), logits.dtype, d)
    call(C.bsr_router_bwd, "bsr_router_bwd", d, lp, kind, T, E, k, int(renormalize), ip, wp, gp, out.data_ptr())
    return out


class ExpertPlan:
    """Which rows belong to which expert, on the device: offsets [E+1], row_token [T*k], slot_row [T, k] (int32).
    The three tensors are not to be replaced or moved afterwards (their addresses are kept)."""

    __slots__ = ("offsets", "row_token", "slot_row", "T", "k", "E", "R", "device", "_offsets", "_token", "_row")

    def __init__(self, offsets: torch.Tensor, row_token: torch.Tensor, slot_row: torch.Tensor):
        T, k = _sizes(slot_row, "slot_row", 2)
        E = _sizes(offsets, "offsets", 1)[0] - 1
        d = device_of(offsets, "offsets")
        self.T, self.k, self.R, self.E, self.device = T, k, T * k, E, d
        self._offsets = pointer(offsets, "offsets", (E + 1,), _I32, d)
        self._token = pointer(row_token, "row_token", (T * k,), _I32, d)
        self._row = pointer(slot_row, "slot_row", (T, k), _I32, d)
        self.offsets, self.row_token, self.slot_row = offsets, row_token, slot_row

    @classmethod
    def from_index(cls, index: torch.Tensor, E: int) -> "ExpertPlan":
        """The plan of index [T, k] int32 (entries outside [0, E) are dropped), via bsr_expert_plan."""
        T, k = _sizes(index, "index", 2)
        d = device_of(index, "index")
        ip = pointer(index, "index", (T, k), _I32, d)
        self = cls.__new__(cls)
        self.T, self.k, self.R, self.E, self.device = T, k, T * k, E, d
        self.offsets = output(None, "offsets", (max(E, 0) + 1,), _I32, d)
        self.row_token = output(None, "row_token", (T * k,), _I32, d)
        self.slot_row = output(None, "slot_row", (T, k), _I32, d)
        self._offsets, self._token, self._row = self.offsets.data_ptr(), self.row_token.data_ptr(), self.slot_row.data_ptr()
        need = C.bsr_expert_plan_workspace(T, k, E)
        ws = output(None, "workspace", (need,), torch.uint8, d) if need else None
        call(C.bsr_expert_plan, "bsr_expert_plan", d, ip, T, k, E, self._offsets, self._token, self._row,
             ws.data_ptr() if need else None, need)
        return self


def expert_fwd(plan: ExpertPlan, X: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None,
               gather: bool = True, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y [R, N] bf16: row r of expert e is x(r) . W[e]^T + bias[e]; W [E, N, K], bias [E, N] or None, via
    bsr_expert_fwd. gather: X is [T, K] by token; otherwise [R, K], sorted like Y."""
    _, N, K = _sizes(W, "W", 3)
    T, R, E, d = plan.T, plan.R, plan.E, plan.device
    xp = pointer(X, "X", (T if gather else R, K), _BF16, d)
    wp = pointer(W, "W", (E, N, K), _BF16, d)
    bp = None if bias is None else pointer(bias, "bias", (E, N), _BF16, d)
    out = output(out, "out", (R, N), _BF16, d)
    call(C.bsr_expert_fwd, "bsr_expert_fwd", d, xp, T, R, E, N, K, plan._offsets, plan._token if gather else None, wp, bp,
         out.data_ptr())
    return out


def expert_bwd_input(plan: ExpertPlan, dY: torch.Tensor, W: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dX [R, K] = dY . W[e] by rows sorted like dY [R, N], via bsr_expert_bwd_input. For a gathered X sum a
    token's rows: combine_fwd(plan, dX, None)."""
    _, N, K = _sizes(W, "W", 3)
    R, E, d = plan.R, plan.E, plan.device
    gp = pointer(dY, "dY", (R, N), _BF16, d)
    wp = pointer(W, "W", (E, N, K), _BF16, d)
    out = output(out, "out", (R, K), _BF16, d)
    call(C.bsr_expert_bwd_input, "bsr_expert_bwd_input", d, gp, R, E, N, K, plan._offsets, wp, out.data_ptr())
    return out


def expert_bwd_weight(plan: ExpertPlan, dY: torch.Tensor, X: torch.Tensor, gather: bool = True, want_dbias: bool = False,
                      out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(dW [E, N, K], dbias [E, N] or None) via bsr_expert_bwd_weight; X and gather as for expert_fwd."""
    N, K = _sizes(dY, "dY", 2)[1], _sizes(X, "X", 2)[1]
    T, R, E, d = plan.T, plan.R, plan.E, plan.device
    gp = pointer(dY, "dY", (R, N), _BF16, d)
    xp = pointer(X, "X", (T if gather else R, K), _BF16, d)
    dW = output(out, "out", (E, N, K), _BF16, d)
    db = output(None, "dbias", (E, N), _BF16, d) if want_dbias else None
    call(C.bsr_expert_bwd_weight, "bsr_expert_bwd_weight", d, gp, xp, T, R, E, N, K, plan._offsets,
         plan._token if gather else None, dW.data_ptr(), db.data_ptr() if want_dbias else None)
    return dW, db


def combine_fwd(plan: ExpertPlan, Y: torch.Tensor, weight: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [T, N] = sum over a token's slots of weight [T, k] (f32; None: 1) times its rows of Y [R, N], via
    bsr_expert_combine_fwd."""
    N = _sizes(Y, "Y", 2)[1]
    T, k, d = plan.T, plan.k, plan.device
    yp = pointer(Y, "Y", (plan.R, N), _BF16, d)
    wp = None if weight is None else pointer(weight, "weight", (T, k), _F32, d)
    out = output(out, "out", (T, N), _BF16, d)
    call(C.bsr_expert_combine_fwd, "bsr_expert_combine_fwd", d, yp, T, k, N, plan._row, wp, out.data_ptr())
    return out


def combine_bwd(plan: ExpertPlan, dout: torch.Tensor, Y: torch.Tensor,
                weight: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dY [R, N] bf16, dweight [T, k] f32) of combine_fwd, via bsr_expert_combine_bwd."""
    N = _sizes(Y, "Y", 2)[1]
    T, k, R, d = plan.T, plan.k, plan.R, plan.device
    gp = pointer(dout, "dout", (T, N), _BF16, d)
    yp = pointer(Y, "Y", (R, N), _BF16, d)
    wp = None if weight is None else pointer(weight, "weight", (T, k), _F32, d)
    dY = output(None, "dY", (R, N), _BF16, d)
    dw = output(None, "dweight", (T, k), _F32, d)
    call(C.bsr_expert_combine_bwd, "bsr_expert_combine_bwd", d, gp, yp, T, k, plan.E, N, plan._offsets, plan._row, wp,
         dY.data_ptr(), dw.data_ptr())
    return dY, dw
