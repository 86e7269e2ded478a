"""ExpertFFN: a feed-forward layer whose tokens each use k of E experts, with autograd over the library's
router, grouped products and sum. It can train with products in 8 bits, its experts can be held in 4 or 8 bits for serving, and a few
tokens can take the whole layer in one call. Gradients of the first order: a second derivative raises."""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch
from torch import nn
from torch.nn import functional as F

from . import experts, few_tokens, fp8, mx4
from .autograd import first_order, no_tangents
from .experts import ExpertPlan


def _whole(t: torch.Tensor) -> torch.Tensor:
    """t as the library takes it: contiguous and 16-byte aligned. A slice of odd sizes (of [T, k], of logits with an odd E, or the
    gradient of a concatenation's part) is contiguous without being aligned."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


class _RouteFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, renormalize):
        index, weight = experts.router_fwd(logits, k, renormalize)
        ctx.renormalize = renormalize
        ctx.save_for_backward(logits, index, weight)
        ctx.mark_non_differentiable(index)
        return index, weight

    @staticmethod
    @first_order
    def backward(ctx, _, dweight):
        logits, index, weight = ctx.saved_tensors
        return experts.router_bwd(logits, index, weight, _whole(dweight.float()), ctx.renormalize), None, None


def route(logits: torch.Tensor, k: int, renormalize: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
    """(index [T, k], weight [T, k]) of logits [T, E]; weight carries the gradient."""
    return _RouteFn.apply(_whole(logits), k, renormalize)


class _ExpertLinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, bias, plan, gather):
        ctx.plan, ctx.gather, ctx.has_bias = plan, gather, bias is not None
        ctx.save_for_backward(x, W)
        return experts.expert_fwd(plan, x, W, bias, gather)

    @staticmethod
    @first_order
    def backward(ctx, dY):
        x, W = ctx.saved_tensors
        plan = ctx.plan
        dY = _whole(dY.to(torch.bfloat16))
        dX = dW = db = None
        if ctx.needs_input_grad[0]:
            dX = experts.expert_bwd_input(plan, dY, W)
            if ctx.gather:
                dX = experts.combine_fwd(plan, dX)
        if ctx.needs_input_grad[1] or (ctx.has_bias and ctx.needs_input_grad[2]):
            dW, db = experts.expert_bwd_weight(plan, dY, x, ctx.gather, ctx.has_bias and ctx.needs_input_grad[2],
                                               want_dW=ctx.needs_input_grad[1])
        return dX, dW, db, None, None


def expert_linear(plan: ExpertPlan, x: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None,
                  gather: bool = True) -> torch.Tensor:
    """Rows [R, N] of x [T, K] (gather) or [R, K] times each expert's W [E, N, K], with gradients."""
    return _ExpertLinearFn.apply(_whole(x), W, bias, plan, gather)


class _ExpertLinearFp8Fn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, bias, plan, gather, want_dx):
        ctx.plan, ctx.gather, ctx.has_bias = plan, gather, bias is not None
        # backward takes W's codes, W itself is only what they came from: a parameter is not saved, so that it may change in place; a
        # weight computed for this call is, so that it is released with the rest
        ctx.sources = (W,) if W.requires_grad and W.is_leaf else ()
        saved = [x, W] if W.requires_grad and not W.is_leaf else [x]
        if want_dx:
            Wq, Wt = fp8.quantize_blocks(W, transposed=True)
            saved += [Wt.codes, Wt.scales]
        else:
            Wq = fp8.quantize_blocks(W)
        ctx.save_for_backward(*saved)
        return fp8.expert_fwd(plan, fp8.quantize_rows(x), Wq, bias, gather)

    @staticmethod
    @first_order
    def backward(ctx, dY):
        x, *rest = ctx.saved_tensors
        plan = ctx.plan
        dY = _whole(dY.to(torch.bfloat16))
        dX = dW = db = None
        if ctx.needs_input_grad[0]:
            dX = fp8.expert_fwd(plan, fp8.quantize_rows(dY), fp8.Fp8Blocks(*rest[-2:]), gather=False)
            if ctx.gather:
                dX = experts.combine_fwd(plan, dX)
        if ctx.needs_input_grad[1] or (ctx.has_bias and ctx.needs_input_grad[2]):
            dW, db = experts.expert_bwd_weight(plan, dY, x, ctx.gather, ctx.has_bias and ctx.needs_input_grad[2],
                                               want_dW=ctx.needs_input_grad[1])
        return dX, dW, db, None, None, None


def expert_linear_fp8(plan: ExpertPlan, x: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None,
                      gather: bool = True) -> torch.Tensor:
    """expert_linear with its products in 8 bits, for training on bf16 weights: x is quantised by row and W by block (fp8.quantize_rows,
    fp8.quantize_blocks; N and K multiples of 16) in every call, and so is the incoming gradient for the input gradient
    q(dY) . q(W). The weight and bias gradients are expert_linear's, on x and dY in bf16: they contract over the rows, along which
    neither has scales. The rounding to codes counts as the identity in the gradients. A gathered x's gradient is rounded to bf16 for
    each of a token's k rows before they are added, as expert_linear's is. The matrix cores drop what lies below 2^-13 of the largest of
    eight neighbouring products (include/bsr_fp8_blocks.h)."""
    x = _whole(x)
    return _ExpertLinearFp8Fn.apply(x, W, bias, plan, gather, torch.is_grad_enabled() and x.requires_grad)


def expert_ffn(x: torch.Tensor, router: torch.Tensor, up, down, k: int, renormalize: bool = True,
               up_bias: Optional[torch.Tensor] = None, down_bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A whole layer of experts for up to 16 tokens x [T, dim] in one call, few_tokens.expert_ffn: weights in bf16, Mx4 or
    Fp8Blocks, forward only (raises where a gradient is wanted, in reverse or forward mode). Against the single calls it keeps the
    router's logits and each expert's result in 32 bits, and rounds silu(gate) * up to bf16 once."""
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in (x, router, up, down, up_bias, down_bias)):
        raise RuntimeError("expert_ffn has no backward pass")
    no_tangents("expert_ffn", x, router, up, down, up_bias, down_bias)
    return few_tokens.expert_ffn(_whole(x), router, up, down, k, renormalize, up_bias, down_bias)


class _CombineFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Y, weight, plan):
        ctx.plan = plan
        ctx.save_for_backward(Y, weight)
        return experts.combine_fwd(plan, Y, weight)

    @staticmethod
    @first_order
    def backward(ctx, dout):
        Y, weight = ctx.saved_tensors
        dY, dw = experts.combine_bwd(ctx.plan, _whole(dout.to(torch.bfloat16)), Y, weight)
        return dY, dw, None


def combine(plan: ExpertPlan, Y: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
    """out [T, N]: a token's rows of Y [R, N], weighted and summed, with gradients."""
    return _CombineFn.apply(_whole(Y), _whole(weight), plan)


class ExpertFFN(nn.Module):
    """y = sum over a token's k experts of weight * down_e(silu(gate_e x) * up_e x).

    The router's logits are x . router^T, a library product rounded to bf16 like the layer's other results (the router itself
    takes f32 logits too); silu(gate), its product with up and each product of the experts are rounded to bf16 once. up holds gate and up weights one after the other ([E, 2 * hidden, dim]).
    quantize_() replaces the expert weights by their 4-bit form for serving: batches of up to `prompt_tokens` tokens
    then keep their activations in bf16, larger ones quantise them too: faster, and less exact by the activations'
    own rounding to 4 bits (up layer 4096 -> 14336 of 8 experts, k = 2: 16 tokens 44 against 46 us, 64 tokens 53 against
    46, 256 tokens 114 against 50). quantize_("fp8") does the same in 8 bits (there 16 tokens 90 against 110 us, 64 tokens 124
    against 110, 256 tokens 135 against 116).
    fp8: the products of the experts in 8 bits while the layer trains on its bf16 weights (expert_linear_fp8; dim and hidden
    multiples of 16). Every call quantises the weights of all experts, also one without gradients and of one token (100 us for 8 x 4096
    x 4096); between training steps few tokens can take decode_tokens instead, and longer evaluations a copy under quantize_("fp8").
    decode_tokens: batches of up to so many tokens (16 at most) whose gradient nobody wants take expert_ffn, in any form of the weights.
    A reentrant checkpoint hides in its first pass that it wants one: such a batch then takes expert_ffn there and the single calls
    when it is recomputed, whose roundings differ."""

    fp8, decode_tokens = False, 0   # of layers stored before these existed

    def __init__(self, dim: int, hidden: int, num_experts: int, k: int, renormalize: bool = True, bias: bool = False,
                 prompt_tokens: int = 64, device=None, fp8: bool = False, decode_tokens: int = 0):
        super().__init__()
        if fp8 and (dim % 16 or hidden % 16):
            raise ValueError("products in 8 bits need dim and hidden to be multiples of 16")
        if not 0 <= decode_tokens <= few_tokens.TOKENS:
            raise ValueError(f"decode_tokens must lie in [0, {few_tokens.TOKENS}]")
        self.dim, self.hidden, self.num_experts, self.k, self.renormalize = dim, hidden, num_experts, k, renormalize
        self.prompt_tokens, self.fp8, self.decode_tokens = prompt_tokens, fp8, decode_tokens
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        mk = lambda *s: nn.Parameter(torch.empty(s, dtype=torch.bfloat16, device=device))  # noqa: E731
        self.router = mk(num_experts, dim)
        self.up, self.down = mk(num_experts, 2 * hidden, dim), mk(num_experts, dim, hidden)
        self.up_bias = mk(num_experts, 2 * hidden) if bias else None
        self.down_bias = mk(num_experts, dim) if bias else None
        for name in ("up_codes", "up_scales", "down_codes", "down_scales"):
            self.register_buffer(name, None)
        self.reset_parameters()

    def reset_parameters(self) -> None:
        with torch.no_grad():
            for p, fan in ((self.router, self.dim), (self.up, self.dim), (self.down, self.hidden),
                           (self.up_bias, self.dim), (self.down_bias, self.hidden)):
                if p is not None:
                    p.uniform_(-1.0 / math.sqrt(fan), 1.0 / math.sqrt(fan))

    @property
    def quantized(self) -> bool:
        return self.up_codes is not None

    @property
    def form(self) -> str:
        """How the expert weights are held: "bf16", "mx4" or "fp8"."""
        return "bf16" if not self.quantized else "mx4" if self.up_scales.dim() == 4 else "fp8"

    @torch.no_grad()
    def quantize_(self, form: str = "mx4") -> "ExpertFFN":
        """Hold the expert weights in 4 bits ("mx4": bsr_mx4_quantize) or 8 ("fp8": bsr_fp8_quantize_blocks) and drop the bf16
        ones; forward only from then on, with the router and the biases frozen."""
        if form not in ("mx4", "fp8"):
            raise ValueError(f"form must be 'mx4' or 'fp8', got {form!r}")
        if self.quantized and form != self.form:
            raise RuntimeError(f"the weights are held as {self.form} already")
        if not self.quantized:
            quantize = mx4.quantize if form == "mx4" else fp8.quantize_blocks
            up, down = quantize(self.up.data), quantize(self.down.data)
            self.up_codes, self.up_scales, self.down_codes, self.down_scales = up.codes, up.scales, down.codes, down.scales
            self.up = self.down = None
            self.requires_grad_(False)
        return self

    def _held(self):
        """The compact up and down weights."""
        make = mx4.Mx4 if self.form == "mx4" else fp8.Fp8Blocks
        return make(self.up_codes, self.up_scales), make(self.down_codes, self.down_scales)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if self.quantized and torch.is_grad_enabled() and (x.requires_grad or any(
                p is not None and p.requires_grad for p in (self.router, self.up_bias, self.down_bias))):
            raise RuntimeError("a quantised ExpertFFN has no backward pass")
        lead = x.shape[:-1]
        x = _whole(x.reshape(-1, self.dim).to(torch.bfloat16))
        if 0 < x.shape[0] <= self.decode_tokens and not (torch.is_grad_enabled() and any(   # (the tensors in use, parameters or not)
                t is not None and t.requires_grad for t in (x, self.router, self.up, self.down, self.up_bias, self.down_bias))):
            held = (self.up, self.down) if not self.quantized else self._held()
            return expert_ffn(x, self.router, *held, self.k, self.renormalize, self.up_bias, self.down_bias).reshape(*lead, self.dim)
        index, weight = route(F.linear(x, self.router), self.k, self.renormalize)
        plan = ExpertPlan.from_index(index, self.num_experts)
        if not self.quantized:
            linear = expert_linear_fp8 if self.fp8 else expert_linear
            gate, up = linear(plan, x, self.up, self.up_bias).chunk(2, dim=1)
            y = linear(plan, F.silu(gate) * up, self.down, self.down_bias, gather=False)
            return combine(plan, y, weight).reshape(*lead, self.dim)
        no_tangents("a quantised ExpertFFN", self.up_bias, self.down_bias)   # (those of x and the router are refused by route)
        held, (quantize, expert_fwd) = self._held(), {"mx4": (mx4.quantize, mx4.expert_fwd),
                                                      "fp8": (fp8.quantize_rows, fp8.expert_fwd)}[self.form]
        form = quantize if x.shape[0] > self.prompt_tokens else (lambda t: t)
        h = expert_fwd(plan, form(x), held[0], self.up_bias)
        gate, up = h.chunk(2, dim=1)
        h = form((F.silu(gate) * up).contiguous())
        y = expert_fwd(plan, h, held[1], self.down_bias, gather=False)
        return experts.combine_fwd(plan, y, weight.detach()).reshape(*lead, self.dim)

    def extra_repr(self) -> str:
        return (f"dim={self.dim}, hidden={self.hidden}, num_experts={self.num_experts}, k={self.k}, "
                f"bias={self.up_bias is not None}, quantized={self.quantized}")
