"""ExpertFFN: a feed-forward layer whose tokens each use k of E experts, with autograd over the library's
router, grouped products and sum; its experts can be held in 4 bits for serving. Gradients of the first order: a second
derivative raises."""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch
from torch import nn
from torch.nn import functional as F

from . import experts, mx4
from .autograd import first_order
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
    46, 256 tokens 114 against 50)."""

    def __init__(self, dim: int, hidden: int, num_experts: int, k: int, renormalize: bool = True, bias: bool = False,
                 prompt_tokens: int = 64, device=None):
        super().__init__()
        self.dim, self.hidden, self.num_experts, self.k, self.renormalize = dim, hidden, num_experts, k, renormalize
        self.prompt_tokens = prompt_tokens
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

    @torch.no_grad()
    def quantize_(self) -> "ExpertFFN":
        """Hold the expert weights in 4 bits (bsr_mx4_quantize) and drop the bf16 ones; forward only from then on, with the
        router and the biases frozen."""
        if not self.quantized:
            up, down = mx4.quantize(self.up.data), mx4.quantize(self.down.data)
            self.up_codes, self.up_scales, self.down_codes, self.down_scales = up.codes, up.scales, down.codes, down.scales
            self.up = self.down = None
            self.requires_grad_(False)
        return self

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if self.quantized and torch.is_grad_enabled() and (x.requires_grad or any(
                p is not None and p.requires_grad for p in (self.router, self.up_bias, self.down_bias))):
            raise RuntimeError("a quantised ExpertFFN has no backward pass")
        lead = x.shape[:-1]
        x = _whole(x.reshape(-1, self.dim).to(torch.bfloat16))
        index, weight = route(F.linear(x, self.router), self.k, self.renormalize)
        plan = ExpertPlan.from_index(index, self.num_experts)
        if not self.quantized:
            gate, up = expert_linear(plan, x, self.up, self.up_bias).chunk(2, dim=1)
            y = expert_linear(plan, F.silu(gate) * up, self.down, self.down_bias, gather=False)
            return combine(plan, y, weight).reshape(*lead, self.dim)
        form = mx4.quantize if x.shape[0] > self.prompt_tokens else (lambda t: t)
        h = mx4.expert_fwd(plan, form(x), mx4.Mx4(self.up_codes, self.up_scales), self.up_bias)
        gate, up = h.chunk(2, dim=1)
        h = form((F.silu(gate) * up).contiguous())
        y = mx4.expert_fwd(plan, h, mx4.Mx4(self.down_codes, self.down_scales), self.down_bias, gather=False)
        return experts.combine_fwd(plan, y, weight.detach()).reshape(*lead, self.dim)

    def extra_repr(self) -> str:
        return (f"dim={self.dim}, hidden={self.hidden}, num_experts={self.num_experts}, k={self.k}, "
                f"bias={self.up_bias is not None}, quantized={self.quantized}")
