"""Block-sparse linear layer on AMD MI355X (gfx950): BSR weights, bf16 MFMA kernels, C ABI.

Public names (loaded on first use, so that importing the package does not load the HIP
library):
  Pattern, linear_fwd, linear_bwd_input, linear_bwd_weight   -- sparse_gemm_amd.binding
  BlockSparseLinear, bsr_linear                              -- sparse_gemm_amd.linear
  ExpertPlan, router_fwd, router_bwd, expert_fwd, expert_bwd_input, expert_bwd_weight,
  combine_fwd, combine_bwd                                   -- sparse_gemm_amd.experts
  Mx4                                                        -- sparse_gemm_amd.mx4 (quantize, dequantize, expert_fwd)
  Fp8Rows, Fp8Blocks                                         -- sparse_gemm_amd.fp8 (quantize_rows, quantize_blocks, dequantize,
                                                                expert_fwd)
  ExpertFFN, route, expert_linear, expert_linear_fp8, expert_ffn, combine
                                                             -- sparse_gemm_amd.expert_layer
Build the library with `python -m sparse_gemm_amd.build`.
"""
__all__ = ["Pattern", "linear_fwd", "linear_bwd_input", "linear_bwd_weight", "BlockSparseLinear", "bsr_linear",
           "ExpertPlan", "router_fwd", "router_bwd", "expert_fwd", "expert_bwd_input", "expert_bwd_weight",
           "combine_fwd", "combine_bwd", "Mx4", "Fp8Rows", "Fp8Blocks", "ExpertFFN", "route", "expert_linear", "expert_linear_fp8",
           "expert_ffn", "combine"]

_BINDING = {"Pattern", "linear_fwd", "linear_bwd_input", "linear_bwd_weight"}
_LINEAR = {"BlockSparseLinear", "bsr_linear"}
_EXPERTS = {"ExpertPlan", "router_fwd", "router_bwd", "expert_fwd", "expert_bwd_input", "expert_bwd_weight",
            "combine_fwd", "combine_bwd"}
_EXPERT_LAYER = {"ExpertFFN", "route", "expert_linear", "expert_linear_fp8", "expert_ffn", "combine"}


def __getattr__(name):
    if name in _BINDING:
        from . import binding
        return getattr(binding, name)
    if name in _LINEAR:
        from . import linear
        return getattr(linear, name)
    if name in _EXPERTS:
        from . import experts
        return getattr(experts, name)
    if name == "Mx4":
        from .mx4 import Mx4
        return Mx4
    if name in ("Fp8Rows", "Fp8Blocks"):
        from . import fp8
        return getattr(fp8, name)
    if name in _EXPERT_LAYER:
        from . import expert_layer
        return getattr(expert_layer, name)
    raise AttributeError(name)
