"""Routed weight-only-quantized (WNA16) MoE layer for AMD Instinct MI355X.

The layer runs in hand-written gfx950 HIP kernels behind the C ABI of
include/moe_wna16.h (libmoe_wna16.so, built in-tree by
`python -m weight_only_bit_moe_amd.build`).  This package binds that ABI;
`inputs` draws seeded synthetic layers; `block_ops` holds the operators around
the layer (residual norm, expert routing, the shared expert's 8-bit products), `expert_ops` those
for experts in 8-bit floating point.
"""
from .binding import (EXPORTED, LIB_PATH, SYNC_BYTES, MoeWna16Error, align, forward, load_library,
                      moe_wna16_align, moe_wna16_forward, moe_wna16_forward_profiled,
                      moe_wna16_plan, moe_wna16_quantize, quantize, moe_wna16_prepare,
                      moe_wna16_forward_prepared, moe_wna16_forward_noalloc, prepare,
                      moe_wna16_status_string, moe_wna16_workspace_f32_offset,
                      moe_wna16_workspace_layout, moe_wna16_workspace_size, workspace_f32_sum,
                      workspace_for, workspace_meta, workspace_sort)

#: operators around the layer, imported on first use (block_ops imports torch at module level), so not
#: in __all__: importing all of that needs neither torch nor the compiled module
_BLOCK_OPS = ("add_rmsnorm", "route_topk", "gemm_w8a8", "gemm_w8a8_workspace_for", "swiglu_quant",
              "moe_wna16_add_rmsnorm", "moe_wna16_route_topk", "moe_wna16_gemm_w8a8",
              "moe_wna16_gemm_w8a8_workspace_size", "moe_wna16_swiglu_quant")
#: operators for experts in 8-bit floating point, imported in the same way
_EXPERT_OPS = ("quant_fp8", "swiglu_quant_fp8", "gemm_fp8", "gemm_fp8_workspace_for", "gemm_fp8_grouped",
               "sort_tokens", "combine_tokens", "forward_fp8", "moe_wna16_quant_fp8",
               "moe_wna16_swiglu_quant_fp8", "moe_wna16_gemm_fp8_workspace_size", "moe_wna16_gemm_fp8",
               "moe_wna16_gemm_fp8_grouped", "moe_wna16_sort_tokens_workspace_size",
               "moe_wna16_sort_tokens", "moe_wna16_combine_tokens", "moe_wna16_combine_tokens_grad")


def __getattr__(name):
    if name in _BLOCK_OPS:
        from . import block_ops
        for n in _BLOCK_OPS:
            globals()[n] = getattr(block_ops, n)
        return globals()[name]
    if name in _EXPERT_OPS:
        from . import expert_ops
        for n in _EXPERT_OPS:
            globals()[n] = getattr(expert_ops, n)
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def __dir__():
    return sorted({*globals(), *_BLOCK_OPS, *_EXPERT_OPS})


__all__ = ["EXPORTED", "LIB_PATH", "SYNC_BYTES", "MoeWna16Error", "align", "forward", "load_library",
           "moe_wna16_align", "moe_wna16_forward", "moe_wna16_forward_profiled", "moe_wna16_plan", "moe_wna16_quantize", "quantize",
           "moe_wna16_prepare", "moe_wna16_forward_prepared", "moe_wna16_forward_noalloc", "prepare",
           "moe_wna16_status_string",
           "moe_wna16_workspace_f32_offset", "moe_wna16_workspace_layout",
           "moe_wna16_workspace_size", "workspace_f32_sum", "workspace_for", "workspace_meta",
           "workspace_sort"]
