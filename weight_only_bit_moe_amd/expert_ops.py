"""Operators for experts in 8-bit floating point (include/moe_wna16.h), on torch tensors.

    quant_fp8          rows in e4m3 with a power-of-two scale for each 128 elements
    swiglu_quant_fp8   the same of their SwiGLU
    gemm_fp8           product of such rows with a weight that has a scale for each 128 x 128 block
    gemm_fp8_grouped   the same for rows sorted by expert, each expert with a weight of its own
    sort_tokens        tokens' rows in the order of their experts, with its gradient
    combine_tokens     experts' rows back to their tokens, weighted and added up, with its gradient
    forward_fp8        the routed layer on such experts, from all of them

Each runs in the library's gfx950 kernels on the current stream; argument checks,
allocation and the library call are in the compiled module _block_ops, as for the
operators around the layer.  The raw entry points take integer device addresses.

sort_tokens and combine_tokens give gradients to x, y, the weights and the addend where they
require one (a gradient's own graph is refused, and so is a forward-mode tangent of theirs); the
others take tensors as values.  A step captured into a graph has its forward and its backward in the
one capture, and no eager graph of the same leaves may be alive then: torch ends the process over the
stream it was made on.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .binding import OK, MoeWna16Error, load_library
from .block_ops import _block_ops


def moe_wna16_quant_fp8(x, T, K, x_stride, dtype, q_out, q_stride, scale_out, s_stride, stream) -> int:
    """Raw entry point on integer device addresses; returns the status."""
    return load_library().moe_wna16_quant_fp8(x, T, K, x_stride, dtype, q_out, q_stride, scale_out,
                                              s_stride, stream)


def moe_wna16_swiglu_quant_fp8(gu, T, I, gu_stride, dtype, alpha, beta, clamp, q_out, q_stride,
                               scale_out, s_stride, stream) -> int:
    """Raw entry point on integer device addresses; returns the status."""
    return load_library().moe_wna16_swiglu_quant_fp8(gu, T, I, gu_stride, dtype, alpha, beta, clamp,
                                                     q_out, q_stride, scale_out, s_stride, stream)


def moe_wna16_gemm_fp8_workspace_size(T: int, N: int, K: int) -> int:
    n = ctypes.c_size_t(0)
    st = load_library().moe_wna16_gemm_fp8_workspace_size(T, N, K, ctypes.byref(n))
    if st != OK:
        raise MoeWna16Error(st, "moe_wna16_gemm_fp8_workspace_size")
    return n.value


def moe_wna16_gemm_fp8(a, a_scale, w, w_scale, addend, T, N, K, lda, lda_s, ldw, ldw_s, ld_add, ldo,
                       out_dtype, out, workspace, workspace_bytes, stream) -> int:
    """Raw entry point on integer device addresses; returns the status."""
    return load_library().moe_wna16_gemm_fp8(a, a_scale, w, w_scale, addend, T, N, K, lda, lda_s, ldw,
                                             ldw_s, ld_add, ldo, out_dtype, out, workspace,
                                             workspace_bytes, stream)


def moe_wna16_gemm_fp8_grouped(a, a_scale, w, w_scale, offsets, rows, E, a_rows, R, N, K, lda, lda_s,
                               ldw, ldw_s, w_expert, ws_expert, ldo, out_dtype, out, stream) -> int:
    """Raw entry point on integer device addresses; returns the status."""
    return load_library().moe_wna16_gemm_fp8_grouped(a, a_scale, w, w_scale, offsets, rows, E, a_rows,
                                                     R, N, K, lda, lda_s, ldw, ldw_s, w_expert,
                                                     ws_expert, ldo, out_dtype, out, stream)


def moe_wna16_sort_tokens_workspace_size(T: int, topk: int, E: int) -> int:
    n = ctypes.c_size_t(0)
    st = load_library().moe_wna16_sort_tokens_workspace_size(T, topk, E, ctypes.byref(n))
    if st != OK:
        raise MoeWna16Error(st, "moe_wna16_sort_tokens_workspace_size")
    return n.value


def moe_wna16_sort_tokens(ids, T, topk, E, x, H, x_stride, dtype, tokens_out, slots_out, offsets_out,
                          xs_out, xs_stride, workspace, workspace_bytes, stream) -> int:
    """Raw entry point on integer device addresses; returns the status."""
    return load_library().moe_wna16_sort_tokens(ids, T, topk, E, x, H, x_stride, dtype, tokens_out,
                                                slots_out, offsets_out, xs_out, xs_stride, workspace,
                                                workspace_bytes, stream)


def moe_wna16_combine_tokens(y, slots, weights, addend, T, topk, H, R, y_stride, add_stride,
                             out_stride, dtype, out, stream) -> int:
    """Raw entry point on integer device addresses; returns the status."""
    return load_library().moe_wna16_combine_tokens(y, slots, weights, addend, T, topk, H, R, y_stride,
                                                   add_stride, out_stride, dtype, out, stream)


def moe_wna16_combine_tokens_grad(dout, y, slots, weights, used, T, topk, H, R, d_stride, y_stride,
                                  dy_stride, dtype, dy, dw, stream) -> int:
    """Raw entry point on integer device addresses; returns the status."""
    return load_library().moe_wna16_combine_tokens_grad(dout, y, slots, weights, used, T, topk, H, R,
                                                        d_stride, y_stride, dy_stride, dtype, dy, dw,
                                                        stream)


quant_fp8 = _block_ops.quant_fp8
swiglu_quant_fp8 = _block_ops.swiglu_quant_fp8
gemm_fp8 = _block_ops.gemm_fp8
gemm_fp8_grouped = _block_ops.gemm_fp8_grouped


def gemm_fp8_workspace_for(T: int, N: int, K: int, device) -> Optional[torch.Tensor]:
    """A workspace for products of these sizes, zeroed; None where none is needed."""
    n = moe_wna16_gemm_fp8_workspace_size(T, N, K)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def _wants_grad(*tensors) -> bool:
    return torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad
                                           for t in tensors)


def sort_tokens(ids: torch.Tensor, experts: int, x: Optional[torch.Tensor] = None, *,
                out: Optional[torch.Tensor] = None) -> dict:
    """sort_tokens(ids, experts, x=None, *, out=None) -> dict

    The pairs of a token and an expert, sorted by expert (stable), and tokens' rows in that order.

    ids int32 [T, k]; the ones outside [0, experts) are left out (another GPU's experts, or none).
    Returns "offsets" int32 [experts + 1], the sorted pairs before each expert and their number;
    "tokens" int32 [T * k], the token of each sorted pair, -1 behind the last; "slots" int32
    [T, k], the place of each pair, -1 for one left out; and, with x [T, H] (bf16, fp16 or fp32; rows
    may be strided), "x" [T * k, H], row tokens[i] of x at i.  Rows of "x" behind the last sorted
    pair are not written; zeros where x requires a gradient.  out: memory for "x", not where x
    requires a gradient.

    The gradient of x is the sum of its rows' (combine_tokens without weights)."""
    if _wants_grad(x):
        if out is not None:
            raise ValueError("out is given, and x requires a gradient")
        return _block_ops.sort_tokens_graph(ids, experts, x)
    return _block_ops.sort_tokens(ids, experts, x, out=out)


def combine_tokens(y: torch.Tensor, slots: torch.Tensor, weights: Optional[torch.Tensor] = None, *,
                   offsets: Optional[torch.Tensor] = None, addend: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """combine_tokens(y, slots, weights=None, *, offsets=None, addend=None, out=None) -> out

    Experts' rows back to their tokens: out[t] = sum over j of weights[t, j] * y[slots[t, j]], plus
    addend[t], in FP32, rounded to y's type at the end.

    y [R, H] (bf16, fp16 or fp32), slots int32 [T, k] as sort_tokens returns them (those outside
    [0, R) are left out), weights float32 [T, k] (ones without), addend [T, H] of y's type; rows
    of y and the addend may be strided.  out may be the addend; not where a gradient is required.
    H up to 2^20, with a gradient of y or the weights 32768.

    Gradients of y, weights and the addend; for those no two slots may name the same row of y.
    Rows of y that no slot names have a gradient of zero.  offsets: sort_tokens', where its slots are
    used as they are: then only the gradient's rows behind the last sorted one are cleared, and each
    before it has to be named by a slot.  Where pairs have been left out since (slots set to -1),
    give none: all of the gradient is cleared first."""
    if _wants_grad(y, weights, addend):
        if out is not None:
            raise ValueError("out is given, and a gradient is required")
        return _block_ops.combine_tokens_graph(y, slots, weights, addend=addend, offsets=offsets)
    return _block_ops.combine_tokens(y, slots, weights, addend=addend, out=out, offsets=offsets)


def forward_fp8(x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, w13: torch.Tensor,
                w13_scale: torch.Tensor, w2: torch.Tensor, w2_scale: torch.Tensor, *,
                alpha: float = 1.0, beta: float = 0.0, clamp: Optional[float] = None, addend=None,
                out=None, codes=None) -> torch.Tensor:
    """The routed layer with experts in 8-bit floating point: forward() for weights that are e4m3
    codes with a scale for each 128 x 128 block.

    x [T, H] (bf16 or fp16); topk_ids int32, topk_w float32 [T, k]; w13 float8_e4m3fn [E, 2I, H],
    gate rows then up rows, w13_scale float32 [E, ceil(2I / 128), ceil(H / 128)]; w2 [E, H, I],
    w2_scale [E, ceil(H / 128), ceil(I / 128)]; H and I multiples of 16.  Ids outside [0, E) are
    left out.  addend [T, H] is added before the rounding; out may be it.  codes: quant_fp8(x), where
    the caller has it.  Returns [T, H] of x's type.  Activations are quantized by quant_fp8 and
    swiglu_quant_fp8; the gate and up rows and the experts' rows are rounded to x's type in between.
    No gradient.

    Rows of experts that are elsewhere cost memory and a pass of the activation, but no product.
    T * k up to 2^21, T * H below 2^32."""
    q, scale = quant_fp8(x) if codes is None else codes
    s = _block_ops.sort_tokens(topk_ids, w13.shape[0])
    # what no single operator sees: rows of other tokens would be read, or left out
    T, H = x.shape
    if topk_ids.shape[0] != T:
        raise ValueError(f"topk_ids has {topk_ids.shape[0]} rows, x {T}")
    if q.shape != x.shape:
        raise ValueError("codes are of another shape than x")
    if w13.dim() != 3 or w2.shape != (w13.shape[0], H, w13.shape[1] // 2):
        raise ValueError("w2 must be [E, H, I] where w13 is [E, 2I, H]")
    gu = gemm_fp8_grouped(q, scale, w13, w13_scale, s["offsets"], rows=s["tokens"], out_dtype=x.dtype)
    q, scale = swiglu_quant_fp8(gu, alpha=alpha, beta=beta, clamp=clamp)
    y = gemm_fp8_grouped(q, scale, w2, w2_scale, s["offsets"], out_dtype=x.dtype)
    return _block_ops.combine_tokens(y, s["slots"], topk_w, addend=addend, out=out)
