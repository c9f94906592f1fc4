"""Operators around the routed layer (include/moe_wna16.h), on torch tensors.

    add_rmsnorm    residual addition, root-mean-square norm, normed rows in 16 and 8 bits
    route_topk     router logits -> the ids and weights forward() reads
    gemm_w8a8      product in 8-bit integers with scales for each token and channel
    swiglu_quant   SwiGLU in 8 bits with a scale for each token

Each runs in the library's gfx950 kernels on the current stream.  Argument
checks, allocation and the library call are in the compiled module _block_ops
(csrc/block_ops_module.cpp): decode steps call these every few microseconds.
The raw entry points take integer device addresses, as the others of binding do.

Inference only, as the rest of the package: tensors that require a gradient are
taken as values, and no output carries a graph.
"""
from __future__ import annotations

import ctypes
import importlib
from typing import Optional

import torch

from .binding import OK, MoeWna16Error, load_library

try:
    _block_ops = importlib.import_module("._block_ops", __package__)
except ModuleNotFoundError as e:
    raise RuntimeError("the module _block_ops is missing: build it with "
                       "`python -m weight_only_bit_moe_amd.build`") from e
except ImportError as e:
    raise RuntimeError(f"the module _block_ops does not load ({e}); if torch has changed since, build "
                       "it again with `python -m weight_only_bit_moe_amd.build`") from e

#: element types of the operators' 16- and 32-bit tensors (moe_wna16_dtype)
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
#: score functions of route_topk (moe_wna16_score)
SCORES = {"softmax": 0, "sigmoid": 1}
#: leading bytes of a product's workspace that start at zero (MOE_WNA16_GEMM_SYNC_BYTES)
GEMM_SYNC_BYTES = 4096


def moe_wna16_add_rmsnorm(x, residual, weight, T, H, x_stride, r_stride, dtype, eps, residual_out,
                          y_out, q_out, q_stride, scale_out, stream) -> int:
    """Raw entry point on integer device addresses; returns the status."""
    return load_library().moe_wna16_add_rmsnorm(x, residual, weight, T, H, x_stride, r_stride,
                                                dtype, eps, residual_out, y_out, q_out, q_stride,
                                                scale_out, stream)


def moe_wna16_route_topk(logits, bias, T, E, stride_elems, dtype, topk, score, groups, topk_groups,
                         renormalize, scale, ids_out, w_out, stream) -> int:
    """Raw entry point on integer device addresses; returns the status."""
    return load_library().moe_wna16_route_topk(logits, bias, T, E, stride_elems, dtype, topk,
                                               score, groups, topk_groups, renormalize, scale,
                                               ids_out, w_out, stream)


def moe_wna16_gemm_w8a8(a, a_scale, w, w_scale, addend, T, N, K, lda, ldw, ld_add, ldo, out_dtype,
                        out, workspace, workspace_bytes, stream) -> int:
    """Raw entry point on integer device addresses; returns the status."""
    return load_library().moe_wna16_gemm_w8a8(a, a_scale, w, w_scale, addend, T, N, K, lda, ldw,
                                              ld_add, ldo, out_dtype, out, workspace,
                                              workspace_bytes, stream)


def moe_wna16_gemm_w8a8_workspace_size(T: int, N: int, K: int) -> int:
    n = ctypes.c_size_t(0)
    st = load_library().moe_wna16_gemm_w8a8_workspace_size(T, N, K, ctypes.byref(n))
    if st != OK:
        raise MoeWna16Error(st, "moe_wna16_gemm_w8a8_workspace_size")
    return n.value


def moe_wna16_swiglu_quant(gu, T, I, gu_stride, dtype, alpha, beta, clamp, q_out, q_stride,
                           scale_out, stream) -> int:
    """Raw entry point on integer device addresses; returns the status."""
    return load_library().moe_wna16_swiglu_quant(gu, T, I, gu_stride, dtype, alpha, beta, clamp,
                                                 q_out, q_stride, scale_out, stream)


#: the library's functions that the module calls, in the order of its table
_FUNCTIONS = ("add_rmsnorm", "route_topk", "gemm_w8a8", "gemm_w8a8_workspace_size", "swiglu_quant",
              "quant_fp8", "swiglu_quant_fp8", "gemm_fp8", "gemm_fp8_workspace_size",
              "gemm_fp8_grouped", "sort_tokens", "sort_tokens_workspace_size", "combine_tokens",
              "combine_tokens_grad")


def _load():
    """Loads the library and gives the module its functions; raises if it is not built."""
    lib = load_library()
    _block_ops.bind(_load, MoeWna16Error, tuple(
        ctypes.cast(getattr(lib, "moe_wna16_" + f), ctypes.c_void_p).value for f in _FUNCTIONS))


_block_ops.bind(_load, MoeWna16Error, (0,) * len(_FUNCTIONS))
add_rmsnorm = _block_ops.add_rmsnorm
route_topk = _block_ops.route_topk
gemm_w8a8 = _block_ops.gemm_w8a8
swiglu_quant = _block_ops.swiglu_quant


def gemm_w8a8_workspace_for(T: int, N: int, K: int, device) -> Optional[torch.Tensor]:
    """A workspace for products of these sizes, zeroed; None where none is needed."""
    n = moe_wna16_gemm_w8a8_workspace_size(T, N, K)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None
