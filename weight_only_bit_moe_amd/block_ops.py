"""Operators around the routed layer (include/moe_wna16.h), on torch tensors.

    add_rmsnorm    residual addition, root-mean-square norm, normed rows in 16 and 8 bits
    route_topk     router logits -> the ids and weights forward() reads
    gemm_w8a8      product in 8-bit integers with scales for each token and channel
    swiglu_quant   SwiGLU in 8 bits with a scale for each token

Argument checks, allocation and marshalling only: the work runs in the
library's gfx950 kernels on the current stream.  Decode steps call these every
few microseconds, so the checks touch each tensor once and outputs can be
passed in.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from .binding import OK, MoeWna16Error, load_library

#: element types of the operators' 16- and 32-bit tensors (moe_wna16_dtype)
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
#: score functions of route_topk (moe_wna16_score)
SCORES = {"softmax": 0, "sigmoid": 1}

_INT8 = torch.int8
_F32 = torch.float32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device_now = getattr(torch._C, "_cuda_getDevice", None)


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


def _rows(t, name, shape, dtype, dev):
    """Checks a matrix of contiguous rows; returns its row stride."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    ld, inner = t.stride()
    if inner != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    # a single row's stride means nothing; rows never overlap
    if shape[0] <= 1:
        return shape[1]
    if ld < shape[1]:
        raise ValueError(f"{name} has overlapping rows (stride {ld} < {shape[1]})")
    return ld


def _flat(t, name, shape, dtype, dev):
    """Checks a contiguous tensor; returns its address."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _matrix(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    return t.shape


def _dtype_code(dtype, name):
    code = DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"{name} has dtype {dtype}, expected one of {list(DTYPES)}")
    return code


def _call(fn, dev, *args):
    """Launch on dev's current stream, with dev as the current device."""
    if _device_now() == dev.index:
        return fn(*args, _raw_stream(dev.index))
    with torch.cuda.device(dev):
        return fn(*args, _raw_stream(dev.index))


def add_rmsnorm(x, weight, residual=None, *, eps: float = 1e-6, quant: bool = False,
                normed: bool = True, residual_out=None, out=None, q=None, scale=None) -> dict:
    """Residual addition and root-mean-square norm of rows x [T, H].

    Returns a dict: "residual" (the sum h, if a residual is given: rounded to x's type), "y"
    (h * weight / rms(h), if normed) and, with quant, "q" int8 [T, H] and "scale" float32 [T]
    with y about q * scale.  x, residual: bf16, fp16 or fp32, rows may be strided; weight [H] of
    the same type.  Outputs are contiguous; pass them in to reuse memory (residual_out may be x
    or residual itself).
    """
    T, H = shape = _matrix(x, "x")
    dt, dev = x.dtype, x.device
    code = _dtype_code(dt, "x")
    xs = _rows(x, "x", shape, dt, dev)
    wp = _flat(weight, "weight", (H,), dt, dev)
    rp, rs, hp = None, H, None
    r = {}
    if residual is not None:
        rs = _rows(residual, "residual", shape, dt, dev)
        rp = residual.data_ptr()
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=dt, device=dev)
        hp = _flat(residual_out, "residual_out", shape, dt, dev)
        r["residual"] = residual_out
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    yp = qp = sp = None
    if normed:
        if out is None:
            out = torch.empty(shape, dtype=dt, device=dev)
        yp = _flat(out, "out", shape, dt, dev)
        r["y"] = out
    qs = H
    if quant:
        if q is None:
            q = torch.empty(shape, dtype=_INT8, device=dev)
        if scale is None:
            scale = torch.empty(T, dtype=_F32, device=dev)
        qs = _rows(q, "q", shape, _INT8, dev)
        qp, sp = q.data_ptr(), _flat(scale, "scale", (T,), _F32, dev)
        r["q"], r["scale"] = q, scale
    st = _call(load_library().moe_wna16_add_rmsnorm, dev, x.data_ptr(), rp, wp, T, H, xs, rs, code,
               eps, hp, yp, qp, qs, sp)
    if st != OK:
        raise MoeWna16Error(st, "moe_wna16_add_rmsnorm")
    return r


def route_topk(logits, topk: int, *, bias=None, score: str = "softmax", groups: int = 1,
               topk_groups: int = 1, renormalize: bool = True, scale: float = 1.0, ids=None,
               weights=None):
    """Expert ids int32 [T, topk] and routing weights float32 [T, topk], as forward() reads them,
    of router logits [T, E] (bf16, fp16 or fp32; rows may be strided).

    score "softmax" or "sigmoid"; bias [E] float32 is added for picking only; with groups > 1 only
    the experts of the topk_groups best groups (by the sum of their two largest) are picked.
    Experts with a logit of -inf or NaN are never picked; slots without an expert get id -1 and
    weight 0.
    """
    T, E = shape = _matrix(logits, "logits")
    dev = logits.device
    code = _dtype_code(logits.dtype, "logits")
    ls = _rows(logits, "logits", shape, logits.dtype, dev)
    sc = SCORES.get(score)
    if sc is None:
        raise ValueError(f"score is {score!r}, expected one of {list(SCORES)}")
    bp = None if bias is None else _flat(bias, "bias", (E,), _F32, dev)
    if ids is None:
        ids = torch.empty((T, topk), dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty((T, topk), dtype=_F32, device=dev)
    st = _call(load_library().moe_wna16_route_topk, dev, logits.data_ptr(), bp, T, E, ls, code,
               topk, sc, groups, topk_groups, renormalize, scale,
               _flat(ids, "ids", (T, topk), torch.int32, dev),
               _flat(weights, "weights", (T, topk), _F32, dev))
    if st != OK:
        raise MoeWna16Error(st, "moe_wna16_route_topk")
    return ids, weights


def gemm_w8a8_workspace_for(T: int, N: int, K: int, device) -> Optional[torch.Tensor]:
    """A workspace for products of these sizes, zeroed; None where none is needed."""
    n = moe_wna16_gemm_w8a8_workspace_size(T, N, K)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def gemm_w8a8(a, a_scale, w, w_scale, *, addend=None, out_dtype=torch.bfloat16, out=None,
              workspace=None):
    """(a @ w.T) * a_scale[:, None] * w_scale + addend, the sum exact in int32, rounded once.

    a int8 [T, K], a_scale float32 [T]; w int8 [N, K], w_scale float32 [N]; addend [T, N] of
    out_dtype (bf16, fp16, fp32).  Rows may be strided.  out may be the addend.  workspace: from
    gemm_w8a8_workspace_for, kept by the caller and used by one call at a time; allocated here
    when it is needed and not given.
    """
    T, K = shape = _matrix(a, "a")
    dev = a.device
    N = w.shape[0]
    code = _dtype_code(out_dtype, "out_dtype")
    lda = _rows(a, "a", shape, _INT8, dev)
    ldw = _rows(w, "w", (N, K), _INT8, dev)
    sa = _flat(a_scale, "a_scale", (T,), _F32, dev)
    sw = _flat(w_scale, "w_scale", (N,), _F32, dev)
    ap, lad = None, N
    if addend is not None:
        lad = _rows(addend, "addend", (T, N), out_dtype, dev)
        ap = addend.data_ptr()
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype, device=dev)
        ldo = N
    else:
        ldo = _rows(out, "out", (T, N), out_dtype, dev)
    if workspace is None:
        workspace = gemm_w8a8_workspace_for(T, N, K, dev)
    wp, wn = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    st = _call(load_library().moe_wna16_gemm_w8a8, dev, a.data_ptr(), sa, w.data_ptr(), sw, ap, T,
               N, K, lda, ldw, lad, ldo, code, out.data_ptr(), wp, wn)
    if st != OK:
        raise MoeWna16Error(st, "moe_wna16_gemm_w8a8")
    return out


def swiglu_quant(gu, *, alpha: float = 1.0, beta: float = 0.0, clamp: Optional[float] = None,
                 q=None, scale=None):
    """SwiGLU of rows gu = [gate (I), up (I)] [T, 2I] (bf16, fp16 or fp32; rows may be strided) in
    8 bits: codes int8 [T, I] and scale float32 [T].  alpha, beta, clamp as in forward()."""
    T, two = shape = _matrix(gu, "gu")
    if two % 2:
        raise ValueError("gu must hold gate and up halves of equal length")
    I, dev = two // 2, gu.device
    code = _dtype_code(gu.dtype, "gu")
    gs = _rows(gu, "gu", shape, gu.dtype, dev)
    if q is None:
        q = torch.empty((T, I), dtype=_INT8, device=dev)
    if scale is None:
        scale = torch.empty(T, dtype=_F32, device=dev)
    qs = _rows(q, "q", (T, I), _INT8, dev)
    sp = _flat(scale, "scale", (T,), _F32, dev)
    st = _call(load_library().moe_wna16_swiglu_quant, dev, gu.data_ptr(), T, I, gs, code, alpha,
               beta, math.inf if clamp is None else clamp, q.data_ptr(), qs, sp)
    if st != OK:
        raise MoeWna16Error(st, "moe_wna16_swiglu_quant")
    return q, scale
