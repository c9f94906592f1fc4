"""Refusals of the operators around the routed layer: on the host, before any
device call, by the library and by the torch conveniences."""
import math

import pytest
import torch

import weight_only_bit_moe_amd as M
from weight_only_bit_moe_amd import binding as Bd

NAN, INF = float("nan"), math.inf
REACHED = (Bd.EHIP, Bd.EARCH)       # valid arguments end at the device check (no GPU here)
P = 4096                            # aligned, never dereferenced: the calls return first

CALLS = {
    "norm": (lambda: M.moe_wna16_add_rmsnorm,
             dict(x=P, residual=P, weight=P, T=4, H=64, xs=64, rs=64, dtype=0, eps=1e-6, ro=P, y=P,
                  q=P, qs=64, s=P, stream=None)),
    "route": (lambda: M.moe_wna16_route_topk,
              dict(l=P, bias=P, T=4, E=64, ld=64, dtype=2, k=6, score=1, groups=8, kg=4, renorm=1,
                   scale=1.0, ids=P, w=P, stream=None)),
    "gemm": (lambda: M.moe_wna16_gemm_w8a8,
             dict(a=P, sa=P, w=P, sw=P, add=P, T=4, N=64, K=128, lda=128, ldw=128, ladd=64, ldo=64,
                  dtype=0, out=P, ws=P, wsn=1 << 30, stream=None)),
    "swiglu": (lambda: M.moe_wna16_swiglu_quant,
               dict(gu=P, T=4, I=64, ld=128, dtype=0, alpha=1.0, beta=0.0, clamp=INF, q=P, qs=64,
                    s=P, stream=None)),
}


def call(name, **over):
    fn, ok = CALLS[name]
    assert set(over) <= set(ok)
    return fn()(*dict(ok, **over).values())


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses are not real")


@no_gpu
@pytest.mark.parametrize("name", sorted(CALLS))
def test_valid_arguments_reach_the_device_check(name):
    assert call(name) in REACHED
    assert call(name, T=0) == Bd.OK


@no_gpu
@pytest.mark.parametrize("name,over,status", [
    ("norm", dict(T=-1), Bd.EINVAL), ("norm", dict(H=0), Bd.EINVAL), ("norm", dict(dtype=3), Bd.EINVAL),
    ("norm", dict(dtype=-1), Bd.EINVAL), ("norm", dict(eps=NAN), Bd.EINVAL),
    ("norm", dict(eps=-1e-6), Bd.EINVAL), ("norm", dict(eps=INF), Bd.EINVAL),
    ("norm", dict(xs=63), Bd.EINVAL), ("norm", dict(rs=63), Bd.EINVAL), ("norm", dict(qs=1), Bd.EINVAL),
    ("norm", dict(rs=0, residual=None), None), ("norm", dict(qs=0, q=None), None),
    ("norm", dict(H=32769, xs=32769, rs=32769, qs=32769), Bd.EUNSUPPORTED),
    ("norm", dict(T=(1 << 21) + 1), Bd.EUNSUPPORTED), ("norm", dict(T=1 << 21), None),
    ("route", dict(T=(1 << 21) + 1), Bd.EUNSUPPORTED),
    ("swiglu", dict(T=(1 << 21) + 1), Bd.EUNSUPPORTED),
    ("norm", dict(x=0), Bd.EINVAL), ("norm", dict(weight=0), Bd.EINVAL),
    ("norm", dict(y=0, q=0), Bd.EINVAL), ("norm", dict(s=0), Bd.EINVAL),
    ("norm", dict(q=0, s=0), None), ("norm", dict(ro=0), None), ("norm", dict(y=0), None),
    ("norm", dict(x=P + 1), Bd.EALIGN), ("norm", dict(x=P + 2), None),
    ("norm", dict(x=P + 2, dtype=2), Bd.EALIGN), ("norm", dict(s=P + 2), Bd.EALIGN),
    ("norm", dict(ro=P + 1), Bd.EALIGN), ("norm", dict(q=P + 1), None),
    ("route", dict(T=-1), Bd.EINVAL), ("route", dict(E=0), Bd.EINVAL), ("route", dict(k=0), Bd.EINVAL),
    ("route", dict(k=65, E=64, ld=64), Bd.EINVAL), ("route", dict(score=2), Bd.EINVAL),
    ("route", dict(groups=0), Bd.EINVAL), ("route", dict(groups=7), Bd.EINVAL),
    ("route", dict(kg=0), Bd.EINVAL), ("route", dict(kg=9), Bd.EINVAL), ("route", dict(ld=63), Bd.EINVAL),
    ("route", dict(scale=NAN), Bd.EINVAL), ("route", dict(dtype=5), Bd.EINVAL),
    ("route", dict(E=1032, ld=1032), Bd.EUNSUPPORTED),
    ("route", dict(E=1024, ld=1024, k=65), Bd.EUNSUPPORTED),
    ("route", dict(E=1024, ld=1024, groups=128), Bd.EUNSUPPORTED),
    ("route", dict(l=0), Bd.EINVAL), ("route", dict(ids=0), Bd.EINVAL), ("route", dict(w=0), Bd.EINVAL),
    ("route", dict(bias=0), None), ("route", dict(l=P + 2), Bd.EALIGN),
    ("route", dict(l=P + 2, dtype=1), None), ("route", dict(bias=P + 2), Bd.EALIGN),
    ("gemm", dict(T=-1), Bd.EINVAL), ("gemm", dict(N=-1), Bd.EINVAL), ("gemm", dict(K=0), Bd.EINVAL),
    ("gemm", dict(N=0), Bd.OK), ("gemm", dict(K=131072, lda=131072, ldw=131072), Bd.EUNSUPPORTED),
    ("gemm", dict(K=131071, lda=131071, ldw=131071), None),
    ("gemm", dict(T=(1 << 21) + 1), Bd.EUNSUPPORTED), ("gemm", dict(lda=127), Bd.EINVAL),
    ("gemm", dict(ldw=127), Bd.EINVAL), ("gemm", dict(ladd=63), Bd.EINVAL),
    ("gemm", dict(ladd=0, add=0), None), ("gemm", dict(ldo=63), Bd.EINVAL),
    ("gemm", dict(lda=1 << 23), Bd.EUNSUPPORTED), ("gemm", dict(ldo=1 << 23), Bd.EUNSUPPORTED),
    ("gemm", dict(dtype=4), Bd.EINVAL), ("gemm", dict(a=0), Bd.EINVAL), ("gemm", dict(sa=0), Bd.EINVAL),
    ("gemm", dict(w=0), Bd.EINVAL), ("gemm", dict(sw=0), Bd.EINVAL), ("gemm", dict(out=0), Bd.EINVAL),
    ("gemm", dict(a=P + 1), None), ("gemm", dict(sa=P + 2), Bd.EALIGN),
    ("gemm", dict(out=P + 1), Bd.EALIGN), ("gemm", dict(out=P + 2, dtype=2), Bd.EALIGN),
    ("gemm", dict(add=P + 1), Bd.EALIGN), ("gemm", dict(ws=P + 16), Bd.EALIGN),
    ("swiglu", dict(T=-1), Bd.EINVAL), ("swiglu", dict(I=0), Bd.EINVAL), ("swiglu", dict(ld=127), Bd.EINVAL),
    ("swiglu", dict(qs=63), Bd.EINVAL), ("swiglu", dict(alpha=NAN), Bd.EINVAL),
    ("swiglu", dict(beta=INF), Bd.EINVAL), ("swiglu", dict(clamp=0.0), Bd.EINVAL),
    ("swiglu", dict(clamp=NAN), Bd.EINVAL), ("swiglu", dict(clamp=-1.0), Bd.EINVAL),
    ("swiglu", dict(I=32769, ld=65538, qs=32769), Bd.EUNSUPPORTED),
    ("swiglu", dict(gu=0), Bd.EINVAL), ("swiglu", dict(q=0), Bd.EINVAL), ("swiglu", dict(s=0), Bd.EINVAL),
    ("swiglu", dict(gu=P + 1), Bd.EALIGN), ("swiglu", dict(gu=P + 2), None),
    ("swiglu", dict(s=P + 1), Bd.EALIGN),
])
def test_refusals(name, over, status):
    st = call(name, **over)
    if status is None:
        assert st in REACHED
    else:
        assert st == status


def test_product_workspace_size():
    lib = M.load_library()
    assert M.moe_wna16_gemm_w8a8_workspace_size(0, 64, 64) == 0
    assert M.moe_wna16_gemm_w8a8_workspace_size(8192, 4096, 4096) >= 0
    for bad in ((-1, 64, 64), (4, 64, 0), (4, 64, 131072), (1 << 22, 64, 64)):
        with pytest.raises(M.MoeWna16Error):
            M.moe_wna16_gemm_w8a8_workspace_size(*bad)
    assert lib.moe_wna16_gemm_w8a8_workspace_size(4, 64, 64, None) == Bd.EINVAL


@no_gpu
def test_product_workspace_is_checked():
    """Every plan that asks for a workspace refuses a missing or smaller one."""
    for T in (1, 4, 16, 64, 65, 128, 256, 512, 1024, 4096):
        for N in (64, 512, 2048, 4096):
            for K in (128, 2048, 4096, 16384):
                need = M.moe_wna16_gemm_w8a8_workspace_size(T, N, K)
                over = dict(T=T, N=N, K=K, lda=K, ldw=K, ladd=N, ldo=N)
                assert call("gemm", wsn=need, **over) in REACHED
                if need:
                    assert call("gemm", wsn=need - 1, **over) == Bd.EWORKSPACE
                    assert call("gemm", ws=0, **over) == Bd.EINVAL
                else:
                    assert call("gemm", ws=0, wsn=0, **over) in REACHED


def test_conveniences_refuse_what_is_not_on_the_gpu():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    i8, f = x.to(torch.int8), x[:, 0].float()
    for call in (lambda: M.add_rmsnorm(x, x[0]), lambda: M.route_topk(x, 2), lambda: M.swiglu_quant(x),
                 lambda: M.gemm_w8a8(i8, f, i8, f)):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
    with pytest.raises(ValueError, match="2-D"):
        M.route_topk(x[0], 2)


@pytest.mark.parametrize("call", [
    lambda x: M.add_rmsnorm([1.0], x), lambda x: M.add_rmsnorm(None, x), lambda x: M.add_rmsnorm(x),
    lambda x: M.add_rmsnorm(x, x, x, 1e-6), lambda x: M.add_rmsnorm(x, x, x=x),
    lambda x: M.add_rmsnorm(x, x, epsilon=1e-6), lambda x: M.route_topk(x),
    lambda x: M.route_topk(x, 2, None), lambda x: M.gemm_w8a8(x, x, x), lambda x: M.swiglu_quant(),
    lambda x: M.swiglu_quant(x, 1.0), lambda x: M.gemm_w8a8(x, x, x, x, x)])
def test_conveniences_refuse_other_arguments(call):
    with pytest.raises(TypeError):
        call(torch.zeros(2, 64))


def test_conveniences_are_documented():
    for f in (M.add_rmsnorm, M.route_topk, M.gemm_w8a8, M.swiglu_quant):
        assert f.__doc__.startswith(f.__name__ + "(")
