"""Refusals of the operators for experts in 8-bit floating point: on the host, before any device
call, by the library and by the torch conveniences."""
import math

import pytest
import torch

import weight_only_bit_moe_amd as M
from weight_only_bit_moe_amd import binding as Bd
from weight_only_bit_moe_amd import block, expert_ops

NAN, INF = float("nan"), math.inf
REACHED = (Bd.EHIP, Bd.EARCH)       # valid arguments end at the device check (no GPU here)
P = 4096                            # aligned, never dereferenced: the calls return first

CALLS = {
    "quant": (lambda: M.moe_wna16_quant_fp8,
              dict(x=P, T=4, K=256, xs=256, dtype=0, q=P, qs=256, s=P, ss=2, stream=None)),
    "swiglu": (lambda: M.moe_wna16_swiglu_quant_fp8,
               dict(gu=P, T=4, I=256, ld=512, dtype=0, alpha=1.0, beta=0.0, clamp=INF, q=P, qs=256, s=P,
                    ss=2, stream=None)),
    "gemm": (lambda: M.moe_wna16_gemm_fp8,
             dict(a=P, sa=P, w=P, sw=P, add=P, T=4, N=200, K=256, lda=256, ldas=2, ldw=256, ldws=2, ladd=200,
                  ldo=200, dtype=0, out=P, ws=P, wsn=1 << 30, stream=None)),
    "grouped": (lambda: M.moe_wna16_gemm_fp8_grouped,
                dict(a=P, sa=P, w=P, sw=P, off=P, rows=P, E=8, arows=4, R=24, N=200, K=256, lda=256, ldas=2,
                     ldw=256, ldws=2, we=200 * 256, se=4, ldo=200, dtype=0, out=P, stream=None)),
    "sort": (lambda: M.moe_wna16_sort_tokens,
             dict(ids=P, T=4, k=6, E=8, x=P, H=100, xs=100, dtype=0, tok=P, slots=P, off=P, out=P, os=100,
                  ws=P, wsn=1 << 30, stream=None)),
    "combine": (lambda: M.moe_wna16_combine_tokens,
                dict(y=P, slots=P, w=P, add=P, T=4, k=6, H=100, R=24, ys=100, adds=100, os=100, dtype=0, out=P,
                     stream=None)),
    "grad": (lambda: M.moe_wna16_combine_tokens_grad,
             dict(d=P, y=P, slots=P, w=P, used=P, T=4, k=6, H=100, R=24, ds=100, ys=100, dys=100, dtype=0, dy=P,
                  dw=P, stream=None)),
}


def call(name, **over):
    fn, ok = CALLS[name]
    assert set(over) <= set(ok)
    return fn()(*dict(ok, **over).values())


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses are not real")
INV, UNS, ALI, WSP, OK = Bd.EINVAL, Bd.EUNSUPPORTED, Bd.EALIGN, Bd.EWORKSPACE, Bd.OK
BIG = 1 << 23


@no_gpu
@pytest.mark.parametrize("name", sorted(CALLS))
def test_valid_arguments_reach_the_device_check(name):
    assert call(name) in REACHED


@no_gpu
@pytest.mark.parametrize("name,over,status", [
    ("quant", dict(T=-1), INV), ("quant", dict(K=0), INV), ("quant", dict(dtype=3), INV), ("quant", dict(xs=255), INV),
    ("quant", dict(qs=255), INV), ("quant", dict(ss=1), INV), ("quant", dict(x=0), INV), ("quant", dict(q=0), INV),
    ("quant", dict(s=0), INV), ("quant", dict(T=0, x=0), OK), ("quant", dict(x=P + 1), ALI),
    ("quant", dict(x=P + 2), None), ("quant", dict(x=P + 2, dtype=2), ALI), ("quant", dict(q=P + 1), None),
    ("quant", dict(s=P + 2), ALI), ("quant", dict(T=(1 << 21) + 1), UNS),
    ("quant", dict(K=131073, xs=131073, qs=131073, ss=1025), UNS),
    ("quant", dict(T=1 << 21, K=131072, xs=131072, qs=131072, ss=1024), UNS),
    ("swiglu", dict(ld=511), INV), ("swiglu", dict(alpha=NAN), INV), ("swiglu", dict(beta=INF), INV),
    ("swiglu", dict(clamp=0.0), INV), ("swiglu", dict(clamp=NAN), INV), ("swiglu", dict(clamp=7.0), None),
    ("swiglu", dict(gu=0), INV), ("swiglu", dict(T=0), OK),
    ("gemm", dict(T=-1), INV), ("gemm", dict(N=-1), INV), ("gemm", dict(K=0), INV), ("gemm", dict(T=0), OK),
    ("gemm", dict(N=0), OK), ("gemm", dict(K=255, lda=256, ldw=256), UNS), ("gemm", dict(K=240), None),
    ("gemm", dict(lda=255), INV), ("gemm", dict(lda=264), ALI), ("gemm", dict(ldw=264), ALI), ("gemm", dict(lda=272), None),
    ("gemm", dict(a=P + 8), ALI), ("gemm", dict(w=P + 8), ALI), ("gemm", dict(sa=P + 2), ALI), ("gemm", dict(sw=P + 2), ALI),
    ("gemm", dict(out=P + 1), ALI), ("gemm", dict(add=P + 1), ALI), ("gemm", dict(ws=P + 16), ALI),
    ("gemm", dict(ldas=1), INV), ("gemm", dict(ldws=1), INV), ("gemm", dict(ldas=1 << 20), UNS),
    ("gemm", dict(ldws=1 << 20), UNS), ("gemm", dict(ladd=199), INV), ("gemm", dict(ladd=0, add=0), None),
    ("gemm", dict(ldo=199), INV), ("gemm", dict(lda=BIG), UNS), ("gemm", dict(ldw=BIG), UNS), ("gemm", dict(ldo=BIG), UNS),
    ("gemm", dict(ladd=BIG), UNS), ("gemm", dict(dtype=5), INV), ("gemm", dict(a=0), INV), ("gemm", dict(sa=0), INV),
    ("gemm", dict(w=0), INV), ("gemm", dict(sw=0), INV), ("gemm", dict(out=0), INV),
    ("gemm", dict(T=(1 << 21) + 1), UNS), ("gemm", dict(K=131088, lda=131088, ldw=131088, ldas=1025, ldws=1025), UNS),
    ("grouped", dict(R=-1), INV), ("grouped", dict(E=0), INV), ("grouped", dict(E=1025), UNS), ("grouped", dict(R=0), OK),
    ("grouped", dict(N=0), OK), ("grouped", dict(arows=0), INV), ("grouped", dict(rows=0), INV),
    ("grouped", dict(rows=0, arows=24), None), ("grouped", dict(we=200 * 256 - 1), INV), ("grouped", dict(we=200 * 256 + 8), ALI),
    ("grouped", dict(se=3), INV), ("grouped", dict(E=1, we=0, se=0), None), ("grouped", dict(off=0), INV),
    ("grouped", dict(off=P + 2), ALI), ("grouped", dict(rows=P + 2), ALI), ("grouped", dict(K=200), UNS),
    ("grouped", dict(R=(1 << 21) + 1), UNS), ("grouped", dict(arows=1 << 20, lda=4096), UNS),
    ("grouped", dict(arows=1 << 20, lda=4080), None), ("grouped", dict(arows=1 << 20, ldas=1024), UNS),
    ("sort", dict(T=-1), INV), ("sort", dict(k=0), INV), ("sort", dict(E=0), INV), ("sort", dict(k=65), UNS),
    ("sort", dict(E=1025), UNS), ("sort", dict(T=(1 << 21) + 1), UNS), ("sort", dict(T=1 << 20, k=17), UNS),
    ("sort", dict(ids=0), INV), ("sort", dict(tok=0), INV), ("sort", dict(slots=0), INV), ("sort", dict(off=0), INV),
    ("sort", dict(out=0), INV), ("sort", dict(x=0, out=0, H=0, xs=0, os=0), None), ("sort", dict(xs=99), INV),
    ("sort", dict(os=99), INV), ("sort", dict(H=0, xs=0, os=0), INV), ("sort", dict(dtype=3), INV), ("sort", dict(x=P + 1), ALI),
    ("sort", dict(ids=P + 2), ALI), ("sort", dict(T=0, ids=0, tok=0, slots=0, x=0), None),
    ("sort", dict(H=(1 << 20) + 1, xs=1 << 21, os=1 << 21), UNS), ("sort", dict(T=20000, ws=0), INV),
    ("sort", dict(T=20000, wsn=16), WSP), ("sort", dict(ws=0, wsn=0), None),
    ("combine", dict(T=-1), INV), ("combine", dict(T=0), OK), ("combine", dict(k=0), INV), ("combine", dict(H=0), INV),
    ("combine", dict(R=-1), INV), ("combine", dict(R=0, y=0), None), ("combine", dict(y=0), INV), ("combine", dict(slots=0), INV),
    ("combine", dict(out=0), INV), ("combine", dict(w=0, add=0, adds=0), None), ("combine", dict(ys=99), INV),
    ("combine", dict(adds=99), INV), ("combine", dict(os=99), INV), ("combine", dict(k=65), UNS), ("combine", dict(y=P + 1), ALI),
    ("combine", dict(w=P + 2), ALI), ("combine", dict(dtype=-1), INV), ("combine", dict(R=(1 << 24) + 1), UNS),
    ("grad", dict(T=-1), INV), ("grad", dict(T=0, used=0), OK), ("grad", dict(T=0, d=0, slots=0), None),
    ("grad", dict(T=0, R=0), OK), ("grad", dict(d=0), INV), ("grad", dict(slots=0), INV), ("grad", dict(dy=0, dw=0, used=0), INV),
    ("grad", dict(dy=0, used=0, dys=0), None), ("grad", dict(dy=0), INV), ("grad", dict(dw=0, y=0, ys=0), None),
    ("grad", dict(y=0), INV), ("grad", dict(H=32769, ds=40000, ys=40000, dys=40000), UNS), ("grad", dict(dys=99), INV),
    ("grad", dict(used=P + 2), ALI), ("grad", dict(dw=P + 2), ALI), ("grad", dict(w=0), None),
])
def test_refusals(name, over, status):
    st = call(name, **over)
    assert st in REACHED if status is None else st == status


def test_workspace_sizes():
    lib = M.load_library()
    assert M.moe_wna16_gemm_fp8_workspace_size(0, 64, 64) == 0
    assert M.moe_wna16_gemm_fp8_workspace_size(4, 4096, 4096) == 0
    for bad in ((-1, 64, 64), (4, 64, 0), (4, 64, 24), (1 << 22, 64, 64)):
        with pytest.raises(M.MoeWna16Error):
            M.moe_wna16_gemm_fp8_workspace_size(*bad)
    assert lib.moe_wna16_gemm_fp8_workspace_size(4, 64, 64, None) == INV
    assert M.moe_wna16_sort_tokens_workspace_size(4, 6, 256) == 0
    assert M.moe_wna16_sort_tokens_workspace_size(20000, 8, 256) >= 4 * 256
    assert lib.moe_wna16_sort_tokens_workspace_size(4, 6, 256, None) == INV
    with pytest.raises(M.MoeWna16Error):
        M.moe_wna16_sort_tokens_workspace_size(4, 65, 256)


@no_gpu
def test_product_workspace_is_checked():
    """Every plan that asks for a workspace refuses a missing or smaller one, and some do ask."""
    asked = 0
    for T in (1, 33, 65, 128, 256, 512, 1024, 4096):
        for N in (64, 512, 2048, 4096):
            for K in (128, 2048, 4096, 16384):
                need = M.moe_wna16_gemm_fp8_workspace_size(T, N, K)
                over = dict(T=T, N=N, K=K, lda=K, ldas=K // 128, ldw=K, ldws=K // 128, ladd=N, ldo=N)
                assert call("gemm", wsn=need, **over) in REACHED
                if need:
                    asked += 1
                    assert call("gemm", wsn=need - 1, **over) == WSP
                    assert call("gemm", ws=0, **over) == INV
                else:
                    assert call("gemm", ws=0, wsn=0, **over) in REACHED
    assert asked


def test_conveniences_refuse_what_is_not_on_the_gpu():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    ids = torch.zeros(2, 3, dtype=torch.int32)
    q, s = x.to(torch.float8_e4m3fn), torch.ones(2, 1)
    for f in (lambda: M.quant_fp8(x), lambda: M.swiglu_quant_fp8(x), lambda: M.gemm_fp8(q, s, q, s),
              lambda: M.gemm_fp8_grouped(q, s, q[None], s[None], ids[0]), lambda: M.sort_tokens(ids, 4, x),
              lambda: M.combine_tokens(x, ids), lambda: M.forward_fp8(x, ids, s, q[None], s[None], q[None], s[None])):
        with pytest.raises(ValueError, match="on the GPU"):
            f()
    with pytest.raises(ValueError, match="2-D"):
        M.quant_fp8(x[0])


@pytest.mark.parametrize("f", [
    lambda x: M.quant_fp8(), lambda x: M.quant_fp8(None), lambda x: M.quant_fp8(x, x), lambda x: M.quant_fp8(x, code=x),
    lambda x: M.swiglu_quant_fp8(x, 1.0), lambda x: M.gemm_fp8(x, x, x), lambda x: M.gemm_fp8(x, x, x, x, x),
    lambda x: M.gemm_fp8_grouped(x, x, x, x), lambda x: M.sort_tokens(x), lambda x: M.combine_tokens(x)])
def test_conveniences_refuse_other_arguments(f):
    with pytest.raises(TypeError):
        f(torch.zeros(2, 64))


def test_names_and_documentation():
    names = ("quant_fp8", "swiglu_quant_fp8", "gemm_fp8", "gemm_fp8_grouped", "sort_tokens", "combine_tokens", "forward_fp8")
    assert set(names) <= set(dir(M))
    for n in names[:-1]:
        assert getattr(M, n).__doc__.startswith(n + "("), n
    for n in ("quant_fp8", "swiglu_quant_fp8", "gemm_fp8", "gemm_fp8_grouped", "forward_fp8"):
        assert "No" in M.__getattr__(n).__doc__ and "gradient" in getattr(M, n).__doc__
    for n in names:
        assert n in expert_ops.__doc__


@pytest.mark.parametrize("shape", [(1, 1), (130, 257), (3, 200, 128)])
def test_block_codes(shape):
    g = torch.Generator()
    g.manual_seed(1)
    w = torch.randn(*shape, generator=g) * torch.exp(torch.randn(shape[-1], generator=g))
    c, s = block.block_codes(w)
    assert c.dtype == torch.float8_e4m3fn and c.shape == w.shape and c.is_contiguous()
    assert s.shape == (*shape[:-2], -(-shape[-2] // 128), -(-shape[-1] // 128))
    step = s.repeat_interleave(128, -2)[..., :shape[-2], :].repeat_interleave(128, -1)[..., :shape[-1]]
    # half a step of e4m3: 2^-4 of the value, or 2^-10 of the scale below the normal ones; the quotient
    # and the product are rounded once each
    off = (c.float() * step - w).abs()
    assert bool((off <= (2.0 ** -4 + 2.0 ** -22) * w.abs() + 2.0 ** -10 * step).all())


def test_block_codes_of_blocks_that_vanish_or_are_not_finite():
    w = torch.ones(256, 256)
    w[5, 7] = NAN
    w[200, 3] = INF
    w[:128, 128:] = 2.0 ** -101
    c, s = block.block_codes(w)
    assert torch.isnan(s).tolist() == [[True, False], [True, False]]
    assert float(s[0, 1]) == 0 and float(s[1, 1]) == torch.tensor(1.0) / 448
    assert not c[:, :128].float().any() and not c[:128].float().any()
    assert bool((c[128:, 128:].float() == 448).all())
