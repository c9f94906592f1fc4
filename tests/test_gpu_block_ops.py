"""The operators around the routed layer on the GPU against 64-bit references
(tests/_block.py), over types, sizes, strides, masks and non-finite values."""
import math
import zlib

import numpy as np
import pytest
import torch

import weight_only_bit_moe_amd as M
from tests import _block as R

pytestmark = pytest.mark.gpu

BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


def gen(*key):
    g = torch.Generator()
    g.manual_seed(zlib.crc32(str(key).encode()))
    return g


def strided(t, dev, pad, offset=0):
    """t on the GPU inside a wider buffer: rows pad elements further apart, the first one at
    `offset`; the gaps hold NaN (or 99)."""
    T, n = t.shape
    fill = 99 if t.dtype == torch.int8 else float("nan")
    buf = torch.full((T * (n + pad) + offset,), fill, dtype=t.dtype, device=dev)
    v = buf[offset:].view(T, n + pad)[:, :n]
    v.copy_(t)
    return v


# ---- residual norm -----------------------------------------------------------

# FP32 steps behind y and scale: the sum of squares adds at most 8 values per thread and chunk
# (64 in a row) and then at most 16 partial sums by trees (10 steps), half of which survives the
# square root; the division, root, product with the weight and with rstd add one rounding each.
NORM_U = (64 + 10 + 2) / 2 + 6


def check_norm(x, r, w, eps, got, quant=True):
    h, y, q, scale, top = R.rmsnorm(x, r, w, eps)
    dt = x.dtype
    if r is not None:
        assert torch.equal(got["residual"].cpu(), h)
    e = got["y"].cpu().to(R.F) - y
    bound = (R.half_step(dt) + NORM_U * R.U) * y.abs() + R.smallest(dt)
    assert bool((e.abs() <= bound).all()), float((e.abs() - bound).max())
    if quant:
        assert torch.equal(got["q"].cpu(), q)
        live = top >= 2.0 ** -100
        s = torch.where(live, scale, torch.zeros_like(scale))
        assert bool(((got["scale"].cpu().to(R.F) - s).abs() <= (NORM_U + 2) * R.U * s).all())


@pytest.mark.parametrize("dt", [BF, HF, FF])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 7), (2, 8), (3, 130), (4, 512), (5, 513), (4, 1000),
                                 (3, 2047), (4, 4096), (2, 5120), (3, 8191), (2, 16384), (2, 20001),
                                 (2, 32767), (2, 32768), (1031, 96)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(dev, dt, T, H, residual):
    g = gen("norm", T, H, residual)
    x = (torch.randn(T, H, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).to(dt)
    r = torch.randn(T, H, generator=g).to(dt) if residual else None
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(dt)
    got = M.add_rmsnorm(x.to(dev), w.to(dev), None if r is None else r.to(dev), eps=1e-6, quant=True)
    assert ("residual" in got) == residual
    check_norm(x, r, w, 1e-6, got)


@pytest.mark.parametrize("dt", [BF, FF])
@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 5), (8, 8), (64, 1)])
def test_norm_strided_unaligned_and_in_place(dev, dt, pad, offset):
    g = gen("strided", pad, offset)
    T, H = 6, 777
    x, r = torch.randn(T, H, generator=g).to(dt), torch.randn(T, H, generator=g).to(dt)
    w = torch.randn(H, generator=g).to(dt)
    q = strided(torch.zeros(T, H, dtype=torch.int8), dev, pad, offset)
    rr = r.to(dev)
    got = M.add_rmsnorm(strided(x, dev, pad, offset), w.to(dev), strided(r, dev, pad, offset),
                        quant=True, q=q)
    check_norm(x, r, w, 1e-6, got)
    assert got["q"] is q
    gap = torch.as_strided(q, (T - 1, pad), (H + pad, 1), q.storage_offset() + H)
    assert bool((gap == 99).all())
    got = M.add_rmsnorm(x.to(dev), w.to(dev), rr, quant=True, residual_out=rr)
    assert got["residual"] is rr
    check_norm(x, r, w, 1e-6, got)


def test_norm_outputs_on_request(dev):
    x = torch.randn(3, 64).to(BF).to(dev)
    w = torch.ones(64, dtype=BF, device=dev)
    assert set(M.add_rmsnorm(x, w)) == {"y"}
    assert set(M.add_rmsnorm(x, w, x, quant=True, normed=False)) == {"residual", "q", "scale"}
    with pytest.raises(M.MoeWna16Error):
        M.add_rmsnorm(x, w, normed=False)
    with pytest.raises(ValueError):
        M.add_rmsnorm(x, w, residual_out=x)


def test_norm_zero_tiny_and_non_finite_rows(dev):
    T, H = 8, 300
    x = torch.randn(T, H, generator=gen("edge"))
    x[0] = 0
    x[1] = 2.0 ** -110
    x[2, 17] = float("nan")
    x[3, 299] = float("inf")
    x[4, 0] = -float("inf")
    x[5] = 0
    x[5, 3] = 1e-8
    w = torch.ones(H)
    for dt in (FF, BF):
        xd = x.to(dt)
        got = M.add_rmsnorm(xd.to(dev), w.to(dt).to(dev), eps=0.0 if dt == FF else 1e-6, quant=True)
        q, s, y = got["q"].cpu(), got["scale"].cpu(), got["y"].cpu()
        assert not q[:5].any() and float(s[1]) == 0
        assert bool(torch.isnan(s[2:5]).all()) and bool(torch.isfinite(s[5:]).all())
        assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3, 299]))
        assert int(q[5, 3]) == 127 and not q[5, :3].any()
        if dt == BF:
            assert float(s[0]) == 0 and not y[0].any()
            check_norm(xd[5:], None, w.to(dt), 1e-6, {k: v[5:] for k, v in got.items()})


def test_norm_row_offsets_past_32_bits(dev):
    """Three rows 1.2e9 elements apart: the last one starts past 2^32 bytes."""
    H, ld = 520, 1_200_000_000
    buf = torch.empty(2 * ld + H, dtype=BF, device=dev)
    x = torch.as_strided(buf, (3, H), (ld, 1))
    src = torch.randn(3, H, generator=gen("far")).to(BF)
    x.copy_(src)
    w = torch.ones(H, dtype=BF)
    check_norm(src, None, w, 1e-6, M.add_rmsnorm(x, w.to(dev), quant=True))


# ---- SwiGLU in 8 bits ----------------------------------------------------------

def check_swiglu(gu, alpha, beta, clamp, q, s):
    a, g = R.swiglu(gu, alpha, beta, clamp)
    # alpha g is rounded before the exponential (|alpha g| U relative in it), the exponential is
    # good to 2 ulp, and the sum, reciprocal, two products and u + beta add one rounding each
    # (the reciprocal two)
    rel = (10 + (alpha * g).abs().amax(-1)) * R.U
    m = a.abs().amax(-1)
    s = s.cpu().to(R.F)
    assert bool(((s - m / 127).abs() <= (rel + 2 * R.U) * m / 127).all())
    live = m >= 2.0 ** -99
    ideal = torch.where(live[:, None], a * 127 / m.clamp(min=2.0 ** -200)[:, None],
                        torch.zeros_like(a))
    off = (q.cpu().to(R.F) - ideal).abs()
    assert bool((off <= 0.5 + 127 * (2 * rel + 4 * R.U)[:, None]).all()), float(off.max())


@pytest.mark.parametrize("dt", [BF, HF, FF])
@pytest.mark.parametrize("T,I", [(1, 1), (2, 9), (3, 128), (4, 513), (5, 1000), (4, 2048), (2, 4097),
                                 (2, 16384), (1, 32768), (999, 64)])
@pytest.mark.parametrize("alpha,beta,clamp", [(1.0, 0.0, None), (1.702, 1.0, 7.0)])
def test_swiglu(dev, dt, T, I, alpha, beta, clamp):
    gu = (4 * torch.randn(T, 2 * I, generator=gen("sw", T, I))).to(dt)
    q, s = M.swiglu_quant(gu.to(dev), alpha=alpha, beta=beta, clamp=clamp)
    check_swiglu(gu, alpha, beta, clamp, q, s)


def test_swiglu_strided(dev):
    gu = (3 * torch.randn(7, 2 * 333, generator=gen("sws"))).to(BF)
    q = strided(torch.zeros(7, 333, dtype=torch.int8), dev, 5, 3)
    got, s = M.swiglu_quant(strided(gu, dev, 7, 1), q=q)
    assert got is q
    check_swiglu(gu, 1.0, 0.0, None, q, s)


def test_swiglu_far_values_and_non_finite_rows(dev):
    I = 200
    gu = torch.randn(6, 2 * I, generator=gen("swe"))
    gu[0] = 0
    gu[1, :I] = -1e4               # sigmoid underflows: exact zeros
    gu[2, 5] = float("nan")
    gu[3, I + 9] = float("inf")
    gu[4, :I] = 90.0               # sigmoid saturates
    q, s = M.swiglu_quant(gu.to(dev))
    q, s = q.cpu(), s.cpu()
    assert not q[:4].any() and float(s[0]) == 0 and float(s[1]) == 0
    assert bool(torch.isnan(s[2:4]).all())
    check_swiglu(gu[4:], 1.0, 0.0, None, q[4:], s[4:])
    # a clamp bounds an infinite up value, and a NaN stays one
    q, s = M.swiglu_quant(gu.to(dev), clamp=7.0)
    assert bool(torch.isnan(s[2])) and bool(torch.isfinite(s[3]))


# ---- routing -------------------------------------------------------------------

def check_route(logits, k, ids, w, bias=None, score="softmax", groups=1, topk_groups=1,
                renormalize=True, scale=1.0):
    ri, rw = R.route(logits, k, bias, score, groups, topk_groups, renormalize, scale)
    assert np.array_equal(ids.cpu().numpy(), ri)
    # carried in 64 bits, rounded once to FP32
    got = w.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - rw) <= 1.01 * R.U * np.abs(rw) + 2.0 ** -149)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,kg", [
    (1, 1, 1, 1, 1), (3, 2, 2, 1, 1), (5, 7, 3, 1, 1), (4, 63, 4, 1, 1), (4, 64, 6, 8, 4),
    (9, 65, 65 - 1, 1, 1), (4, 160, 6, 8, 3), (4, 160, 8, 160 // 20, 2), (64, 256, 6, 1, 1),
    (33, 256, 8, 8, 4), (7, 256, 64, 4, 2), (5, 384, 8, 1, 1), (3, 384, 8, 64, 32),
    (2, 512, 9, 16, 16), (5, 1000, 7, 8, 1), (3, 1024, 64, 64, 9), (2, 6, 2, 6, 3)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route(dev, score, T, E, k, groups, kg, with_bias):
    g = gen("route", T, E, k)
    logits = 1.5 * torch.randn(T, E, generator=g)
    bias = 0.2 * torch.randn(E, generator=g) if with_bias else None
    for renorm, scale in ((True, 2.5), (False, 1.0)):
        ids, w = M.route_topk(logits.to(dev), k, bias=None if bias is None else bias.to(dev),
                              score=score, groups=groups, topk_groups=kg, renormalize=renorm,
                              scale=scale)
        check_route(logits, k, ids, w, bias, score, groups, kg, renorm, scale)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("groups,kg", [(1, 1), (8, 4)])
def test_route_ties_go_to_the_lower_index(dev, dt, groups, kg):
    """Coarse logits: many experts share a value, within and across groups."""
    g = gen("ties", groups)
    logits = (torch.randint(-3, 3, (50, 256), generator=g) * 0.5).to(dt)
    for score in ("softmax", "sigmoid"):
        ids, w = M.route_topk(logits.to(dev), 8, score=score, groups=groups, topk_groups=kg)
        check_route(logits, 8, ids, w, None, score, groups, kg)
        b = torch.full((256,), 0.25)
        ids, w = M.route_topk(logits.to(dev), 8, score=score, groups=groups, topk_groups=kg,
                              bias=b.to(dev))
        check_route(logits, 8, ids, w, b, score, groups, kg)


def test_route_near_ties_follow_64_bits(dev):
    """Scores that FP32 cannot tell apart: bias moves by less than its last bit would at 1."""
    g = gen("near")
    T, E = 200, 128
    logits = torch.full((T, E), 0.5) + torch.randint(-40, 40, (T, E), generator=g) * 2.0 ** -23
    bias = torch.randint(-40, 40, (E,), generator=g) * 2.0 ** -27
    ids, w = M.route_topk(logits.to(dev), 8, bias=bias.to(dev), score="sigmoid")
    check_route(logits, 8, ids, w, bias, "sigmoid")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kg", [(1, 1), (4, 2)])
def test_route_masked_and_non_finite(dev, score, groups, kg):
    INF = math.inf
    g = gen("mask")
    E, k = 64, 8
    logits = torch.randn(9, E, generator=g)
    logits[0] = -INF                                  # nothing left
    logits[1] = -INF
    logits[1, [3, 40]] = torch.tensor([0.5, -2.0])    # two of eight left
    logits[2] = torch.finfo(FF).min                   # masked by the lowest value: all equal
    logits[3] = torch.finfo(FF).min
    logits[3, 50] = 1.0
    logits[4, 7] = float("nan")                       # a NaN expert is out
    logits[5] = float("nan")
    logits[6, 9] = INF                                # counts as the largest finite
    logits[7, 16:48] = -INF                           # whole groups out
    bias = 0.1 * torch.randn(E, generator=g)
    for b in (None, bias):
        ids, w = M.route_topk(logits.to(dev), k, bias=None if b is None else b.to(dev), score=score,
                              groups=groups, topk_groups=kg)
        check_route(logits, k, ids, w, b, score, groups, kg)
        assert bool((ids[0] == -1).all()) and not bool(w[0].any())
        assert bool(torch.isfinite(w).all())
    out = torch.zeros(E)
    out[::2] = -INF                                   # experts taken out by the bias
    out[3] = INF
    ids, w = M.route_topk(logits[8:].to(dev), k, bias=out.to(dev), score=score)
    check_route(logits[8:], k, ids, w, out, score)
    assert int(ids[0, 0]) == 3 and bool((ids % 2 == 1).all())
    many = torch.zeros(256)                           # experts that are always on, all equal
    many[[5, 70, 71, 133, 200, 202, 255]] = INF
    wide = torch.randn(9, 256, generator=g)
    for gr, kgr in ((1, 1), (8, 3), (4, 4)):
        ids, w = M.route_topk(wide.to(dev), k, bias=many.to(dev), score=score, groups=gr,
                              topk_groups=kgr)
        check_route(wide, k, ids, w, many, score, gr, kgr)


@pytest.mark.parametrize("E", [128, 256, 1000])
def test_route_negative_and_equal_scores(dev, E):
    """A bias below zero turns the scores negative; a constant one leaves ties and zeros."""
    g = gen("negative", E)
    logits = torch.randn(40, E, generator=g)
    logits[:, ::7] = logits[:, :1]
    for bias in (torch.randn(E, generator=g) - 2, torch.full((E,), -0.5), -torch.rand(E, generator=g) * 1e4):
        for score in ("softmax", "sigmoid"):
            ids, w = M.route_topk(logits.to(dev), 7, bias=bias.to(dev), score=score)
            check_route(logits, 7, ids, w, bias, score)
    flat = torch.zeros(3, E)
    flat[1] = -0.0
    flat[2, ::2] = -0.0                               # -0 and +0 are one logit
    ids, w = M.route_topk(flat.to(dev), 9)
    check_route(flat, 9, ids, w)


def test_route_strided_rows(dev):
    logits = torch.randn(37, 100, generator=gen("rs"))
    ids, w = M.route_topk(strided(logits, dev, 3, 1), 5)
    check_route(logits, 5, ids, w)
    ld = 1_200_000_000
    buf = torch.empty(ld + 100, dtype=FF, device=dev)
    x = torch.as_strided(buf, (2, 100), (ld, 1))
    x.copy_(logits[:2])
    ids, w = M.route_topk(x, 5, score="sigmoid")
    check_route(logits[:2], 5, ids, w, None, "sigmoid")


# ---- 8-bit product ---------------------------------------------------------------

def check_gemm(a, sa, w, sw, add, out):
    p, ref = R.gemm(a, sa, w, sw, add)
    dt = out.dtype
    # int -> FP32, two scales: 3 roundings of the product; the addition one of the result; then
    # one to the output type
    bound = (R.half_step(dt) if dt != FF else 0) * ref.abs() + 4 * R.U * (p.abs() + ref.abs())
    bound = bound * (1 + 2.0 ** -8) + R.smallest(dt)
    off = (out.cpu().to(R.F) - ref).abs()
    assert bool((off <= bound).all()), float((off - bound).max())


def operands(T, N, K, key):
    g = gen("gemm", T, N, K, key)
    a = torch.randint(-127, 128, (T, K), generator=g, dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8)
    sa = torch.rand(T, generator=g) * 0.02 + 1e-3
    sw = torch.rand(N, generator=g) * 0.01 / math.sqrt(K) + 1e-4
    return a, sa, w, sw, g


SIZES = [(1, 1, 1), (1, 16, 64), (3, 5, 7), (4, 64, 128), (1, 4096, 4096), (4, 1000, 4096),
         (15, 33, 1024), (16, 48, 320), (17, 128, 2048), (33, 16, 16), (63, 40, 8192), (64, 256, 2048),
         (65, 128, 256), (100, 257, 512), (127, 127, 127), (128, 128, 128), (129, 130, 144),
         (200, 511, 1040), (256, 256, 4096), (300, 2056, 320), (513, 384, 2048), (1, 7, 131071),
         (70, 20, 131056), (1000, 24, 48), (2049, 300, 256), (70, 70, 100)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("dt", [BF, HF, FF])
def test_gemm(dev, T, N, K, dt):
    a, sa, w, sw, g = operands(T, N, K, "")
    ws = M.gemm_w8a8_workspace_for(T, N, K, dev)
    d = [v.to(dev) for v in (a, sa, w, sw)]
    out = M.gemm_w8a8(*d, out_dtype=dt, workspace=ws)
    check_gemm(a, sa, w, sw, None, out)
    add = torch.randn(T, N, generator=g).to(dt)
    out = M.gemm_w8a8(*d, addend=add.to(dev), out_dtype=dt, workspace=ws)
    check_gemm(a, sa, w, sw, add, out)
    acc = add.to(dev)
    assert M.gemm_w8a8(*d, addend=acc, out=acc, out_dtype=dt) is acc     # own workspace, in place
    assert torch.equal(acc, out)


@pytest.mark.parametrize("T,N,K", [(4200, 2050, 512), (4096, 4096, 272), (6200, 2304, 144),
                                   (2040, 2050, 4112), (4090, 4090, 1040), (1020, 4070, 2064),
                                   (510, 4080, 2064), (250, 2000, 2064), (2040, 4090, 1040),
                                   (2047, 2056, 400), (1900, 3000, 784)])
def test_gemm_large_tiles(dev, T, N, K):
    a, sa, w, sw, g = operands(T, N, K, "large")
    add = torch.randn(T, N, generator=g).to(BF)
    out = M.gemm_w8a8(a.to(dev), sa.to(dev), w.to(dev), sw.to(dev), addend=add.to(dev))
    check_gemm(a, sa, w, sw, add, out)


@pytest.mark.parametrize("T,N,K", [(128, 512, 4112), (66, 150, 16400), (300, 130, 6160), (100, 64, 8208),
                                   (70, 20, 131056)])
def test_gemm_split_k(dev, T, N, K):
    """Few output tiles and a long K: K is split, and the sums are joined in the workspace, whose
    counters are back at zero after every call."""
    assert M.moe_wna16_gemm_w8a8_workspace_size(T, N, K) > 0
    ws = M.gemm_w8a8_workspace_for(T, N, K, dev)
    ws[4096:] = 0x5A                                    # only the counters start at zero
    for i in range(4):
        a, sa, w, sw, g = operands(T, N, K, i)
        add = torch.randn(T, N, generator=g).to(HF) if i % 2 else None
        out = M.gemm_w8a8(a.to(dev), sa.to(dev), w.to(dev), sw.to(dev), out_dtype=HF, workspace=ws,
                          addend=None if add is None else add.to(dev))
        check_gemm(a, sa, w, sw, add, out)
        assert not bool(ws[:4096].any())
    assert torch.equal(out, M.gemm_w8a8(a.to(dev), sa.to(dev), w.to(dev), sw.to(dev), out_dtype=HF,
                                        addend=add.to(dev)))     # a workspace of its own


def test_gemm_split_k_graph_replays(dev):
    T, N, K = 90, 130, 8192
    a, sa, w, sw, g = operands(T, N, K, "graph")
    d = [v.to(dev) for v in (a, sa, w, sw)]
    for ws in (M.gemm_w8a8_workspace_for(T, N, K, dev), None):
        M.gemm_w8a8(*d, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = M.gemm_w8a8(*d, workspace=ws)
        for _ in range(4):
            d[0].copy_(torch.randint(-127, 128, (T, K), generator=g, dtype=torch.int8))
            want = M.gemm_w8a8(*d)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(want, held)
            check_gemm(d[0].cpu(), sa, w, sw, None, held)


def test_gemm_extreme_codes_fill_int32(dev):
    """All products at -128 * -128 over the longest K: the sum is 2147467264, just inside int32."""
    K = 131071
    for T in (2, 70):
        a = torch.full((T, K), -128, dtype=torch.int8)
        w = torch.full((18, K), -128, dtype=torch.int8)
        sa, sw = torch.full((T,), 2.0 ** -20), torch.ones(18)
        out = M.gemm_w8a8(a.to(dev), sa.to(dev), w.to(dev), sw.to(dev), out_dtype=FF)
        check_gemm(a, sa, w, sw, None, out)


@pytest.mark.parametrize("T", [5, 40, 300, 2100])
@pytest.mark.parametrize("pad,offset", [(16, 0), (16, 32), (1, 0), (0, 1), (7, 3)])
def test_gemm_strided_and_unaligned(dev, T, pad, offset):
    N, K = 150, 336
    a, sa, w, sw, g = operands(T, N, K, "strided")
    add = torch.randn(T, N, generator=g).to(BF)
    out = strided(torch.zeros(T, N, dtype=BF), dev, 6, 1)
    got = M.gemm_w8a8(strided(a, dev, pad, offset), sa.to(dev), strided(w, dev, pad, offset),
                      sw.to(dev), addend=strided(add, dev, 3, 2), out=out)
    assert got is out
    check_gemm(a, sa, w, sw, add, out)
    gap = torch.as_strided(out, (T - 1, 6), (N + 6, 1), out.storage_offset() + N)
    assert bool(torch.isnan(gap).all())


@pytest.mark.parametrize("T,N,K", [(1, 40, 1), (3, 5000, 4090), (8, 100, 15), (13, 100, 2063), (16, 4200, 777),
                                   (27, 333, 3001), (64, 130, 2050), (64, 40, 16399),
                                   (65, 40, 17), (100, 700, 127), (90, 300, 129), (128, 512, 4090),
                                   (66, 20, 131071), (300, 130, 6161), (513, 384, 257), (510, 4080, 1030),
                                   (2047, 2056, 401), (2040, 2050, 1001), (4090, 4090, 385), (4200, 2050, 523),
                                   (6200, 2304, 133), (1020, 4070, 2063), (2040, 4090, 1039)])
def test_gemm_odd_lengths(dev, T, N, K):
    """K at which no row but the first begins at a multiple of 16 bytes, for every tile and split: what
    follows a row in memory (the next row's codes) is not counted."""
    a, sa, w, sw, g = operands(T, N, K, "odd")
    ws = M.gemm_w8a8_workspace_for(T, N, K, dev)
    if ws is not None:
        ws[4096:] = 0x5A
    add = torch.randn(T, N, generator=g).to(BF)
    d = [v.to(dev) for v in (a, sa, w, sw)]
    for _ in range(2):
        out = M.gemm_w8a8(*d, addend=add.to(dev), workspace=ws)
        check_gemm(a, sa, w, sw, add, out)
    assert ws is None or not bool(ws[:4096].any())
    # operands at odd addresses, and one aligned with the other not
    o = torch.empty(T * K + 1, dtype=torch.int8, device=dev)[1:].view(T, K).copy_(a)
    assert torch.equal(out, M.gemm_w8a8(o, *d[1:], addend=add.to(dev)))


def test_gemm_row_offsets_past_32_bits(dev):
    T, N, K, ld = 620, 80, 160, (1 << 23) - 16
    a, sa, w, sw, _ = operands(T, N, K, "far")
    buf = torch.empty((T - 1) * ld + K, dtype=torch.int8, device=dev)
    far = torch.as_strided(buf, (T, K), (ld, 1))
    far.copy_(a)
    out = M.gemm_w8a8(far, sa.to(dev), w.to(dev), sw.to(dev), out_dtype=FF)
    check_gemm(a, sa, w, sw, None, out)


def test_gemm_non_finite_scales_stay_in_their_row(dev):
    for T in (6, 90):
        a, sa, w, sw, _ = operands(T, 48, 256, "nan")
        sa[2] = float("nan")
        out = M.gemm_w8a8(a.to(dev), sa.to(dev), w.to(dev), sw.to(dev)).cpu()
        assert bool(torch.isnan(out[2]).all())
        out[2] = 0
        assert bool(torch.isfinite(out).all())


# ---- refusals, empty calls, streams, graphs --------------------------------------------------

def test_refusals_name_the_argument(dev):
    x = torch.zeros(4, 64, dtype=BF, device=dev)
    w, f = torch.ones(64, dtype=BF, device=dev), torch.ones(4, device=dev)
    i8 = torch.zeros(4, 64, dtype=torch.int8, device=dev)
    for call, kind, what in (
            (lambda: M.add_rmsnorm(x, w.float()), TypeError, "weight"),
            (lambda: M.add_rmsnorm(x, w[:32]), ValueError, "weight"),
            (lambda: M.add_rmsnorm(x, w.cpu()), ValueError, "weight"),
            (lambda: M.add_rmsnorm(x.double(), w.double()), TypeError, "x"),
            (lambda: M.add_rmsnorm(x, w, x[:2]), ValueError, "residual"),
            (lambda: M.add_rmsnorm(x.t(), w[:4]), ValueError, "x"),
            (lambda: M.add_rmsnorm(x[:1].expand(4, 64), w), ValueError, "x"),
            (lambda: M.add_rmsnorm(x, w, out=x[:, :32]), ValueError, "out"),
            (lambda: M.add_rmsnorm(x, w, quant=True, q=x), TypeError, "q"),
            (lambda: M.add_rmsnorm(x, w, quant=True, scale=f[:3]), ValueError, "scale"),
            (lambda: M.add_rmsnorm(x, w, eps="a"), TypeError, "number"),
            (lambda: M.add_rmsnorm(x, w, eps=-1.0), M.MoeWna16Error, "moe_wna16_add_rmsnorm"),
            (lambda: M.route_topk(x, 65), M.MoeWna16Error, "moe_wna16_route_topk"),
            (lambda: M.route_topk(x, 0), ValueError, "topk"),
            (lambda: M.route_topk(x, 2, score="tanh"), ValueError, "score"),
            (lambda: M.route_topk(x, 2, score=3), TypeError, "score"),
            (lambda: M.route_topk(x, 2, bias=w), TypeError, "bias"),
            (lambda: M.route_topk(x, 2, groups=3), M.MoeWna16Error, "route_topk"),
            (lambda: M.route_topk(x, 2, ids=torch.zeros(4, 2, device=dev)), TypeError, "ids"),
            (lambda: M.gemm_w8a8(x, f, i8, f), TypeError, "a has"),
            (lambda: M.gemm_w8a8(i8, f, i8[:, :32], f), ValueError, "w"),
            (lambda: M.gemm_w8a8(i8, f[:2], i8, f), ValueError, "a_scale"),
            (lambda: M.gemm_w8a8(i8, f, i8, f, addend=x[:, :4].float()), TypeError, "addend"),
            (lambda: M.gemm_w8a8(i8, f, i8, f, out_dtype=torch.int8), TypeError, "out_dtype"),
            (lambda: M.gemm_w8a8(i8, f, i8, f, out_dtype=2), TypeError, "out_dtype"),
            (lambda: M.gemm_w8a8(i8, f, i8, f, out=x), ValueError, "out"),
            (lambda: M.gemm_w8a8(i8, f, i8, f, workspace=f), TypeError, "workspace"),
            (lambda: M.swiglu_quant(x[:, :63]), ValueError, "gu"),
            (lambda: M.swiglu_quant(x, clamp=-1.0), M.MoeWna16Error, "swiglu_quant"),
            (lambda: M.swiglu_quant(x, q=i8), ValueError, "q")):
        with pytest.raises(kind, match=what):
            call()


def test_empty(dev):
    z = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device=dev)  # noqa: E731
    got = M.add_rmsnorm(z(0, 64), z(64), z(0, 64), quant=True)
    assert got["q"].shape == (0, 64) and got["scale"].shape == (0,)
    ids, w = M.route_topk(z(0, 16), 2)
    assert ids.shape == w.shape == (0, 2)
    i8, f = torch.int8, FF
    assert M.gemm_w8a8(z(0, 32, dtype=i8), z(0, dtype=f), z(8, 32, dtype=i8), z(8, dtype=f)).shape == (0, 8)
    assert M.gemm_w8a8(z(3, 32, dtype=i8), z(3, dtype=f), z(0, 32, dtype=i8), z(0, dtype=f)).shape == (3, 0)
    q, s = M.swiglu_quant(z(0, 64))
    assert q.shape == (0, 32) and s.shape == (0,)


def block(x, r, wn, gate, bias, w13, s13, w2, s2):
    """Norm, routing and shared expert, as a step runs them."""
    n = M.add_rmsnorm(x, wn, r, quant=True)
    ids, w = M.route_topk(torch.mm(n["y"].float(), gate), 4, bias=bias, score="sigmoid", groups=4,
                          topk_groups=2)
    gu = M.gemm_w8a8(n["q"], n["scale"], w13, s13)
    q, s = M.swiglu_quant(gu)
    return n["residual"], ids, w, M.gemm_w8a8(q, s, w2, s2, addend=n["y"])


def block_inputs(T, dev):
    H, I, E = 512, 256, 32
    g = gen("block", T)
    i8 = lambda n, k: torch.randint(-127, 128, (n, k), generator=g, dtype=torch.int8).to(dev)  # noqa: E731
    sc = lambda n, k: (torch.rand(n, generator=g) * 0.02 / math.sqrt(k)).to(dev)  # noqa: E731
    return [torch.randn(T, H, generator=g).to(BF).to(dev), torch.randn(T, H, generator=g).to(BF).to(dev),
            torch.ones(H, dtype=BF, device=dev), (torch.randn(H, E, generator=g) / 20).to(dev),
            (0.1 * torch.randn(E, generator=g)).to(dev), i8(2 * I, H), sc(2 * I, H), i8(H, I), sc(H, I)]


@pytest.mark.parametrize("T", [3, 200])
def test_another_stream(dev, T):
    args = block_inputs(T, dev)
    want = block(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        moved = [a.clone() for a in args]       # produced on the stream that consumes them
        got = block(*moved)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [2, 48, 130])
def test_graph_replays(dev, T):
    args = block_inputs(T, dev)
    block(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(*args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block(*args)
    g = gen("replay", T)
    for _ in range(4):
        args[0].copy_(torch.randn(args[0].shape, generator=g).to(BF))
        args[1].copy_(torch.randn(args[1].shape, generator=g).to(BF))
        want = block(*args)                     # eager work between replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, held):
            assert torch.equal(a, b)
