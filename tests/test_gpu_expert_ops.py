"""The operators for experts in 8-bit floating point on the GPU against 64-bit
references (tests/_expert.py), over types, sizes, strides, masks and non-finite
values."""
import pytest
import torch

import weight_only_bit_moe_amd as M
from tests import _expert as R
from tests.test_gpu_block_ops import gen

pytestmark = pytest.mark.gpu

BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


def padded(t, dev, pad, fill=float("nan")):
    """t [.., T, n] on the GPU with rows pad elements further apart; the gaps hold `fill`."""
    T, n = t.shape[-2:]
    if t.dtype == R.E4M3:
        buf = torch.full((*t.shape[:-2], T, n + pad), 0x7f, dtype=torch.uint8, device=dev)
        v = buf[..., :n]
        v.copy_(t.view(torch.uint8))
        return v.view(R.E4M3)
    buf = torch.full((*t.shape[:-2], T, n + pad), fill, dtype=t.dtype, device=dev)
    buf[..., :n].copy_(t)
    return buf[..., :n]


def numbers(q):
    return q.cpu().to(FF).to(R.F)


# ---- rows in e4m3 ----------------------------------------------------------------

@pytest.mark.parametrize("dt", [BF, HF, FF])
@pytest.mark.parametrize("T,K", [(1, 1), (3, 7), (2, 127), (5, 128), (4, 129), (7, 1000), (3, 4096),
                                 (2, 5119), (1, 32769), (1030, 96), (2, 131072)])
def test_quant(dev, dt, T, K):
    x = (torch.randn(T, K, generator=gen("q8", T, K)) * 3).to(dt)
    x[0, 0] = 448 if K < 200 else 1.75            # a largest value that just fits its scale
    q, s = M.quant_fp8(x.to(dev))
    rq, rs = R.codes(x.to(R.F))
    assert q.dtype == R.E4M3 and s.shape == (T, R.blocks(K))
    assert torch.equal(s.cpu().to(R.F), rs) and torch.equal(numbers(q), rq)


@pytest.mark.parametrize("dt", [BF, HF])
def test_quant_of_every_value(dev, dt):
    """All finite values of the type, each in blocks of its own exponents' range, and ties."""
    bits = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16)
    v = bits.view(dt)
    v = v[torch.isfinite(v)]
    v = torch.cat([v, v[:-v.numel() % 128]]) if v.numel() % 128 else v
    x = v[:v.numel() // 128 * 128].view(-1, 128)
    q, s = M.quant_fp8(x.to(dev))
    rq, rs = R.codes(x.to(R.F))
    assert torch.equal(s.cpu().to(R.F), rs) and torch.equal(numbers(q), rq)


def test_quant_strided_zero_tiny_and_non_finite(dev):
    x = torch.randn(6, 300, generator=gen("q8e"))
    x[0] = 0
    x[1] = 2.0 ** -140                              # below what the smallest scale holds
    x[2, 17] = float("nan")
    x[3, 299] = -float("inf")
    x[4] = 3.0e38
    q = padded(torch.zeros(6, 300).to(R.E4M3), dev, 5)
    s = padded(torch.zeros(6, 3), dev, 2)
    got = M.quant_fp8(padded(x, dev, 7), q=q, scale=s)
    assert got[0] is q and got[1] is s
    rq, rs = R.codes(x.to(R.F))
    assert torch.equal(numbers(q), rq)
    assert torch.equal(torch.nan_to_num(s.cpu().to(R.F), nan=-1), torch.nan_to_num(rs, nan=-1))
    assert bool(torch.isnan(s[2, 0])) and bool(torch.isnan(s[3, 2])) and not bool(torch.isnan(s[3, 0]))
    gap = torch.as_strided(q.view(torch.uint8), (6, 5), (305, 1), 300)
    assert bool((gap == 0x7f).all())
    gap = torch.as_strided(s, (6, 2), (5, 1), 3)
    assert bool(torch.isnan(gap).all())


@pytest.mark.parametrize("dt", [BF, HF, FF])
@pytest.mark.parametrize("T,I", [(1, 1), (3, 130), (4, 512), (5, 777), (2, 2048), (700, 64)])
@pytest.mark.parametrize("alpha,beta,clamp", [(1.0, 0.0, None), (1.702, 1.0, 7.0)])
def test_swiglu_quant(dev, dt, T, I, alpha, beta, clamp):
    gu = (4 * torch.randn(T, 2 * I, generator=gen("sq8", T, I))).to(dt)
    q, s = M.swiglu_quant_fp8(padded(gu, dev, 3), alpha=alpha, beta=beta, clamp=clamp)
    a, g = R.swiglu(gu, alpha, beta, clamp)
    # as for the activation in 8-bit integers: alpha g rounded before the exponential, and ten steps
    rel = (10 + (alpha * g).abs().amax()) * R.U
    s = s.cpu().to(R.F)
    top = torch.zeros(T, R.blocks(I) * 128, dtype=R.F)
    top[:, :I] = a.abs()
    top = top.view(T, -1, 128).amax(-1)
    # a power of two under which the block fits (up to the error of its largest value), half of which
    # it would not; blocks whose largest value is below the smallest scale's reach have that
    assert torch.equal(torch.exp2(torch.round(torch.log2(s))), s)
    assert bool((top <= 448 * s * (1 + 2 * rel)).all())
    small = s == 2.0 ** -126
    assert bool((small | (top * (1 + 2 * rel) > 224 * s)).all())
    step = s.repeat_interleave(128, 1)[:, :I]
    # half a step of e4m3: 2^-4 of the value, or 2^-10 below the normal ones
    off = (numbers(q) * step - a).abs()
    assert bool((off <= (2.0 ** -4 + 2 * rel) * a.abs() + 2.0 ** -10 * step + rel * a.abs()).all())


def test_swiglu_quant_non_finite(dev):
    gu = torch.randn(3, 512, generator=gen("sqn"))
    gu[0, 3] = float("nan")
    gu[1, 256 + 200] = float("inf")
    q, s = M.swiglu_quant_fp8(gu.to(dev))
    nan = torch.isnan(s.cpu())
    assert nan.tolist() == [[True, False], [False, True], [False, False]]
    assert not numbers(q)[0, :128].any() and not numbers(q)[1, 128:].any()
    assert bool(numbers(q)[0, 128:].any())


# ---- product ---------------------------------------------------------------------

def operands(key, T, N, K, E=None, wide=False):
    g = gen("g8", key, T, N, K)
    a, sa = R.random_codes(g, T, K), torch.exp2(torch.randint(-9, 3, (T, R.blocks(K)), generator=g).float())
    n = (E, N, K) if E else (N, K)
    w = R.random_codes(g, *n)
    sw = torch.rand(*n[:-2], R.blocks(N), R.blocks(K), generator=g) * 1e-2
    if wide:                                        # scales far apart, negative and zero ones
        sa = sa * torch.randn(sa.shape, generator=g)
        sw = torch.where(torch.rand(sw.shape, generator=g) < 0.2, torch.zeros_like(sw), sw)
    return a, sa, w, sw, g


def check_product(got, a, sa, w, sw, dt, add=None):
    exact, terms, groups = R.product(a, sa, w, sw, add)
    assert got.dtype == dt and got.shape == exact.shape
    off = (got.cpu().to(R.F) - exact).abs()
    b = R.product_bound(exact, terms, groups, a.shape[1], dt, add)
    assert bool((off <= b).all()), float((off - b).max())


SIZES = [(1, 1, 16), (1, 16, 128), (2, 17, 144), (3, 130, 256), (7, 256, 2048), (8, 100, 400), (9, 129, 1040),
         (16, 64, 4096), (17, 256, 512), (31, 33, 640), (33, 200, 1008), (64, 512, 2048), (65, 70, 112),
         (65, 130, 1024), (100, 257, 272), (128, 512, 4096), (129, 300, 1936), (200, 1025, 528),
         (257, 256, 1152), (300, 640, 4064), (513, 1100, 384), (1000, 264, 2048), (1111, 2049, 400),
         (2048, 2048, 1024), (3, 8200, 256), (12, 4500, 128), (2500, 2500, 144),
         (1280, 4096, 272), (3000, 1536, 400), (1500, 3000, 528), (4100, 4097, 144), (2047, 2057, 4048)]


@pytest.mark.parametrize("T,N,K", SIZES)
def test_gemm(dev, T, N, K):
    a, sa, w, sw, g = operands("p", T, N, K)
    for dt in (BF, FF):
        check_product(M.gemm_fp8(a.to(dev), sa.to(dev), w.to(dev), sw.to(dev), out_dtype=dt),
                      a, sa, w, sw, dt)
    add = (torch.randn(T, N, generator=g) * 20).to(HF)
    out = add.to(dev)
    got = M.gemm_fp8(a.to(dev), sa.to(dev) * 2.0 ** -8, w.to(dev), sw.to(dev), addend=out, out=out, out_dtype=HF)
    assert got is out
    check_product(got, a, sa * 2.0 ** -8, w, sw, HF, add)


@pytest.mark.parametrize("T,N,K", [(5, 200, 272), (40, 129, 1040), (150, 300, 528), (700, 1025, 1936)])
def test_gemm_strided(dev, T, N, K):
    a, sa, w, sw, g = operands("s", T, N, K, wide=True)
    add = torch.randn(T, N, generator=g).to(BF)
    out = padded(torch.zeros(T, N, dtype=BF), dev, 3)
    got = M.gemm_fp8(padded(a, dev, 16), padded(sa, dev, 1), padded(w, dev, 48), padded(sw, dev, 2),
                     addend=padded(add, dev, 5), out=out, out_dtype=BF)
    check_product(got, a, sa, w, sw, BF, add)
    gap = torch.as_strided(out, (T, 3), (N + 3, 1), N)
    assert bool(torch.isnan(gap).all())


@pytest.mark.parametrize("T,N,K", [(4, 64, 256), (70, 140, 400), (600, 520, 1040)])
def test_gemm_carries_nan_where_it_belongs(dev, T, N, K):
    a, sa, w, sw, _ = operands("n", T, N, K)
    a.view(torch.uint8)[1, K - 1] = 0x7f                # a token's last code
    sa[2, 0] = float("nan")                             # what quant_fp8 gives a block it cannot hold
    w.view(torch.uint8)[3, 5] = 0xff                    # a channel's
    got = M.gemm_fp8(a.to(dev), sa.to(dev), w.to(dev), sw.to(dev), out_dtype=FF).cpu()
    want = torch.zeros(T, N, dtype=torch.bool)
    want[1:3] = True
    want[:, 3] = True
    assert torch.equal(torch.isnan(got), want)


def test_gemm_every_finite_code_pair_is_exact(dev):
    """One product a sum: a[t] = 2^i-scaled codes against one code of w, exact in FP32."""
    c = torch.arange(256, dtype=torch.int32)
    c = c[(c & 127) != 127].to(torch.uint8).view(R.E4M3)            # 254 codes
    a = torch.zeros(254, 128).to(R.E4M3)
    a.view(torch.uint8)[:, 77] = c.view(torch.uint8)
    w = torch.zeros(254, 128).to(R.E4M3)
    w.view(torch.uint8)[:, 77] = c.view(torch.uint8)
    one = torch.ones(254, 1)
    got = M.gemm_fp8(a.to(dev), one.to(dev), w.to(dev), torch.ones(2, 1, device=dev), out_dtype=FF)
    v = numbers(c)
    assert torch.equal(got.cpu().to(R.F), v[:, None] * v)


def test_gemm_gives_the_same_bits(dev):
    for T, N, K in ((4, 512, 4096), (128, 512, 16384), (300, 700, 2048)):
        a, sa, w, sw, _ = operands("b", T, N, K)
        a, sa, w, sw = (t.to(dev) for t in (a, sa, w, sw))
        first = M.gemm_fp8(a, sa, w, sw, out_dtype=FF)
        ws = M.gemm_fp8_workspace_for(T, N, K, dev)
        for _ in range(3):
            assert torch.equal(M.gemm_fp8(a, sa, w, sw, out_dtype=FF, workspace=ws), first)
        if ws is not None:
            assert not ws[:4096].any()


# ---- product by expert -------------------------------------------------------------

def counts_of(key, E, R_, g):
    """Rows of each expert: some none, some many."""
    if key == "even":
        return torch.full((E,), R_ // E)
    if key == "one":
        c = torch.zeros(E, dtype=torch.int64)
        c[E // 2] = R_
        return c
    w = torch.rand(E, generator=g) ** 4
    c = torch.floor(w / w.sum() * R_).long()
    c[0] = 0
    return c


@pytest.mark.parametrize("E,N,K", [(1, 130, 272), (8, 256, 512), (65, 144, 128), (256, 33, 144), (130, 260, 1040)])
@pytest.mark.parametrize("R_", [1, 5, 40, 300, 1500, 4000])
@pytest.mark.parametrize("key", ["even", "one", "skewed"])
def test_grouped(dev, E, N, K, R_, key):
    g = gen("gr", E, N, K, R_, key)
    counts = counts_of(key, E, R_, g)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32)
    used = int(off[-1])
    tokens = max(1, R_ // 3)
    a, sa, w, sw, _ = operands("gr", tokens, N, K, E, wide=True)
    rows = torch.full((R_,), -1, dtype=torch.int32)
    rows[:used] = torch.randint(0, tokens, (used,), generator=g, dtype=torch.int32)
    out = torch.full((R_, N), 7.0, dtype=BF, device=dev)
    got = M.gemm_fp8_grouped(a.to(dev), sa.to(dev), w.to(dev), sw.to(dev), off.to(dev), rows=rows.to(dev), out=out)
    assert got is out and bool((out[used:] == 7).all())
    xs, ss = a[rows[:used].long()], sa[rows[:used].long()]
    for e in torch.nonzero(counts).view(-1).tolist():
        part = slice(int(off[e]), int(off[e + 1]))
        check_product(out[part], xs[part], ss[part], w[e], sw[e], BF)
    if R_ <= 300 and used:                              # rows already in order, strided, FP32
        full = torch.zeros(R_, K).to(R.E4M3)
        full.view(torch.uint8)[:used] = xs.view(torch.uint8)
        fs = torch.ones(R_, R.blocks(K))
        fs[:used] = ss
        got = M.gemm_fp8_grouped(padded(full, dev, 32), padded(fs, dev, 1), padded(w, dev, 16), padded(sw, dev, 3),
                                 off.to(dev), out_dtype=FF)
        for e in torch.nonzero(counts).view(-1).tolist():
            part = slice(int(off[e]), int(off[e + 1]))
            check_product(got[part], xs[part], ss[part], w[e], sw[e], FF)


def test_grouped_offsets_and_rows_out_of_range_are_held_inside(dev):
    """Offsets past the rows end at them; rows outside a are read as its row 0."""
    a, sa, w, sw, _ = operands("oob", 4, 64, 128, 3)
    off = torch.tensor([-5, 2, 99, 50], dtype=torch.int32)
    rows = torch.tensor([0, 1, 400, -7, 3], dtype=torch.int32)
    out = M.gemm_fp8_grouped(a.to(dev), sa.to(dev), w.to(dev), sw.to(dev), off.to(dev), rows=rows.to(dev))
    check_product(out[:2], a[:2], sa[:2], w[0], sw[0], BF)
    at = torch.tensor([0, 0, 3])
    check_product(out[2:], a[at], sa[at], w[1], sw[1], BF)


# ---- sort and combine ----------------------------------------------------------------

def some_ids(key, T, k, E, out_of=True):
    g = gen("ids", key, T, k, E)
    lo, hi = (-1, E + 2) if out_of else (0, E)
    return torch.randint(lo, hi, (T, k), generator=g, dtype=torch.int32)


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 6, 256), (3, 2, 3), (4, 6, 256), (64, 6, 256), (63, 64, 7),
                                   (129, 8, 1024), (700, 1, 5), (1024, 8, 64), (1025, 8, 64), (1366, 6, 256),
                                   (2048, 6, 1000), (3000, 3, 1), (5000, 8, 256), (20000, 1, 300), (300, 64, 16)])
@pytest.mark.parametrize("H", [0, 1, 96, 1031])
def test_sort(dev, T, k, E, H):
    ids = some_ids("s", T, k, E)
    x = torch.randn(T, H, generator=gen("sx", T)).to(BF) if H else None
    out = torch.full((T * k, H), 7.0, dtype=BF, device=dev) if H else None
    r = M.sort_tokens(ids.to(dev), E, None if x is None else padded(x, dev, 5), out=out)
    tokens, slots, offsets = R.sort(ids, E)
    assert torch.equal(r["offsets"].cpu(), offsets)
    assert torch.equal(r["tokens"].cpu(), tokens) and torch.equal(r["slots"].cpu(), slots)
    assert ("x" in r) == bool(H)
    if H:
        used = int(offsets[-1])
        assert torch.equal(r["x"][:used].cpu(), x[tokens[:used].long()])
        assert bool((r["x"][used:] == 7).all())


@pytest.mark.parametrize("dt", [BF, HF, FF])
@pytest.mark.parametrize("T,k,E,H", [(5, 3, 4, 33), (4, 6, 256, 4096), (700, 8, 64, 520), (2000, 6, 16, 128)])
def test_sort_gradient(dev, dt, T, k, E, H):
    g = gen("sg", T, k)
    ids = some_ids("sg", T, k, E)
    x = torch.randn(T, H, generator=g).to(dt).to(dev).requires_grad_()
    r = M.sort_tokens(ids.to(dev), E, x)
    tokens, slots, offsets = R.sort(ids, E)
    used = int(offsets[-1])
    assert torch.equal(r["x"][:used].cpu(), x.detach().cpu()[tokens[:used].long()])
    assert not r["slots"].requires_grad
    d = torch.randn(T * k, H, generator=g).to(dt)
    d[used:] = float("nan")                             # of rows that nobody has
    (dx,) = torch.autograd.grad(r["x"], x, d.to(dev))
    exact, terms = R.combine(d, slots)
    off = (dx.cpu().to(R.F) - exact).abs()
    assert dx.dtype == dt
    assert bool((off <= k * R.U * terms + 1.001 * R.half_step(dt) * exact.abs() + R.smallest(dt)).all())


def combine_case(key, dt, T, k, R_, H):
    """Slots that name a row of y at most once, some none."""
    g = gen("cc", key, T, k, R_, H)
    perm = torch.randperm(max(R_, T * k), generator=g)[:T * k].to(torch.int32).view(T, k)
    slots = torch.where(perm < R_, perm, torch.full_like(perm, -1))
    slots = torch.where(torch.rand(T, k, generator=g) < 0.1, torch.full_like(slots, R_ + 3), slots)
    y = torch.randn(R_, H, generator=g).to(dt)
    w = torch.randn(T, k, generator=g)
    return g, slots, y, w


COMBINE = [(1, 1, 1, 1), (3, 2, 6, 9), (4, 6, 24, 4096), (5, 9, 40, 33), (64, 8, 700, 513), (300, 6, 1500, 2050),
           (7, 64, 448, 100), (2, 3, 0, 16), (9, 2, 18, 9000), (3, 2, 5, 32768)]


@pytest.mark.parametrize("dt", [BF, HF, FF])
@pytest.mark.parametrize("T,k,R_,H", COMBINE)
def test_combine(dev, dt, T, k, R_, H):
    g, slots, y, w = combine_case("c", dt, T, k, R_, H)
    add = torch.randn(T, H, generator=g).to(dt)
    for weights, addend in ((w, None), (w, add), (None, None)):
        out = padded(torch.zeros(T, H, dtype=dt), dev, 2)
        if addend is not None:
            out.copy_(addend)
        got = M.combine_tokens(padded(y, dev, 3), slots.to(dev), None if weights is None else weights.to(dev),
                               addend=None if addend is None else out, out=out)
        assert got is out
        exact, terms = R.combine(y, slots, weights, addend)
        off = (got.cpu().to(R.F) - exact).abs()
        assert bool((off <= (k + 1) * R.U * terms + 1.001 * R.half_step(dt) * exact.abs() + R.smallest(dt)).all())


@pytest.mark.parametrize("dt", [BF, HF, FF])
@pytest.mark.parametrize("T,k,R_,H", COMBINE)
@pytest.mark.parametrize("with_offsets", [False, True])
def test_combine_gradient(dev, dt, T, k, R_, H, with_offsets):
    g, slots, y, w = combine_case("cg", dt, T, k, R_, H)
    if with_offsets:                                    # the first `used` rows have slots, as after a sort
        used = min(R_, T * k)
        slots = torch.full((T * k,), -1, dtype=torch.int32)
        slots[:used] = torch.randperm(used, generator=g).to(torch.int32)
        slots = slots.view(T, k)
        used -= used // 3
        slots[slots >= used] = -1
    add = torch.randn(T, H, generator=g).to(dt)
    yd, wd, ad = (t.to(dev).requires_grad_() for t in (y, w, add))
    off = torch.tensor([0, used // 2, used], dtype=torch.int32, device=dev) if with_offsets else None
    out = M.combine_tokens(yd, slots.to(dev), wd, offsets=off, addend=ad)
    d = torch.randn(T, H, generator=g).to(dt)
    dy, dw, dadd = torch.autograd.grad(out, (yd, wd, ad), d.to(dev))
    here = (slots >= 0) & (slots < R_)
    rows = torch.zeros(T, k, H, dtype=R.F)
    rows[here] = y.to(R.F)[slots[here].long()]
    edw = (rows * d.to(R.F)[:, None]).sum(-1)
    # dot products of H terms: each of at most H additions and products rounds once
    bound = (H + 1) * R.U * (rows * d.to(R.F)[:, None]).abs().sum(-1)
    assert dw.dtype == FF and bool(((dw.cpu().to(R.F) - edw).abs() <= bound).all())
    edy = torch.zeros(R_, H, dtype=R.F)
    t, j = torch.nonzero(here, as_tuple=True)
    edy[slots[t, j].long()] = w.to(R.F)[t, j][:, None] * d.to(R.F)[t]
    err = (dy.cpu().to(R.F) - edy).abs()
    assert bool((err <= (1.001 * R.half_step(dt) + R.U) * edy.abs() + R.smallest(dt)).all())
    assert torch.equal(dadd.cpu(), d)


def test_gradients_one_at_a_time(dev):
    _, slots, y, w = combine_case("one", FF, 6, 2, 12, 40)
    y, w, s = y.to(dev), w.to(dev), slots.to(dev)
    full = M.combine_tokens(y, s, w)
    for which in ("y", "w"):
        a, b = y.clone().requires_grad_(which == "y"), w.clone().requires_grad_(which == "w")
        out = M.combine_tokens(a, s, b)
        assert torch.equal(out.detach(), full)
        out.sum().backward()                            # an expanded gradient
        assert (a.grad is None) == (which == "w") and (b.grad is None) == (which == "y")
    with torch.no_grad():
        assert not M.combine_tokens(a.requires_grad_(), s, b).requires_grad


@pytest.mark.parametrize("T,k,E,H", [(7, 2, 5, 24)])
def test_gradients_against_differences(dev, T, k, E, H):
    """Sort, scale by expert, combine: derivatives along a direction against differences.  All of it is
    linear in x and in w, so central differences have the roundings of two results only."""
    g = gen("diff")
    ids = some_ids("diff", T, k, E).to(dev)
    x, dx = (torch.randn(T, H, generator=g).to(dev) for _ in range(2))
    w, dw = (torch.randn(T, k, generator=g).to(dev) for _ in range(2))
    c = torch.randn(T, H, generator=g).to(dev)

    def f(x, w):
        s = M.sort_tokens(ids, E, x)
        y = torch.where((s["tokens"] >= 0)[:, None], s["x"] * 1.5, torch.zeros_like(s["x"]))
        return M.combine_tokens(y, s["slots"], w, offsets=s["offsets"])

    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    gx, gw = torch.autograd.grad((f(xr, wr) * c).sum(), (xr, wr))
    F = torch.float64
    for direction, grad, at in ((dx, gx, lambda h: f(x + h * dx, w)), (dw, gw, lambda h: f(x, w + h * dw))):
        diff = ((at(1.0).to(F) - at(-1.0).to(F)) * c.to(F)).sum() / 2
        assert abs(float(diff - (grad.to(F) * direction.to(F)).sum())) <= 40 * R.U * T * k * H
