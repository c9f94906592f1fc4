"""The operators for experts in 8-bit floating point together: the routed layer and a block from
them, a training step through sort and combine, streams and captured graphs."""
import pytest
import torch

import weight_only_bit_moe_amd as M
from tests import _block as RB
from tests import _expert as R
from tests import _gpu as G
from tests.test_gpu_block_ops import gen
from weight_only_bit_moe_amd import block as B
from weight_only_bit_moe_amd.inputs import LayerSpec

pytestmark = pytest.mark.gpu

BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


def experts(key, E, H, I, dev):
    g = gen("experts", key, E, H, I)
    w13, s13 = B.block_codes(torch.randn(E, 2 * I, H, generator=g) * H ** -0.5)
    w2, s2 = B.block_codes(torch.randn(E, H, I, generator=g) * I ** -0.5)
    return [t.to(dev) for t in (w13, s13, w2, s2)], g


def routed_bound(x, ids, w, w13, s13, w2, s2, alpha, beta, clamp, dt):
    """The layer in 64 bits on the defined codes of x, and how far a result may be off: what the first
    product and the rounding of its rows may be off moves the activation by its derivatives, the
    activation's code is off by half a step of e4m3 more (2^-4 of the value, or 2^-10 of the scale, which
    may be the next power of two), and the second product adds its own."""
    q, s = R.codes(x.to(R.F))
    q8 = q.to(FF).to(R.E4M3)
    out, bound = torch.zeros(*x.shape, dtype=R.F), torch.zeros(*x.shape, dtype=R.F)
    I = w2.shape[2]
    for e in range(w13.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        gu, terms, groups = R.product(q8[t], s[t], w13[e], s13[e])
        d = R.product_bound(gu, terms, groups, x.shape[1], dt)
        a, _ = R.swiglu(gu, alpha, beta, clamp)
        g, u = gu[:, :I], gu[:, I:]
        if clamp is not None:
            g, u = g.clamp(max=clamp), u.clamp(-clamp, clamp)
        sig = torch.sigmoid(alpha * g)
        slope = sig + (alpha * g).abs() * sig * (1 - sig)
        da = 1.05 * (slope * (u + beta).abs() * d[:, :I] + (g * sig).abs() * d[:, I:]) + 2.0 ** -18 * a.abs()
        _, sa = R.codes(a)
        step = 2 * sa.repeat_interleave(128, 1)[:, :I]
        da = da + 2.0 ** -4 * (a.abs() + da) + 2.0 ** -10 * step
        v = R.values(w2[e], s2[e], 128)
        y = a @ v.t()
        # magnitudes of the terms for the second product's own errors: of codes up to a + da
        top = (a.abs() + da) @ v.abs().t()
        dy = da @ v.abs().t() + 7 * 2.0 ** -13 * 2 * top + 100 * R.U * top + 1.01 * R.half_step(dt) * (y.abs() + da @ v.abs().t())
        ww = w[t, j].to(R.F)[:, None]
        out.index_add_(0, t, ww * y)
        bound.index_add_(0, t, ww.abs() * dy * (1 + 2.0 ** -20))
    return out, bound + 1.01 * R.half_step(dt) * (out.abs() + bound) + R.smallest(dt)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("T,k,E,H,I", [(1, 1, 1, 16, 16), (4, 6, 32, 512, 256), (9, 2, 5, 272, 144), (130, 4, 16, 256, 384),
                                       (700, 3, 8, 400, 128)])
@pytest.mark.parametrize("alpha,beta,clamp", [(1.0, 0.0, None), (1.702, 1.0, 7.0)])
def test_routed_layer(dt, T, k, E, H, I, alpha, beta, clamp):
    dev = G.device()
    ws, g = experts("layer", E, H, I, dev)
    x = (torch.randn(T, H, generator=g) * torch.exp(0.5 * torch.randn(T, 1, generator=g))).to(dt)
    ids = torch.argsort(torch.rand(T, E, generator=g), 1)[:, :k].to(torch.int32)
    ids[torch.rand(T, k, generator=g) < 0.1] = -1
    w = torch.rand(T, k, generator=g)
    act = dict(alpha=alpha, beta=beta, clamp=clamp)
    out = M.forward_fp8(x.to(dev), ids.to(dev), w.to(dev), *ws, **act)
    exact, bound = routed_bound(x, ids, w, *(t.cpu() for t in ws), alpha, beta, clamp, dt)
    off = (out.cpu().to(R.F) - exact).abs()
    assert out.dtype == dt and bool((off <= bound).all()), float((off / bound).max())
    # from its parts, with the codes at hand and added to something
    codes = M.quant_fp8(x.to(dev))
    s = M.sort_tokens(ids.to(dev), E)
    gu = M.gemm_fp8_grouped(*codes, ws[0], ws[1], s["offsets"], rows=s["tokens"], out_dtype=dt)
    y = M.gemm_fp8_grouped(*M.swiglu_quant_fp8(gu, **act), ws[2], ws[3], s["offsets"], out_dtype=dt)
    assert torch.equal(out, M.combine_tokens(y, s["slots"], w.to(dev)))
    add = torch.randn(T, H, generator=g).to(dt).to(dev)
    want = M.combine_tokens(y, s["slots"], w.to(dev), addend=add)
    got = M.forward_fp8(x.to(dev), ids.to(dev), w.to(dev), *ws, **act, codes=codes, addend=add, out=add)
    assert got is add and torch.equal(got, want)


def test_routed_layer_without_tokens_and_without_experts():
    dev = G.device()
    ws, g = experts("none", 4, 64, 32, dev)
    x = torch.randn(3, 64, generator=g).to(BF).to(dev)
    ids = torch.full((3, 2), -1, dtype=torch.int32, device=dev)
    assert not M.forward_fp8(x, ids, torch.ones(3, 2, device=dev), *ws).any()
    assert M.forward_fp8(x[:0], ids[:0], torch.ones(0, 2, device=dev), *ws).shape == (0, 64)


def test_routed_layer_gives_a_share_of_the_experts():
    """Two halves of the experts, each with ids of its own, add up to all of them."""
    dev = G.device()
    ws, g = experts("share", 8, 256, 128, dev)
    x = torch.randn(50, 256, generator=g).to(BF).to(dev)
    ids = torch.argsort(torch.rand(50, 8, generator=g), 1)[:, :3].to(torch.int32).to(dev)
    w = torch.rand(50, 3, generator=g).to(dev)
    full = M.forward_fp8(x, ids, w, *ws)
    lo = M.forward_fp8(x, ids, w, *(t[:4] for t in ws))
    hi = M.forward_fp8(x, ids - 4, w, *(t[4:] for t in ws))
    exact = lo.float() + hi.float()
    # each of the three results is rounded once
    bound = R.half_step(BF) * 1.01 * (lo.float().abs() + hi.float().abs() + full.float().abs()) + 1e-6
    assert bool(((full.float() - exact).abs() <= bound).all())


# ---- block -----------------------------------------------------------------------------

def spec(**kw):
    base = dict(name="block", T=1, H=512, I=256, E=16, topk=4, bits13=2, group13=128, bits2=2, group2=128,
                scale_lo=0.005, scale_hi=0.02)
    return LayerSpec(**dict(base, **kw))


@pytest.mark.parametrize("T", [1, 6, 90, 260])
@pytest.mark.parametrize("clamped", [False, True])
def test_block_in_8_bit_floating_point(T, clamped):
    dev = G.device()
    act = dict(alpha=1.702, beta=1.0, clamp=7.0) if clamped else {}
    block = B.synthetic(spec(**act), 7, dev, shared=384, fp8=True)
    x, r = (torch.randn(T, 512, generator=gen("b8", T, i)).to(BF) for i in range(2))
    out, h = block(x.to(dev), r.to(dev))
    hr = RB.rmsnorm(x, r, block.norm.cpu(), block.eps)[0]
    assert torch.equal(h.cpu(), hr)
    n = M.add_rmsnorm(x.to(dev), block.norm, r.to(dev))
    ids, w = block.route(n["y"])
    act = dict(alpha=block.alpha, beta=block.beta, clamp=block.clamp)
    routed = M.forward_fp8(n["y"], ids, w, block.w13, block.s13, block.w2, block.s2, **act)
    gu = M.gemm_fp8(*M.quant_fp8(n["y"]), block.shared13, block.shared13_scale)
    want = M.gemm_fp8(*M.swiglu_quant_fp8(gu, **act), block.shared2, block.shared2_scale, addend=routed)
    assert torch.equal(out, want)
    # and the shared expert against 64 bits
    y = n["y"].cpu()
    zero = torch.zeros(T, 1, dtype=torch.int32)
    exact, bound = routed_bound(y, zero, torch.ones(T, 1), *(t.cpu()[None] for t in (
        block.shared13, block.shared13_scale, block.shared2, block.shared2_scale)), block.alpha, block.beta,
        block.clamp, BF)
    total = exact + routed.cpu().to(R.F)
    bound = bound + 1.01 * R.half_step(BF) * (total.abs() + bound + exact.abs())
    assert bool(((out.cpu().to(R.F) - total).abs() <= bound).all())


def test_block_with_one_kind_in_8_bit_floating_point():
    """Routed experts in 2-bit integers with a shared one in 8-bit floating point, and the other way round."""
    dev = G.device()
    ints, floats = B.synthetic(spec(), 3, dev), B.synthetic(spec(), 3, dev, fp8=True)
    x = torch.randn(5, 512, device=dev).to(BF)
    shared = [n for n in ("shared13", "shared13_scale", "shared2", "shared2_scale")]
    one = B.synthetic(spec(), 3, dev)
    other = B.synthetic(spec(), 3, dev, fp8=True)
    for n in shared:
        setattr(one, n, getattr(floats, n))
        setattr(other, n, getattr(ints, n))
    for block in (one, other):
        out, _ = block(x)
        n = M.add_rmsnorm(x, block.norm, quant=True)
        ids, w = block.route(n["y"])
        if block.routed_fp8:
            want = M.forward_fp8(n["y"], ids, w, block.w13, block.s13, block.w2, block.s2)
            want = block.shared(n["q"], n["scale"], want)
            assert torch.equal(out, want)
        else:
            want = M.forward(n["y"], ids, w, block.w13, block.s13, block.w2, block.s2, bits=block.bits,
                             group=block.group)
            want = block.shared(*M.quant_fp8(n["y"]), want)
            # the routed sum's FP32 additions have no fixed order
            assert torch.allclose(out.float(), want.float(), rtol=2 ** -6, atol=1e-2)


# ---- streams and graphs ------------------------------------------------------------------

def test_calls_on_two_streams():
    dev = G.device()
    ws, g = experts("streams", 16, 512, 256, dev)
    xs = [torch.randn(90, 512, generator=g).to(BF).to(dev) for _ in range(2)]
    ids = torch.argsort(torch.rand(90, 16, generator=g), 1)[:, :4].to(torch.int32).to(dev)
    w = torch.rand(90, 4, generator=g).to(dev)
    want = [M.forward_fp8(x, ids, w, *ws) for x in xs]
    a, s13 = M.quant_fp8(torch.randn(128, 4096, device=dev).to(BF))      # a product that splits K
    wa, ws13 = B.block_codes(torch.randn(512, 4096, device=dev))
    assert M.moe_wna16_gemm_fp8_workspace_size(200, 512, 16384) > 0
    product = M.gemm_fp8(a, s13, wa, ws13)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append((M.forward_fp8(xs[i], ids, w, *ws), M.gemm_fp8(a, s13, wa, ws13)))
    torch.cuda.synchronize()
    for i in range(2):
        for y, p in got[i]:
            assert torch.equal(y, want[i]) and torch.equal(p, product)


@pytest.mark.parametrize("T", [3, 200])
def test_captured_block(T):
    """Two graphs of steps of one block, replayed in turn with eager work in between."""
    dev = G.device()
    block = B.synthetic(spec(), 5, dev, fp8=True)
    xs = [torch.randn(T, 512, device=dev).to(BF) for _ in range(2)]
    inputs = [torch.randn(T, 512, device=dev).to(BF) for _ in range(4)]
    want = [block(x)[0] for x in inputs]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(block(x)[0])
        graphs.append(graph)
    for i in range(8):
        which, data = i % 2, i % 4
        xs[which].copy_(inputs[data])
        graphs[which].replay()
        eager = block(inputs[(data + 1) % 4])[0]
        torch.cuda.synchronize()
        assert torch.equal(outs[which], want[data]) and torch.equal(eager, want[(data + 1) % 4])


def test_captured_products_that_split_share_nothing():
    """Each captured product that splits K clears and counts in memory of its own graph."""
    dev = G.device()
    T, N, K = 600, 512, 16384
    assert M.moe_wna16_gemm_fp8_workspace_size(T, N, K) > 0
    w, sw = B.block_codes(torch.randn(N, K, device=dev) * K ** -0.5)
    codes = [M.quant_fp8(torch.randn(T, K, device=dev).to(BF)) for _ in range(3)]
    want = [M.gemm_fp8(*c, w, sw) for c in codes]
    x = [torch.empty_like(t) for t in codes[0]]
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(M.gemm_fp8(x[0], x[1], w, sw))
        graphs.append(graph)
    for i in range(6):
        for a, b in zip(x, codes[i % 3]):
            a.view(torch.uint8).copy_(b.view(torch.uint8)) if a.dtype == R.E4M3 else a.copy_(b)
        graphs[i % 2].replay()
        eager = M.gemm_fp8(*codes[(i + 1) % 3], w, sw)
        torch.cuda.synchronize()
        assert torch.equal(outs[i % 2], want[i % 3]) and torch.equal(eager, want[(i + 1) % 3])


@pytest.mark.parametrize("T,k,E", [(40, 4, 8), (3000, 4, 64)])
def test_captured_training_step(T, k, E):
    """Sort, an expert's function, combine and their gradients in one graph, against the eager step."""
    dev = G.device()
    H = 96
    g = gen("train", T)
    scale = torch.randn(H, generator=g).to(dev)

    def step(x, ids, w, d):
        s = M.sort_tokens(ids, E, x)
        y = torch.tanh(s["x"] * scale)
        out = M.combine_tokens(y, s["slots"], w, offsets=s["offsets"])
        return (out, *torch.autograd.grad(out, (x, w), d))

    data = [(torch.randn(T, H, generator=g).to(dev), torch.argsort(torch.rand(T, E, generator=g), 1)[:, :k].to(torch.int32).to(dev),
             torch.rand(T, k, generator=g).to(dev), torch.randn(T, H, generator=g).to(dev)) for _ in range(3)]
    want = [step(x.clone().requires_grad_(), ids, w.clone().requires_grad_(), d) for x, ids, w, d in data]
    # by hand: every pair's row is tanh(x scale), weighted
    x, ids, w, d = data[0]
    exact = torch.tanh(x.double() * scale.double()) * w.double().sum(1, keepdim=True)
    assert bool(((want[0][0].double() - exact).abs() <= 2e-6 * (1 + exact.abs())).all())
    held = [t.clone() for t in data[0]]
    held[0].requires_grad_()
    held[2].requires_grad_()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*held)
    for i in range(6):
        with torch.no_grad():
            for a, b in zip(held, data[i % 3]):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want[i % 3]):
            assert torch.equal(a, b)


def test_a_gradients_step_learns_through_sort_and_combine():
    """Linear experts: the gradient of each expert's weight and of x against dense 64-bit ones."""
    dev = G.device()
    T, k, E, H = 60, 2, 4, 32
    g = gen("dense")
    x = torch.randn(T, H, generator=g)
    W = torch.randn(E, H, H, generator=g) * H ** -0.5
    ids = torch.argsort(torch.rand(T, E, generator=g), 1)[:, :k].to(torch.int32)
    w = torch.rand(T, k, generator=g)
    c = torch.randn(T, H, generator=g)
    xd, Wd, wd = (t.to(dev).requires_grad_() for t in (x, W, w))
    s = M.sort_tokens(ids.to(dev), E, xd)
    off = s["offsets"].tolist()
    y = torch.cat([s["x"][off[e]:off[e + 1]] @ Wd[e] for e in range(E)])
    out = M.combine_tokens(y, s["slots"], wd, offsets=s["offsets"])
    got = torch.autograd.grad((out * c.to(dev)).sum(), (xd, Wd, wd))
    xr, Wr, wr = (t.to(R.F).requires_grad_() for t in (x, W, w))
    rows = torch.einsum("th,tkhj->tkj", xr, Wr[ids.long()])
    ref = torch.autograd.grad(((rows * wr[..., None]).sum(1) * c.to(R.F)).sum(), (xr, Wr, wr))
    for a, b in zip(got, ref):
        # sums of at most T * H FP32 products of numbers of size one
        assert bool(((a.cpu().to(R.F) - b).abs() <= T * H * R.U * (1 + b.abs().max())).all())
