"""Operators for experts in 8-bit floating point on long inputs: tensors whose bytes pass 2^32, where the
rows behind that place are what they would be in a small tensor, and the first ones too; and sorts of many
pairs."""
import pytest
import torch

from tests import _expert as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
MANY = 1_100_000                                        # rows: times 4096 bytes more than 2^32
ENDS = [0, 1, 77, MANY - 66, MANY - 2, MANY - 1]


@pytest.fixture(scope="module")
def M():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    import weight_only_bit_moe_amd as M
    yield M
    torch.cuda.empty_cache()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def close(got, want, tol):
    off = (got.double() - want).abs() / tol
    assert bool((off <= 1).all()), f"{float(off.max())} of the allowed"


def at(i):
    return torch.tensor(i, device="cuda")


def test_quant(M):
    x = torch.zeros(MANY, 4096, dtype=BF, device="cuda")
    some = torch.randn(len(ENDS), 4096, generator=gen(1)).to(BF)
    x[at(ENDS)] = some.cuda()
    q, s = M.quant_fp8(x)
    want_q, want_s = R.codes(some.to(torch.float64))
    assert torch.equal(q.view(torch.uint8)[at(ENDS)].cpu().view(R.E4M3).float().double(), want_q)
    assert torch.equal(s[at(ENDS)].cpu().double(), want_s)
    assert not q.view(torch.uint8)[100:MANY - 100:997].any()


def test_gemm_of_many_strided_rows(M):
    N, K = 2048, 128
    g = gen(2)
    a, w = R.random_codes(g, len(ENDS), K), R.random_codes(g, N, K)
    sa, sw = torch.rand(len(ENDS), 1, generator=g), torch.rand(N // 128, 1, generator=g)
    buf = torch.zeros(MANY, 4096, dtype=torch.uint8, device="cuda")
    buf[at(ENDS), :K] = a.view(torch.uint8).cuda()
    scale = torch.zeros(MANY, 1, device="cuda")
    scale[at(ENDS)] = sa.cuda()
    out = M.gemm_fp8(buf.view(R.E4M3)[:, :K], scale, w.cuda(), sw.cuda())
    exact, terms, groups = R.product(a, sa, w, sw)
    close(out[at(ENDS)].cpu(), exact, R.product_bound(exact, terms, groups, K, BF))
    assert not out[100:MANY - 100:997].any()


@pytest.mark.parametrize("rows", [6, 600])
def test_grouped_with_the_weights_of_many_experts(M, rows):
    E, N, K = 300, 4096, 4096
    g = gen(3)
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    sw = torch.zeros(E, N // 128, K // 128, device="cuda")
    last, last_s = R.random_codes(g, N, K), torch.rand(N // 128, K // 128, generator=g)
    w[E - 1], sw[E - 1] = last.view(torch.uint8).cuda(), last_s.cuda()
    a, sa = R.random_codes(g, 2 * rows, K), torch.rand(2 * rows, K // 128, generator=g)
    offsets = torch.full((E + 1,), rows, dtype=torch.int32)
    offsets[0], offsets[E] = 0, 2 * rows
    out = M.gemm_fp8_grouped(a.cuda(), sa.cuda(), w.view(R.E4M3), sw, offsets.cuda()).cpu()
    assert not out[:rows].any()
    show = [rows, rows + 1, 2 * rows - 1]
    exact, terms, groups = R.product(a[show], sa[show], last, last_s)
    close(out[show], exact, R.product_bound(exact, terms, groups, K, BF))


def test_grouped_with_many_rows_out(M):
    T, N, K = 2_000_000, 1104, 128                      # out: 4.4e9 bytes
    ends = [0, 3, T - 300, T - 1]
    g = gen(4)
    a, w = R.random_codes(g, 5, K), R.random_codes(g, 2 * N, K).view(torch.uint8).view(2, N, K).view(R.E4M3)
    sa, sw = torch.rand(5, 1, generator=g), torch.rand(2, R.blocks(N), 1, generator=g)
    offsets = torch.tensor([0, T // 2 + 1, T], dtype=torch.int32, device="cuda")
    rows = torch.arange(T, device="cuda", dtype=torch.int32) % 5
    out = M.gemm_fp8_grouped(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), offsets, rows=rows)
    for e, part in ((0, ends[:2]), (1, ends[2:])):
        from_rows = [i % 5 for i in part]
        exact, terms, groups = R.product(a[from_rows], sa[from_rows], w[e], sw[e])
        close(out[at(part)].cpu(), exact, R.product_bound(exact, terms, groups, K, BF))


def test_sort_and_its_gradient(M):
    T, k, E, H = 140_000, 8, 64, 2048                   # the sorted rows: 4.6e9 bytes
    g = gen(5)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    x = torch.randn(T, 1, generator=g).to(BF).cuda().expand(T, H).contiguous()
    x[:, 1::2] *= 2
    x.requires_grad_()
    s = M.sort_tokens(ids.cuda(), E, x)
    assert int(s["offsets"][-1]) == T * k
    tokens = s["tokens"].long()
    order = torch.sort(ids.view(-1).cuda(), stable=True)[1]
    assert torch.equal(tokens, order // k)
    for columns in (0, 1, H - 1):
        assert torch.equal(s["x"].detach()[:, columns], x.detach()[:, columns][tokens])
    d = torch.zeros(T * k, H, dtype=BF, device="cuda")
    t = [0, 5, T - 2, T - 1]
    slots = s["slots"][at(t)].long()
    rows = torch.randn(len(t), k, H, generator=g).to(BF)
    d[slots.view(-1)] = rows.view(-1, H).cuda()
    s["x"].backward(d)
    exact, terms = rows.double().sum(1), rows.double().abs().sum(1)
    close(x.grad[at(t)].cpu(), exact, (k - 1) * R.U * terms + R.half_step(BF) * 1.001 * exact.abs() + R.smallest(BF))


@pytest.mark.parametrize("T,k", [(8193, 8), (70_000, 1), (20_011, 64), (200_000, 6)])
@pytest.mark.parametrize("E", [1, 64, 65, 1000])
def test_sort_of_many_pairs(M, T, k, E):
    H = 24
    ids = torch.randint(-2, E + 2, (T, k), generator=gen(T + E), dtype=torch.int32).cuda()
    x = torch.arange(T * H, device="cuda", dtype=torch.float32).view(T, H)
    s = M.sort_tokens(ids, E, x)
    flat = ids.view(-1).long()
    here = (flat >= 0) & (flat < E)
    order = torch.sort(torch.where(here, flat, E), stable=True)[1]
    n = int(here.sum())
    counts = torch.bincount(flat[here], minlength=E)
    assert torch.equal(s["offsets"].long(), torch.cat([counts.new_zeros(1), counts.cumsum(0)]))
    assert torch.equal(s["tokens"][:n].long(), order[:n] // k) and bool((s["tokens"][n:] == -1).all())
    slots = torch.full_like(flat, -1)
    slots[order[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(s["slots"].view(-1).long(), slots)
    assert torch.equal(s["x"][:n], x[order[:n] // k])


def test_combine_and_its_gradient(M):
    T, k, H = MANY // 2, 2, 2048                        # y: 4.5e9 bytes
    g = gen(6)
    t = [0, 9, T - 3, T - 1]
    slots = torch.arange(T * k, dtype=torch.int32).flip(0).view(T, k)
    weights = torch.rand(T, k, generator=g)
    rows = torch.randn(len(t), k, H, generator=g).to(BF)
    y = torch.zeros(T * k, H, dtype=BF, device="cuda")
    y[slots[t].long().view(-1).cuda()] = rows.view(-1, H).cuda()
    y.requires_grad_()
    wd = weights.cuda().requires_grad_()
    out = M.combine_tokens(y, slots.cuda(), wd)
    exact = (rows.double() * weights[t].double()[..., None])
    terms, exact = exact.abs().sum(1), exact.sum(1)
    close(out.detach()[at(t)].cpu(), exact, k * R.U * terms + R.half_step(BF) * 1.001 * exact.abs() + R.smallest(BF))
    d = torch.zeros(T, H, dtype=BF, device="cuda")
    dt = torch.randn(len(t), H, generator=g).to(BF)
    d[at(t)] = dt.cuda()
    out.backward(d)
    dy = (weights[t].double()[..., None] * dt.double()[:, None])
    got = y.grad[slots[t].long().view(-1).cuda()].cpu().view(len(t), k, H)
    close(got, dy, R.U * dy.abs() + R.half_step(BF) * 1.001 * dy.abs() + R.smallest(BF))
    dots = rows.double() * dt.double()[:, None]
    close(wd.grad[at(t)].cpu(), dots.sum(-1), H * R.U * dots.abs().sum(-1))
