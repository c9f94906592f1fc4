"""Every tile of the 8-bit floating point products, whole and with K split, against 64 bits at sizes of
many blocks of K with remainders in every direction (tests/_expert_products.py).  The references of these
sizes are computed on the GPU, in float64."""
import pytest
import torch

import weight_only_bit_moe_amd as M
from tests import _expert as R
from tests import _expert_products as S
from tests.test_gpu_block_ops import gen
from tests.test_gpu_expert_ops import padded

pytestmark = pytest.mark.gpu

BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    yield torch.device("cuda:0")
    torch.cuda.empty_cache()


def operands(key, dev, T, N, K, E=None):
    """All finite codes; scales far apart, negative and zero ones among the weight's."""
    g = torch.Generator(device=dev)
    g.manual_seed(gen("products", key, T, N, K, E).initial_seed())

    def codes(*shape):
        c = torch.randint(0, 254, shape, generator=g, device=dev, dtype=torch.int16)
        return (c + (c >= 127)).to(torch.uint8).view(R.E4M3)    # 127 and 255 are NaN
    rand = lambda *s: torch.rand(*s, generator=g, device=dev)  # noqa: E731
    e = () if E is None else (E,)
    sa = torch.exp2(torch.floor(12 * rand(T, R.blocks(K))) - 9)
    sw = (rand(*e, R.blocks(N), R.blocks(K)) - 0.3) * 1e-2
    sw[sw.abs() < 5e-4] = 0
    return codes(T, K), sa, codes(*e, N, K), sw, g


def check(got, reference, K, dt, scale=1.0, add=None):
    """reference: of R.product, for scale = 1 and no addend; scale: a power of two on all of it."""
    exact, terms, groups = (v * scale for v in reference)
    if add is not None:
        exact = exact + add.to(R.F)
    assert got.dtype == dt and got.shape == exact.shape
    off = (got.to(R.F) - exact).abs()
    b = R.product_bound(exact, terms, groups, K, dt, add)
    assert bool((off <= b).all()), (float((off - b).max()), int((off > b).sum()))


def forms(dev, T, N, K):
    """One product in every output type, with and without an addend in place."""
    a, sa, w, sw, g = operands("plain", dev, T, N, K)
    reference = R.product(a, sa, w, sw)
    ws = M.gemm_fp8_workspace_for(T, N, K, dev)
    if ws is not None:
        ws[4096:] = 0x5A                                # only the counters start at zero
    small = 2.0 ** -8                                   # for float16
    for dt in (FF, BF, HF):
        f = small if dt == HF else 1.0
        got = M.gemm_fp8(a, sa * f, w, sw, out_dtype=dt, workspace=ws)
        check(got, reference, K, dt, f)
        assert torch.equal(M.gemm_fp8(a, sa * f, w, sw, out_dtype=dt), got)   # a workspace of its own
        add = (torch.randn(T, N, generator=g, device=dev) * 20).to(dt)
        out = add.clone()
        assert M.gemm_fp8(a, sa * f, w, sw, addend=out, out=out, out_dtype=dt, workspace=ws) is out
        check(out, reference, K, dt, f, add)
        assert ws is None or not bool(ws[:4096].any())
    add = torch.randn(T, N, generator=g, device=dev).to(BF)
    out = padded(torch.zeros(T, N, dtype=BF, device=dev), dev, 3)
    M.gemm_fp8(padded(a, dev, 16), padded(sa, dev, 1), padded(w, dev, 48), padded(sw, dev, 2),
               addend=padded(add, dev, 5), out=out, workspace=ws)
    check(out, reference, K, BF, 1.0, add)
    assert bool(torch.isnan(torch.as_strided(out, (T, 3), (N + 3, 1), N)).all())


@pytest.mark.parametrize("tile,split", S.PLAIN)
def test_every_tile(dev, tile, split):
    size = S.PLAIN[tile, split]
    p = S.plan(*size)
    assert (p.tile, p.split) == (tile, split)
    forms(dev, *size)


@pytest.mark.parametrize("size", S.STREAMED)
def test_streamed(dev, size):
    forms(dev, *size)


@pytest.mark.parametrize("tile,size", S.GROUPED)
@pytest.mark.parametrize("gather", [True, False])
def test_every_grouped_tile(dev, tile, size, gather):
    E, rows_out, N, K = size
    assert S.grouped_tile(*size) == tile
    tokens = max(1, rows_out // 3) if gather else rows_out
    a, sa, w, sw, g = operands("grouped", dev, tokens, N, K, E)
    # experts without rows, with one, with a part of a tile and with several
    share = torch.rand(E, generator=g, device=dev) ** 3
    counts = torch.floor(share / share.sum() * (rows_out - 1)).long().cpu()
    if E > 2:
        counts[0], counts[E // 2] = 0, min(1, int(counts[E // 2]))
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    used = int(off[-1])
    assert 0 < used < rows_out
    rows = None
    if gather:
        rows = torch.full((rows_out,), -1, dtype=torch.int32, device=dev)
        rows[:used] = torch.randint(0, tokens, (used,), generator=g, device=dev, dtype=torch.int32)
    at = torch.arange(rows_out, device=dev) if rows is None else rows.long()
    offsets = off.to(torch.int32).to(dev)
    outs = {dt: torch.full((rows_out, N), 7.0, dtype=dt, device=dev) for dt in (FF, BF, HF)}
    f = {FF: 1.0, BF: 1.0, HF: 2.0 ** -8}
    for dt, out in outs.items():
        M.gemm_fp8_grouped(a, sa * f[dt], w, sw, offsets, rows=rows, out_dtype=dt, out=out)
    strided = M.gemm_fp8_grouped(padded(a, dev, 32), padded(sa, dev, 1), padded(w, dev, 16), padded(sw, dev, 3),
                                 offsets, rows=rows, out=padded(torch.zeros(rows_out, N, dtype=BF, device=dev), dev, 5))
    assert torch.equal(strided[:used], outs[BF][:used])
    for e in torch.nonzero(counts).view(-1).tolist():
        part = slice(int(off[e]), int(off[e + 1]))
        reference = R.product(a[at[part]], sa[at[part]], w[e], sw[e])
        for dt, out in outs.items():
            check(out[part], reference, K, dt, f[dt])
    for out in outs.values():
        assert bool((out[used:] == 7).all())


def test_split_products_on_two_streams(dev):
    """Each call's sums meet in a workspace of its own."""
    sizes = [(200, 517, 16400), (1130, 933, 5424)]
    data, want = [], []
    for size in sizes:
        p = S.plan(*size)
        assert p.split > 1 and M.moe_wna16_gemm_fp8_workspace_size(*size) > 0
        data.append(operands("streams", dev, *size)[:4])
        want.append(M.gemm_fp8(*data[-1], out_dtype=FF))
        check(want[-1], R.product(*data[-1]), size[2], FF)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(M.gemm_fp8(*data[i], out_dtype=FF))
                got[i].append(M.gemm_fp8(*data[1 - i], out_dtype=FF))
    torch.cuda.synchronize()
    for i in range(2):
        for j, y in enumerate(got[i]):
            assert torch.equal(y, want[i if j % 2 == 0 else 1 - i])
