"""Pairs left out of a sort (ids of experts elsewhere, padding) in training: the rows behind the last
sorted pair reach no gradient."""
import pytest
import torch

import weight_only_bit_moe_amd as M
from tests import _expert as R
from tests.test_gpu_block_ops import gen
from tests.test_gpu_expert_ops import some_ids

pytestmark = pytest.mark.gpu

BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


def leave_nan(dev, *shape, dtype=FF):
    """Memory that the allocator hands out next holds NaN."""
    t = [torch.full(shape, float("nan"), dtype=dtype, device=dev) for _ in range(3)]
    del t


@pytest.mark.parametrize("dt", [BF, HF, FF])
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 1), (5, 3, 4, 33), (64, 6, 64, 4096), (700, 8, 64, 520), (2000, 6, 16, 129),
                                     (70000, 2, 9, 24), (6, 2, 3, 32769), (3, 2, 5, 1 << 18)])
@pytest.mark.parametrize("which", ["some", "none", "all"])
def test_rows_behind_the_last_pair_are_zeros_in_a_graph(dev, dt, T, k, E, H, which):
    ids = some_ids("absent", T, k, E) if which == "some" else torch.full((T, k), E if which == "none" else E - 1, dtype=torch.int32)
    x = torch.randn(T, H, generator=gen("ab", T)).to(dt).to(dev).requires_grad_()
    tokens, _, offsets = R.sort(ids, E)
    used = int(offsets[-1])
    leave_nan(dev, T * k, H, dtype=dt)
    s = M.sort_tokens(ids.to(dev), E, x)
    assert torch.equal(s["x"][:used].detach().cpu(), x.detach().cpu()[tokens[:used].long()])
    assert not s["x"][used:].detach().cpu().any()       # a NaN counts as something


@pytest.mark.parametrize("T,k,E", [(40, 4, 8), (3000, 4, 64)])
def test_an_experts_parameters_have_finite_gradients(dev, T, k, E):
    """A function of all rows with parameters, between sort and combine, some ids elsewhere."""
    H = 96
    g = gen("abs", T)
    ids = some_ids("abs", T, k, E)
    x, c = torch.randn(T, H, generator=g), torch.randn(T, H, generator=g)
    w, scale, bias = torch.randn(T, k, generator=g), torch.randn(H, generator=g), torch.randn(H, generator=g)
    xd, wd, sd, bd = (t.to(dev).requires_grad_() for t in (x, w, scale, bias))
    leave_nan(dev, T * k, H)
    s = M.sort_tokens(ids.to(dev), E, xd)
    leave_nan(dev, T * k, H)
    out = M.combine_tokens(s["x"] * sd + bd, s["slots"], wd, offsets=s["offsets"])
    leave_nan(dev, T * k, H)
    got = torch.autograd.grad((out * c.to(dev)).sum(), (xd, wd, sd, bd))
    here = ((ids >= 0) & (ids < E)).to(R.F)
    xr, wr, sr, br = (t.to(R.F).requires_grad_() for t in (x, w, scale, bias))
    total = ((wr * here).sum(1, keepdim=True) * (xr * sr + br) * c.to(R.F)).sum()
    want = torch.autograd.grad(total, (xr, wr, sr, br))
    for a, b in zip(got, want):
        # sums of at most T * k * H FP32 products of numbers of size one
        assert bool(torch.isfinite(a).all())
        assert bool(((a.cpu().to(R.F) - b).abs() <= T * k * H * R.U * (1 + b.abs().max())).all())


def test_captured(dev):
    """Each replay clears the rows behind its own last pair."""
    T, k, E, H = 300, 4, 8, 64
    x = torch.randn(T, H, device=dev)
    data = [some_ids(i, T, k, E).to(dev) for i in range(3)] + [torch.full((T, k), -1, dtype=torch.int32, device=dev)]
    held, ids = x.clone().requires_grad_(), data[0].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        M.sort_tokens(ids, E, held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = M.sort_tokens(ids, E, held)
    for i in range(8):
        ids.copy_(data[i % 4])
        with torch.no_grad():
            s["x"].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = M.sort_tokens(data[i % 4], E, x)
        n = int(want["offsets"][-1])
        assert torch.equal(s["x"][:n], want["x"][:n]) and not s["x"][n:].any()


@pytest.mark.parametrize("T,k,E", [(40, 4, 8), (3000, 4, 64)])
def test_captured_training_step(dev, T, k, E):
    """Sort, a function of all rows with parameters, combine and their gradients in one graph, with other
    pairs left out in each replay, against the eager step."""
    H = 96
    g = gen("absent step", T)
    # a parameter for each row, so that no sum of torch's is in the graph
    d, scale = torch.randn(T, H, generator=g).to(dev), torch.randn(T * k, H, generator=g).to(dev)

    def step(ids, x, w, p):
        s = M.sort_tokens(ids, E, x)
        out = M.combine_tokens(torch.tanh(s["x"] * p), s["slots"], w, offsets=s["offsets"])
        return (out, *torch.autograd.grad(out, (x, w, p), d))

    data = [(some_ids((i, "step"), T, k, E).to(dev), torch.randn(T, H, generator=g).to(dev),
             torch.rand(T, k, generator=g).to(dev), scale * (i + 1)) for i in range(3)]
    leaves = lambda c: (c[0].clone(), *(t.clone().requires_grad_() for t in c[1:]))  # noqa: E731
    want = [step(*leaves(c)) for c in data]
    held = leaves(data[0])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*held)
    for i in range(7):
        with torch.no_grad():
            for a, b in zip(held, data[i % 3]):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        eager = step(*leaves(data[(i + 1) % 3]))
        torch.cuda.synchronize()
        for a, b in zip((*outs, *eager), (*want[i % 3], *want[(i + 1) % 3])):
            assert bool(torch.isfinite(a).all()) and torch.equal(a, b)
