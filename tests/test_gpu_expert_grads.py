"""The graphs of sort_tokens and combine_tokens: which gradients exist, what they are made from, and
what is refused."""
import threading

import pytest
import torch

import weight_only_bit_moe_amd as M
from tests import _expert as R
from tests.test_gpu_block_ops import gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


def case(dev, T=9, k=3, E=5, H=20, dtype=torch.float32):
    g = gen("graph", T, k, E, H)
    ids = torch.argsort(torch.rand(T, E, generator=g), 1)[:, :k].to(torch.int32).to(dev)
    x = torch.randn(T, H, generator=g).to(dtype).to(dev).requires_grad_()
    w = torch.rand(T, k, generator=g).to(dev).requires_grad_()
    return ids, x, w, E


def test_sums_hand_over_expanded_gradients(dev):
    ids, x, w, E = case(dev)
    s = M.sort_tokens(ids, E, x)
    s["x"].sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 3.0))         # three rows of each token
    y = s["x"].detach().requires_grad_()
    M.combine_tokens(y, s["slots"], w).sum().backward()
    assert torch.equal(y.grad[s["slots"].long()], w.detach()[..., None].expand(*w.shape, x.shape[1]))
    rows = y.detach().double()[s["slots"].long()].sum(-1)
    assert bool(((w.grad.double() - rows).abs() <= 20 * R.U * y.detach().double().abs()[s["slots"].long()].sum(-1)).all())


def test_which_results_are_in_the_graph(dev):
    ids, x, w, E = case(dev)
    s = M.sort_tokens(ids, E, x)
    assert s["x"].requires_grad and not any(s[n].requires_grad for n in ("tokens", "slots", "offsets"))
    assert not M.sort_tokens(ids, E, x.detach())["x"].requires_grad
    with torch.no_grad():
        assert not M.sort_tokens(ids, E, x)["x"].requires_grad
        assert not M.combine_tokens(s["x"], s["slots"], w).requires_grad
    y = s["x"].detach()
    assert not M.combine_tokens(y, s["slots"], w.detach()).requires_grad
    only_w = M.combine_tokens(y, s["slots"], w)
    assert only_w.requires_grad
    only_w.sum().backward()
    assert w.grad is not None and y.grad is None


def test_a_gradient_of_a_gradient_is_refused(dev):
    ids, x, w, E = case(dev)
    s = M.sort_tokens(ids, E, x)
    out = M.combine_tokens(s["x"] * s["x"], s["slots"], w, offsets=s["offsets"])
    dx, dw = torch.autograd.grad(out.square().sum(), (x, w), create_graph=True)
    assert dx.requires_grad and dw.requires_grad
    for d in (dx, dw):
        with pytest.raises(RuntimeError, match="have no gradient"):
            d.sum().backward(retain_graph=True)
        # towards x alone torch does not come past the refusal: it finds no way at all
        with pytest.raises(RuntimeError):
            torch.autograd.grad(d.sum(), x, retain_graph=True)


def test_what_a_gradient_is_made_from_must_not_change(dev):
    ids, x, w, E = case(dev)
    s = M.sort_tokens(ids, E, x.detach())
    for change in (lambda y: y.add_(1), lambda y: s["slots"].add_(0)):
        y = s["x"].clone().requires_grad_()
        z = y * 1.0
        out = M.combine_tokens(z, s["slots"], w, offsets=s["offsets"])
        with torch.no_grad():
            change(z)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out.sum().backward()


def test_a_graph_used_twice_gives_the_same(dev):
    ids, x, w, E = case(dev, T=700, k=4, E=16, H=264, dtype=torch.bfloat16)
    s = M.sort_tokens(ids, E, x)
    out = M.combine_tokens(s["x"], s["slots"], w, offsets=s["offsets"])
    d = torch.randn_like(out)
    a = torch.autograd.grad(out, (x, w), d, retain_graph=True)
    b = torch.autograd.grad(out, (x, w), d)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    with pytest.raises(RuntimeError):
        torch.autograd.grad(out, (x, w), d)


def test_refusals_where_a_gradient_is_required(dev):
    ids, x, w, E = case(dev)
    s = M.sort_tokens(ids, E, x)
    y = s["x"]
    for call in (lambda: M.sort_tokens(ids, E, x, out=torch.empty_like(y)),
                 lambda: M.combine_tokens(y, s["slots"], w, out=torch.empty_like(x)),
                 lambda: M.combine_tokens(y, s["slots"], w, offsets=s["offsets"][:0]),
                 lambda: M.combine_tokens(y, s["slots"], w, offsets=s["offsets"].cpu()),
                 lambda: M.combine_tokens(y, s["slots"], w[:-1]),
                 lambda: M.combine_tokens(y, s["slots"], w, addend=x[:, :-1])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: M.combine_tokens(y, s["slots"], w, offsets=s["offsets"].long()),
                 lambda: M.combine_tokens(y, s["slots"], w.double()),
                 lambda: M.sort_tokens(ids.long(), E, x)):
        with pytest.raises(TypeError):
            call()


def test_gradients_on_another_stream_and_from_two_threads(dev):
    """A gradient runs on its forward's stream, behind it; two threads' graphs keep apart."""
    data = [case(dev, T=300 + i, k=4, E=16, H=136) for i in range(4)]

    def step(ids, x, w, E):
        s = M.sort_tokens(ids, E, x)
        out = M.combine_tokens(torch.tanh(s["x"]), s["slots"], w, offsets=s["offsets"])
        return torch.autograd.grad(out.square().sum(), (x, w))

    want = [step(*c) for c in data]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(5):
                got[i] = step(*data[i])
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_nothing_to_sort_or_combine(dev):
    x = torch.zeros(0, 8, device=dev, requires_grad=True)
    s = M.sort_tokens(torch.zeros(0, 2, dtype=torch.int32, device=dev), 3, x)
    out = M.combine_tokens(s["x"], s["slots"])
    out.sum().backward()
    assert x.grad.shape == (0, 8)
    y = torch.ones(4, 8, device=dev, requires_grad=True)        # rows that nobody names
    out = M.combine_tokens(y, torch.full((3, 2), -1, dtype=torch.int32, device=dev))
    assert not out.any()
    out.sum().backward()
    assert not y.grad.any()
