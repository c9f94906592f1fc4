"""A gradient of combine computes what it is asked for."""
import itertools

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


def make(dev, given, T=1024, k=4, H=2048):
    g = gen("asked", T, k, H)
    t = dict(y=torch.randn(T * k, H, generator=g).to(dev).requires_grad_())
    if "w" in given:
        t["w"] = torch.randn(T, k, generator=g).to(dev).requires_grad_()
    if "a" in given:
        t["a"] = torch.randn(T, H, generator=g).to(dev).requires_grad_()
    slots = torch.randperm(T * k, generator=g).to(torch.int32).view(T, k).to(dev)
    out = M.combine_tokens(t["y"], slots, t.get("w"), addend=t.get("a"))
    return t, slots, out, torch.randn(T, H, generator=g).to(dev)


@pytest.mark.parametrize("given", ["", "w", "a", "wa"])
def test_each_choice_of_gradients(dev, given):
    t, slots, out, d = make(dev, given)
    names = ["y", *given]
    full = dict(zip(names, torch.autograd.grad(out, [t[n] for n in names], d, retain_graph=True)))
    rows = d.double()[:, None] * (t["w"].detach().double()[..., None] if "w" in given else 1.0)
    rows = rows.expand(*slots.shape, -1)
    got = full["y"].double()[slots.long()]
    assert bool(((got - rows).abs() <= 2 * R.U * rows.abs()).all())
    for n in range(1, len(names) + 1):
        for asked in itertools.combinations(names, n):
            part = torch.autograd.grad(out, [t[a] for a in asked], d, retain_graph=True)
            assert all(torch.equal(p, full[a]) for p, a in zip(part, asked))


def test_no_memory_for_a_gradient_that_nobody_asked_for(dev):
    t, _, out, d = make(dev, "wa")
    def peak(names):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        grads = torch.autograd.grad(out, [t[n] for n in names], d, retain_graph=True)
        torch.cuda.synchronize()
        del grads
        return torch.cuda.max_memory_allocated() - before
    rows = t["y"].numel() * 4
    assert peak("y") >= rows and peak("wy") >= rows
    assert peak("w") < rows // 2 and peak("a") < rows // 2 and peak("wa") < rows // 2
