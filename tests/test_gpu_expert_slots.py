"""Gradients of combine where slots have been changed since the sort."""
import pytest
import torch

import weight_only_bit_moe_amd as M
from tests import _expert as R
from tests.test_gpu_block_ops import gen

pytestmark = pytest.mark.gpu

FF = torch.float32


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


def data(T, k, H, dev):
    g = gen("slots", T, k, H)
    y, w, d = torch.randn(T * k, H, generator=g), torch.randn(T, k, generator=g), torch.randn(T, H, generator=g)
    slots = torch.randperm(T * k, generator=g).to(torch.int32).view(T, k)
    return g, y, w, d, slots


def gradients(y, w, d, slots, dev, offsets=None):
    y, w = y.to(dev).requires_grad_(), w.to(dev).requires_grad_()
    left = [torch.full_like(y, float("nan")) for _ in range(3)]         # what the allocator hands out next
    del left
    out = M.combine_tokens(y, slots.to(dev), w, offsets=offsets)
    return [t.cpu().to(R.F) for t in torch.autograd.grad(out, (y, w), d.to(dev))]


def check(got, y, w, d, slots, upto):
    """Rows of dy from `upto` on are zeros; a dot product of H terms rounds at most H + 1 times."""
    dy, dw = got
    T, k = slots.shape
    want = torch.zeros(y.shape, dtype=R.F)
    for t, j in torch.nonzero((slots >= 0) & (slots < upto)).tolist():
        want[slots[t, j]] = w[t, j].to(R.F) * d[t].to(R.F)
    assert bool(((dy - want).abs() <= 2 * R.U * want.abs()).all())
    rows = torch.where((slots >= 0)[..., None], y.to(R.F)[slots.clamp(min=0).long()], torch.zeros(1, dtype=R.F))
    dots = rows * d.to(R.F)[:, None]
    assert bool(((dw - dots.sum(-1)).abs() <= (y.shape[1] + 1) * R.U * dots.abs().sum(-1)).all())


@pytest.mark.parametrize("T,k,H", [(3, 2, 9), (64, 4, 520), (1000, 8, 64)])
def test_pairs_left_out_since_the_sort(dev, T, k, H):
    g, y, w, d, slots = data(T, k, H, dev)
    slots[torch.rand(T, k, generator=g) < 0.4] = -1
    check(gradients(y, w, d, slots, dev), y, w, d, slots, T * k)


@pytest.mark.parametrize("T,k,H", [(3, 2, 9), (64, 4, 520), (1000, 8, 64)])
@pytest.mark.parametrize("used", [0, 1, "most", "more", -3])
def test_a_slot_behind_the_last_sorted_row_gets_nothing(dev, T, k, H, used):
    """It is cleared there, whichever comes first."""
    _, y, w, d, slots = data(T, k, H, dev)
    n = T * k - T * k // 3 if used == "most" else T * k + 5 if used == "more" else used
    offsets = torch.tensor([0, n], dtype=torch.int32, device=dev)
    for _ in range(3):
        check(gradients(y, w, d, slots, dev, offsets), y, w, d, slots, max(0, min(n, T * k)))
