"""Calls of the operators for experts in 8-bit floating point that are refused before anything runs."""
import pytest
import torch

import weight_only_bit_moe_amd as M
from tests.test_gpu_expert_grads import case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


@pytest.mark.parametrize("grad", [False, True])
def test_offsets_are_checked_with_and_without_a_gradient(dev, grad):
    ids, x, w, E = case(dev)
    s = M.sort_tokens(ids, E, x.detach())
    y, off = s["x"].requires_grad_(grad), s["offsets"]
    for bad, kind in ((off.long(), TypeError), (off.cpu(), ValueError), (off[:0], ValueError), (off[::2], ValueError),
                      ([0, 1], TypeError)):
        out = torch.full_like(x.detach(), 7.0)
        with pytest.raises(kind):
            M.combine_tokens(y, s["slots"], offsets=bad, **({} if grad else dict(out=out)))
        assert bool((out == 7).all())
    assert M.combine_tokens(y, s["slots"], offsets=off).requires_grad == grad


def test_rows_too_long_for_a_gradient_are_refused_at_the_call(dev):
    H = 32769
    y, w, add = torch.randn(4, H, device=dev), torch.ones(2, 2, device=dev), torch.randn(2, H, device=dev)
    slots = torch.arange(4, dtype=torch.int32, device=dev).view(2, 2)
    for a, b in ((y.clone().requires_grad_(), w), (y, w.clone().requires_grad_())):
        with pytest.raises(ValueError, match="up to 32768"):
            M.combine_tokens(a, slots, b)
        with torch.no_grad():
            assert M.combine_tokens(a, slots, b).shape == (2, H)
    added = add.clone().requires_grad_()                # its gradient is the output's, of any length
    M.combine_tokens(y, slots, w, addend=added).sum().backward()
    assert torch.equal(added.grad, torch.ones_like(add))
    a = y[:, 1:].clone().requires_grad_()
    M.combine_tokens(a, slots, w).sum().backward()
    assert torch.equal(a.grad, torch.ones_like(a))


def test_forward_mode_is_refused(dev):
    import torch.autograd.forward_ad as forward
    ids, x, w, E = case(dev)
    x, w = x.detach(), w.detach()
    s = M.sort_tokens(ids, E, x)
    y, slots = s["x"], s["slots"]
    with forward.dual_level():
        for asked in (False, True):
            def dual(t):
                return forward.make_dual(t.clone().requires_grad_(asked), torch.ones_like(t))
            for call in (lambda: M.sort_tokens(ids, E, dual(x)), lambda: M.combine_tokens(dual(y), slots, w),
                         lambda: M.combine_tokens(y, slots, dual(w)), lambda: M.combine_tokens(y, slots, w, addend=dual(x))):
                with pytest.raises(NotImplementedError, match="tangent"):
                    call()
                with torch.no_grad(), pytest.raises(NotImplementedError, match="tangent"):
                    call()
        assert torch.equal(M.sort_tokens(ids, E, x)["x"], y)        # without one, inside a level
    assert torch.equal(M.sort_tokens(ids, E, x)["x"], y)


def test_the_layer_checks_its_arguments_against_each_other(dev):
    from tests.test_gpu_expert_layer import experts
    (w13, s13, w2, s2), g = experts("sizes", 4, 64, 32, dev)
    x = torch.randn(5, 64, generator=g).bfloat16().to(dev)
    ids, w = torch.zeros(5, 2, dtype=torch.int32, device=dev), torch.ones(5, 2, device=dev)
    full = M.forward_fp8(x, ids, w, w13, s13, w2, s2)
    assert torch.equal(M.forward_fp8(x, ids, w, w13, s13, w2, s2, codes=M.quant_fp8(x)), full)
    more = lambda t: torch.cat([t, t[:2]])  # noqa: E731
    for call in (lambda: M.forward_fp8(x, ids[:3], w[:3], w13, s13, w2, s2), lambda: M.forward_fp8(x, more(ids), more(w), w13, s13, w2, s2),
                 lambda: M.forward_fp8(x, ids, w, w13, s13, w2, s2, codes=M.quant_fp8(more(x))),
                 lambda: M.forward_fp8(x, ids, w, w13, s13, w2, s2, codes=M.quant_fp8(x[:4])),
                 lambda: M.forward_fp8(x, ids, w, w13, s13, w2[:, :48], s2), lambda: M.forward_fp8(x, ids, w, w13, s13, w2[:3], s2[:3]),
                 lambda: M.forward_fp8(x, ids, w, w13, s13, w2[..., :16], s2), lambda: M.forward_fp8(x, ids, w, w13[0], s13, w2, s2),
                 lambda: M.forward_fp8(x, ids, w[:, :1], w13, s13, w2, s2), lambda: M.forward_fp8(x, ids, w, w13, s13, w2, s2, addend=x[:4]),
                 lambda: M.forward_fp8(x, ids, w, w13, s13, w2, s2, out=more(x))):
        with pytest.raises(ValueError):
            call()
    # codes of a view with its tokens' own rows
    assert torch.equal(M.forward_fp8(x[1:4], ids[1:4], w[1:4], w13, s13, w2, s2), full[1:4])
