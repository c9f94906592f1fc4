"""A whole mixture-of-experts block: norm, routing, routed experts and shared expert together,
against the oracle's layer and 64-bit references of the other steps."""
import numpy as np
import pytest
import torch

import weight_only_bit_moe_amd as M
from oracle import oracle as O
from tests import _block as R
from tests import _gpu as G
from weight_only_bit_moe_amd import block as B
from weight_only_bit_moe_amd.inputs import LayerSpec, make_layer

pytestmark = pytest.mark.gpu


def spec(**kw):
    base = dict(name="block", T=1, H=512, I=256, E=16, topk=4, bits13=2, group13=128, bits2=2,
                group2=128, scale_lo=0.005, scale_hi=0.02)
    base.update(kw)
    return LayerSpec(**base)


@pytest.mark.parametrize("T", [1, 6, 90, 260])
@pytest.mark.parametrize("groups,kg", [(1, 1), (4, 2)])
@pytest.mark.parametrize("first", [False, True])
def test_block(T, groups, kg, first):
    dev = G.device()
    sp = spec(alpha=1.702, beta=1.0, clamp=7.0)
    block = B.synthetic(sp, 7, dev, shared=384)
    block.groups, block.topk_groups = groups, kg
    g = torch.Generator()
    g.manual_seed(T)
    x, r = (torch.randn(T, sp.H, generator=g).bfloat16() for _ in range(2))
    r = None if first else r
    out, h = block(x.to(dev), None if first else r.to(dev))
    n = M.add_rmsnorm(x.to(dev), block.norm, None if first else r.to(dev), quant=True)
    hr, y, q, scale, _ = R.rmsnorm(x, r, block.norm.cpu(), block.eps)
    assert torch.equal(h.cpu(), hr) and torch.equal(n["q"].cpu(), q)
    logits = torch.nn.functional.linear(n["y"], block.gate)
    ids, w = block.route(n["y"])
    ri, rw = R.route(logits.cpu(), sp.topk, block.bias.cpu(), "sigmoid", groups, kg, True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), ri)
    # routed experts: the oracle on the block's own normed rows and routing
    L = make_layer(sp, 7)
    L.x = n["y"].view(torch.int16).cpu().numpy().view(np.uint16)
    L.topk_ids, L.topk_w = ids.cpu().numpy(), w.cpu().numpy()
    L.spec = spec(T=T, alpha=1.702, beta=1.0, clamp=7.0)
    routed = torch.from_numpy(O.forward_layer(L))
    # shared expert in 64 bits without the roundings in between
    d = lambda c, s: c.cpu().to(R.F) * s.cpu().to(R.F)[:, None]  # noqa: E731
    gu = d(n["q"], n["scale"]) @ d(block.shared13, block.shared13_scale).t()
    a, _ = R.swiglu(gu, 1.702, 1.0, 7.0)
    shared = a @ d(block.shared2, block.shared2_scale).t()
    # the layer's own bound on the routed part; the shared part's error is dominated by the 8-bit
    # rounding of the activation (half a code of a row's largest, random over Is channels, 6 sigma)
    # and of its 16-bit input (half a step, to first order the same size)
    code = a.abs().amax(-1, keepdim=True) / 127 / 12 ** 0.5
    inputs = a.abs().pow(2).mean(-1, keepdim=True).sqrt() * R.half_step(torch.bfloat16) * 4
    w2 = d(block.shared2, block.shared2_scale).pow(2).sum(-1).sqrt()
    bound = 6 * (code.pow(2) + inputs.pow(2)).sqrt() * w2
    rms = float(routed.pow(2).mean().sqrt())
    total = routed + shared
    bound = bound + 2e-2 * rms + 1e-3 + 2 * R.half_step(torch.bfloat16) * (total.abs() + routed.abs())
    off = (out.cpu().to(R.F) - total).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


def test_block_steps_follow_each_other():
    """A second step on the same block (kept workspaces) gives what a new block gives."""
    dev = G.device()
    x = torch.randn(5, 512, device=dev).bfloat16()
    one, two = B.synthetic(spec(), 3, dev), B.synthetic(spec(), 3, dev)
    out, h = one(x)
    again, h2 = one(out, h)
    fresh, f2 = two(out, h)
    assert torch.equal(h2, f2)
    # the routed sum's FP32 additions have no fixed order
    assert torch.allclose(again.float(), fresh.float(), rtol=2 ** -6, atol=1e-2)


def test_tokens_whose_experts_are_all_masked_get_the_shared_expert_only():
    """Router logits of -inf (experts taken out of service) reach the layer as ids of -1."""
    dev = G.device()
    block = B.synthetic(spec(), 5, dev)
    y = torch.randn(3, 512, device=dev).bfloat16()
    logits = torch.nn.functional.linear(y, block.gate)
    logits[1] = -float("inf")
    ids, w = M.route_topk(logits, 4)
    out = M.forward(y, ids, w, block.w13, block.s13, block.w2, block.s2, bits=block.bits,
                    group=block.group)
    assert bool((ids[1] == -1).all()) and not bool(out[1].any())
    assert bool(out[0].any()) and bool(out[2].any())
