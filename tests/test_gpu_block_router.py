"""A block's router in 32 bits: logits that bf16 could not tell apart pick the experts."""
import numpy as np
import pytest
import torch

from tests import _block as R
from tests import _gpu as G
from weight_only_bit_moe_amd import block as B
from weight_only_bit_moe_amd.inputs import LayerSpec

pytestmark = pytest.mark.gpu


def make():
    return B.synthetic(LayerSpec(name="block", T=1, H=512, I=256, E=16, topk=4, bits13=2, group13=128,
                                 bits2=2, group2=128, scale_lo=0.005, scale_hi=0.02), 3, G.device())


def test_float32_router():
    block = make()
    g = torch.Generator()
    g.manual_seed(1)
    y = torch.randn(60, 512, generator=g).bfloat16()
    one = torch.randn(1, 512, generator=g) * 512 ** -0.5
    # all experts' logits are nearly equal: within a bf16 step, many FP32 ones apart
    gate = one * (1 + torch.randperm(16, generator=g)[:, None] * 2.0 ** -13)
    block.gate, block.bias = gate.to(G.device()), None
    logits = (y.double() @ gate.double().t())
    ids, w = block.route(y.to(G.device()))
    far = logits.sum(1).abs() > 0.8             # 16 logits of 0.05 and more: steps of 6e-6, errors of 1e-6
    assert int(far.sum()) > 40
    want, _ = R.route(logits[far], 4, None, "sigmoid", 1, 1, True, 1.0)
    assert np.array_equal(ids.cpu()[far].numpy(), want)
    x = y.to(G.device())
    out, h = block(x)
    assert out.shape == x.shape and bool(torch.isfinite(out).all()) and h is x


def test_bf16_router_as_before():
    block = make()
    y = torch.randn(9, 512, device=G.device()).bfloat16()
    logits = torch.nn.functional.linear(y, block.gate)
    assert logits.dtype == torch.bfloat16
    ids, w = block.route(y)
    want, _ = R.route(logits.cpu(), 4, block.bias.cpu(), "sigmoid", 1, 1, True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), want)
