"""Routing weights of experts whose scores are all tiny."""
import math

import numpy as np
import pytest
import torch

import weight_only_bit_moe_amd as M
from tests import _block as R

pytestmark = pytest.mark.gpu

F = np.float64
INF = math.inf


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


def check_weights(w, logp, alive):
    """Weights against exp(log p) / sum, the sum over the picked; 1.01 roundings to FP32."""
    logp = np.where(alive, logp, -INF)
    with np.errstate(all="ignore"):
        e = np.exp(logp - logp.max(-1, keepdims=True))
        want = np.where(alive.any(-1, keepdims=True), e / e.sum(-1, keepdims=True), 0.0)
    got = w.cpu().numpy().astype(F)
    assert np.all(np.abs(got - want) <= 1.01 * R.U * want + 2.0 ** -149), np.abs(got - want).max()


@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("with_bias", [False, True])
def test_renormalized_weights_of_tiny_sigmoids(dev, groups, with_bias):
    """The weights are ratios: sigmoid(-695) of four experts is a quarter each."""
    rng = np.random.default_rng([groups, with_bias])
    E, k = 16, 4
    rows = [np.full(E, v) for v in (-69.0, -690.0, -695.0, -705.0, -709.5)]
    rows += [np.full(E, -720.0), np.full(E, float(np.finfo(np.float32).min))]    # p is 0 in 64 bits
    rows += [rng.uniform(lo, hi, E) for lo, hi in ((-80, -60), (-709, -600), (-709, -690), (-708, -707),
                                                   (-1000, -650), (-120, 3), (-700, -75), (-800, 0))]
    l = np.array(rows, np.float32)
    bias = torch.zeros(E) if with_bias else None
    ids, w = M.route_topk(torch.from_numpy(l).to(dev), k, score="sigmoid", groups=groups,
                          topk_groups=groups, bias=None if bias is None else bias.to(dev))
    picked = np.take_along_axis(l, ids.cpu().numpy(), 1).astype(F)
    with np.errstate(over="ignore"):
        alive = np.isfinite(np.exp(-picked))            # the sigmoid is not 0 in 64 bits
    check_weights(w, picked - np.log1p(np.exp(picked)), alive)


def test_renormalized_weights_of_tiny_softmaxes(dev):
    """Experts picked by the bias far below the row's largest logit, which the bias takes out."""
    rng = np.random.default_rng(5)
    E, k, rows = 64, 4, []
    for lo, hi in ((-80, -60), (-700, -690), (-740, -700), (-650, -600), (-709, -100), (-30, 0)):
        r = rng.uniform(lo, hi, E)
        r[7] = 0.0
        rows.append(r)
    rows.append(np.where(np.arange(E) == 7, 0.0, -760.0))           # exp(-760) is 0 in 64 bits
    l = np.array(rows, np.float32)
    bias = torch.from_numpy(rng.uniform(1, 2, E).astype(np.float32))
    bias[7] = -INF
    ids, w = M.route_topk(torch.from_numpy(l).to(dev), k, bias=bias.to(dev))
    assert not (ids == 7).any()
    picked = np.take_along_axis(l, ids.cpu().numpy(), 1).astype(F)
    check_weights(w, picked, np.exp(picked) > 0)
