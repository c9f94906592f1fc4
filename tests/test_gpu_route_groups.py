"""Group-limited expert routing where the 32-bit sum of a group's two scores is off by more than the
sum itself shows: the groups kept have to be those of the 64-bit sums."""
import numpy as np
import pytest
import torch

import weight_only_bit_moe_amd as M
from tests import _block as R

pytestmark = pytest.mark.gpu

F = np.float64


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


def sigmoid(l):
    return 1.0 / (1.0 + np.exp(-l.astype(F)))


def logit(p):
    return np.log(p / (1.0 - p)).astype(np.float32)


# groups that are runs of whole lanes (merged by permutes), and others (through LDS)
@pytest.mark.parametrize("E,groups", [(16, 8), (256, 8), (512, 16), (160, 8), (96, 32)])
@pytest.mark.parametrize("size", [0.5, 10.0, 100.0, 1000.0, 1e4])
def test_groups_whose_two_scores_cancel(dev, E, groups, size):
    """A group's two largest scores are p + size and p - size: the 32-bit sum is off by the rounding
    of either, not of the sum."""
    rng = np.random.default_rng([E, groups, int(size * 10)])
    T, per = 3000, E // groups
    b = (size * (1 + 0.1 * rng.uniform(-1, 1, groups))).astype(np.float32)
    bias = np.full((groups, per), -20 * size - 5 * groups, np.float32)
    bias[:, 0], bias[:, per - 1] = b, -b
    bias[1:-1, per - 1] -= 3 + 2 * np.arange(groups - 2, dtype=np.float32)  # all but the first and last: far
    l = np.full((T, groups, per), -40.0, np.float32)
    t, a = np.arange(T), np.tile([0, groups - 1], (T, 1))
    p = rng.uniform(0.3, 0.7, (T, 3))
    l[t, a[:, 0], 0], l[t, a[:, 0], per - 1], l[t, a[:, 1], 0] = logit(p).T
    total = sigmoid(l[t, a[:, 0], 0]) + sigmoid(l[t, a[:, 0], per - 1])
    near = rng.uniform(-1, 1, T) * 2.0 ** -23 * (1 + size)
    rest = total + near - sigmoid(l[t, a[:, 1], 0])
    l[t, a[:, 1], per - 1] = logit(np.clip(rest, 0.01, 0.99))
    logits, bias = torch.from_numpy(l.reshape(T, E)), torch.from_numpy(bias.reshape(E))
    want, _ = R.route(logits, 2, bias, "sigmoid", groups, 1, True, 1.0)
    ids, _ = M.route_topk(logits.to(dev), 2, bias=bias.to(dev), score="sigmoid", groups=groups,
                          topk_groups=1)
    wrong = (ids.cpu().numpy() != want).any(1)
    assert not wrong.any(), int(wrong.sum())


def test_two_groups_apart_by_less_than_their_scores(dev):
    """32-bit sums 1.354065 and 1.3540573, 64-bit sums the other way round."""
    logits = torch.tensor([[0.004597960, 1.757609248, 0.004603488, 1.757599115]])
    bias = torch.tensor([100.0, -100.0, 100.3, -100.3])
    ids, _ = M.route_topk(logits.to(dev), 1, bias=bias.to(dev), score="sigmoid", groups=2,
                          topk_groups=1)
    want, _ = R.route(logits, 1, bias, "sigmoid", 2, 1, True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("E,groups", [(4, 2), (64, 4), (60, 4), (256, 8), (160, 8)])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_groups_of_finite_scores_whose_sum_overflows_32_bits(dev, E, groups, sign):
    """Biases near the largest float: the sum of two is an infinity in 32 bits, and a group of them
    is neither empty nor equal to the others."""
    rng = np.random.default_rng([E, groups])
    bias = torch.from_numpy((sign * rng.uniform(2e38, 3.4e38, E)).astype(np.float32))
    logits = torch.from_numpy(rng.normal(size=(20, E)).astype(np.float32))
    for score in ("softmax", "sigmoid"):
        for kg in (1, 2):
            k = min(4, E // groups * kg)
            want, _ = R.route(logits, k, bias, score, groups, kg, True, 1.0)
            ids, _ = M.route_topk(logits.to(dev), k, bias=bias.to(dev), score=score, groups=groups,
                                  topk_groups=kg)
            assert np.array_equal(ids.cpu().numpy(), want)
