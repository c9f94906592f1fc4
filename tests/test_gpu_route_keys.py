"""Expert routing where two scores differ by less than their 32-bit keys: the order has to be that of
the 64-bit scores.  Experts are placed on either side of the borders at which a key changes."""
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


# (experts, experts a lane): a 32-bit key gives its lowest bits to the expert's place in its lane, so
# two scores next to a multiple of that many units in the last place are told apart the other way
@pytest.mark.parametrize("E,per_lane", [(128, 2), (256, 4), (384, 8), (1024, 16)])
@pytest.mark.parametrize("level", [0.0, 3.5, 7.5, 8.2, 15.5, 33.0, 64.0, -3.5, -9.0, -33.0])
def test_two_scores_on_either_side_of_a_key_border(dev, E, per_lane, level):
    rng = np.random.default_rng([E, int(level * 10) & 0xffff])
    T = 60000
    bias = (level + rng.uniform(-0.4, 0.4, E)).astype(np.float32)
    # the first or the last place in its lane: the largest shift of the key either way
    places = np.array([e for e in range(E) if e % per_lane in (0, per_lane - 1)])
    pair = np.stack([rng.choice(places, T), rng.choice(places, T)], 1)
    same = pair[:, 0] == pair[:, 1]
    pair[same, 1] = (pair[same, 0] + per_lane) % E
    ulp = 2.0 ** (np.floor(np.log2(abs(level + 0.6))) - 23)
    border = np.round((level + 0.6 + rng.uniform(-0.15, 0.15, T)) / (ulp * per_lane)) * ulp * per_lane
    b = bias[pair].astype(F)
    p = border[:, None] + rng.uniform(-0.8, -0.2, (T, 2)) * ulp - b
    l = logit(np.clip(p, 0.02, 0.98))
    c = sigmoid(l) + b
    # every other expert stays below: its score is its bias, at most level + 0.4
    ok = (p > 0.02) & (p < 0.98) & (c > level + 0.42)
    l[~ok.all(1)] = 1.0
    logits = torch.full((T, E), -40.0, device=dev)
    logits.scatter_(1, torch.from_numpy(pair).to(dev), torch.from_numpy(l).to(dev))
    ids, _ = M.route_topk(logits, 1, bias=torch.from_numpy(bias).to(dev), score="sigmoid")
    first = (c[:, 0] > c[:, 1]) | ((c[:, 0] == c[:, 1]) & (pair[:, 0] < pair[:, 1]))
    want = np.where(first, pair[:, 0], pair[:, 1])
    keep = ok.all(1)
    assert keep.mean() > 0.5
    wrong = (ids[:, 0].cpu().numpy() != want) & keep
    assert not wrong.any(), (int(wrong.sum()), int(keep.sum()))


def test_two_scores_apart_by_less_than_their_keys(dev):
    """Experts 0 and 31 of 1024: keys 4.367637 and 4.3676224, the 64-bit scores the other way."""
    logits, bias = torch.zeros(1, 1024), torch.zeros(1024)
    logits[0, 0], bias[0] = 1.4788669, 3.5532284
    logits[0, 31], bias[31] = -1.5739268, 4.1959724
    ids, _ = M.route_topk(logits.to(dev), 1, bias=bias.to(dev), score="sigmoid")
    want, _ = R.route(logits, 1, bias, "sigmoid", 1, 1, True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), want)
