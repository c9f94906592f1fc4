"""The residual norm and the SwiGLU in 8 bits against the errors that their steps can add up to,
element by element."""
import numpy as np
import pytest
import torch

import weight_only_bit_moe_amd as M
from tests import _block as R
from tests import _swiglu_bound as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


@pytest.mark.parametrize("alpha", [1.0, 1.702])
def test_swiglu_elements(dev, alpha):
    """Rows of one element: the scale is the element's magnitude / 127."""
    g = B.samples(2)
    gu = torch.from_numpy(np.stack([g, np.ones_like(g)], 1)).to(dev)
    q, scale = M.swiglu_quant(gu, alpha=alpha)
    x = g.astype(np.float64) * np.float32(alpha).astype(np.float64)
    a = g.astype(np.float64) / (1.0 + np.exp(-x))
    live = np.abs(a) >= 2.0 ** -99
    off = np.abs(scale.cpu().numpy().astype(np.float64) * 127 - np.abs(a))
    over = (off > B.element_bound(x, alpha == 1.0) * np.abs(a)) & live
    assert not over.any(), (int(over.sum()), float((off[live] / np.abs(a[live])).max() / R.U))
    assert np.array_equal(q[:, 0].cpu().numpy()[live], np.sign(a[live]).astype(np.int8) * 127)


# a thread adds up to 4 chunks of 8 squares, a wave and the row's waves 6 and 4 steps: 42 roundings
# and the mean's two, half of which survive the square root; root, division, weight, rstd: 6
NORM_U = (32 + 10 + 2) / 2 + 6


@pytest.mark.parametrize("H", [8, 512, 4096, 8192, 8200, 16384, 20001, 32768])
def test_norm_elements(dev, H):
    g = torch.Generator()
    g.manual_seed(H)
    x = torch.randn(64, H, generator=g) * torch.exp(torch.randn(64, 1, generator=g))
    w = 1 + 0.3 * torch.randn(H, generator=g)
    got = M.add_rmsnorm(x.to(dev), w.to(dev), quant=True)
    _, y, q, scale, _ = R.rmsnorm(x, None, w, 1e-6)
    off = ((got["y"].cpu().to(R.F) - y).abs() / y.abs().clamp(min=2.0 ** -120)).max()
    assert float(off) <= NORM_U * R.U, float(off) / R.U
    assert torch.equal(got["q"].cpu(), q)
    assert bool(((got["scale"].cpu().to(R.F) - scale).abs() <= (NORM_U + 2) * R.U * scale).all())
