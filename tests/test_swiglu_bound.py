"""The bound that the GPU test holds the SwiGLU's elements to sees the exponent's correction."""
import numpy as np

from tests import _swiglu_bound as B


def test_bound_holds_with_the_correction_and_fails_without():
    g = B.samples(1)
    ref = B.silu(g)
    bound = B.element_bound(g.astype(np.float64), True) * np.abs(ref)
    assert (np.abs(B.silu_fp32(g, True) - ref) <= bound).all()
    assert (np.abs(B.silu_fp32(g, False) - ref) > bound).mean() > 0.1
