"""Error of one element of the SwiGLU kernels' FP32 arithmetic, in roundings of 2^-24.

With x = alpha g: exp2 and the reciprocal are good to a unit in the last place (two roundings each);
the correction of the exponent's rounding, the product with it, 1 + p, g s, u + beta and their
product add one each; alpha g adds |x| where alpha is not 1.  The scale's division adds one more."""
import numpy as np

from tests import _block as R


def element_bound(x, alpha_is_one):
    return (2 + 2 + 6 + 1 + (0 if alpha_is_one else np.abs(x))) * R.U * (1 + 2.0 ** -20)


def silu_fp32(g, compensated):
    """The kernel's steps for alpha = 1, u = 1 in numpy, with or without the exponent's correction."""
    f = np.float32
    log2e, low, ln2 = f(1.44269502), f(1.92596303e-8), f(0.693147181)
    t = (-g * log2e).astype(f)
    e = (-g.astype(np.float64) * log2e - t).astype(f)                # exact, as the fused product
    e = (-g.astype(np.float64) * low + e).astype(f)
    p = np.exp2(t.astype(np.float64)).astype(f)
    if compensated:
        p = (p * (e.astype(np.float64) * ln2 + 1.0).astype(f)).astype(f)
    s = (f(1) / (f(1) + p)).astype(f)
    return (g * s).astype(f)


def samples(seed, n=20000):
    return np.random.default_rng(seed).uniform(-60, 60, n).astype(np.float32)


def silu(g):
    g = g.astype(np.float64)
    return g / (1.0 + np.exp(-g))
