"""What the operators' documentation has to say: they give no gradient."""
import pytest

import weight_only_bit_moe_amd as M
from weight_only_bit_moe_amd import block_ops


@pytest.mark.parametrize("name", ["add_rmsnorm", "route_topk", "gemm_w8a8", "swiglu_quant"])
def test_no_gradient_is_documented(name):
    assert "No gradient" in getattr(M, name).__doc__
    assert "no output carries a graph" in block_ops.__doc__


def test_the_products_roundings_are_documented():
    assert "rounded\nonce" not in M.gemm_w8a8.__doc__ and "FP32" in M.gemm_w8a8.__doc__
