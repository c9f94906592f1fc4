"""Workspaces of the 8-bit product: exactly none where K is not split."""
import pytest

import weight_only_bit_moe_amd as M


@pytest.mark.parametrize("T,N,K,split", [
    (0, 64, 64, False), (4, 4096, 4096, False), (64, 4096, 2048, False), (2047, 2056, 4096, False),
    (8192, 4096, 4096, False), (128, 512, 16384, True), (128, 512, 4096, True)])
def test_product_workspace(T, N, K, split):
    n = M.moe_wna16_gemm_w8a8_workspace_size(T, N, K)
    if split:       # counters, and int32 sums of two slices or more
        assert n >= 4096 + 2 * 4 * T * N
    else:
        assert n == 0
