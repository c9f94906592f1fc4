"""The sizes that tests compare with 64 bits reach every tile of the 8-bit floating point products."""
import pytest
import torch

import weight_only_bit_moe_amd as M
from tests import _expert as R
from tests import _expert_products as S


@pytest.mark.parametrize("want,size", S.PLAIN.items())
def test_plain(want, size):
    p = S.plan(*size)
    assert (p.tile, p.split) == want
    assert p.workspace == M.moe_wna16_gemm_fp8_workspace_size(*size)
    assert (p.workspace > 4096) == (p.split > 1) and (p.workspace == 0) == (p.split == 1)
    # more blocks than stages, with a part of one; remainders of every tile height and width
    assert size[2] > 8 * 128 and size[2] % 128 and size[0] % 64 and size[1] % 64


def test_every_tile_is_among_them():
    assert {t for t, s in S.PLAIN if s == 1} == set(range(S.TILES))
    assert {t for t, s in S.PLAIN if s > 1} == set(range(S.TILES))
    assert {s for _, s in S.PLAIN} == {1, 2, 4, 8, 16}
    assert {t for t, _ in S.GROUPED} == set(range(S.GROUPED_TILES))


@pytest.mark.parametrize("size", S.STREAMED)
def test_streamed(size):
    assert S.plan(*size).tile == -1 and M.moe_wna16_gemm_fp8_workspace_size(*size) == 0


@pytest.mark.parametrize("tile,size", S.GROUPED)
def test_grouped(tile, size):
    assert S.grouped_tile(*size) == tile
    assert size[3] > 8 * 128 and size[3] % 128


@pytest.mark.parametrize("split,K", [(2, 2192), (4, 8480), (16, 35888)])
def test_a_slice_that_is_missing_exceeds_the_bound(split, K):
    """Of a sum without one slice of K, most elements are further off than the tests allow."""
    g = torch.Generator()
    g.manual_seed(K)
    a, w = R.random_codes(g, 33, K), R.random_codes(g, 18, K)
    sa = torch.exp2(torch.floor(12 * torch.rand(33, R.blocks(K), generator=g)) - 9)
    sw = (torch.rand(1, R.blocks(K), generator=g) - 0.3) * 1e-2
    exact, terms, groups = R.product(a, sa, w, sw)
    bound = R.product_bound(exact, terms, groups, K, torch.bfloat16)
    for i in (0, split - 1):
        cut = slice(i * R.blocks(K) // split * 128, (i + 1) * R.blocks(K) // split * 128)
        part = R.values(a, sa)[:, cut] @ R.values(w, sw, 128)[:, cut].t()
        assert float((part.abs() > bound).double().mean()) > 0.5
