"""The workspaces that a block's steps take: how much of them is kept, and steps on several streams
and in captured graphs."""
import pytest
import torch

from tests import _gpu as G
from weight_only_bit_moe_amd import block as B
from weight_only_bit_moe_amd.inputs import LayerSpec

pytestmark = pytest.mark.gpu


def make(seed=3, shared=0, **kw):
    base = dict(name="block", T=1, H=512, I=256, E=16, topk=4, bits13=2, group13=128, bits2=2,
                group2=128, scale_lo=0.005, scale_hi=0.02)
    return B.synthetic(LayerSpec(**dict(base, **kw)), seed, G.device(), shared=shared)


def rows(T, seed=0):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(T, 512, generator=g).bfloat16().to(G.device())


def same(a, b):
    # the routed sum's FP32 additions have no fixed order
    return torch.allclose(a.float(), b.float(), rtol=2 ** -6, atol=1e-2)


def kept_bytes(block, counts):
    make()(rows(2))                                     # the libraries' own memory
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for T in counts:
        block(rows(T))
    torch.cuda.synchronize()
    return torch.cuda.memory_allocated() - before


def test_many_token_counts_keep_the_largest_workspace_only():
    """Steps of many token counts leave no more allocated than one of the largest."""
    one, many = make(), make()
    need = kept_bytes(one, [400])
    assert 0 < kept_bytes(many, list(range(1, 400, 7)) + [400, 3, 250]) <= need


def test_blocks_share_workspaces():
    a, b = make(3), make(4)
    one = kept_bytes(a, [300])
    b.workspaces = a.workspaces
    assert kept_bytes(b, [300, 17, 300]) == 0 < one
    fresh = make(4)
    for T in (300, 5, 70):
        a(rows(T))
        assert same(b(rows(T))[0], fresh(rows(T))[0])


@pytest.mark.parametrize("order", [(400, 3, 130, 90, 400), (3, 90, 130, 400, 64, 65), (1, 600, 1, 66)])
def test_steps_of_other_sizes_on_one_workspace(order):
    """Sizes that grow, shrink, run the layer in one launch and split the products' K."""
    block = make(shared=4096)
    for i, T in enumerate(order):
        x = rows(T, seed=i)
        assert same(block(x)[0], make(shared=4096)(x)[0]), T


def test_another_stream_has_its_own():
    block = make()
    x = rows(90)
    want = block(x)[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = block(x)[0]
    again = block(x)[0]                                 # both may run at once
    torch.cuda.synchronize()
    assert same(want, got) and same(want, again)


@pytest.mark.parametrize("T", [3, 130])
@pytest.mark.parametrize("given", [False, True])
def test_captured_steps_and_eager_ones_between(T, given):
    """A graph captured from a block's first step of this size; eager steps before the first replay
    and between replays, and larger ones, whose workspace takes the place of a smaller."""
    block = make(shared=4096)
    block(rows(2))                                # code loading is no part of a capture
    make(shared=4096)(rows(T))
    x = rows(T, seed=1)
    ws = block.workspace_for(T) if given else None
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block(x, workspace=ws)[0]
    fresh = make(shared=4096)
    for i in range(5):
        assert same(block(x)[0], fresh(x)[0])           # eager, the first before any replay
        graph.replay()
        torch.cuda.synchronize()
        assert same(held, fresh(x)[0])
        block(rows(T + 200 * i))                  # grows
        x.copy_(rows(T, seed=i + 2))


def test_workspace_given_by_the_caller():
    block = make()
    x = rows(100)
    ws = block.workspace_for(100)
    assert same(block(x, workspace=ws)[0], make()(x)[0])
    assert same(block(x[:3], workspace=ws)[0], make()(x[:3])[0])
    with pytest.raises(ValueError, match="too small"):
        block(rows(2000), workspace=ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        x.mul_(1)                                       # a graph is not empty
        with pytest.raises(RuntimeError, match="capture"):
            block.workspace_for(100)
