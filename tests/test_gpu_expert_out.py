"""Memory handed in for results: autograd learns that it has changed."""
import pytest
import torch

import weight_only_bit_moe_amd as M
from tests import _expert as R
from tests.test_gpu_expert_grads import case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


def test_a_buffer_used_again_before_its_gradient(dev):
    """Rows sorted into one buffer twice, with parameters behind each: the first step's gradient needs
    the first step's rows."""
    ids, x, w, E = case(dev)
    x = x.detach()
    buf = torch.empty(ids.numel(), x.shape[1], device=dev)
    scale = torch.ones(x.shape[1], device=dev, requires_grad=True)
    y = M.sort_tokens(ids, E, x, out=buf)["x"] * scale
    M.sort_tokens(ids, E, 2 * x, out=buf)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    total = torch.empty_like(x)
    s = M.sort_tokens(ids, E, x)
    z = M.combine_tokens(s["x"], s["slots"], out=total) * scale
    M.combine_tokens(s["x"], s["slots"], addend=x, out=total)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.sum().backward()


def test_every_result_counts_as_changed(dev):
    x = torch.randn(4, 256, device=dev)
    q, s = M.quant_fp8(x)
    w, ws = torch.zeros(64, 256, device=dev).to(R.E4M3), torch.ones(1, 2, device=dev)
    q2, s2 = M.swiglu_quant_fp8(x)
    out, rows = torch.empty(4, 64, device=dev), torch.empty(4, 64, device=dev)
    off = torch.tensor([0, 4], dtype=torch.int32, device=dev)
    calls = [((q, s), lambda: M.quant_fp8(x, q=q, scale=s)), ((q2, s2), lambda: M.swiglu_quant_fp8(x, q=q2, scale=s2)),
             ((out,), lambda: M.gemm_fp8(q, s, w, ws, out_dtype=torch.float32, out=out)),
             ((rows,), lambda: M.gemm_fp8_grouped(q, s, w[None], ws[None], off, out_dtype=torch.float32, out=rows))]
    for tensors, call in calls:
        before = [t._version for t in tensors]
        call()
        assert [t._version for t in tensors] == [v + 1 for v in before]


def test_inference_tensors_and_modes(dev):
    """Memory made in inference mode is taken inside and outside of it."""
    ids, x, w, E = case(dev)
    x = x.detach()
    want = M.sort_tokens(ids, E, x)["x"]
    with torch.inference_mode():
        buf = torch.zeros_like(want)
        assert M.sort_tokens(ids, E, x, out=buf)["x"] is buf and torch.equal(buf, want)
    buf = torch.zeros_like(buf.clone())
    with torch.inference_mode():
        held = torch.zeros_like(want)
    assert torch.equal(M.sort_tokens(ids, E, x, out=held)["x"], want)


def test_memory_in_a_graph_is_refused(dev):
    ids, x, w, E = case(dev)
    rows = torch.zeros(ids.numel(), x.shape[1], device=dev)
    s = M.sort_tokens(ids, E, x.detach())
    for make in (lambda t: t.clone().requires_grad_(), lambda t: t.clone().requires_grad_() * 1.0):
        a, b = make(rows), make(x.detach())
        with pytest.raises(ValueError, match="out requires a gradient"):
            M.sort_tokens(ids, E, x.detach(), out=a)
        with pytest.raises(ValueError, match="out requires a gradient"):
            M.combine_tokens(s["x"], s["slots"], out=b)
        with torch.no_grad():
            assert torch.equal(M.sort_tokens(ids, E, x, out=a)["x"], s["x"])
            assert M.combine_tokens(s["x"], s["slots"], out=b) is b
