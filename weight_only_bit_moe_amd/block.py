"""One mixture-of-experts block of a decoder, as a serving step runs it:

    h, y, q = residual addition, root-mean-square norm, y in 8 bits   add_rmsnorm
    logits  = y @ gate.T                                              torch
    ids, w  = expert routing                                          route_topk
    out     = routed experts of y                                     forward
    out    += shared expert of q: product, SwiGLU in 8 bits, product  gemm_w8a8, swiglu_quant

and returns out and h, the residual stream that the next norm adds out to.

    python -m weight_only_bit_moe_amd.block --tokens 4      # time of a step on synthetic weights
"""
from __future__ import annotations

import dataclasses
import math
from typing import NamedTuple, Optional, Tuple

import torch

from . import binding, block_ops


def channel_codes(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rows of a weight in 8 bits: codes int8 and a float32 scale for each row (channel), the
    largest magnitude of a row at 127.  As in the operators, a row whose largest magnitude is below
    2^-100 gets zero codes and scale 0, one with a NaN or infinity zero codes and scale NaN.  Done
    once, when weights are loaded."""
    v = w.float()
    top = v.abs().amax(-1)
    finite = torch.isfinite(top)
    live = finite & (top >= 2.0 ** -100)
    mult = torch.where(live, 127.0 / top, torch.zeros_like(top))[:, None]
    codes = torch.where(live[:, None], torch.round(v * mult), torch.zeros_like(mult)).to(torch.int8)
    scale = torch.where(live, top / 127.0, torch.zeros_like(top))
    return codes, torch.where(finite, scale, torch.full_like(top, math.nan))


class StepWorkspace(NamedTuple):
    """Device memory of one step's calls: the routed layer's, and the shared expert's products'."""

    layer: torch.Tensor
    product: Optional[torch.Tensor]

    def holds(self, layer: int, product: int) -> bool:
        return (self.layer.numel() >= layer
                and (not product or (self.product is not None and self.product.numel() >= product)))


def _new_workspace(layer: int, product: int, device) -> StepWorkspace:
    """Of these sizes; the leading bytes that have to start at zero are zeroed on the current stream."""
    def make(n, sync):
        t = torch.empty(n, dtype=torch.uint8, device=device)
        t[:sync].zero_()
        return t
    return StepWorkspace(make(max(layer, binding.SYNC_BYTES), binding.SYNC_BYTES),
                         make(product, block_ops.GEMM_SYNC_BYTES) if product else None)


class Workspaces:
    """Workspaces of steps: one for each stream that steps run on, as large as a step on it has
    needed so far.  Steps on a stream follow each other there, so the blocks of a model can share
    one (MoEBlock's workspaces); two host threads that issue steps on one stream need one each.

    A step that is captured into a graph gets memory of the graph's own instead, cleared by the
    replay: what is kept here is cleared once, when it is made, and a larger one may take its place.
    """

    def __init__(self):
        self._kept = {}

    def get(self, layer: int, product: int, device: torch.device) -> StepWorkspace:
        """A workspace of at least these sizes in bytes, for a step on the device's current stream."""
        if device.index != torch.cuda.current_device():
            with torch.cuda.device(device):
                return self.get(layer, product, device)
        if torch.cuda.is_current_stream_capturing():
            return _new_workspace(layer, product, device)
        key = (device.index, torch._C._cuda_getCurrentRawStream(device.index))
        kept = self._kept.get(key)
        if kept is None or not kept.holds(layer, product):
            if kept is not None:                    # never smaller than the one it takes the place of
                layer = max(layer, kept.layer.numel())
                product = max(product, 0 if kept.product is None else kept.product.numel())
                del kept, self._kept[key]           # released before the new one is made
            kept = self._kept[key] = _new_workspace(layer, product, device)
        return kept


@dataclasses.dataclass
class MoEBlock:
    """Weights and routing of one block.  The routed experts' tensors are forward()'s; the shared
    expert's are int8 codes with a scale for each channel (channel_codes).  Steps take their
    workspace from `workspaces`; pass the same one to all blocks of a model."""

    norm: torch.Tensor                      # [H] bf16
    gate: torch.Tensor                      # [E, H], router: float32, or bf16 (rounds the logits too)
    w13: torch.Tensor                       # routed experts: codes and scales
    s13: torch.Tensor
    w2: torch.Tensor
    s2: torch.Tensor
    bits: Tuple[int, int]
    group: Tuple[int, int]
    shared13: torch.Tensor                  # [2 Is, H] int8, gate rows then up rows
    shared13_scale: torch.Tensor            # [2 Is] float32
    shared2: torch.Tensor                   # [H, Is] int8
    shared2_scale: torch.Tensor             # [H] float32
    topk: int
    bias: Optional[torch.Tensor] = None     # [E] float32, balance
    score: str = "softmax"
    groups: int = 1
    topk_groups: int = 1
    renormalize: bool = True
    route_scale: float = 1.0
    alpha: float = 1.0
    beta: float = 0.0
    clamp: Optional[float] = None
    eps: float = 1e-6
    workspaces: Workspaces = dataclasses.field(default_factory=Workspaces, repr=False)
    _need: dict = dataclasses.field(default_factory=dict, repr=False)   # _sizes, kept

    def _sizes(self, T: int):
        """Bytes that a step's layer and its two products need."""
        n = self._need.get((T, self.topk))
        if n is None:
            H, E, I = self.norm.numel(), self.w13.shape[0], self.w13.shape[1] // 2
            two_is, Is = self.shared13.shape[0], self.shared2.shape[1]
            n = self._need[T, self.topk] = (
                binding.moe_wna16_workspace_size(T, H, I, E, self.topk),
                max(block_ops.moe_wna16_gemm_w8a8_workspace_size(T, two_is, H),
                    block_ops.moe_wna16_gemm_w8a8_workspace_size(T, H, Is)))
        return n

    def workspace_for(self, T: int) -> StepWorkspace:
        """A workspace for steps of T tokens that the caller keeps, and clears by making it: for
        steps captured into a graph, which then need not clear one, one for each graph."""
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("workspace_for inside a capture: its fill would run in replays only")
        return _new_workspace(*self._sizes(T), self.norm.device)

    def route(self, y: torch.Tensor):
        """Expert ids and routing weights of normed rows y [T, H] bf16, from logits of gate's type."""
        logits = torch.nn.functional.linear(y.to(self.gate.dtype), self.gate)
        return block_ops.route_topk(logits, self.topk, bias=self.bias, score=self.score,
                                    groups=self.groups, topk_groups=self.topk_groups,
                                    renormalize=self.renormalize, scale=self.route_scale)

    def shared(self, q, scale, addend, workspaces=(None, None)):
        """The shared expert of rows in 8 bits, added to `addend` [T, H] bf16 in place.  workspaces:
        the two products', which may be one."""
        gu = block_ops.gemm_w8a8(q, scale, self.shared13, self.shared13_scale,
                                 workspace=workspaces[0])
        aq, ascale = block_ops.swiglu_quant(gu, alpha=self.alpha, beta=self.beta, clamp=self.clamp)
        return block_ops.gemm_w8a8(aq, ascale, self.shared2, self.shared2_scale, addend=addend,
                                   out=addend, workspace=workspaces[1])

    def __call__(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                 workspace: Optional[StepWorkspace] = None):
        """x [T, H] bf16, the block's input, and the residual stream it is added to (None at the
        start of the stack).  Returns (out, residual stream).  workspace: from workspace_for, used by
        one step at a time; one of `workspaces` if not given."""
        sizes = self._sizes(x.shape[0])
        if workspace is None:
            workspace = self.workspaces.get(*sizes, x.device)
        elif not workspace.holds(*sizes):
            raise ValueError(f"the workspace is too small for {x.shape[0]} tokens")
        n = block_ops.add_rmsnorm(x, self.norm, residual, eps=self.eps, quant=True)
        ids, w = self.route(n["y"])
        out = binding.forward(n["y"], ids, w, self.w13, self.s13, self.w2, self.s2, bits=self.bits,
                              group=self.group, alpha=self.alpha, beta=self.beta, clamp=self.clamp,
                              workspace=workspace.layer)
        out = self.shared(n["q"], n["scale"], out, (workspace.product, workspace.product))
        return out, n.get("residual", x)


def synthetic(spec, seed: int, device, shared: int = 0) -> MoEBlock:
    """A block with the random routed experts of an inputs.LayerSpec (its T and routing are not
    used) and random other weights; shared: the shared expert's intermediate size (0: spec.I)."""
    import numpy as np

    from .inputs import make_layer
    L = make_layer(dataclasses.replace(spec, T=1), seed)
    Is = shared or spec.I
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    c13, sc13 = channel_codes(randn(2 * Is, spec.H) * spec.H ** -0.5)
    c2, sc2 = channel_codes(randn(spec.H, Is) * Is ** -0.5)
    dev = lambda a: torch.from_numpy(a).to(device)  # noqa: E731
    return MoEBlock(
        norm=(1 + 0.1 * randn(spec.H)).bfloat16(), gate=(randn(spec.E, spec.H) * spec.H ** -0.5).bfloat16(),
        w13=dev(L.w13.view(np.int32)), s13=dev(L.s13), w2=dev(L.w2.view(np.int32)), s2=dev(L.s2),
        bits=(spec.bits13, spec.bits2), group=(spec.group13, spec.group2), shared13=c13,
        shared13_scale=sc13, shared2=c2, shared2_scale=sc2, topk=spec.topk, bias=0.05 * randn(spec.E),
        score="sigmoid", route_scale=1.0, alpha=spec.alpha, beta=spec.beta,
        clamp=None if math.isinf(spec.clamp) else spec.clamp)


def main() -> None:
    import argparse
    import time

    from .inputs import CONFIGS
    ap = argparse.ArgumentParser(description="Time of one block's step on synthetic weights "
                                             "(hidden 4096, 256 experts of 2048, 2-bit codes).")
    ap.add_argument("--tokens", type=int, default=4)
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    block = synthetic(CONFIGS[2], 1, dev)
    H = CONFIGS[2].H
    x, r = (torch.randn(a.tokens, H, device=dev).bfloat16() for _ in range(2))
    for _ in range(5):
        out, h = block(x, r)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        out, h = block(x, r)
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens: {(time.perf_counter() - t) / a.steps * 1e6:.1f} us a step")


if __name__ == "__main__":
    main()
