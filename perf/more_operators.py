"""Measured cases of the operators for experts in 8-bit floating point.

A routed or shared expert whose weights are e4m3 codes with a scale for each 128 x 128 block
runs, next to the operators of perf/operators.py:

    quant    rows in e4m3 with a power-of-two scale for each 128 elements, of the rows themselves
             (weight_only_bit_moe_amd.quant_fp8) or of their SwiGLU (swiglu_quant_fp8)
    gemm     the product of such rows with such weights (gemm_fp8)
    grouped  the same for rows sorted by expert, each expert with weights of its own
             (gemm_fp8_grouped)
    sort     tokens' rows in the order of their experts, and its gradient (sort_tokens)
    combine  experts' rows back to their tokens, weighted and added up, and its gradient
             (combine_tokens)

`run` computes a case in its plain form with elementary torch operations, or, with `own`
set, through the package's entry points.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_E4M3 = torch.float8_e4m3fn
_TOP = 448.0                                    # largest e4m3 value


def listed():
    return [
        # an odd chunk's normed rows in half precision, before the gate/up product
        dict(name="quant-T2047-fp16", op="quant", T=2047, K=4096, dtype="fp16", swiglu=False),
        # the large prefill chunk's activation, before the shared expert's down product
        dict(name="swiglu-prefill-T8192", op="quant", T=8192, K=2048, dtype="bf16", swiglu=True,
             alpha=1.702, beta=1.0, clamp=7.0),
        # the shared expert's gate/up product of four decode tokens: streams the weights
        dict(name="gemm-decode-T4", op="gemm", T=4, N=4096, K=4096, out="bf16", addend=False),
        # an odd chunk, an odd share of the columns, a last block that is a part, an addend
        dict(name="gemm-T2047-fp16", op="gemm", T=2047, N=2057, K=4048, out="fp16", addend=True),
        # the large prefill chunk's gate/up product
        dict(name="gemm-prefill-T8192", op="gemm", T=8192, N=4096, K=4096, out="bf16",
             addend=False),
        # decode: gate/up products of four tokens with the six experts of each
        dict(name="grouped-decode-T4", op="grouped", T=4, topk=6, E=256, here=256, N=4096, K=4096,
             out="bf16", gather=True),
        # batched decode: down products, the rows already in the experts' order
        dict(name="grouped-down-T64", op="grouped", T=64, topk=6, E=256, here=256, N=4096, K=2048,
             out="bf16", gather=False),
        # the large prefill chunk's gate/up products
        dict(name="grouped-prefill-T8192", op="grouped", T=8192, topk=8, E=256, here=256, N=4096,
             K=4096, out="bf16", gather=True),
        # batched decode on a GPU that holds a quarter of the experts
        dict(name="sort-T64", op="sort", T=64, topk=6, E=256, here=64, H=4096, dtype="bf16",
             grad=False),
        # a training step's chunk, forward and backward
        dict(name="sort-train-T4096", op="sort", T=4096, topk=8, E=256, here=256, H=4096,
             dtype="bf16", grad=True),
        # batched decode, added to the shared expert's rows
        dict(name="combine-T64", op="combine", T=64, topk=6, E=256, here=256, H=4096,
             dtype="bf16", addend=True, grad=False),
        # a training step's chunk, forward and backward to the rows and the weights
        dict(name="combine-train-T4096", op="combine", T=4096, topk=8, E=256, here=256, H=4096,
             dtype="bf16", addend=False, grad=True),
    ]


def _spread(rng, lo, hi):
    """An odd integer or a power of two in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    if rng.random() < 0.7:
        return min(int(v) | 1, (hi - 1) | 1)
    return min(1 << int(round(math.log2(v))), hi)


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "grouped", "grouped", "sort", "combine"])
    if op == "quant":
        swiglu = rng.random() < 0.5
        case = dict(op=op, T=_spread(rng, 1, 8191), dtype=rng.choice(["bf16", "fp16"]),
                    K=rng.choice([128 * rng.randint(1, 16), _spread(rng, 64, 2048)]),
                    swiglu=swiglu)
        if swiglu:
            case.update(alpha=rng.choice([1.0, 1.702]), beta=rng.choice([0.0, 1.0]),
                        clamp=rng.choice([0.0, 7.0]))
        return case
    if op == "gemm":
        return dict(op=op, T=_spread(rng, 1, 8191),
                    N=rng.choice([128 * rng.randint(2, 32), _spread(rng, 256, 4096)]),
                    K=rng.choice([16 * rng.randint(16, 256), 128 * rng.randint(2, 32)]),
                    out=rng.choice(["bf16", "fp16"]), addend=rng.random() < 0.5)
    E = rng.choice([8, 32, 64, 160, 256])
    topk = rng.randint(1, 8)
    here = rng.choice([E, E, E // 4])
    if op == "grouped":
        return dict(op=op, T=_spread(rng, 1, 4095), topk=topk, E=E, here=here,
                    N=rng.choice([128 * rng.randint(2, 16), _spread(rng, 256, 2047)]),
                    K=rng.choice([16 * rng.randint(16, 128), 128 * rng.randint(2, 16)]),
                    out=rng.choice(["bf16", "fp16"]), gather=rng.random() < 0.5)
    grad = rng.random() < 0.5
    case = dict(op=op, T=_spread(rng, 1, 2047), topk=topk, E=E,
                here=E if op == "sort" and grad else here,
                H=rng.choice([128 * rng.randint(2, 32), _spread(rng, 96, 4096)]),
                dtype=rng.choice(["bf16", "fp16", "fp32"]), grad=grad)
    if op == "combine":
        case["addend"] = rng.random() < 0.5
    return case


# ---- what a program has in hand ----------------------------------------------

def _power(e):
    """2^e in float32 for whole numbers e, -126 <= e <= 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _rows_to_codes(x):
    """Rows in e4m3 with a power-of-two scale for each 128 elements (the last part may be less)."""
    T, K = x.shape
    blocks = -(-K // 128)
    v = torch.zeros(T, blocks * 128, device=x.device)
    v[:, :K] = x
    v = v.view(T, blocks, 128)
    mant, expo = torch.frexp(v.abs().amax(-1))          # top = mant 2^expo, mant in [1/2, 1)
    # the smallest power of two s with top <= 448 s = 0.875 2^9 s
    s = _power(torch.where(mant <= 0.875, expo - 9, expo - 8).clamp(min=-126))
    q = (v / s.unsqueeze(-1)).to(_E4M3)
    return q.view(T, blocks * 128)[:, :K].contiguous(), s


def _weight_to_codes(w):
    """A weight in e4m3 with a float32 scale for each 128 x 128 block, as checkpoints have it."""
    N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    v = torch.zeros(nb * 128, kb * 128, device=w.device)
    v[:N, :K] = w
    v = v.view(nb, 128, kb, 128)
    s = v.abs().amax((1, 3)) / _TOP
    q = (v / s[:, None, :, None]).to(_E4M3).view(nb * 128, kb * 128)[:N, :K]
    return q.contiguous(), s


def _ids(case, randn):
    """Distinct expert ids of each token; some experts are drawn to more than others."""
    pull = 0.4 * randn(case["E"])
    return torch.topk(randn(case["T"], case["E"]) + pull, case["topk"], -1)[1].to(torch.int32)


def _order(ids, here):
    """tokens, slots and offsets of a stable sort of the pairs by expert; ids from `here` on are
    other GPUs' experts."""
    T, topk = ids.shape
    flat = ids.reshape(-1).long()
    mine = (flat >= 0) & (flat < here)
    key = torch.where(mine, flat, torch.full_like(flat, here))
    order = torch.sort(key, stable=True)[1]
    at = torch.arange(T * topk, device=ids.device)
    slots = torch.empty_like(flat)
    slots[order] = at
    slots = torch.where(mine, slots, torch.full_like(slots, -1)).view(T, topk)
    counts = (key[:, None] == torch.arange(here, device=ids.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    tokens = torch.where(at < offsets[-1], order // topk, torch.full_like(order, -1))
    return tokens.to(torch.int32), slots.to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    op, T = case["op"], case["T"]
    s = dict(case)
    if op == "quant":
        # activations with a few outlier channels, tokens of different sizes
        n = 2 * case["K"] if case["swiglu"] else case["K"]
        s["x"] = (1.5 * randn(T, n) * torch.exp(0.5 * randn(n)) *
                  (1.0 if case["swiglu"] else torch.exp(0.5 * randn(T, 1)))).to(_DT[case["dtype"]])
        return s
    if op == "gemm":
        N, K = case["N"], case["K"]
        s["a"], s["sa"] = _rows_to_codes(randn(T, K) * torch.exp(0.5 * randn(K)))
        s["w"], s["sw"] = _weight_to_codes(randn(N, K) * torch.exp(0.3 * randn(N, 1)) * K ** -0.5)
        s["add"] = randn(T, N).to(_DT[case["out"]]) if case["addend"] else None
        s["ws"] = None
        if own:
            import weight_only_bit_moe_amd as M
            s["ws"] = M.gemm_fp8_workspace_for(T, N, K, dev)  # kept by a serving program
        return s
    ids = _ids(case, randn)
    P = T * case["topk"]
    if op == "sort":
        H, dt = case["H"], _DT[case["dtype"]]
        s["ids"] = ids
        s["x"] = randn(T, H).to(dt).requires_grad_(case["grad"])
        s["dxs"] = randn(P, H).to(dt) if case["grad"] else None
        # rows of other GPUs' experts are not written
        s["out"] = None if case["grad"] else torch.zeros(P, H, dtype=dt, device=dev)
        return s
    tokens, slots, offsets = _order(ids, case["here"])
    if op == "combine":
        H, dt = case["H"], _DT[case["dtype"]]
        s["slots"], s["offsets"] = slots, offsets
        s["y"] = randn(P, H).to(dt).requires_grad_(case["grad"])
        w = torch.exp(randn(T, case["topk"]))
        s["weights"] = (w / w.sum(-1, keepdim=True)).requires_grad_(case["grad"])
        s["add"] = randn(T, H).to(dt) if case["addend"] else None
        s["dout"] = randn(T, H).to(dt) if case["grad"] else None
        return s
    N, K, here = case["N"], case["K"], case["here"]
    s["w"] = torch.empty(here, N, K, dtype=_E4M3, device=dev)
    s["sw"] = torch.empty(here, -(-N // 128), -(-K // 128), device=dev)
    for e in range(here):
        s["w"][e], s["sw"][e] = _weight_to_codes(randn(N, K) * K ** -0.5)
    s["a"], s["sa"] = _rows_to_codes(randn(T if case["gather"] else P, K) * torch.exp(0.5 * randn(K)))
    s["rows"] = tokens if case["gather"] else None
    s["offsets"] = offsets
    s["out_rows"] = torch.zeros(P, N, dtype=_DT[case["out"]], device=dev)
    # for the plain form: the experts that have rows, and the most rows of one
    counts = offsets[1:] - offsets[:-1]
    s["active"], s["most"] = torch.nonzero(counts).view(-1), int(counts.max())
    return s


# ---- the calls ---------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _values(q, scale):
    """Codes and their blocks' scales as the bfloat16 values they stand for (exact)."""
    T, K = q.shape
    v = q.to(torch.bfloat16)
    if K % 128 == 0:
        v.view(T, K // 128, 128).mul_(scale.unsqueeze(-1))
        return v
    return v.mul_(scale.repeat_interleave(128, 1)[:, :K])


def _run_own(s):
    import weight_only_bit_moe_amd as M
    op = s["op"]
    if op == "quant":
        if s["swiglu"]:
            return _values(*M.swiglu_quant_fp8(s["x"], alpha=s["alpha"], beta=s["beta"],
                                               clamp=s["clamp"] or None))
        q, scale = M.quant_fp8(s["x"])
        return dict(q=q, scale=scale)
    if op == "gemm":
        return M.gemm_fp8(s["a"], s["sa"], s["w"], s["sw"], addend=s["add"],
                          out_dtype=_DT[s["out"]], workspace=s["ws"])
    if op == "grouped":
        return M.gemm_fp8_grouped(s["a"], s["sa"], s["w"], s["sw"], s["offsets"], rows=s["rows"],
                                  out_dtype=_DT[s["out"]], out=s["out_rows"])
    if op == "sort":
        r = M.sort_tokens(s["ids"], s["here"], s["x"], out=s["out"])
        if s["grad"]:
            r["dx"] = torch.autograd.grad(r["x"], s["x"], s["dxs"])[0]
        return r
    out = M.combine_tokens(s["y"], s["slots"], s["weights"], offsets=s["offsets"], addend=s["add"])
    if not s["grad"]:
        return out
    dy, dw = torch.autograd.grad(out, (s["y"], s["weights"]), s["dout"])
    return dict(out=out, dy=dy, dweights=dw)


def _scaled(q, scale):
    """Codes [.., n, K] times their scales [.., n or blocks of 128 n, blocks of 128 K], float32."""
    v = q.float()
    n, K = q.shape[-2:]
    if scale.shape[-2] != n:
        scale = scale.repeat_interleave(128, -2)[..., :n, :]
    if K % 128 == 0:
        v.view(*q.shape[:-1], K // 128, 128).mul_(scale.unsqueeze(-1))
        return v
    return v.mul_(scale.repeat_interleave(128, -1)[..., :K])


def _run_plain(s):
    op = s["op"]
    if op == "quant":
        x = s["x"].float()
        if not s["swiglu"]:
            q, scale = _rows_to_codes(x)
            return dict(q=q, scale=scale)
        g, u = x.chunk(2, dim=-1)
        if s["clamp"]:
            g, u = torch.clamp(g, max=s["clamp"]), torch.clamp(u, -s["clamp"], s["clamp"])
        return _values(*_rows_to_codes(g / (1.0 + torch.exp(-s["alpha"] * g)) * (u + s["beta"])))
    if op == "gemm":
        y = _scaled(s["a"], s["sa"]) @ _scaled(s["w"], s["sw"]).t()
        if s["add"] is not None:
            y = y + s["add"].float()
        return y.to(_DT[s["out"]])
    if op == "grouped":
        # each active expert's rows, filled up to the most that one has
        off = s["offsets"].long()
        P, act, most = s["out_rows"].shape[0], s["active"], s["most"]
        if not most:
            return s["out_rows"]
        at = torch.arange(P, device=off.device)
        a = _scaled(s["a"], s["sa"])
        place = off[act][:, None] + torch.arange(most, device=off.device)
        place = torch.minimum(place, off[-1] - 1)
        src = place if s["rows"] is None else s["rows"].long()[place]
        y = torch.bmm(a[src], _scaled(s["w"][act], s["sw"][act]).transpose(1, 2))
        e = (at[:, None] >= off[act + 1]).sum(-1).clamp(max=act.numel() - 1)
        y = y[e, (at - off[act][e]).clamp(max=most - 1)].to(_DT[s["out"]])
        s["out_rows"].copy_(torch.where((at < off[-1])[:, None], y, torch.zeros_like(y)))
        return s["out_rows"]
    if op == "sort":
        x = s["x"].detach()
        tokens, slots, offsets = _order(s["ids"], s["here"])
        xs = x[tokens.clamp(min=0).long()]
        if not s["grad"]:
            s["out"].copy_(torch.where(tokens[:, None] >= 0, xs, torch.zeros_like(xs)))
            return dict(tokens=tokens, slots=slots, offsets=offsets, x=s["out"])
        dx = _gathered(s["dxs"], slots).sum(1).to(x.dtype)
        return dict(tokens=tokens, slots=slots, offsets=offsets, x=xs, dx=dx)
    y, w, slots = s["y"].detach(), s["weights"].detach(), s["slots"]
    rows = _gathered(y, slots)
    out = (rows * w.unsqueeze(-1)).sum(1)
    if s["add"] is not None:
        out = out + s["add"].float()
    out = out.to(y.dtype)
    if not s["grad"]:
        return out
    d = s["dout"].float()
    R = y.shape[0]
    dy = torch.zeros(R + 1, y.shape[1], dtype=y.dtype, device=y.device)
    to = torch.where(slots >= 0, slots, torch.full_like(slots, R)).long().view(-1)
    dy[to] = (d[:, None, :] * w.unsqueeze(-1)).to(y.dtype).flatten(0, 1)
    return dict(out=out, dy=dy[:R], dweights=(rows * d[:, None, :]).sum(-1))


def _gathered(y, slots):
    """Each token's rows [T, k, H] in float32; zeros where a slot is -1."""
    rows = y[slots.clamp(min=0).long()].float()
    return torch.where(slots[..., None] >= 0, rows, torch.zeros_like(rows))


# ---- what a pass cannot do without ---------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    if op == "quant":
        K = case["K"]
        n = 2 * K if case["swiglu"] else K
        return {"bytes": T * (n * _BYTES[case["dtype"]] + K + 4 * -(-K // 128)),
                "flops": T * K * (14 if case["swiglu"] else 3)}
    if op == "gemm":
        N, K, b = case["N"], case["K"], _BYTES[case["out"]]
        kb = -(-K // 128)
        return {"bytes": T * K + N * K + T * N * b * (2 if case["addend"] else 1) +
                4 * kb * (T + -(-N // 128)), "flops": 2 * T * N * K}
    P = T * case["topk"]
    rows = -(-P * case["here"] // case["E"])            # of experts that are here, on average
    if op == "grouped":
        N, K, b = case["N"], case["K"], _BYTES[case["out"]]
        # experts that have rows: about here (1 - (1 - 1/E)^P)
        used = case["here"] * (1 - (1 - case["topk"] / case["E"]) ** T)
        a = T if case["gather"] else rows
        return {"bytes": int(used * N * K) + a * K + rows * N * b, "flops": 2 * rows * N * K}
    H, b = case["H"], _BYTES[case["dtype"]]
    if op == "sort":
        return {"bytes": ((T + rows) * H * b) * (2 if case["grad"] else 1) + 12 * P,
                "flops": rows * H if case["grad"] else P}
    fwd = (rows + T * (2 if case["addend"] else 1)) * H * b + 8 * P
    bwd = (2 * rows + T) * H * b + 8 * P if case["grad"] else 0
    return {"bytes": fwd + bwd, "flops": rows * H * (6 if case["grad"] else 2)}


# ---- 64 bits -------------------------------------------------------------------

def _two_to(e):
    """2^e in float64, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(v):
    """The nearest e4m3 value of |v| <= 448, ties to even: three bits behind the leading one,
    steps of 2^-9 below 2^-6."""
    expo = torch.frexp(v)[1].clamp(min=-5) - 1
    step = _two_to(expo - 3)
    return torch.round(v / step) * step


def _exact_codes(v):
    """Codes (as numbers) and scales of rows in 64 bits."""
    T, K = v.shape
    pad = -K % 128
    v = torch.nn.functional.pad(v, (0, pad)).view(T, -1, 128)
    m, e = torch.frexp(v.abs().max(-1)[0] / 448)
    s = _two_to(torch.where(m == 0.5, e - 1, e).clamp(min=-126))
    q = _e4m3(v / s[..., None])
    return q.view(T, -1)[:, :K], s


def _exact_values(q, scale, rows_a_scale=1):
    """q [n, K] times its scales, in 64 bits."""
    n, K = q.shape
    row = torch.arange(n, device=q.device) // rows_a_scale
    col = torch.arange(K, device=q.device) // 128
    return q.double() * scale.double()[row[:, None], col]


def exact(case, seed):
    s = prepare(case, seed)
    op, f = case["op"], torch.float64
    if op == "quant":
        x = s["x"].to(f)
        if not case["swiglu"]:
            q, scale = _exact_codes(x)
            return dict(q=q, scale=scale)
        gate, up = x[:, :case["K"]], x[:, case["K"]:]
        if case["clamp"]:
            gate, up = gate.clamp(max=case["clamp"]), up.clamp(-case["clamp"], case["clamp"])
        q, scale = _exact_codes(gate * torch.sigmoid(case["alpha"] * gate) * (up + case["beta"]))
        return _exact_values(q, scale)
    if op == "gemm":
        y = _exact_values(s["a"], s["sa"]) @ _exact_values(s["w"], s["sw"], 128).t()
        return y if s["add"] is None else y + s["add"].to(f)
    if op == "grouped":
        off = s["offsets"].tolist()
        y = torch.zeros(case["T"] * case["topk"], case["N"], dtype=f, device=s["a"].device)
        a = _exact_values(s["a"], s["sa"])
        for e in range(case["here"]):
            if off[e + 1] > off[e]:
                part = slice(off[e], off[e + 1])
                rows = a[part] if s["rows"] is None else a[s["rows"][part].long()]
                y[part] = rows @ _exact_values(s["w"][e], s["sw"][e], 128).t()
        return y
    if op == "sort":
        if not case["grad"]:
            return None
        slots = _order(s["ids"], case["here"])[1].long()
        dx = s["dxs"].to(f)[slots.clamp(min=0)] * (slots >= 0)[..., None]
        return dict(tokens=None, slots=None, offsets=None, x=None, dx=dx.sum(1))
    y, w, slots = s["y"].detach().to(f), s["weights"].detach().to(f), s["slots"].long()
    here = (slots >= 0)[..., None]
    rows = y[slots.clamp(min=0)] * here
    out = torch.einsum("tkh,tk->th", rows, w)
    if s["add"] is not None:
        out = out + s["add"].to(f)
    if not case["grad"]:
        return out
    d = s["dout"].to(f)
    dy = torch.zeros_like(y)
    to = slots.view(-1)[slots.view(-1) >= 0]
    dy[to] = (w[..., None] * d[:, None]).flatten(0, 1)[slots.view(-1) >= 0]
    return dict(out=out, dy=dy, dweights=torch.einsum("tkh,th->tk", rows, d))
