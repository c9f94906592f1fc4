"""Measured cases of the operators around the routed layer.

A serving step of a mixture-of-experts block runs, besides the routed layer itself:

    norm    residual addition, root-mean-square norm, and the normed rows in 8 bits with a
            scale for each token (weight_only_bit_moe_amd.add_rmsnorm)
    route   router logits -> the expert ids and weights the routed layer reads
            (weight_only_bit_moe_amd.route_topk)
    gemm    the shared expert's products in 8-bit integers with scales for each token and
            channel (weight_only_bit_moe_amd.gemm_w8a8)
    swiglu  the shared expert's activation, in 8 bits with a scale for each token
            (weight_only_bit_moe_amd.swiglu_quant)

`run` computes a case in its plain form with elementary torch operations, or, with `own`
set, through the package's entry points.  8-bit outputs are returned as the values they
stand for (code times scale, in bfloat16).
"""
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # a decode step of four tokens, before the block
        dict(name="norm-decode-T4", op="norm", T=4, H=4096, dtype="bf16", residual=True),
        # an odd chunk in half precision, a hidden size at the single launch's limit; the
        # first norm of a stack has no residual yet
        dict(name="norm-T2047-fp16", op="norm", T=2047, H=5120, dtype="fp16", residual=False),
        # the large prefill chunk
        dict(name="norm-prefill-T8192", op="norm", T=8192, H=4096, dtype="bf16", residual=True),
        # decode: sigmoid scores, balance bias, 4 of 8 groups
        dict(name="route-decode-T4", op="route", T=4, E=256, k=6, score="sigmoid", bias=True,
             groups=8, topk_groups=4, dtype="fp32"),
        # batched decode with plain softmax routing and half-precision logits
        dict(name="route-softmax-T64", op="route", T=64, E=256, k=6, score="softmax", bias=False,
             groups=1, topk_groups=1, dtype="bf16"),
        # the large prefill chunk, grouped
        dict(name="route-prefill-T8192", op="route", T=8192, E=256, k=8, score="sigmoid",
             bias=True, groups=8, topk_groups=4, dtype="fp32"),
        # the shared expert's gate/up product of four decode tokens: streams the weights
        dict(name="gemm-decode-T4", op="gemm", T=4, N=4096, K=4096, out="bf16", addend=False),
        # batched decode: down product, added to the routed experts' sum
        dict(name="gemm-decode-T64", op="gemm", T=64, N=4096, K=2048, out="bf16", addend=True),
        # an odd chunk, one GPU's share of the gate/up columns, half precision out
        dict(name="gemm-T2047-fp16", op="gemm", T=2047, N=2056, K=4096, out="fp16", addend=False),
        # the large prefill chunk's gate/up product
        dict(name="gemm-prefill-T8192", op="gemm", T=8192, N=4096, K=4096, out="bf16",
             addend=False),
        # batched decode, clamped activation as some checkpoints have it
        dict(name="swiglu-T64", op="swiglu", T=64, I=2048, dtype="bf16", alpha=1.702, beta=1.0,
             clamp=7.0),
        # the large prefill chunk, plain SiLU
        dict(name="swiglu-prefill-T8192", op="swiglu", T=8192, I=2048, dtype="bf16", alpha=1.0,
             beta=0.0, clamp=0.0),
    ]


def _spread(rng, lo, hi):
    """An odd integer or a power of two in [lo, hi], spread over the logarithm."""
    import math
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    if rng.random() < 0.7:
        return min(int(v) | 1, (hi - 1) | 1)
    return min(1 << int(round(math.log2(v))), hi)


def draw(rng):
    op = rng.choice(["norm", "route", "gemm", "gemm", "swiglu"])
    if op == "norm":
        # hidden sizes: multiples of 128 as the layer takes them, and odd ones
        H = rng.choice([128 * rng.randint(2, 23), 128 * rng.randint(25, 40), _spread(rng, 96, 5120)])
        return dict(op=op, T=_spread(rng, 1, 6553), H=H, dtype=rng.choice(["bf16", "fp16"]),
                    residual=rng.random() < 0.7)
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = rng.choice([64, 128, 160, 256])
        kg = rng.randint(1, groups)
        return dict(op=op, T=_spread(rng, 1, 8191), E=E, k=rng.randint(1, min(8, E // groups * kg)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6,
                    groups=groups, topk_groups=kg, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "gemm":
        N = rng.choice([16 * rng.randint(16, 191), 128 * rng.randint(25, 32), _spread(rng, 256, 4096)])
        K = rng.choice([64 * rng.randint(4, 47), 128 * rng.randint(25, 32)])
        return dict(op=op, T=_spread(rng, 1, 8191), N=N, K=K,
                    out=rng.choice(["bf16", "fp16"]), addend=rng.random() < 0.5)
    return dict(op=op, T=_spread(rng, 1, 8191),
                I=rng.choice([128 * rng.randint(1, 11), 128 * rng.randint(13, 16),
                              _spread(rng, 64, 2048)]),
                dtype=rng.choice(["bf16", "fp16"]), alpha=rng.choice([1.0, 1.702]),
                beta=rng.choice([0.0, 1.0]), clamp=rng.choice([0.0, 7.0]))


def _rows_to_codes(v):
    """Rows of v in 8 bits: codes as int8, and the scale of each row."""
    amax = v.abs().amax(-1)
    return torch.round(v * (127.0 / amax).unsqueeze(-1)).to(torch.int8), amax / 127.0


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    op, T = case["op"], case["T"]
    s = dict(case)
    if op == "norm":
        # activations with a few outlier channels, tokens of different sizes
        H, dt = case["H"], _DT[case["dtype"]]
        chan = torch.exp(0.8 * randn(H))
        tok = torch.exp(0.5 * randn(T, 1))
        s["x"] = (randn(T, H) * chan * tok).to(dt)
        s["r"] = (randn(T, H) * chan * 2).to(dt) if case["residual"] else None
        s["w"] = (1 + 0.2 * randn(H)).to(dt)
        s["eps"] = 1e-6
    elif op == "route":
        # some experts are drawn to more than others; the bias pushes back in part
        E = case["E"]
        pull = 0.7 * randn(E)
        s["logits"] = (1.5 * randn(T, E) + pull).to(_DT[case["dtype"]])
        s["b"] = (0.1 * randn(E) - 0.05 * pull) if case["bias"] else None
    elif op == "gemm":
        N, K = case["N"], case["K"]
        a = randn(T, K) * torch.exp(0.5 * randn(K))
        s["a"], s["sa"] = _rows_to_codes(a)
        w = randn(N, K) * torch.exp(0.3 * randn(N, 1)) * K ** -0.5
        s["w"], s["sw"] = _rows_to_codes(w)
        s["add"] = randn(T, N).to(_DT[case["out"]]) if case["addend"] else None
        s["ws"] = None
        if own:
            import weight_only_bit_moe_amd as M
            s["ws"] = M.gemm_w8a8_workspace_for(T, N, K, dev)  # kept by a serving program
    else:
        chan = torch.exp(0.5 * randn(2 * case["I"]))
        s["gu"] = (1.5 * randn(T, 2 * case["I"]) * chan).to(_DT[case["dtype"]])
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _values(q, scale):
    """Codes [T, n] and the scale of each row as the values they stand for."""
    return torch.mul(q, scale.unsqueeze(-1), out=torch.empty(q.shape, dtype=torch.bfloat16,
                                                             device=q.device))


def _run_own(s):
    import weight_only_bit_moe_amd as M
    op = s["op"]
    if op == "norm":
        r = M.add_rmsnorm(s["x"], s["w"], s["r"], eps=s["eps"], quant=True)
        out = dict(y=r["y"], scale=r["scale"], values=_values(r["q"], r["scale"]))
        if s["r"] is not None:
            out["h"] = r["residual"]
        return out
    if op == "route":
        ids, w = M.route_topk(s["logits"], s["k"], bias=s["b"], score=s["score"],
                              groups=s["groups"], topk_groups=s["topk_groups"], scale=2.5)
        return dict(ids=ids, weights=w)
    if op == "gemm":
        return M.gemm_w8a8(s["a"], s["sa"], s["w"], s["sw"], addend=s["add"],
                           out_dtype=_DT[s["out"]], workspace=s["ws"])
    q, scale = M.swiglu_quant(s["gu"], alpha=s["alpha"], beta=s["beta"],
                              clamp=s["clamp"] or None)
    return dict(scale=scale, values=_values(q, scale))


def _plain_codes(v):
    """Rows of v (float32) in 8 bits: the codes as floats, and each row's largest magnitude."""
    amax = v.abs().amax(-1, keepdim=True)
    mult = torch.where(amax > 0, torch.full_like(amax, 127.0) / amax, torch.zeros_like(amax))
    return torch.round(v * mult), amax


def _run_plain(s):
    op = s["op"]
    if op == "norm":
        dt, out = s["x"].dtype, {}
        h = s["x"]
        if s["r"] is not None:
            h = (s["x"].float() + s["r"].float()).to(dt)
            out["h"] = h
        h, w = h.float(), s["w"].float()
        rstd = torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"])
        v = h * w
        codes, amax = _plain_codes(v)
        scale = amax * rstd / 127.0
        out.update(y=(v * rstd).to(dt), scale=scale.squeeze(-1), values=(codes * scale).bfloat16())
        return out
    if op == "route":
        # in 64 bits: which of two nearly equal scores is ahead has to come out the same
        x = s["logits"].double()
        T, E = x.shape
        if s["score"] == "softmax":
            p = torch.exp(x - x.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
        else:
            p = 1.0 / (1.0 + torch.exp(-x))
        c = p if s["b"] is None else p + s["b"].double()
        if s["groups"] > 1:
            per = E // s["groups"]
            two = torch.sort(c.view(T, s["groups"], per), dim=-1, descending=True)[0][..., :2]
            best = torch.sort(two.sum(-1), dim=-1, descending=True, stable=True)[1]
            keep = torch.zeros(T, s["groups"], dtype=torch.bool, device=x.device)
            keep.scatter_(1, best[:, :s["topk_groups"]], True)
            c = torch.where(keep.repeat_interleave(per, 1), c, torch.full_like(c, -torch.inf))
        ids = torch.sort(c, dim=-1, descending=True, stable=True)[1][:, :s["k"]]
        w = torch.gather(p, 1, ids)
        w = w / w.sum(-1, keepdim=True) * 2.5
        return dict(ids=ids.to(torch.int32), weights=w.float())
    if op == "gemm":
        y = s["a"].float() @ s["w"].float().t()
        y = y * s["sa"].unsqueeze(-1) * s["sw"]
        if s["add"] is not None:
            y = y + s["add"].float()
        return y.to(_DT[s["out"]])
    g, u = s["gu"].float().chunk(2, dim=-1)
    if s["clamp"]:
        g, u = torch.clamp(g, max=s["clamp"]), torch.clamp(u, -s["clamp"], s["clamp"])
    act = g / (1.0 + torch.exp(-s["alpha"] * g)) * (u + s["beta"])
    codes, amax = _plain_codes(act)
    scale = amax / 127.0
    return dict(scale=scale.squeeze(-1), values=(codes * scale).bfloat16())


def work(case):
    op, T = case["op"], case["T"]
    if op == "norm":
        H, b = case["H"], _BYTES[case["dtype"]]
        per = 2 * b + 1 + (2 * b if case["residual"] else 0)  # x, y, codes; residual in and out
        return {"bytes": T * H * per + H * b + 4 * T, "flops": T * H * 8}
    if op == "route":
        E, k = case["E"], case["k"]
        return {"bytes": T * (E * _BYTES[case["dtype"]] + 8 * k) + 4 * E, "flops": T * E * 10}
    if op == "gemm":
        N, K = case["N"], case["K"]
        b = _BYTES[case["out"]]
        return {"bytes": T * K + N * K + T * N * b * (2 if case["addend"] else 1) + 4 * (T + N),
                "flops": 2 * T * N * K}
    return {"bytes": T * (case["I"] * (2 * _BYTES[case["dtype"]] + 1) + 4),
            "flops": T * case["I"] * 12}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = torch.float64
    if op == "norm":
        out = {}
        h = s["x"].to(f)
        if s["r"] is not None:
            # the residual stream is defined as the stored, rounded sum
            h = (h + s["r"].to(f)).to(s["x"].dtype).to(f)
            out["h"] = h
        v = h * s["w"].to(f)
        root = torch.sqrt((h * h).sum(-1, keepdim=True) / h.shape[1] + s["eps"])
        step = v.abs().max(-1, keepdim=True)[0] / 127
        codes = torch.where(step > 0, torch.round(v / step), torch.zeros_like(v))
        out.update(y=v / root, scale=(step / root).squeeze(-1), values=codes * (step / root))
        return out
    if op == "route":
        x = s["logits"].to(f)
        p = torch.softmax(x, -1) if case["score"] == "softmax" else torch.sigmoid(x)
        c = p if s["b"] is None else p + s["b"].to(f)
        T, E = x.shape
        G = case["groups"]
        if G > 1:
            grouped = c.reshape(T, G, E // G)
            group = grouped.topk(min(2, E // G), -1)[0].sum(-1)
            order = group.neg().argsort(dim=-1, stable=True)[:, :case["topk_groups"]]
            allowed = torch.full((T, G, 1), -torch.inf, dtype=f, device=x.device)
            allowed.scatter_(1, order.unsqueeze(-1), 0.0)
            c = (grouped + allowed).reshape(T, E)
        ids = c.neg().argsort(dim=-1, stable=True)[:, :case["k"]]
        chosen = p.gather(1, ids)
        return dict(ids=None, weights=2.5 * chosen / chosen.sum(-1, keepdim=True))
    if op == "gemm":
        a = s["a"].to(f) * s["sa"].to(f)[:, None]
        w = s["w"].to(f) * s["sw"].to(f)[:, None]
        y = torch.mm(a, w.t())
        return y if s["add"] is None else y + s["add"].to(f)
    I = case["I"]
    gate, up = s["gu"][:, :I].to(f), s["gu"][:, I:].to(f)
    if case["clamp"]:
        gate, up = gate.clamp(max=case["clamp"]), up.clamp(-case["clamp"], case["clamp"])
    act = gate * torch.sigmoid(case["alpha"] * gate) * (up + case["beta"])
    step = act.abs().max(-1, keepdim=True)[0] / 127
    codes = torch.where(step > 0, torch.round(act / step), torch.zeros_like(act))
    return dict(scale=step.squeeze(-1), values=codes * step)
