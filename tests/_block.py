"""64-bit references of the operators around the routed layer, from their
formulas, on the CPU.  Rounding counts: a result rounded to a type is off by at
most half a step, finfo.eps / 2 relative (or half the smallest subnormal)."""
import numpy as np
import torch

F = torch.float64
U = 2.0 ** -24                      # one FP32 rounding
INT8_TOP = 127


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """Half the distance between the values next to zero."""
    fi = torch.finfo(dtype)
    return fi.tiny * fi.eps / 2


def codes_fp32(v):
    """The defined codes of FP32 rows v: every operation is one IEEE rounding, so
    the kernel's codes equal them bit for bit."""
    v = v.numpy().astype(np.float32)
    top = np.abs(v).max(-1, keepdims=True).astype(np.float32)
    live = (top >= np.float32(2.0 ** -100)) & np.isfinite(top)
    with np.errstate(all="ignore"):
        mult = np.where(live, np.float32(127) / top, np.float32(0))
        q = np.rint(np.where(live, v * mult, 0)).astype(np.int8)
    return torch.from_numpy(q), torch.from_numpy(top[:, 0])


def rmsnorm(x, r, w, eps):
    """h (in x's type) and y, scale in 64 bits, codes by definition."""
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    hd = h.to(F)
    rstd = 1.0 / torch.sqrt((hd * hd).mean(-1, keepdim=True) + eps)
    y = hd * w.to(F) * rstd
    q, top = codes_fp32(h.float() * w.float())
    scale = (hd * w.to(F)).abs().amax(-1) * rstd[:, 0] / INT8_TOP
    return h, y, q, scale, top


def swiglu(gu, alpha, beta, clamp):
    I = gu.shape[1] // 2
    g, u = gu[:, :I].to(F), gu[:, I:].to(F)
    if clamp is not None:
        g, u = g.clamp(max=clamp), u.clamp(-clamp, clamp)
    return g * torch.sigmoid(alpha * g) * (u + beta), g


def gemm(a, sa, w, sw, add=None):
    s = a.to(F) @ w.to(F).t()       # integers below 2^53: exact
    p = s * sa.to(F)[:, None] * sw.to(F)
    return p, (p if add is None else p + add.to(F))


def route(logits, k, bias, score, groups, topk_groups, renormalize, scale):
    l = logits.to(F).numpy().copy()
    out = ~(l > -np.inf)            # -inf and NaN
    l[out] = -np.inf
    l = np.minimum(l, np.finfo(np.float32).max)
    T, E = l.shape
    ids = np.full((T, k), -1, np.int32)
    wts = np.zeros((T, k))
    for t in range(T):
        with np.errstate(all="ignore"):
            if out[t].all():
                continue
            if score == "softmax":
                e = np.where(out[t], 0.0, np.exp(l[t] - l[t].max()))
                p = e / e.sum()
            else:
                p = np.where(out[t], 0.0, 1.0 / (1.0 + np.exp(-l[t])))
        c = p + (0.0 if bias is None else bias.to(F).numpy())
        if bias is None and groups == 1:
            c = l[t].copy()         # the same order, also where p saturates
        c[out[t] | ~(c > -np.inf)] = -np.inf
        if groups > 1:
            per = E // groups
            two = np.sort(c.reshape(groups, per), -1)[:, ::-1][:, :2]
            gs = np.where(np.isfinite(two[:, -1]) | (two[:, -1] == np.inf), two.sum(-1), two[:, 0])
            keep = np.argsort(-gs, kind="stable")[:topk_groups]
            drop = np.ones(groups, bool)
            drop[keep] = False
            c[np.repeat(drop, per)] = -np.inf
        order = [e for e in np.argsort(-c, kind="stable")[:k] if c[e] > -np.inf]
        w = p[order]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else w * 0
        ids[t, :len(order)] = order
        wts[t, :len(order)] = w * scale
    return ids, wts
