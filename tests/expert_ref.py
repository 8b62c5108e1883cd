"""64-bit references of the group norm, the router and the experts' feed-forward, and
how far a kernel that follows their contract may be from them: as in block_ref, each
function returns {output: (value, bound)} and the bounds propagate every rounding to
the dtype that the contract names and the fp32 errors of the sums.
"""
from __future__ import annotations

import math

import torch

from block_ref import E, EXTRA, TINY, U, acc, act_pair


def act_of(name, z):
    return (z, torch.ones_like(z)) if name == "none" else act_pair(name, z)


# ---------------------------------------------------------------- group norm
def group_norm_all(x, G, w, b, act, eps, dtype, dy=None):
    """x [N, P, C] in float64. A sum over n elements is cut over threads and joined
    pairwise or by warps; ks allows 16 roundings and one for each 64 elements, which is above
    the longest run of any thread (8 positions a batch, 16-bit types up to 4096 batches)."""
    un, tiny = U[dtype], TINY[dtype]
    N, P, C = x.shape
    D = C // G
    v = x.reshape(N, P, G, D)
    n = P * D
    ks = E * (16 + n / 64)
    mean = v.mean((1, 3), keepdim=True)
    dev = v - mean
    var = (dev * dev).mean((1, 3), keepdim=True)
    inv = 1 / torch.sqrt(var + eps)
    # the mean is made of means of batches of deviations: its error is that of the values near it
    em = ks * v.abs().mean((1, 3), keepdim=True) + E * 8 * mean.abs()
    hat = dev * inv
    ed = em + 4 * E * (v.abs() + mean.abs())
    # relative error of 1 / deviation: half of the variance's, whose deviations are off by ed
    ei = ks + EXTRA + (dev.abs() * ed).mean((1, 3), keepdim=True) * inv ** 2 + (ed * ed).mean((1, 3), keepdim=True) * inv ** 2
    eh = ed * inv * (1 + ei) + hat.abs() * ei
    one, zero = torch.ones(C, dtype=x.dtype), torch.zeros(C, dtype=x.dtype)
    wv = (one if w is None else w).reshape(1, 1, G, D)
    bv = (zero if b is None else b).reshape(1, 1, G, D)
    z = hat * wv + bv
    ez = eh * wv.abs() + 4 * E * ((hat * wv).abs() + bv.abs())
    a, slope = act_of(act, z)
    ea = 1.2 * ez + EXTRA * (a.abs() + slope.abs() * z.abs())

    def rounded(value, e, shape):
        return value.reshape(shape), (e + un * (value.abs() + e) + tiny).reshape(shape)

    out = {"y": rounded(a, ea, x.shape)}
    if dy is None:
        return out
    d = dy.reshape(N, P, G, D)
    es = 1.2 * ez + EXTRA * (slope.abs() + 1)
    if act == "relu":
        es = es + (z.abs() <= ez).to(z.dtype)
    if act == "none":
        es = torch.zeros_like(z)
    dz = d * slope
    edz = d.abs() * es + 2 * E * dz.abs()
    g, eg = dz * wv, edz * wv.abs() + 2 * E * (dz * wv).abs()
    m1, m2 = g.mean((1, 3), keepdim=True), (g * hat).mean((1, 3), keepdim=True)
    em1 = eg.mean((1, 3), keepdim=True) + ks * g.abs().mean((1, 3), keepdim=True)
    em2 = (eg * hat.abs() + (g.abs() + eg) * eh).mean((1, 3), keepdim=True) + ks * (g * hat).abs().mean((1, 3), keepdim=True)
    dx = inv * (g - m1 - hat * m2)
    edx = inv * (1 + ei) * (eg + em1 + eh * (m2.abs() + em2) + hat.abs() * em2 + 4 * E * (g.abs() + m1.abs() + (hat * m2).abs()))
    edx = edx + ei * dx.abs()
    out["dx"] = rounded(dx, edx, x.shape)
    kc = E * (16 + N * P / 8)
    if w is not None:
        t = dz * hat
        out["dw"] = rounded(t.sum((0, 1)), (edz * hat.abs() + (dz.abs() + edz) * eh).sum((0, 1)) + kc * t.abs().sum((0, 1)), (C,))
    if b is not None:
        out["db"] = rounded(dz.sum((0, 1)), edz.sum((0, 1)) + kc * dz.abs().sum((0, 1)), (C,))
    return out


# ---------------------------------------------------------------- router
def route(logits, k):
    """Indexes of the k largest of each row of float64 logits, equal ones by the lower index, -1 where none may be taken."""
    at = torch.argsort(logits, dim=-1, descending=True, stable=True)[..., :k]
    return torch.where(logits.gather(-1, at) == -math.inf, -1, at)


def route_all(logits, k, over, dtype, dweights=None, experts=None):
    """logits [T, E] in float64. An exponential of a difference of logits errs by the rounding of that difference,
    up to 2^-24 of |l| + |top|, and by its own few roundings; a sum of E of them by acc(E)."""
    un, tiny = U[dtype], TINY[dtype]
    T, E_ = logits.shape
    if experts is None:
        experts = route(logits, k)
    took = (experts >= 0) & (experts < E_)
    safe = experts.clamp(0, E_ - 1).long()
    chosen = torch.where(took, logits.gather(-1, safe), torch.full((), -math.inf, dtype=torch.float64))
    top = (logits if over == "all" else chosen).amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(logits - top)
    e = torch.exp(chosen - top)
    total = (p if over == "all" else e).sum(-1, keepdim=True)
    total = torch.where(total == 0, torch.ones_like(total), total)
    finite = torch.where(logits.isfinite(), logits, torch.zeros_like(logits))
    rel = E * (finite.abs().amax(-1, keepdim=True) + top.abs()) + EXTRA
    ks = acc(E_) + 2 * rel
    w = e / total
    ew = w * (rel + ks) + 2.0 ** -140
    out = {"weights": (w, ew + un * (w + ew) + tiny)}
    if dweights is None:
        return experts, out
    dw = torch.where(took, dweights, torch.zeros_like(dweights))
    s = (w * dw).sum(-1, keepdim=True)
    es = (ew * dw.abs()).sum(-1, keepdim=True) + ks * (w * dw).abs().sum(-1, keepdim=True)
    z = lambda v: torch.zeros_like(logits).scatter_add(-1, safe, torch.where(took, v, torch.zeros_like(v)))  # noqa: E731
    if over == "all":
        q, add = p / total, z(dw)
        v = q * (add - s)
        ev = q * (rel + ks) * (add.abs() + s.abs()) + q * (es + 4 * E * (z(dw.abs()) + s.abs()))
    else:
        v = z(w * (dw - s))
        ev = z(ew * (dw - s).abs() + w * (es + 4 * E * (dw.abs() + s.abs())))
    ev = ev + 2.0 ** -120
    out["dlogits"] = (v, ev + un * (v.abs() + ev) + tiny)
    return experts, out
