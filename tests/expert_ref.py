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


# ---------------------------------------------------------------- experts' feed-forward
def expert_ffn(x, experts, weights, wg, wu, wd, act):
    y = torch.zeros_like(x)
    for e in range(wg.shape[0]):
        t, j = (experts == e).nonzero(as_tuple=True)
        h = act_pair(act, x[t] @ wg[e].T)[0] * (x[t] @ wu[e].T)
        y.index_add_(0, t, weights[t, j].unsqueeze(-1) * (h @ wd[e].T))
    return y


def experts_all(x, experts, weights, wg, wu, wd, act, dtype, dy=None):
    """x [T, C], experts and weights [T, k], the matrices [E, ...], all but experts in float64. As
    block_ref.ffn_all for each expert's rows, with the weights applied in fp32 and the rounding of
    weights * h, dw_down's operand."""
    un, tiny = U[dtype], TINY[dtype]
    T, C = x.shape
    E_, F, k = wg.shape[0], wg.shape[1], experts.shape[1]

    def product(p, ep, q, K):
        """p q^T, its error from p's and the sum's."""
        return p @ q.T, (0 if ep is None else ep @ q.abs().T) + acc(K) * (p.abs() @ q.abs().T)

    def both(p, ep, q, eq, K):
        v, e = product(p, ep, q, K)
        return v, e + (0 if eq is None else (p.abs() + (0 if ep is None else ep)) @ eq.T)

    def rounded(v, e):
        return v, e + un * (v.abs() + e) + tiny

    y, ey, my = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    out = {}
    if dy is not None:
        dx, edx, mdx = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
        dwt, edwt = torch.zeros_like(weights), torch.zeros_like(weights)
        dws = {n: [] for n in ("dw_gate", "dw_up", "dw_down")}
    for e in range(E_):
        t, j = (experts == e).nonzero(as_tuple=True)
        xe, w = x[t], weights[t, j].unsqueeze(-1)
        (g, eg), (u, eu) = product(xe, None, wg[e], C), product(xe, None, wu[e], C)
        a, d = act_pair(act, g)
        ea = 1.2 * eg + EXTRA * (a.abs() + d.abs() * g.abs())
        h = a * u
        exact_h, eh = h, ea * u.abs() + a.abs() * eu + ea * eu + EXTRA * h.abs()
        h, eh = rounded(h, eh)
        ys, eys = product(h, eh, wd[e], F)
        y.index_add_(0, t, w * ys)
        ey.index_add_(0, t, w.abs() * eys)
        my.index_add_(0, t, (w * ys).abs())
        if dy is None:
            continue
        dye = dy[t]
        dwt[t, j] = (dye * ys).sum(-1)
        edwt[t, j] = (dye.abs() * eys).sum(-1) + acc(C) * (dye * ys).abs().sum(-1)
        dh, edh = product(dye, None, wd[e].T, C)
        dh, edh = w * dh, w.abs() * edh + E * (w * dh).abs()
        hw, ehw = rounded(w * exact_h, w.abs() * (eh + E * exact_h.abs()))
        ed = 1.2 * eg + EXTRA * (d.abs() + 1)
        if act == "relu":
            ed = (g.abs() <= eg).to(g.dtype)
        dg, du = dh * u * d, dh * a
        edg = edh * (u * d).abs() + (dh.abs() + edh) * (eu * (d.abs() + ed) + u.abs() * ed) + EXTRA * dg.abs()
        edu = edh * a.abs() + (dh.abs() + edh) * ea + EXTRA * du.abs()
        dg, edg = rounded(dg, edg)
        du, edu = rounded(du, edu)
        v1, e1 = product(dg, edg, wg[e].T, 2 * F)
        v2, e2 = product(du, edu, wu[e].T, 2 * F)
        dxs, edxs = v1 + v2, e1 + e2
        dx.index_add_(0, t, dxs)
        edx.index_add_(0, t, edxs)
        mdx.index_add_(0, t, dxs.abs())
        rows = max(1, t.numel())
        dws["dw_gate"].append(rounded(*both(dg.T, edg.T, xe.T, None, rows)))
        dws["dw_up"].append(rounded(*both(du.T, edu.T, xe.T, None, rows)))
        dws["dw_down"].append(rounded(*both(dye.T, None, hw.T, ehw.T, rows)))
    out["y"] = rounded(y, ey + k * E * my)
    if dy is not None:
        out["dx"] = rounded(dx, edx + k * E * mdx)
        out["dweights"] = rounded(dwt, edwt)
        for n, pairs in dws.items():
            out[n] = tuple(torch.stack([p[i] for p in pairs]) for i in range(2))
    return out
