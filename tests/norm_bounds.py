"""The group norm in 64 bits with bounds that follow its sums: the mean is the mean of deviations that were
formed from a mean of their own, and no sum of the kernels has a longer chain of additions than `run` (a thread's
positions, the joins over a block's rows, a lane's chunks and channels of a group) or `run_params` (the same, and an
eighth of the rows of partial sums) for the shapes that a test names. As in block_ref, a chain of K additions errs by
acc(K) of the sum of its absolute terms."""
from __future__ import annotations

import torch

from block_ref import E, EXTRA, TINY, U, acc
from expert_ref import act_of


def group_norm(x, G, w, b, act, eps, dtype, dy=None, run=256, run_params=512, roundings=2):
    """{output: (value, bound)} of x [N, P, C] in float64, also of the statistics that the forward call keeps."""
    un, tiny = U[dtype], TINY[dtype]
    N, P, C = x.shape
    D = C // G
    v = x.reshape(N, P, G, D)
    ks = acc(run)
    mean = v.mean((1, 3), keepdim=True)
    dev = v - mean
    var = (dev * dev).mean((1, 3), keepdim=True)
    inv = 1 / torch.sqrt(var + eps)
    # the means of parts, each rounded and then averaged, and the result's own rounding; 1: there is one part
    em = ks * dev.abs().mean((1, 3), keepdim=True) + roundings * E * mean.abs()
    ed = em + 2 * E * dev.abs()
    ei = ks / 2 + 8 * E + (em * inv) ** 2
    hat = dev * inv
    eh = ed * inv * (1 + ei) + hat.abs() * (ei + 2 * E)
    one, zero = torch.ones(C, dtype=x.dtype, device=x.device), torch.zeros(C, dtype=x.dtype, device=x.device)
    wv = (one if w is None else w).reshape(1, 1, G, D)
    bv = (zero if b is None else b).reshape(1, 1, G, D)
    z = hat * wv + bv
    ez = eh * wv.abs() + 4 * E * ((hat * wv).abs() + bv.abs())
    a, slope = act_of(act, z)
    ea = 1.2 * ez + (0 if act == "none" else EXTRA) * (a.abs() + slope.abs() * z.abs())

    def rounded(value, e, shape):
        return value.reshape(shape), (e + un * (value.abs() + e) + tiny).reshape(shape)

    pair = lambda m, i: torch.cat([m.reshape(N, G, 1), i.reshape(N, G, 1)], -1)  # noqa: E731
    out = {"y": rounded(a, ea, x.shape), "stats": (pair(mean, inv), pair(em, inv * (ei + E)))}
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
    out["dx"] = rounded(dx, edx + ei * dx.abs(), x.shape)
    kc = acc(run_params)
    if w is not None:
        t = dz * hat
        out["dw"] = rounded(t.sum((0, 1)), (edz * hat.abs() + (dz.abs() + edz) * eh).sum((0, 1)) + kc * t.abs().sum((0, 1)), (C,))
    if b is not None:
        out["db"] = rounded(dz.sum((0, 1)), edz.sum((0, 1)) + kc * dz.abs().sum((0, 1)), (C,))
    return out
