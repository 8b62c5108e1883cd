"""64-bit references of the residual-block operators, and how far a kernel that
follows their contract may be from them.

Each function takes float64 tensors holding exactly the kernel's inputs and
returns {output: (value, bound)}. The bounds propagate, element by element,
 - U[dtype] * |v| (+ half the smallest subnormal) for every rounding to the dtype
   that the contract names: the outputs, and h, dg and du between products;
 - the fp32 error of a sum of K products, at most acc(K) * sum |a||b|. The
   worst case over any order is K * 2^-24; partial sums of random terms err by
   about sqrt(K) * 2^-24, and acc() allows eight times that plus 16 roundings;
 - the errors of the operands through each formula's derivatives, with |act'| <=
   1.2 and |act''| <= 1.2 (relu: its step at 0 counts whole where g is within its
   error of 0).
Quantities rounded once in fp32 along the way are covered by EXTRA roundings.
"""
from __future__ import annotations

import math

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
E = 2.0 ** -24
EXTRA = 16 * E


def acc(K: int) -> float:
    return E * (16 + 8 * math.sqrt(K))


def act_pair(name, g):
    """act(g), act'(g)."""
    if name == "relu":
        return torch.where(g > 0, g, torch.zeros_like(g)), (g > 0).to(g.dtype)
    if name in ("silu", "sigmoid"):
        p = 1 / (1 + torch.exp(-g))
        return (g * p, p * (1 + g * (1 - p))) if name == "silu" else (p, p * (1 - p))
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def ffn(x, wg, wu, wd, act):
    g, u = x @ wg.T, x @ wu.T
    return (act_pair(act, g)[0] * u) @ wd.T


def ffn_all(x, wg, wu, wd, act, dtype, dy=None):
    R, C = x.shape
    F = wg.shape[0]
    un, tiny = U[dtype], TINY[dtype]
    g, u = x @ wg.T, x @ wu.T
    eg, eu = acc(C) * (x.abs() @ wg.abs().T), acc(C) * (x.abs() @ wu.abs().T)
    a, d = act_pair(act, g)
    ea = 1.2 * eg + EXTRA * (a.abs() + d.abs() * g.abs())
    h = a * u
    eh = ea * u.abs() + a.abs() * eu + ea * eu + EXTRA * h.abs()
    eh = eh + un * (h.abs() + eh) + tiny

    def product(p, ep, q, eq, K):
        """p q^T with the operands' errors, the sum's and the output's rounding."""
        v = p @ q.T
        e = ep @ q.abs().T if eq is None else p.abs() @ eq.T if ep is None else None
        e = e + acc(K) * (p.abs() @ q.abs().T)
        return v, e

    def rounded(v, e):
        return v, e + un * (v.abs() + e) + tiny

    out = {"y": rounded(*product(h, eh, wd, None, F))}
    if dy is None:
        return out
    dh = dy @ wd
    edh = acc(C) * (dy.abs() @ wd.abs())
    ed = 1.2 * eg + EXTRA * (d.abs() + 1)
    if act == "relu":
        ed = (g.abs() <= eg).to(g.dtype)
    dg, du = dh * u * d, dh * a
    edg = (edh * (u * d).abs() + (dh.abs() + edh) * (eu * (d.abs() + ed) + u.abs() * ed)) + EXTRA * dg.abs()
    edu = edh * a.abs() + (dh.abs() + edh) * ea + EXTRA * du.abs()
    edg, edu = edg + un * (dg.abs() + edg) + tiny, edu + un * (du.abs() + edu) + tiny
    v1, e1 = product(dg, edg, wg.T, None, 2 * F)
    v2, e2 = product(du, edu, wu.T, None, 2 * F)
    out["dx"] = rounded(v1 + v2, e1 + e2)
    out["dw_gate"] = rounded(*product(dg.T, edg.T, x.T, None, R))
    out["dw_up"] = rounded(*product(du.T, edu.T, x.T, None, R))
    out["dw_down"] = rounded(*product(dy.T, None, h.T, eh.T, R))
    return out


# ---------------------------------------------------------------- norms
def _moments(kind, v, ev, eps):
    """hat, inv and hat's error of a row given v's."""
    C = v.shape[-1]
    k = E * (16 + C / 32)  # a column's sum is cut over at least 32 lanes
    if kind == "none":
        return v, torch.ones_like(v[..., :1]), ev
    m = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
    em = (ev.mean(-1, keepdim=True) + k * v.abs().mean(-1, keepdim=True)) if kind == "layer" else 0.0
    inv = 1 / torch.sqrt(((v - m) ** 2).mean(-1, keepdim=True) + eps)
    hat = (v - m) * inv
    ed = ev + em + EXTRA * (v.abs() + m.abs())
    einv = ((hat.abs() * ed).mean(-1, keepdim=True) * inv + (ed * ed).mean(-1, keepdim=True) * inv ** 2 + k)  # relative
    return hat, inv, ed * inv * (1 + einv) + hat.abs() * einv


def residual_norm(x, y, p):
    """(r, n) in the inputs' type; p: the keyword arguments of the call."""
    R = x.shape[0]

    def norm(kind, v, w, b):
        if kind == "none":
            return v
        if kind == "layer":
            v = v - v.mean(-1, keepdim=True)
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + p["eps"])
        v = v if w is None else v * w
        return v if b is None else v + b

    r = x if p["res_scale"] is None else x * p["res_scale"]
    if y is not None:
        post = norm(p["post"], y, p["w_post"], p["b_post"])
        if p["gate"] is not None:
            at = torch.arange(R) // (p["rows_per_gate"] or max(R, 1))
            post = post * p["gate"][at.to(x.device)]
        r = r + post
    return r, None if p["pre"] == "none" else norm(p["pre"], r, p["w_pre"], p["b_pre"])


def residual_norm_all(x, y, p, dtype, dr=None, dn=None, backward=False):
    un, tiny = U[dtype], TINY[dtype]
    R, C = x.shape
    one, zero = torch.ones(C, dtype=x.dtype), torch.zeros(C, dtype=x.dtype)
    rs = one if p["res_scale"] is None else p["res_scale"]
    wq = one if p["w_post"] is None else p["w_post"]
    bq = zero if p["b_post"] is None else p["b_post"]
    wp = one if p["w_pre"] is None else p["w_pre"]
    per = p["rows_per_gate"] or max(R, 1)
    at = torch.arange(R) // per

    def rounded(v, e):
        return v, e + un * (v.abs() + e) + tiny

    r, ea = x * rs, EXTRA * (x * rs).abs()
    if y is not None:
        gate = one.expand(R, C) if p["gate"] is None else p["gate"][at]
        yh, yi, eyh = _moments(p["post"], y, torch.zeros_like(y), p["eps"])
        post = yh * wq + bq
        epost = eyh * wq.abs() + EXTRA * ((yh * wq).abs() + bq.abs())
        r = r + gate * post
        ea = ea + gate.abs() * epost + EXTRA * (gate * post).abs()
    ea = ea + EXTRA * r.abs()
    out = {"r": rounded(r, ea)}
    rh, ri, erh = _moments(p["pre"], r, ea, p["eps"])
    if p["pre"] != "none":
        n = rh * wp + (0 if p["b_pre"] is None else p["b_pre"])
        out["n"] = rounded(n, erh * wp.abs() + EXTRA * ((rh * wp).abs() + n.abs()))
    if not backward:
        return out

    def norm_back(kind, e, ee, hat, ehat, inv):
        """Gradient of the normed row from e = d * w with error ee."""
        if kind == "none":
            return e, ee
        k = E * (16 + C / 32)
        c = (e * hat).mean(-1, keepdim=True)
        ec = (ee * hat.abs() + (e.abs() + ee) * ehat).mean(-1, keepdim=True) + k * (e * hat).abs().mean(-1, keepdim=True)
        m = e.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(c)
        em = ee.mean(-1, keepdim=True) + k * e.abs().mean(-1, keepdim=True)
        v = inv * (e - m - hat * c)
        ev = inv * (ee + em + ehat * (c.abs() + ec) + hat.abs() * ec + EXTRA * (e.abs() + m.abs() + (hat * c).abs()))
        # the inverse deviation's own relative error is within hat's at |hat| >= 1
        return v, ev + v.abs() * (k + ehat.amax(-1, keepdim=True))

    dt = torch.zeros_like(x) if dr is None else dr.clone()
    edt = EXTRA * dt.abs()
    if dn is not None:
        v, ev = norm_back(p["pre"], dn * wp, EXTRA * (dn * wp).abs(), rh, erh, ri)
        dt, edt = dt + v, edt + ev
    edt = edt + EXTRA * dt.abs()
    kr = E * (16 + R / 8)  # a column's sum over rows, cut over at least 8 lanes

    def col(v, e):
        return rounded(v.sum(0), e.sum(0) + kr * v.abs().sum(0))

    out["dx"] = rounded(dt * rs, edt * rs.abs() + EXTRA * (dt * rs).abs())
    if p["res_scale"] is not None:
        out["dres_scale"] = col(x * dt, x.abs() * edt)
    if y is not None:
        dp, edp = gate * dt, gate.abs() * edt + EXTRA * (gate * dt).abs()
        out["dy"] = rounded(*norm_back(p["post"], dp * wq, edp * wq.abs() + EXTRA * (dp * wq).abs(), yh, eyh, yi))
        if p["gate"] is not None:
            t, et = post * dt, epost * (dt.abs() + edt) + post.abs() * edt
            G = p["gate"].shape[0]
            z = lambda v: torch.zeros(G, C, dtype=x.dtype).index_add_(0, at, v)  # noqa: E731
            out["dgate"] = rounded(z(t), z(et) + kr * z(t.abs()))
        if p["w_post"] is not None:
            out["dw_post"] = col(dp * yh, edp * (yh.abs() + eyh) + dp.abs() * eyh)
        if p["b_post"] is not None:
            out["db_post"] = col(dp, edp)
    if p["w_pre"] is not None:
        d = torch.zeros_like(x) if dn is None else dn
        out["dw_pre"] = col(d * rh, d.abs() * erh)
    if p["b_pre"] is not None:
        d = torch.zeros_like(x) if dn is None else dn
        out["db_pre"] = col(d, EXTRA * d.abs())
    return out


def check(got, want, what=""):
    """got: {name: tensor} against {name: (value, bound)}: every output, every element."""
    assert {k for k, v in got.items() if v is not None} == set(want), (sorted(got), sorted(want))
    for name, (v, e) in want.items():
        g = got[name].detach().double().cpu().reshape(v.shape)
        err = (g - v).abs()
        bad = ~(err <= e)
        assert not bad.any(), (f"{what} {name}: {int(bad.sum())} of {bad.numel()} elements out of bounds; worst ratio "
                               f"{float((err / e).nan_to_num(float('inf')).max()):.3g}")
