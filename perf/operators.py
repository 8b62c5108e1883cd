"""Timed cases of the residual-block operators: the gated feed-forward, the
norms around a block with its gate and residual scale, and the clipping of
gradients by their global norm. `run` computes a case in elementary torch
operations, or, where `own` is true, by the framework's entry points."""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


def listed():
    return [
        # one position through a small block: a single image's pooled features, or one generated token; latency only
        dict(name="ffn_one_row", op="ffn", train=False, R=1, C=512, F=2048, act="silu", dtype="bf16"),
        # a handful of positions at the widest block: every weight is read for five rows
        dict(name="ffn_few_rows_wide", op="ffn", train=False, R=5, C=4096, F=10240, act="silu", dtype="bf16"),
        # inference over a short ragged batch; the hidden width is no multiple of a vector
        dict(name="ffn_ragged", op="ffn", train=False, R=777, C=1000, F=2730, act="gelu_tanh", dtype="bf16"),
        # inference over the 56 x 56 x 128 channels-last maps of 64 images (the sweep layers' batch)
        dict(name="ffn_maps", op="ffn", train=False, R=64 * 56 * 56, C=128, F=512, act="gelu", dtype="f16"),
        # a training step over 28 x 28 maps of 16 images
        dict(name="ffn_train_maps", op="ffn", train=True, R=16 * 28 * 28, C=256, F=1024, act="gelu", dtype="f16"),
        # a full-precision training step of odd sizes
        dict(name="ffn_train_f32", op="ffn", train=True, R=1569, C=384, F=1001, act="silu", dtype="f32"),
        # the largest training step: many rows at the widest block
        dict(name="ffn_train_wide", op="ffn", train=True, R=8192, C=4096, F=10240, act="silu", dtype="bf16"),
        # one row between two blocks while serving; latency only
        dict(name="norm_one_row", op="norm", train=False, R=1, C=512, per_gate=1, post="rms", pre="rms",
             affine=True, scale=True, dtype="bf16"),
        # training over 56 x 56 x 128 maps, a gate for each image and channel
        dict(name="norm_train_maps", op="norm", train=True, R=64 * 56 * 56, C=128, per_gate=56 * 56, post="layer",
             pre="layer", affine=True, scale=True, dtype="f16"),
        # training over wide rows with one gate for all rows
        dict(name="norm_train_wide", op="norm", train=True, R=8192, C=4096, per_gate=8192, post="rms", pre="rms",
             affine=True, scale=True, dtype="bf16"),
        # the gradients of a small convolutional network: filters, norms' weights, biases
        dict(name="clip_small_net", op="clip", count=53, total=3_200_000, mixed=False, dtype="f32", max_norm=1.0),
        # the gradients of twelve of the widest blocks, with some in full precision
        dict(name="clip_wide_net", op="clip", count=48, total=1_500_000_000, mixed=True, dtype="bf16", max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "norm", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "ffn":
        train = rng.random() < 0.5
        most_r, most_c = (4096, 1024) if dtype == "f32" else (200704, 4096)
        C = _log(rng, 64, most_c)
        if rng.random() < 0.6:
            C = max(64, C // 8 * 8)
        F = int(C * rng.uniform(1.0, 4.0))
        if rng.random() < 0.6:
            F = F // 8 * 8
        F = min(F, 10240)
        most = 18 * 8192 * 4096 * 10240 // ((18 if train else 6) * C * F)
        R = min(_log(rng, 1, most_r), most)
        return dict(op="ffn", train=train, R=R, C=C, F=F, act=rng.choice(["silu", "gelu", "gelu_tanh", "relu", "sigmoid"]),
                    dtype=dtype)
    if op == "norm":
        C = _log(rng, 32, 8192)
        if rng.random() < 0.6:
            C = C // 8 * 8
        R = min(_log(rng, 1, 200704), 8192 * 4096 // C)
        per_gate = rng.choice([1, _log(rng, 1, R), R])
        return dict(op="norm", train=rng.random() < 0.5, R=R, C=C, per_gate=per_gate,
                    post=rng.choice(["none", "rms", "layer"]), pre=rng.choice(["none", "rms", "layer"]),
                    affine=rng.random() < 0.8, scale=rng.random() < 0.8, dtype=dtype)
    count = _log(rng, 1, 60)
    total = max(_log(rng, 1000, 1_500_000_000 * 2 // SIZE[dtype]), count)
    return dict(op="clip", count=count, total=total, mixed=rng.random() < 0.3 and dtype != "f32", dtype=dtype,
                max_norm=rng.choice([0.5, 1.0, 1e6]))


def _sizes(case):
    """Tensor sizes of a list of gradients: a fixed spread of large, odd and tiny ones."""
    n, total = case["count"], case["total"]
    share = [0.001 if i % 4 == 3 else 1.0 + 0.37 * (i % 5) for i in range(n)]
    size = [max(1, int(total * s / sum(share))) for s in share]
    return [s if s < 4096 or i % 3 else s // 64 * 64 for i, s in enumerate(size)]


def _types(case):
    return [torch.float32 if case["mixed"] and i % 4 == 3 else DT[case["dtype"]] for i in range(case["count"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT.get(case["dtype"])

    def normal(*shape, std=1.0, mean=0.0):
        t = torch.empty(shape, device="cuda", dtype=dt)
        t.normal_(mean, std, generator=g)
        return t

    s = dict(case=case)
    if case["op"] == "ffn":
        R, C, F = case["R"], case["C"], case["F"]
        s["x"] = normal(R, C)
        s["w_gate"], s["w_up"] = normal(F, C, std=C ** -0.5), normal(F, C, std=C ** -0.5)
        s["w_down"] = normal(C, F, std=F ** -0.5)
        if case["train"]:
            s["dy"] = normal(R, C, std=0.1)
    elif case["op"] == "norm":
        R, C = case["R"], case["C"]
        groups = -(-R // case["per_gate"])
        s["x"], s["y"] = normal(R, C, mean=0.1), normal(R, C, std=0.7, mean=-0.2)
        s["gate"] = normal(groups, C, std=0.3, mean=0.5)
        s["res_scale"] = normal(C, std=0.1, mean=1.0) if case["scale"] else None
        for side in ("post", "pre"):
            has = case[side] != "none" and case["affine"]
            s["w_" + side] = normal(C, std=0.2, mean=1.0) if has else None
            s["b_" + side] = normal(C, std=0.2) if has and case[side] == "layer" else None
        if case["train"]:
            s["dr"] = normal(R, C, std=0.1)
            s["dn"] = normal(R, C, std=0.1) if case["pre"] != "none" else None
    else:
        s["grads"] = [torch.empty(n, device="cuda", dtype=t).normal_(0.0, 10.0 ** (-1 - i % 3), generator=g)
                      for i, (n, t) in enumerate(zip(_sizes(case), _types(case)))]
        # the optimizer's buffers for the clipped gradients, which such a program keeps
        s["outs"] = [torch.empty_like(t) for t in s["grads"]]
    return s


# ---------------------------------------------------------------- plain forms (32 bits, one rounding at the end)
def _act(name, g):
    """The activation and its derivative."""
    if name == "relu":
        return g.clamp(min=0), (g > 0).to(g.dtype)
    if name in ("silu", "sigmoid"):
        p = 1 / (1 + torch.exp(-g))
        return (g * p, p + g * p * (1 - p)) if name == "silu" else (p, p * (1 - p))
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(g * 0.5 ** 0.5))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5
    k = (2 / math.pi) ** 0.5
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def _plain_ffn(s):
    c = s["case"]
    dt = s["x"].dtype
    x, wg, wu, wd = s["x"].float(), s["w_gate"].float(), s["w_up"].float(), s["w_down"].float()
    gate, up = x @ wg.t(), x @ wu.t()
    a, da = _act(c["act"], gate)
    h = a * up
    y = (h @ wd.t()).to(dt)
    if not c["train"]:
        return dict(y=y)
    dy = s["dy"].float()
    dh = dy @ wd
    dgate, dup = dh * up * da, dh * a
    return dict(y=y, dx=(dgate @ wg + dup @ wu).to(dt), dw_gate=(dgate.t() @ x).to(dt), dw_up=(dup.t() @ x).to(dt),
                dw_down=(dy.t() @ h).to(dt))


def _norm(kind, v, w, b):
    """(normalised v, 1 / its deviation, the affine result)."""
    if kind == "none":
        return v, None, v
    m = v - v.mean(-1, keepdim=True) if kind == "layer" else v
    inv = 1 / torch.sqrt((m * m).mean(-1, keepdim=True) + EPS)
    hat = m * inv
    out = hat if w is None else hat * w
    return hat, inv, out if b is None else out + b


def _norm_back(kind, d, hat, inv, w):
    if kind == "none":
        return d
    d = d if w is None else d * w
    back = d - hat * (d * hat).mean(-1, keepdim=True)
    return inv * (back - d.mean(-1, keepdim=True) if kind == "layer" else back)


def _group_sum(v, per):
    groups = -(-v.shape[0] // per)
    out = torch.zeros(groups * per, v.shape[1], device=v.device, dtype=v.dtype)
    out[:v.shape[0]] = v
    return out.view(groups, per, -1).sum(1)


def _plain_norm(s):
    c = s["case"]
    dt = s["x"].dtype
    f = {k: None if s.get(k) is None else s[k].float()
         for k in ("x", "y", "gate", "res_scale", "w_post", "b_post", "w_pre", "b_pre", "dr", "dn")}
    gate = f["gate"].repeat_interleave(c["per_gate"], 0)[:c["R"]]
    y_hat, y_inv, p = _norm(c["post"], f["y"], f["w_post"], f["b_post"])
    r = (f["x"] if f["res_scale"] is None else f["x"] * f["res_scale"]) + gate * p
    r_hat, r_inv, n = _norm(c["pre"], r, f["w_pre"], f["b_pre"])
    out = dict(r=r.to(dt), n=n.to(dt) if c["pre"] != "none" else None)
    if not c["train"]:
        return out
    dt_ = f["dr"]
    if c["pre"] != "none":
        dt_ = dt_ + _norm_back(c["pre"], f["dn"], r_hat, r_inv, f["w_pre"])
    dp = gate * dt_
    grads = dict(dx=dt_ if f["res_scale"] is None else dt_ * f["res_scale"],
                 dy=_norm_back(c["post"], dp, y_hat, y_inv, f["w_post"]), dgate=_group_sum(p * dt_, c["per_gate"]),
                 dres_scale=None if f["res_scale"] is None else (f["x"] * dt_).sum(0),
                 dw_post=None if f["w_post"] is None else (dp * y_hat).sum(0),
                 db_post=None if f["b_post"] is None else dp.sum(0),
                 dw_pre=None if f["w_pre"] is None else (f["dn"] * r_hat).sum(0),
                 db_pre=None if f["b_pre"] is None else f["dn"].sum(0))
    out.update({k: None if v is None else v.to(dt) for k, v in grads.items()})
    return out


def _plain_clip(s):
    total = torch.sqrt(torch.stack([(t.float() * t.float()).sum() for t in s["grads"]]).sum())
    factor = torch.clamp(s["case"]["max_norm"] / (total + EPS), max=1.0)
    return dict(norm=total, outs=[(t.float() * factor).to(t.dtype) for t in s["grads"]])


# ---------------------------------------------------------------- the framework's entry points
def _own_ffn(s):
    import memory_efficient_cnn_gb300 as mec
    c = s["case"]
    args = (s["x"], s["w_gate"], s["w_up"], s["w_down"])
    if not c["train"]:
        return dict(y=mec.gated_ffn(*args, act=c["act"]))
    y, saved = mec.gated_ffn_train(*args, act=c["act"])
    dx, dwg, dwu, dwd = mec.gated_ffn_backward(s["dy"], *args, saved, act=c["act"])
    return dict(y=y, dx=dx, dw_gate=dwg, dw_up=dwu, dw_down=dwd)


def _own_norm(s):
    import memory_efficient_cnn_gb300 as mec
    c = s["case"]
    block = dict(post=c["post"], w_post=s["w_post"], b_post=s["b_post"], gate=s["gate"], rows_per_gate=c["per_gate"],
                 res_scale=s["res_scale"], pre=c["pre"], w_pre=s["w_pre"], b_pre=s["b_pre"], eps=EPS)
    r, n = mec.residual_norm(s["x"], s["y"], **block)
    out = dict(r=r, n=n)
    if c["train"]:
        out.update(mec.residual_norm_backward(s["dr"], s["dn"], s["x"], s["y"], **block))
    return out


def _own_clip(s):
    import memory_efficient_cnn_gb300 as mec
    norm = mec.clip_grad_norm(s["grads"], s["case"]["max_norm"], outs=s["outs"], eps=EPS)
    return dict(norm=norm, outs=s["outs"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"ffn": _own_ffn, "norm": _own_norm, "clip": _own_clip}[op](state)
    return {"ffn": _plain_ffn, "norm": _plain_norm, "clip": _plain_clip}[op](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "ffn":
        R, C, F, e = case["R"], case["C"], case["F"], SIZE[case["dtype"]]
        if case["train"]:
            return dict(bytes=e * (4 * R * C + 6 * C * F), flops=18 * R * C * F)
        return dict(bytes=e * (2 * R * C + 3 * C * F), flops=6 * R * C * F)
    if case["op"] == "norm":
        R, C, e = case["R"], case["C"], SIZE[case["dtype"]]
        groups = -(-R // case["per_gate"])
        has_pre = case["pre"] != "none"
        n_par = case["scale"] + sum(0 if case[k] == "none" or not case["affine"] else 2 if case[k] == "layer" else 1
                                    for k in ("post", "pre"))
        maps, times = (3 + has_pre, 1) if not case["train"] else (6 + 2 * has_pre, 2)
        return dict(bytes=e * (maps * R * C + times * (groups + n_par) * C), flops=(20 if not case["train"] else 60) * R * C)
    elems = _sizes(case)
    size = sum(n * (4 if t == torch.float32 else 2) for n, t in zip(elems, _types(case)))
    return dict(bytes=2 * size, flops=3 * sum(elems))


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_ffn(s):
    """Through the chain rule by torch's own differentiation of the forward definition."""
    c = s["case"]
    leaf = {k: s[k].double().requires_grad_(c["train"]) for k in ("x", "w_gate", "w_up", "w_down")}
    gate = torch.einsum("rc,fc->rf", leaf["x"], leaf["w_gate"])
    up = torch.einsum("rc,fc->rf", leaf["x"], leaf["w_up"])
    fn = torch.nn.functional
    act = {"silu": fn.silu, "gelu": fn.gelu, "gelu_tanh": lambda v: fn.gelu(v, approximate="tanh"), "relu": fn.relu,
           "sigmoid": torch.sigmoid}[c["act"]]
    y = torch.einsum("rf,cf->rc", act(gate) * up, leaf["w_down"])
    out = dict(y=y.detach())
    if c["train"]:
        y.backward(s["dy"].double())
        out.update(dx=leaf["x"].grad, dw_gate=leaf["w_gate"].grad, dw_up=leaf["w_up"].grad, dw_down=leaf["w_down"].grad)
    return out


def _exact_norm(s):
    c = s["case"]
    names = ("x", "y", "gate", "res_scale", "w_post", "b_post", "w_pre", "b_pre")
    leaf = {k: None if s[k] is None else s[k].double().requires_grad_(c["train"]) for k in names}

    def normed(kind, v, w, b):
        if kind == "layer":
            return torch.nn.functional.layer_norm(v, v.shape[-1:], w, b, EPS)
        if kind == "rms":
            v = v * (v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS).rsqrt()
            return v if w is None else v * w
        return v

    at = torch.arange(c["R"], device="cuda") // c["per_gate"]
    r = leaf["x"] if leaf["res_scale"] is None else leaf["x"] * leaf["res_scale"]
    r = r + leaf["gate"].index_select(0, at) * normed(c["post"], leaf["y"], leaf["w_post"], leaf["b_post"])
    n = normed(c["pre"], r, leaf["w_pre"], leaf["b_pre"]) if c["pre"] != "none" else None
    out = dict(r=r.detach(), n=None if n is None else n.detach())
    if c["train"]:
        total = (r * s["dr"].double()).sum()
        if n is not None:
            total = total + (n * s["dn"].double()).sum()
        total.backward()
        out.update({"d" + k: None if leaf[k] is None else leaf[k].grad for k in names})
    return out


def _exact_clip(s):
    total, outs = 0.0, []
    for t in s["grads"]:
        total += float(torch.dot(t.double(), t.double()))
    norm = math.sqrt(total)
    factor = min(1.0, s["case"]["max_norm"] / (norm + EPS))
    for t in s["grads"]:
        outs.append(t.double() * factor)
    return dict(norm=norm, outs=outs)


def exact(case, seed):
    if case["op"] == "ffn" and work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    return {"ffn": _exact_ffn, "norm": _exact_norm, "clip": _exact_clip}[case["op"]](s)
