"""Timed cases of the operators of a block of experts after a convolution: the group
norm with its activation over channels-last maps, the router, and the gated
feed-forward grouped by expert. `run` computes a case in elementary torch operations,
or, where `own` is true, by the framework's entry points."""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5


def listed():
    return [
        # the last 7 x 7 maps of one image while serving; latency only
        dict(name="norm_one_image", op="norm", train=False, N=1, H=7, W=7, C=512, G=32, act="silu", affine=True, dtype="bf16"),
        # inference over the 56 x 56 x 128 maps of 64 images (the sweep layers' batch)
        dict(name="norm_maps", op="norm", train=False, N=64, H=56, W=56, C=128, G=32, act="relu", affine=True, dtype="f16"),
        # a training step over the same maps
        dict(name="norm_train_maps", op="norm", train=True, N=64, H=56, W=56, C=128, G=32, act="silu", affine=True, dtype="bf16"),
        # full-precision training over odd maps, groups of no whole vector
        dict(name="norm_train_odd", op="norm", train=True, N=13, H=31, W=37, C=90, G=6, act="gelu", affine=True, dtype="f32"),
        # training over the first, wide maps of large images: one image is more than the SMs of a cluster hold
        dict(name="norm_train_large", op="norm", train=True, N=4, H=448, W=448, C=64, G=8, act="silu", affine=True, dtype="bf16"),
        # the router of one position; latency only
        dict(name="route_one", op="route", train=False, T=1, E=8, k=2, over="top", dtype="bf16"),
        # routing every position of 28 x 28 maps of 64 images, with gradients
        dict(name="route_train_maps", op="route", train=True, T=64 * 28 * 28, E=64, k=4, over="all", dtype="f32"),
        # one position through two of eight experts: a generated token or pooled features; latency only
        dict(name="experts_one", op="experts", train=False, T=1, k=2, E=8, C=512, F=2048, act="silu", dtype="bf16"),
        # a ragged batch for many experts; the hidden width is no multiple of a vector
        dict(name="experts_ragged", op="experts", train=False, T=777, k=2, E=24, C=1000, F=1366, act="gelu_tanh", dtype="bf16"),
        # a training step over 28 x 28 maps of 16 images
        dict(name="experts_train_maps", op="experts", train=True, T=16 * 28 * 28, k=2, E=8, C=256, F=1024, act="gelu", dtype="f16"),
        # a full-precision training step of odd sizes
        dict(name="experts_train_f32", op="experts", train=True, T=1569, k=1, E=5, C=384, F=1001, act="silu", dtype="f32"),
        # the largest training step: many rows, wide experts
        dict(name="experts_train_wide", op="experts", train=True, T=8192, k=2, E=16, C=2048, F=4096, act="silu", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "route", "experts", "experts"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
    train = rng.random() < 0.5
    if op == "norm":
        D = rng.choice([1, 2, 3, 4, 8, 15, 16, 32, 64])
        G = _log(rng, 1, max(1, 2048 // D))
        most = 4 * 448 * 448 * 64 * 2 // SIZE[dtype]
        H, W = _log(rng, 1, 448), _log(rng, 1, 448)
        C = G * D
        while H * W * C > most:
            H = max(1, H // 2)
        N = min(_log(rng, 1, 256), max(1, most // (H * W * C)))
        return dict(op="norm", train=train, N=N, H=H, W=W, C=C, G=G, act=rng.choice(["none", act]),
                    affine=rng.random() < 0.8, dtype=dtype)
    if op == "route":
        E = _log(rng, 2, 256)
        return dict(op="route", train=train, T=_log(rng, 1, 200704), E=E, k=rng.randint(1, min(8, E)),
                    over=rng.choice(["top", "all"]), dtype=dtype)
    E = _log(rng, 1, 64)
    k = rng.randint(1, min(4, E))
    C = _log(rng, 64, 512 if dtype == "f32" else 2048)
    if rng.random() < 0.6:
        C = C // 8 * 8
    F = max(1, int(C * rng.uniform(0.5, 4.0)))
    if rng.random() < 0.6:
        F = max(8, F // 8 * 8)
    E = max(k, min(E, 16 * 2048 * 4096 // (C * F)))
    most = (1 if train else 3) * (8192 * 2 * 2048 * 4096 // (16 if dtype == "f32" else 1)) // (k * C * F)
    T = min(_log(rng, 1, 12544), max(1, most))
    return dict(op="experts", train=train, T=T, k=k, E=E, C=C, F=F, act=act, dtype=dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return torch.empty(shape, device="cuda", dtype=dtype).normal_(mean, std, generator=g)

    s = dict(case=case)
    if case["op"] == "norm":
        N, H, W, C = (case[k] for k in ("N", "H", "W", "C"))
        s["x"] = normal(N, H, W, C, std=1.5, mean=0.4)
        s["w"] = normal(C, std=0.2, mean=1.0) if case["affine"] else None
        s["b"] = normal(C, std=0.2) if case["affine"] else None
        if case["train"]:
            s["dy"] = normal(N, H, W, C, std=0.1)
        return s
    T, k, E = case["T"], case["k"], case["E"]
    # some experts are in more demand than others
    logits = normal(T, E, std=1.0, dtype=torch.float32) + normal(E, std=0.5, dtype=torch.float32)
    if case["op"] == "route":
        s["logits"] = logits.to(dt)
        if case["train"]:
            s["dweights"] = normal(T, k, std=0.1)
        return s
    C, F = case["C"], case["F"]
    top, at = logits.topk(k, dim=-1)
    # a few positions find their expert full and are dropped there
    dropped = torch.rand(T, k, device="cuda", generator=g) < 0.01
    s["experts"] = torch.where(dropped, -1, at).to(torch.int32)
    s["weights"] = torch.softmax(top, -1).to(dt)
    s["x"] = normal(T, C)
    s["w_gate"], s["w_up"] = normal(E, F, C, std=C ** -0.5), normal(E, F, C, std=C ** -0.5)
    s["w_down"] = normal(E, C, F, std=F ** -0.5)
    if case["train"]:
        s["dy"] = normal(T, C, std=0.1)
    return s


# ---------------------------------------------------------------- plain forms (32 bits, one rounding at the end)
def _act(name, g):
    """The activation and its derivative."""
    if name == "none":
        return g, torch.ones_like(g)
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


def _plain_norm(s):
    c = s["case"]
    dt, shape = s["x"].dtype, s["x"].shape
    N, G, D = c["N"], c["G"], c["C"] // c["G"]
    x = s["x"].float().view(N, -1, G, D)
    mean = x.mean((1, 3), keepdim=True)
    m = x - mean
    inv = 1 / torch.sqrt((m * m).mean((1, 3), keepdim=True) + EPS)
    hat = m * inv
    w = None if s["w"] is None else s["w"].float().view(1, 1, G, D)
    z = hat if w is None else hat * w + s["b"].float().view(1, 1, G, D)
    y, slope = _act(c["act"], z)
    out = dict(y=y.to(dt).view(shape))
    if not c["train"]:
        return out
    dz = s["dy"].float().view(N, -1, G, D) * slope
    d = dz if w is None else dz * w
    dx = inv * (d - d.mean((1, 3), keepdim=True) - hat * (d * hat).mean((1, 3), keepdim=True))
    out.update(dx=dx.to(dt).view(shape), dw=None if w is None else (dz * hat).sum((0, 1)).view(-1).to(dt),
               db=None if w is None else dz.sum((0, 1)).view(-1).to(dt))
    return out


def _plain_route(s):
    c = s["case"]
    T, k = c["T"], c["k"]
    logits = s["logits"].float()
    # a stable descending order: equal logits keep the order of their indexes
    experts = torch.sort(logits, dim=-1, descending=True, stable=True)[1][:, :k]
    chosen = logits.gather(-1, experts)
    top = logits.max(-1, keepdim=True)[0]
    e = torch.exp(logits - top)
    total = e.sum(-1, keepdim=True) if c["over"] == "all" else e.gather(-1, experts).sum(-1, keepdim=True)
    weights = torch.exp(chosen - top) / total
    dt = s["logits"].dtype
    out = dict(weights=weights.to(dt), experts=experts.to(torch.int32))
    if c["train"]:
        dweights = s["dweights"].float()
        mean = (weights * dweights).sum(-1, keepdim=True)
        d = torch.zeros_like(logits)
        if c["over"] == "all":
            d = -(e / total) * mean
        d = d.scatter_add(-1, experts, weights * (dweights if c["over"] == "all" else dweights - mean))
        out["dlogits"] = d.to(dt)
    return out


def _plain_experts(s):
    c = s["case"]
    dt = s["x"].dtype
    x = s["x"].float()
    y = torch.zeros_like(x)
    train = c["train"]
    if train:
        dy, dx, dweights = s["dy"].float(), torch.zeros_like(x), torch.zeros(s["weights"].shape, device="cuda")
        dws = {n: torch.zeros_like(s[n]) for n in ("w_gate", "w_up", "w_down")}
    for e in range(c["E"]):
        t, j = (s["experts"] == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        wg, wu, wd = s["w_gate"][e].float(), s["w_up"][e].float(), s["w_down"][e].float()
        xe, p = x[t], s["weights"][t, j].float().unsqueeze(-1)
        gate, up = xe @ wg.t(), xe @ wu.t()
        a, da = _act(c["act"], gate)
        h = a * up
        ye = h @ wd.t()
        y.index_add_(0, t, ye * p)
        if train:
            dweights[t, j] = (dy[t] * ye).sum(-1)
            dye = dy[t] * p
            dh = dye @ wd
            dgate, dup = dh * up * da, dh * a
            dx.index_add_(0, t, dgate @ wg + dup @ wu)
            dws["w_gate"][e], dws["w_up"][e] = (dgate.t() @ xe).to(dt), (dup.t() @ xe).to(dt)
            dws["w_down"][e] = (dye.t() @ h).to(dt)
    out = dict(y=y.to(dt))
    if train:
        out.update(dx=dx.to(dt), dweights=dweights.to(dt), dw_gate=dws["w_gate"], dw_up=dws["w_up"], dw_down=dws["w_down"])
    return out


# ---------------------------------------------------------------- the framework's entry points
def _own_norm(s):
    import memory_efficient_cnn_gb300 as mec
    c = s["case"]
    args = dict(w=s["w"], b=s["b"], act=c["act"])
    if not c["train"]:
        return dict(y=mec.group_norm(s["x"], c["G"], eps=EPS, **args))
    y, stats = mec.group_norm_train(s["x"], c["G"], eps=EPS, **args)
    dx, dw, db = mec.group_norm_backward(s["dy"], s["x"], stats, **args)
    return dict(y=y, dx=dx, dw=dw, db=db)


def _own_route(s):
    import memory_efficient_cnn_gb300 as mec
    c = s["case"]
    weights, experts = mec.expert_route(s["logits"], c["k"], over=c["over"])
    out = dict(weights=weights, experts=experts)
    if c["train"]:
        out["dlogits"] = mec.expert_route_backward(s["dweights"], s["logits"], experts, over=c["over"])
    return out


def _own_experts(s):
    import memory_efficient_cnn_gb300 as mec
    c = s["case"]
    ws = (s["w_gate"], s["w_up"], s["w_down"])
    if not c["train"]:
        return dict(y=mec.expert_ffn(s["x"], s["experts"], s["weights"], *ws, act=c["act"]))
    y, saved = mec.expert_ffn_train(s["x"], s["experts"], s["weights"], *ws, act=c["act"])
    dx, dweights, dwg, dwu, dwd = mec.expert_ffn_backward(s["dy"], s["weights"], *ws, saved, act=c["act"])
    return dict(y=y, dx=dx, dweights=dweights, dw_gate=dwg, dw_up=dwu, dw_down=dwd)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "route": _own_route, "experts": _own_experts}[op](state)
    return {"norm": _plain_norm, "route": _plain_route, "experts": _plain_experts}[op](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    size = SIZE[case["dtype"]]
    if case["op"] == "norm":
        n = case["N"] * case["H"] * case["W"] * case["C"]
        par = case["C"] * (2 if case["affine"] else 0)
        # training: x, dy read; y, dx written
        maps, pars, each = (4, 2, 40) if case["train"] else (2, 1, 15)
        return dict(bytes=size * (maps * n + pars * par), flops=each * n)
    T, k, E = case["T"], case["k"], case["E"]
    if case["op"] == "route":
        if case["train"]:
            return dict(bytes=2 * size * T * E + (2 * size + 4) * T * k, flops=12 * T * E)
        return dict(bytes=size * T * E + (size + 4) * T * k, flops=6 * T * E)
    C, F, pairs = case["C"], case["F"], T * k
    # no more experts than pairs are read
    read = 3 * min(E, pairs) * C * F
    if case["train"]:
        return dict(bytes=size * (4 * T * C + read + 3 * E * C * F) + (2 * size + 4) * pairs, flops=18 * pairs * C * F)
    return dict(bytes=size * (2 * T * C + read) + (size + 4) * pairs, flops=6 * pairs * C * F)


# ---------------------------------------------------------------- the definitions in 64 bits
_TORCH_ACT = {"none": lambda v: v, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
              "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh"), "relu": torch.nn.functional.relu,
              "sigmoid": torch.sigmoid}


def _exact_norm(s):
    """Image by image, through torch's own differentiation of the forward definition."""
    c = s["case"]
    ys, dxs = [], []
    leaf = {n: None if s[n] is None else s[n].double().requires_grad_(c["train"]) for n in ("w", "b")}
    for n in range(c["N"]):
        x = s["x"][n].double().reshape(1, -1, c["C"]).transpose(1, 2).contiguous().requires_grad_(c["train"])
        z = torch.nn.functional.group_norm(x, c["G"], leaf["w"], leaf["b"], EPS)
        y = _TORCH_ACT[c["act"]](z)
        ys.append(y.detach().transpose(1, 2).reshape(s["x"].shape[1:]))
        if c["train"]:
            y.backward(s["dy"][n].double().reshape(1, -1, c["C"]).transpose(1, 2))
            dxs.append(x.grad.transpose(1, 2).reshape(s["x"].shape[1:]))
    out = dict(y=torch.stack(ys))
    if c["train"]:
        out.update(dx=torch.stack(dxs), **{"d" + n: None if v is None else v.grad for n, v in leaf.items()})
    return out


def _exact_route(s):
    c = s["case"]
    logits = s["logits"].double().requires_grad_(c["train"])
    experts = torch.argsort(logits.detach(), dim=-1, descending=True, stable=True)[:, :c["k"]]
    if c["over"] == "all":
        weights = torch.softmax(logits, -1).gather(-1, experts)
    else:
        weights = torch.softmax(logits.gather(-1, experts), -1)
    out = dict(weights=weights.detach(), experts=experts.to(torch.int32))
    if c["train"]:
        weights.backward(s["dweights"].double())
        out["dlogits"] = logits.grad
    return out


def _exact_experts(s):
    """One expert after the other over all positions that chose it, by torch's own differentiation."""
    c = s["case"]
    train = c["train"]
    x = s["x"].double().requires_grad_(train)
    weights = s["weights"].double().requires_grad_(train)
    y = torch.zeros_like(s["x"], dtype=torch.float64)
    grads = {n: [] for n in ("w_gate", "w_up", "w_down")}
    for e in range(c["E"]):
        leaf = {n: s[n][e].double().requires_grad_(train) for n in grads}
        pairs = (s["experts"] == e).reshape(-1).nonzero().reshape(-1)
        at = torch.div(pairs, c["k"], rounding_mode="floor")
        rows = x.index_select(0, at)
        h = _TORCH_ACT[c["act"]](torch.einsum("rc,fc->rf", rows, leaf["w_gate"])) * torch.einsum("rc,fc->rf", rows, leaf["w_up"])
        part = torch.einsum("rf,cf->rc", h, leaf["w_down"]) * weights.reshape(-1, 1).index_select(0, pairs)
        y.index_add_(0, at, part.detach())
        if train:
            part.backward(s["dy"].double().index_select(0, at))
            for n, v in leaf.items():
                grads[n].append(v.grad)
    out = dict(y=y)
    if train:
        out.update(dx=x.grad, dweights=weights.grad, **{"d" + n: torch.stack(v) for n, v in grads.items()})
    return out


def exact(case, seed):
    if case["op"] == "experts" and work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "experts": _exact_experts}[case["op"]](s)
