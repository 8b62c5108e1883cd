"""The norms with gate and residual scale against the 64-bit reference: every
type and pair of norms, absent parts, gates of every extent, odd widths."""
import itertools

import pytest
import torch

import block_ref as ref
import memory_efficient_cnn_gb300 as mec

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
KINDS = ("none", "rms", "layer")


def make(R, C, dt, post="rms", pre="rms", per=None, affine=True, scale=True, gate=True, y=True, eps=1e-6, seed=0, mean=0.3):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0, m=0.0: (torch.randn(*s, generator=g) * std + m).to(DT[dt])  # noqa: E731
    per_ = per or max(R, 1)
    p = dict(post=post, pre=pre, eps=eps, rows_per_gate=per,
             gate=n(-(-R // per_), C, std=0.5, m=0.5) if gate else None,
             res_scale=n(C, std=0.2, m=1.0) if scale else None,
             w_post=n(C, std=0.3, m=1.0) if affine and post != "none" else None,
             b_post=n(C, std=0.3) if affine and post == "layer" else None,
             w_pre=n(C, std=0.3, m=1.0) if affine and pre != "none" else None,
             b_pre=n(C, std=0.3) if affine and pre == "layer" else None)
    return n(R, C, m=mean), n(R, C, std=0.8, m=-mean) if y else None, n(R, C, std=0.5), n(R, C, std=0.5), p


def moved(p, f):
    return {k: f(v) if isinstance(v, torch.Tensor) else v for k, v in p.items()}


def check(x, y, dr, dn, p, dt, what=""):
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    d = lambda t: None if t is None else t.double()  # noqa: E731
    if p["pre"] == "none":
        dn = None
    want = ref.residual_norm_all(d(x), d(y), moved(p, d), DT[dt], d(dr), d(dn), backward=True)
    pc = moved(p, cu)
    r, n = mec.residual_norm(cu(x), cu(y), **pc)
    got = dict(r=r, n=n)
    got.update(mec.residual_norm_backward(cu(dr), cu(dn), cu(x), cu(y), **pc))
    torch.cuda.synchronize()
    ref.check(got, want, what)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("post,pre", list(itertools.product(KINDS, KINDS)))
def test_kinds(dt, post, pre):
    for affine, scale, gate in ((True, True, True), (False, False, False), (True, False, True)):
        x, y, dr, dn, p = make(37, 72, dt, post, pre, per=10, affine=affine, scale=scale, gate=gate)
        if not gate:
            p["rows_per_gate"] = None
        check(x, y, dr, dn, p, dt, f"{dt} {post} {pre} {affine}")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("R,C", [(1, 1), (1, 512), (2, 3), (3, 1000), (5, 33), (64, 128), (65, 130), (7, 4096),
                                 (300, 257), (1000, 64), (129, 8), (2, 8192), (3, 8200), (2, 20000), (9, 2047),
                                 (33, 1024), (40, 3001)])
def test_sizes(dt, R, C):
    x, y, dr, dn, p = make(R, C, dt, "layer", "rms", seed=R + C)
    check(x, y, dr, dn, p, dt, f"{dt} {(R, C)}")
    x, y, dr, dn, p = make(R, C, dt, "rms", "layer", per=max(1, R // 3), seed=R + C)
    check(x, y, dr, dn, p, dt, f"{dt} {(R, C)} grouped")


@pytest.mark.parametrize("per", [1, 2, 63, 64, 65, 100, 700, 699, 701, 5000])
@pytest.mark.parametrize("dt", DT)
def test_gate_extents(dt, per):
    x, y, dr, dn, p = make(700, 48, dt, "rms", "layer", per=per)
    check(x, y, dr, dn, p, dt, f"{dt} per {per}")


@pytest.mark.parametrize("dt", DT)
def test_many_rows(dt):
    x, y, dr, dn, p = make(30000, 40, dt, "layer", "layer", per=784)
    check(x, y, dr, dn, p, dt)
    x, y, dr, dn, p = make(20000, 64, dt, "rms", "rms", per=3)
    check(x, y, dr, dn, p, dt)


@pytest.mark.parametrize("dt", DT)
def test_without_a_branch(dt):
    """The first norm of a stack: no y, no gate."""
    for scale in (False, True):
        x, _, dr, dn, p = make(50, 136, dt, "none", "layer", y=False, gate=False, scale=scale)
        check(x, None, dr, dn, p, dt)


@pytest.mark.parametrize("dt", DT)
def test_absent_gradients(dt):
    x, y, dr, dn, p = make(41, 96, dt, "rms", "rms")
    check(x, y, None, dn, p, dt, "no dr")
    check(x, y, dr, None, p, dt, "no dn")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("post,pre", [("rms", "layer"), ("layer", "rms")])
def test_constant_and_zero_rows(dt, post, pre):
    """Rows without deviation: the eps alone keeps the root from zero."""
    x, y, dr, dn, p = make(6, 64, dt, post, pre, eps=1e-3)
    x[1], y[1] = 0, 0
    y[2] = 0.5
    x[3], y[3] = 2.0, 0
    check(x, y, dr, dn, p, dt)


def test_large_mean():
    """A mean far above the deviation: the second moment is taken about it."""
    x, y, dr, dn, p = make(20, 512, "f32", "layer", "layer", mean=100.0)
    check(x, y, dr, dn, p, "f32")


@pytest.mark.parametrize("dt", DT)
def test_in_place(dt):
    x, y, _, _, p = make(33, 200, dt, "rms", "layer", per=4)
    x, y, p = x.cuda(), y.cuda(), moved(p, lambda t: t.cuda())
    r, n = mec.residual_norm(x, y, **p)
    a = [p[k] for k in ("gate", "rows_per_gate", "res_scale", "post", "w_post", "b_post", "pre", "w_pre", "b_pre", "eps")]
    x2, y2 = x.clone(), y.clone()
    mec.im2win_residual_norm(x2, y2, *a, x2, y2)
    assert torch.equal(x2, r) and torch.equal(y2, n)
    n2 = torch.empty_like(x)
    mec.im2win_residual_norm(x, y, *a, None, n2)  # r not wanted
    assert torch.equal(n2, n)


@pytest.mark.parametrize("dt", DT)
def test_no_rows(dt):
    x, y, dr, dn, p = make(0, 40, dt, "layer", "layer")
    p = moved(p, lambda t: t.cuda())
    x, y, dr, dn = (t.cuda() for t in (x, y, dr, dn))
    r, n = mec.residual_norm(x, y, **p)
    assert r.shape == n.shape == (0, 40)
    g = mec.residual_norm_backward(dr, dn, x, y, **p)
    for k in ("dres_scale", "dw_post", "db_post", "dw_pre", "db_pre"):
        assert bool((g[k] == 0).all()), k


def test_rows_do_not_mix():
    x, y, _, _, p = make(9, 72, "bf16", "rms", "layer")
    p = moved(p, lambda t: t.cuda())
    r, n = mec.residual_norm(x.cuda(), y.cuda(), **p)
    y[4, 7], x[0, 0] = float("nan"), float("inf")
    r2, n2 = mec.residual_norm(x.cuda(), y.cuda(), **p)
    keep = [1, 2, 3, 5, 6, 7, 8]
    assert torch.equal(r2[keep], r[keep]) and torch.equal(n2[keep], n[keep])
    assert bool(n2[4].isnan().all()) and bool(n2[0].isnan().all())


@pytest.mark.parametrize("R,C,per", [(700, 128, 100), (50, 4096, 50), (3000, 33, 7)])
def test_same_bits_every_time(R, C, per):
    for dt in DT:
        x, y, dr, dn, p = make(R, C, dt, "layer", "rms", per=per)
        p = moved(p, lambda t: t.cuda())
        args = [t.cuda() for t in (dr, dn, x, y)]
        a, b = (mec.residual_norm_backward(*args, **p) for _ in range(2))
        assert all(a[k] is b[k] is None or torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("post,pre", [("rms", "layer"), ("layer", "rms"), ("none", "layer")])
def test_gradients_against_differences(post, pre):
    """fp32 gradients along a direction against central differences of the formula
    in 64 bits (their error is of the step's square, 1e-8); each term of the sum is
    held to about 1e-6 of its size."""
    x, y, dr, dn, p = make(12, 40, "f32", post, pre, per=5)
    pc = moved(p, lambda t: t.cuda())
    g = mec.residual_norm_backward(dr.cuda(), dn.cuda(), x.cuda(), y.cuda(), **pc)
    leaves = {"x": x, "y": y, **{k: v for k, v in p.items() if isinstance(v, torch.Tensor)}}
    rnd = torch.Generator().manual_seed(1)
    dirs = {k: torch.randn(v.shape, generator=rnd, dtype=torch.float64) for k, v in leaves.items()}
    s = 1e-4

    def f(k):
        q = {**moved(p, lambda t: t.double()), **{}}
        at = {name: leaves[name].double() + k * s * dirs[name] for name in leaves}
        q.update({name: v for name, v in at.items() if name in p})
        r, n = ref.residual_norm(at["x"], at["y"], q)
        return (r * dr.double()).sum() + (n * dn.double()).sum()

    diff = (f(1) - f(-1)) / (2 * s)
    terms = [g["d" + k].double().cpu() * dirs[k] for k in leaves]
    dot, size = sum(t.sum() for t in terms), sum(t.abs().sum() for t in terms)
    assert abs(float(dot - diff)) <= 1e-5 * float(size)
