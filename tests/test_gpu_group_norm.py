"""Group norm with its activation against the 64-bit reference: types, activations,
groups of one channel to all, odd channels, one position to large maps, parameters left
out, spoiled values, and what the contract says about empty calls and repeatability."""
import pytest
import torch

import block_ref
import expert_ref as ref
import memory_efficient_cnn_gb300 as mec

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def make(N, P, C, dt, seed=0, affine=True):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g) * std + mean).to(DT[dt])  # noqa: E731
    return (n(N, P, C, std=1.5, mean=0.7), n(C, std=0.2, mean=1.0) if affine else None, n(C, std=0.3) if affine else None,
            n(N, P, C, std=0.5))


def dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check(N, P, C, G, dt, act="silu", seed=0, affine=True):
    x, w, b, dy = make(N, P, C, dt, seed, affine)
    want = ref.group_norm_all(x.double(), G, *[None if t is None else t.double() for t in (w, b)], act, EPS, DT[dt],
                              dy.double())
    xd, wd, bd, dyd = dev(x, w, b, dy)
    y, stats = mec.group_norm_train(xd, G, wd, bd, act=act, eps=EPS)
    dx, dw, db = mec.group_norm_backward(dyd, xd, stats, wd, bd, act=act)
    plain = mec.group_norm(xd, G, wd, bd, act=act, eps=EPS)
    what = f"{dt} {act} {(N, P, C, G)}"
    block_ref.check(dict(y=y, dx=dx, dw=dw, db=db), want, what)
    assert torch.equal(plain, y), what


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("act", list(mec.NORM_ACTS))
def test_activations(dt, act):
    check(3, 35, 48, 6, dt, act)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("N,P,C,G", [
    (1, 2, 1, 1), (1, 1, 8, 1), (1, 1, 2, 1), (2, 49, 512, 32), (3, 7, 90, 6), (2, 33, 7, 7), (5, 10, 21, 3), (1, 200, 64, 64),
    (4, 64, 32, 1), (2, 300, 24, 8), (1, 3, 2048, 1), (2, 2, 4100, 10), (1, 1, 3000, 3), (2, 17, 1030, 2), (300, 4, 16, 4),
    (1, 5000, 8, 2), (1, 20001, 6, 3), (7, 784, 128, 32)])
def test_sizes(dt, N, P, C, G):
    check(N, P, C, G, dt, seed=N + P + C)


@pytest.mark.parametrize("N,P,C,G,dt", [(8, 3136, 128, 32, "f16"), (2, 40000, 64, 8, "bf16"), (1, 100000, 16, 1, "bf16"),
                                        (1, 50177, 33, 11, "f32"), (2, 3000, 640, 5, "bf16"), (40, 196, 256, 16, "f32")])
def test_large(N, P, C, G, dt):
    check(N, P, C, G, dt, "gelu", seed=5)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("N,C,G", [(1, 1, 1), (3, 8, 8), (1000, 64, 8), (77, 96, 4), (5000, 30, 6), (300, 512, 2), (64, 1024, 1),
                                   (40, 4096, 4), (33, 4100, 2), (9, 2049, 3), (2100, 2048, 32), (20, 510, 1), (7, 12288, 3)])
def test_one_position(dt, N, C, G):
    """Groups of single rows, of one element to more than the lanes of a warp hold."""
    check(N, 1, C, G, dt, "gelu", seed=N + C)


@pytest.mark.parametrize("dt", DT)
def test_without_parameters(dt):
    check(2, 50, 40, 5, dt, affine=False)
    x, w, b, dy = dev(*make(2, 50, 40, dt))
    y, stats = mec.group_norm_train(x, 5, None, b)
    dx, dw, db = mec.group_norm_backward(dy, x, stats, None, b)
    assert dw is None
    one = torch.ones_like(b)
    y1, stats1 = mec.group_norm_train(x, 5, one, b)
    dx1, _, db1 = mec.group_norm_backward(dy, x, stats1, one, b)
    assert torch.equal(y, y1) and torch.equal(dx, dx1) and torch.equal(db, db1) and torch.equal(stats, stats1)


@pytest.mark.parametrize("P", [40, 30000])
def test_far_mean(P):
    """Values whose mean is four hundred deviations away keep their digits; an outlier in front of
    them does not cost the others theirs."""
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(2, P, 16, generator=g) + 400.0).float()
    want = ref.group_norm_all(x.double(), 4, None, None, "none", EPS, torch.float32)
    block_ref.check(dict(y=mec.group_norm(x.cuda(), 4)), want)
    x = torch.randn(1, P, 16, generator=g).float()
    x[0, 0, 0] = 3000.0
    want = ref.group_norm_all(x.double(), 4, None, None, "none", EPS, torch.float32)
    block_ref.check(dict(y=mec.group_norm(x.cuda(), 4)), want)


@pytest.mark.parametrize("P", [1, 9, 4000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_spoiled_values_stay_in_their_group(P, bad):
    x, w, b, dy = dev(*make(3, P, 24, "bf16"))
    want, stats = mec.group_norm_train(x, 4, w, b)
    dx, _, _ = mec.group_norm_backward(dy, x, stats, w, b)
    x2 = x.clone()
    x2[1, P // 2, 7] = bad  # group 1 of image 1
    y, stats2 = mec.group_norm_train(x2, 4, w, b)
    dx2, _, _ = mec.group_norm_backward(dy, x2, stats2, w, b)
    for got, clean in ((y, want), (dx2, dx)):
        assert got[1, :, 6:12].float().isnan().all()
        keep = torch.ones_like(got, dtype=torch.bool)
        keep[1, :, 6:12] = False
        assert torch.equal(got[keep], clean[keep])


def test_constant_maps():
    x = torch.full((2, 30, 16), 3.0, device="cuda")
    w, b = torch.full((16,), 2.0, device="cuda"), torch.full((16,), 0.25, device="cuda")
    assert torch.equal(mec.group_norm(x, 4, w, b), torch.full_like(x, 0.25))


def test_empty():
    w = torch.ones(8, device="cuda")
    for shape in ((0, 5, 8), (3, 0, 8)):
        x = torch.empty(shape, device="cuda")
        y, stats = mec.group_norm_train(x, 2, w, w)
        dx, dw, db = mec.group_norm_backward(x, x, stats, w, w)
        assert y.shape == dx.shape == x.shape and not dw.any() and not db.any()


def test_shapes_in_place_and_out():
    x, w, b, _ = dev(*make(2, 12, 16, "f16"))
    want = mec.group_norm(x, 4, w, b, act="relu")
    out = torch.full((2, 3, 4, 16), float("nan"), dtype=x.dtype, device="cuda")
    assert mec.group_norm(x.view(2, 3, 4, 16), 4, w, b, act="relu", out=out) is out
    assert torch.equal(out.view(2, 12, 16), want)
    flat = mec.group_norm(x.view(24, 16), 4, w, b)  # a position an image
    assert torch.equal(flat, mec.group_norm(x.view(24, 1, 16), 4, w, b).view(24, 16))
    mec.group_norm(x, 4, w, b, act="relu", out=x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("N,P,C,G", [(1, 49, 512, 32), (4, 3136, 64, 8), (2, 40000, 24, 3)])
@pytest.mark.parametrize("dt", DT)
def test_same_bits_every_time(N, P, C, G, dt):
    x, w, b, dy = dev(*make(N, P, C, dt))

    def once():
        y, stats = mec.group_norm_train(x, G, w, b, act="silu")
        return (y, stats, *mec.group_norm_backward(dy, x, stats, w, b, act="silu"))

    assert all(torch.equal(a, c) for a, c in zip(once(), once()))


def test_gradients_asked_for_alone():
    x, w, b, dy = dev(*make(2, 60, 24, "bf16"))
    _, stats = mec.group_norm_train(x, 3, w, b, act="gelu")
    dx, dw, db = mec.group_norm_backward(dy, x, stats, w, b, act="gelu")
    only = mec.group_norm_backward(dy, x, stats, w, b, act="gelu", need_dw=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    only = mec.group_norm_backward(dy, x, stats, w, b, act="gelu", need_dx=False)
    assert only[0] is None and torch.equal(only[1], dw) and torch.equal(only[2], db)


def test_gradient_by_differences():
    x, w, b, dy = (t.float().double() for t in make(1, 6, 8, "f32", seed=3))
    _, stats = mec.group_norm_train(x.float().cuda(), 2, w.float().cuda(), b.float().cuda(), act="silu", eps=EPS)
    grads = mec.group_norm_backward(dy.float().cuda(), x.float().cuda(), stats, w.float().cuda(), b.float().cuda(), act="silu")

    def value(x, w, b):
        return (ref.group_norm_all(x, 2, w, b, "silu", EPS, torch.float32)["y"][0] * dy).sum()

    h = 1e-5
    for i, got in enumerate(grads):
        args = [x, w, b]
        for at in range(0, args[i].numel(), 5):
            up, down = [t.clone() for t in args], [t.clone() for t in args]
            up[i].view(-1)[at] += h
            down[i].view(-1)[at] -= h
            slope = (value(*up) - value(*down)) / (2 * h)
            # central differences err by h^2 times the third derivative, and by 1e-16 / h
            assert abs(float(got.view(-1)[at]) - float(slope)) < 2e-5 * (1 + abs(float(slope)))


def test_graph_and_streams():
    x, w, b, dy = dev(*make(3, 500, 32, "bf16"))
    side = torch.cuda.Stream()
    out, ws = torch.empty_like(x), torch.empty(max(1, mec.im2win_group_norm_size(False, 3, 500, 32, 4, mec.BF16)), dtype=torch.uint8, device="cuda")
    want, stats = mec.group_norm_train(x, 4, w, b, act="silu")
    want_back = mec.group_norm_backward(dy, x, stats, w, b, act="silu")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mec.group_norm(x, 4, w, b, act="silu")
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mec.group_norm(x, 4, w, b, act="silu", out=out, ws=ws)
        y, s = mec.group_norm_train(x, 4, w, b, act="silu")
        back = mec.group_norm_backward(dy, x, s, w, b, act="silu")
    keep = x.clone()
    x.mul_(2.0)
    out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, mec.group_norm(x, 4, w, b, act="silu"))
    x.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(y, want)
    assert all(torch.equal(a, c) for a, c in zip(back, want_back))
