"""Calls of the group norm that its documentation allows, in each of its three ways (single rows in registers, maps that
stay on the chip, maps that are read twice): parts of a batch, in place, right behind the launch that writes the inputs."""
import pytest
import torch

import block_ref
import memory_efficient_cnn_gb300 as mec
import norm_bounds

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def make(N, P, C, dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, std=1.0, mean=0.0: torch.empty(s, device="cuda", dtype=DT[dt]).normal_(mean, std, generator=g)  # noqa: E731
    return n(N, P, C, std=1.5, mean=0.7), n(C, std=0.2, mean=1.0), n(C, std=0.3), n(N, P, C, std=0.5)


@pytest.mark.parametrize("N,P,C,G", [(6, 1, 24, 3), (4, 50, 24, 3), (3, 180000, 24, 3)])
def test_gradients_of_a_part_of_a_batch(N, P, C, G):
    """The statistics of its later images begin anywhere on 8 bytes."""
    x, w, b, dy = make(N, P, C, "bf16")
    _, stats = mec.group_norm_train(x, G, w, b, act="silu")
    for first in range(1, N):
        part, own = stats[first:], stats[first:].clone()
        got = mec.group_norm_backward(dy[first:], x[first:], part, w, b, act="silu")
        want = mec.group_norm_backward(dy[first:], x[first:], own, w, b, act="silu")
        assert all(torch.equal(a, c) for a, c in zip(got, want))


# ---- maps that are read twice: in each type, vectors of 16 bytes, two and one elements, and more positions a thread than the
# ring of copies holds (8 forward, 4 backward)
LARGE = [("f32", 40, 3000, 64, 8), ("f32", 10, 7000, 66, 11), ("f32", 10, 14000, 33, 3), ("f16", 20, 8000, 64, 8),
         ("f16", 10, 14000, 66, 11), ("f16", 10, 28000, 33, 3), ("bf16", 20, 8000, 64, 4), ("bf16", 10, 14000, 66, 6),
         ("bf16", 10, 28000, 33, 11)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt,N,P,C,G", LARGE)
def test_large_maps(dt, N, P, C, G, act):
    """A thread adds up to 36 positions, a block up to 128 rows in halves, a lane of the statistics up to 32 of a group's chunks and
    channels; dw and db an eighth of 560 rows: chains of 128 and of 256 at most. The gradients' bounds would show a chunk
    left out (test_norm_bounds.py)."""
    x, w, b, dy = make(N, P, C, dt, seed=C)
    want = norm_bounds.group_norm(x.double(), G, w.double(), b.double(), act, EPS, DT[dt], dy.double(), run=128, run_params=256)
    want = {n: (v.cpu(), e.cpu()) for n, (v, e) in want.items()}
    y, stats = mec.group_norm_train(x, G, w, b, act=act, eps=EPS)
    dx, dw, db = mec.group_norm_backward(dy, x, stats, w, b, act=act)
    block_ref.check(dict(y=y, stats=stats, dx=dx, dw=dw, db=db), want, f"{dt} {(N, P, C, G)}")
    assert torch.equal(mec.group_norm(x, G, w, b, act=act, eps=EPS), y)
    # the same bits again, and in place of the inputs
    y2, stats2 = mec.group_norm_train(x, G, w, b, act=act, eps=EPS)
    again = mec.group_norm_backward(dy, x, stats2, w, b, act=act)
    assert torch.equal(y2, y) and torch.equal(stats2, stats)
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))
    in_place(x, G, w, b, dy, act)


def in_place(x, G, w, b, dy, act):
    """y written over x, and dx over dy."""
    y, stats = mec.group_norm_train(x, G, w, b, act=act, eps=EPS)
    dx, dw, db = mec.group_norm_backward(dy, x, stats, w, b, act=act)
    over, dw2, db2 = dy.clone(), torch.empty_like(dw), torch.empty_like(db)
    mec.im2win_group_norm_backward(over, x, stats, w, b, over, dw2, db2, None, act=act)
    assert torch.equal(over, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    out = x.clone()
    assert mec.group_norm(out, G, w, b, act=act, eps=EPS, out=out) is out
    assert torch.equal(out, y)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("N,P,C,G", [(1, 1, 8, 1), (3000, 1, 96, 4), (70, 1, 1000, 1), (4, 49, 512, 32), (2, 3000, 33, 3),
                                     (5000, 2, 12, 2), (1, 30000, 16, 4), (30000, 4, 40, 5)])
def test_in_place(dt, N, P, C, G):
    in_place(*(lambda x, w, b, dy: (x, G, w, b, dy))(*make(N, P, C, dt)), "silu")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dt,N,P,C,G", [("f16", 20, 30000, 24, 8), ("f32", 10, 14000, 33, 11), ("bf16", 10, 14000, 66, 6)])
def test_spoiled_values_stay_in_their_group(dt, N, P, C, G, bad):
    """Maps that are read twice, whose vectors hold channels of two groups or more."""
    x, w, b, dy = make(N, P, C, dt)
    want, stats = mec.group_norm_train(x, G, w, b, act="silu")
    dx, _, _ = mec.group_norm_backward(dy, x, stats, w, b, act="silu")
    D = C // G
    for p in (0, P // 2, P - 1):  # a chunk's first position, one inside, the last
        spoiled = x.clone()
        spoiled[1, p, D] = bad  # group 1 of image 1
        y, stats2 = mec.group_norm_train(spoiled, G, w, b, act="silu")
        dx2, _, _ = mec.group_norm_backward(dy, spoiled, stats2, w, b, act="silu")
        for got, clean in ((y, want), (dx2, dx)):
            assert got[1, :, D:2 * D].isnan().all()
            keep = torch.ones_like(got, dtype=torch.bool)
            keep[1, :, :2 * D] = False
            assert torch.equal(got[keep], clean[keep])
        # The group before shares a pair of channels with it where D is odd: in 16 bits silu's two logistic functions have
        # one reciprocal between them, 1/p = q (1/pq), whose rounding (2^-23, and the product's) follows the other's q. So p
        # differs by 2^-22 twice, y by that and a step of its type, the slope p + z p (1 - p) by 2^-21 (1 + |z|); of dx, so
        # much of w dy, and of its means (whose sums' roundings are as far below).
        un = 0.0 if dt == "f32" else 2 * block_ref.U[DT[dt]]
        f = lambda t: t[1, :, :D].double()  # noqa: E731
        mean, inv = stats[1, 0].double()
        hat = (f(x) - mean) * inv
        z = hat * w[:D].double() + b[:D].double()
        e = 2.0 ** -21 * (f(dy) * w[:D].double()).abs() * (1 + z.abs())
        most = inv * (e + e.mean() + hat.abs() * (e * hat.abs()).mean()) if dt != "f32" else torch.zeros_like(z)
        assert ((f(y) - f(want)).abs() <= (un + (2.0 ** -21 if un else 0)) * f(want).abs() + block_ref.TINY[DT[dt]] * 2).all()
        assert ((f(dx2) - f(dx)).abs() <= un * f(dx).abs() + 4 * most).all()


WAYS = [(3000, 1, 96, 4), (16, 784, 64, 8), (30, 3136, 128, 32), (1, 200000, 64, 8), (9000, 4, 64, 8)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("N,P,C,G", WAYS)
def test_right_behind_what_writes_the_inputs(dt, N, P, C, G):
    """Norms in a row, each of the one before and in its place, with nothing between them: the launches that read ahead of their
    own wait find what the launch before the call has written."""
    x, w, b, dy = make(N, P, C, dt)

    def chain(wait):
        h, d = x.clone(), dy.clone()
        out = []
        for act in ("silu", "none", "relu", "gelu", "none"):
            mec.group_norm(h, G, w, b, act=act, out=h)
            wait()
            y, stats = mec.group_norm_train(h, G, w, b, act=act)
            wait()
            h.copy_(y) if act == "relu" else h.add_(y)  # (another kernel writes them)
            wait()
            _, stats = mec.group_norm_train(h, G, w, b, act=act)
            wait()
            d, dw, db = mec.group_norm_backward(d, h, stats, w, b, act=act)
            wait()
            mec.im2win_group_norm_backward(d, h, stats, w, b, d, dw, db, None, act=act)
            wait()
            d = d.div_(d.float().abs().max().clamp(min=1e-3)).to(d.dtype)
            out += [y, stats, dw, db]
        return [h, d, *out]

    slow = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(chain(lambda: None), slow))


@pytest.mark.parametrize("N,P,C,G", WAYS)
def test_captured_and_on_two_streams(N, P, C, G):
    """Two graphs with one workspace, replayed in turn; and calls at the same time on two streams."""
    dt = "bf16"
    x, w, b, dy = make(N, P, C, dt)
    x2 = make(N, P, C, dt, seed=1)[0]
    code = mec.BF16
    ws = torch.empty(max(1, *(mec.im2win_group_norm_size(back, N, P, C, G, code) for back in (False, True))), dtype=torch.uint8,
                     device="cuda")

    def step(x, ws=None):
        y, stats = mec.group_norm_train(x, G, w, b, act="silu", ws=ws)
        return (y, stats, *mec.group_norm_backward(dy, x, stats, w, b, act="silu", ws=ws))

    want, want2 = step(x), step(x2)
    held, held2 = x.clone(), x2.clone()
    graphs = []
    for v in (held, held2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(v, ws)
        graphs.append((graph, got))
    for turn in range(3):
        for (graph, got), right in zip(graphs, (want, want2) if turn != 1 else (want2, want)):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, right))
        held.copy_((x2, x, x)[turn])
        held2.copy_((x, x2, x2)[turn])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            other = step(x2)
        here = step(x)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(other, want2)) and all(torch.equal(p, q) for p, q in zip(here, want))
