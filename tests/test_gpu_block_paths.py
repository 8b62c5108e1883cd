"""Paths of the residual-block operators that sizes of the other tests do not reach, or that
they reach one call at a time: calls in a row, in graphs and on two streams, buffers that begin
as NaN, blocks of several tiles."""
import pytest
import torch

import block_ref as ref
import memory_efficient_cnn_gb300 as mec
from test_gpu_gated_ffn import DT, check as check_ffn, make
from test_gpu_residual_norm import make as make_norm, moved

pytestmark = pytest.mark.gpu

# sizes of each way through the feed-forward
FFN_PATHS = {
    "few": (5, 520, 1000), "one kernel": (40000, 128, 200), "single tiles": (300, 256, 640),
    "pairs": (8192, 1024, 2048), "pairs, streamed": (512, 4096, 1024), "odd": (777, 1001, 271)}


@pytest.mark.parametrize("path", FFN_PATHS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_calls_in_a_row(dt, path):
    """Launches that begin while the one before ends, fifty calls on: the same bits, and no wait
    of any that gave up."""
    R, C, F = FFN_PATHS[path]
    code = mec._binding._DTYPE[DT[dt]]
    x, wg, wu, wd, dy = (t.cuda() for t in make(R, C, F, dt))
    ws = torch.empty(mec.im2win_gated_ffn_size(mec.FFN_FORWARD, R, C, F, code), dtype=torch.uint8, device="cuda")
    wb = torch.empty(mec.im2win_gated_ffn_size(mec.FFN_BACKWARD, R, C, F, code), dtype=torch.uint8, device="cuda")
    want = mec.gated_ffn(x, wg, wu, wd, ws=ws)
    _, saved = mec.gated_ffn_train(x, wg, wu, wd)
    grads = mec.gated_ffn_backward(dy, x, wg, wu, wd, saved, ws=wb)
    got = [(mec.gated_ffn(x, wg, wu, wd, ws=ws), mec.gated_ffn_backward(dy, x, wg, wu, wd, saved, ws=wb)) for _ in range(50)]
    assert mec.im2win_device_status(ws) == 0 and mec.im2win_device_status(wb) == 0
    for y, g in got:
        assert torch.equal(y, want) and all(torch.equal(a, b) for a, b in zip(g, grads))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("R,C,F", [(5, 512, 10240), (3, 5000, 264), (1, 9744, 512), (16, 256, 9000), (16, 264, 5008),
                                   (17, 128, 256), (24, 512, 1536), (32, 1024, 4096), (32, 264, 5000), (29, 2440, 72),
                                   (11, 2600, 3002)])
def test_few_rows(dt, R, C, F):
    """Blocks of several tiles of weights, on either side; 17 to 32 rows of whole vectors."""
    check_ffn(R, C, F, dt, "silu", seed=R + C)


def test_rows_do_not_mix_f32():
    """A row that is not finite spoils its own outputs only, by every way of fp32."""
    for R, C, F in ((3, 64, 96), (20, 520, 1000), (300, 64, 96), (300, 1000, 250)):
        x, wg, wu, wd, _ = (t.cuda() for t in make(R, C, F, "f32"))
        clean = mec.gated_ffn(x, wg, wu, wd)
        for value in (float("nan"), float("inf")):
            bad = x.clone()
            bad[R // 2, 5] = value
            got = mec.gated_ffn(bad, wg, wu, wd)
            keep = torch.arange(R, device="cuda") != R // 2
            assert torch.equal(got[keep], clean[keep]) and not torch.isfinite(got[R // 2]).any(), (R, C, F, value)


# ---------------------------------------------------------------- buffers that begin as NaN, between guard bytes
def guarded(nbytes):
    """A buffer of 0xFF (NaN in every type) between guard bytes, and its inside."""
    n = (nbytes + 15) // 16 * 16
    buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    inside = buf[256:256 + nbytes]
    inside.fill_(0xFF)
    return buf, inside


class Guards:
    def __init__(self):
        self.all = {}

    def bytes(self, name, n):
        self.all[name] = guarded(n)
        return self.all[name][1]

    def like(self, name, t):
        return self.bytes(name, t.numel() * t.element_size()).view(t.dtype).view(t.shape)

    def check(self):
        torch.cuda.synchronize()
        for name, (buf, inside) in self.all.items():
            n = inside.numel()
            assert bool((buf[:256] == 0xA5).all()) and bool((buf[256 + n:] == 0xA5).all()), name


@pytest.mark.parametrize("path", FFN_PATHS)
@pytest.mark.parametrize("dt", DT)
def test_ffn_buffers(dt, path):
    """Nothing is read that the call has not written, and nothing is written beside the buffers."""
    R, C, F = FFN_PATHS[path]
    code = mec._binding._DTYPE[DT[dt]]
    x, wg, wu, wd, dy = (t.cuda() for t in make(R, C, F, dt))
    want_y = mec.gated_ffn(x, wg, wu, wd)
    want_t, saved = mec.gated_ffn_train(x, wg, wu, wd)
    want = mec.gated_ffn_backward(dy, x, wg, wu, wd, saved)
    size = lambda b: mec.im2win_gated_ffn_size(b, R, C, F, code)  # noqa: E731
    g = Guards()
    y, yt = g.like("y", x), g.like("y of training", x)
    mec.im2win_gated_ffn(x, wg, wu, wd, y, None, g.bytes("forward", size(mec.FFN_FORWARD)))
    kept = g.bytes("saved", size(mec.FFN_SAVED))
    mec.im2win_gated_ffn(x, wg, wu, wd, yt, kept, g.bytes("train", size(mec.FFN_TRAIN)))
    grads = [g.like(n, t) for n, t in (("dx", x), ("dw_gate", wg), ("dw_up", wu), ("dw_down", wd))]
    mec.im2win_gated_ffn_backward(dy, x, wg, wu, wd, kept, *grads, g.bytes("backward", size(mec.FFN_BACKWARD)))
    g.check()
    assert torch.equal(y, want_y) and torch.equal(yt, want_t)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("R,C,per", [(700, 48, 64), (3000, 33, 7), (600, 6000, 1), (310, 6000, 310), (300, 4096, 100),
                                     (50, 8200, 7), (9, 2047, 9), (1, 1, 1)])
def test_norm_buffers(dt, R, C, per):
    code = mec._binding._DTYPE[DT[dt]]
    x, y, dr, dn, p = make_norm(R, C, dt, "layer", "rms", per=per)
    x, y, dr, dn = (t.cuda() for t in (x, y, dr, dn))
    p = moved(p, lambda t: t.cuda())
    want = mec.residual_norm(x, y, **p)
    want_back = mec.residual_norm_backward(dr, dn, x, y, **p)
    args = [x, y, *(p[k] for k in ("gate", "rows_per_gate", "res_scale", "post", "w_post", "b_post", "pre", "w_pre", "b_pre",
                                   "eps"))]
    g = Guards()
    r, n = g.like("r", x), g.like("n", x)
    mec.im2win_residual_norm(*args, r, n)
    back = {k: None if v is None else g.like(k, v) for k, v in want_back.items()}
    ws = g.bytes("ws", mec.im2win_residual_norm_backward_size(R, C, per, code))
    mec.im2win_residual_norm_backward(dr, dn, *args, *back.values(), ws)
    g.check()
    assert torch.equal(r, want[0]) and torch.equal(n, want[1])
    assert all(v is None or torch.equal(v, want_back[k]) for k, v in back.items())


# ---------------------------------------------------------------- graphs and streams
@pytest.mark.parametrize("path", FFN_PATHS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_ffn_in_a_graph(dt, path):
    """Captured once, replayed on other inputs."""
    R, C, F = FFN_PATHS[path]
    first, then = (([t.cuda() for t in make(R, C, F, dt, seed=s)]) for s in (1, 2))

    def step(x, wg, wu, wd, dy):
        y, saved = mec.gated_ffn_train(x, wg, wu, wd)
        return (mec.gated_ffn(x, wg, wu, wd), y, *mec.gated_ffn_backward(dy, x, wg, wu, wd, saved))

    step(*first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*first)
    for a, b in zip(first, then):
        a.copy_(b)
    for _ in range(3):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, step(*then)))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_norm_and_clip_in_a_graph(dt):
    def data(seed):
        x, y, dr, dn, p = make_norm(500, 200, dt, "layer", "rms", per=50, seed=seed)
        return [t.cuda() for t in (x, y, dr, dn)], moved(p, lambda t: t.cuda())

    (first, p), (then, q) = data(1), data(2)

    def step(x, y, dr, dn, p):
        r, n = mec.residual_norm(x, y, **p)
        g = [t for t in mec.residual_norm_backward(dr, dn, x, y, **p).values() if t is not None]
        outs = [torch.empty_like(t) for t in g]
        return [r, n, *g, mec.clip_grad_norm(g, 0.5, outs=outs), *outs]

    step(*first, p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*first, p)
    for a, b in zip(first, then):
        a.copy_(b)
    for k, v in q.items():
        if isinstance(v, torch.Tensor):
            p[k].copy_(v)
    for _ in range(3):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, step(*then, q)))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_two_streams_at_once(dt):
    """Calls of every way on two streams, each with buffers of its own."""
    sets = []
    for path in FFN_PATHS:
        sets.append([t.cuda() for t in make(*FFN_PATHS[path], dt, seed=len(sets))])

    def step(x, wg, wu, wd, dy):
        y, saved = mec.gated_ffn_train(x, wg, wu, wd)
        g = mec.gated_ffn_backward(dy, x, wg, wu, wd, saved)
        r, n = mec.residual_norm(x, y, post="rms", pre="layer")
        b = mec.residual_norm_backward(dy, n, x, y, post="rms", pre="layer")
        norm = mec.clip_grad_norm(list(g), 1.0)
        return (mec.gated_ffn(x, wg, wu, wd), y, *g, r, n, b["dx"], b["dy"], norm)

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for i in range(4 * len(sets)):
        for k, st in enumerate(side):
            j = (i + k * 3) % len(sets)  # never the same way at the same time
            with torch.cuda.stream(st):
                got[k].append((j, step(*sets[j])))
    torch.cuda.synchronize()
    for k in range(2):
        for j, out in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[j])), j


# ---------------------------------------------------------------- offsets past 32 bits
LAST = 300


def test_ffn_beyond_32_bit_offsets():
    """More than 2^31 elements of x, y and dx; dy is zero but for the last rows, which alone then make the dw."""
    R, C, F = 2_200_003, 1000, 24
    x, wg, wu, wd, dy = make(LAST, C, F, "bf16")
    want = ref.ffn_all(*(t.double() for t in (x, wg, wu, wd)), "silu", torch.bfloat16, dy.double())
    w = [t.cuda() for t in (wg, wu, wd)]
    big, bdy = (torch.zeros(R, C, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    big[-LAST:], bdy[-LAST:] = x.cuda(), dy.cuda()
    y, saved = mec.gated_ffn_train(big, *w)
    dx, dwg, dwu, dwd = mec.gated_ffn_backward(bdy, big, *w, saved)
    ref.check(dict(y=y[-LAST:], dx=dx[-LAST:], dw_gate=dwg, dw_up=dwu, dw_down=dwd), want)
    assert not bool(y[:-LAST].any()) and not bool(dx[:-LAST].any())
    got = mec.gated_ffn(big, *w)
    ref.check(dict(y=got[-LAST:]), {"y": want["y"]})


@pytest.mark.parametrize("C,per", [(1000, 1), (1000, 700_000), (8200, 64)])
def test_norm_beyond_32_bit_offsets(C, per):
    """Of zero rows but for the last, which alone then make the sums."""
    R = (1 << 31) // C + 5000
    x, y, dr, dn, p = make_norm(R % per + 2 * per if per < 1000 else LAST, C, "bf16", "rms", "layer", per=per, eps=1e-3)
    rows = x.shape[0]
    if per >= 1000:  # the last rows are of one group
        p["gate"] = p["gate"][:1]
    d = lambda t: t.double()  # noqa: E731
    want = ref.residual_norm_all(d(x), d(y), moved(p, d), torch.bfloat16, d(dr), d(dn), backward=True)
    p["b_post"] = None
    big = []
    for t in (x, y, dr, dn):
        big.append(torch.zeros(R, C, dtype=torch.bfloat16, device="cuda"))
        big[-1][-rows:] = t.cuda()
    pc = moved(p, lambda t: t.cuda())
    groups, own = -(-R // per), p["gate"].shape[0]
    gate = torch.ones(groups, C, dtype=torch.bfloat16, device="cuda")
    gate[-own:] = pc["gate"]
    pc["gate"] = gate
    r, n = mec.residual_norm(big[0], big[1], **pc)
    g = mec.residual_norm_backward(big[2], big[3], big[0], big[1], **pc)
    got = dict(r=r[-rows:], n=n[-rows:], dx=g["dx"][-rows:], dy=g["dy"][-rows:], dgate=g["dgate"][-own:])
    got.update({k: g[k] for k in want if k not in got})
    ref.check(got, want)
    assert not bool(r[:-rows].any()) and not bool(g["dx"][:-rows].any())
