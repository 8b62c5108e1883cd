"""Gated feed-forward against the 64-bit reference: every type and activation,
sizes from one row and one channel to many, odd and ragged ones, and what the
call's contract says about empty batches, optional gradients and repeatability."""
import pytest
import torch

import block_ref as ref
import memory_efficient_cnn_gb300 as mec

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")


def make(R, C, F, dt, seed=0, x_scale=1.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(DT[dt])  # noqa: E731
    return (n(R, C, std=x_scale), n(F, C, std=C ** -0.5), n(F, C, std=C ** -0.5), n(C, F, std=F ** -0.5),
            n(R, C, std=0.5))


def run_train(x, wg, wu, wd, dy, act):
    dev = [t.cuda() for t in (x, wg, wu, wd)]
    y, saved = mec.gated_ffn_train(*dev, act=act)
    dx, dwg, dwu, dwd = mec.gated_ffn_backward(dy.cuda(), *dev, saved, act=act)
    torch.cuda.synchronize()
    return dict(y=y, dx=dx, dw_gate=dwg, dw_up=dwu, dw_down=dwd)


def check(R, C, F, dt, act, seed=0):
    x, wg, wu, wd, dy = make(R, C, F, dt, seed)
    d = [t.double() for t in (x, wg, wu, wd)]
    want = ref.ffn_all(*d, act, DT[dt], dy.double())
    ref.check(run_train(x, wg, wu, wd, dy, act), want, f"{dt} {act} {(R, C, F)}")
    y = mec.gated_ffn(x.cuda(), wg.cuda(), wu.cuda(), wd.cuda(), act=act)
    ref.check(dict(y=y), {"y": want["y"]}, f"inference {dt} {act} {(R, C, F)}")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("act", ACTS)
def test_activations(dt, act):
    check(70, 48, 136, dt, act)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("R,C,F", [
    (1, 1, 1), (1, 64, 128), (1, 512, 1000), (2, 7, 9), (3, 250, 130), (5, 1024, 520), (8, 64, 64), (9, 72, 200),
    (16, 128, 256), (17, 130, 129), (33, 256, 96), (64, 64, 512), (65, 8, 8), (100, 320, 264), (127, 257, 255),
    (128, 128, 128), (129, 136, 120), (255, 512, 64), (256, 64, 256), (257, 264, 136), (500, 1000, 30),
    (1000, 96, 384), (1100, 40, 72)])
def test_sizes(dt, R, C, F):
    check(R, C, F, dt, "silu", seed=R + C + F)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("R,C,F", [(4, 2048, 4096), (2048, 512, 1024), (3000, 1000, 250), (20000, 64, 128),
                                   (40, 4096, 520), (600, 776, 2056)])
def test_large(dt, R, C, F):
    """Long sums, several tiles each way, and splits of long sums over few tiles."""
    check(R, C, F, dt, "gelu", seed=7)


@pytest.mark.parametrize("R,C,F", [(33, 520, 1000), (40, 1000, 700), (72, 1024, 520), (100, 600, 512), (32, 1100, 700),
                                   (128, 360, 363)])
def test_f32_rows_of_less_than_a_tile(R, C, F):
    """Both sides of where the fp32 kernels of few rows end."""
    check(R, C, F, "f32", "silu", seed=R)


def test_leading_axes_and_out():
    x, wg, wu, wd, _ = (t.cuda() for t in make(2 * 3 * 5, 64, 128, "bf16"))
    want = mec.gated_ffn(x, wg, wu, wd)
    out = torch.full((2, 3, 5, 64), float("nan"), dtype=x.dtype, device="cuda")
    got = mec.gated_ffn(x.view(2, 3, 5, 64), wg, wu, wd, out=out)
    assert got is out and torch.equal(got.view(-1, 64), want)


@pytest.mark.parametrize("R,C,F", [(1, 512, 1024), (40, 320, 264), (700, 128, 250), (5000, 64, 128)])
def test_same_bits_every_time(R, C, F):
    for dt in DT:
        args = make(R, C, F, dt)
        a, b = run_train(*args, "silu"), run_train(*args, "silu")
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_gradients_asked_for_alone():
    x, wg, wu, wd, dy = (t.cuda() for t in make(50, 72, 40, "f16"))
    _, saved = mec.gated_ffn_train(x, wg, wu, wd)
    full = mec.gated_ffn_backward(dy, x, wg, wu, wd, saved)
    only_dx = mec.gated_ffn_backward(dy, x, wg, wu, wd, saved, need_dw=False)
    only_dw = mec.gated_ffn_backward(dy, x, wg, wu, wd, saved, need_dx=False)
    assert torch.equal(only_dx[0], full[0]) and only_dx[1:] == (None, None, None)
    assert only_dw[0] is None and all(torch.equal(a, b) for a, b in zip(only_dw[1:], full[1:]))


@pytest.mark.parametrize("dt", DT)
def test_no_rows(dt):
    _, wg, wu, wd, _ = (t.cuda() for t in make(1, 24, 40, dt))
    x = torch.empty(0, 24, dtype=DT[dt], device="cuda")
    y, saved = mec.gated_ffn_train(x, wg, wu, wd)
    assert y.shape == (0, 24)
    dx, *dws = mec.gated_ffn_backward(x, x, wg, wu, wd, saved)
    assert dx.shape == (0, 24) and all(bool((w == 0).all()) for w in dws)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("R", [1, 5, 40, 300])
def test_rows_do_not_mix(dt, R):
    """An infinite or NaN row spoils its own outputs only."""
    x, wg, wu, wd, _ = make(R + 2, 64, 96, dt)
    clean = mec.gated_ffn(x.cuda(), wg.cuda(), wu.cuda(), wd.cuda())
    bad = x.clone()
    bad[0, 3], bad[R + 1, 5] = float("nan"), float("inf")
    got = mec.gated_ffn(bad.cuda(), wg.cuda(), wu.cuda(), wd.cuda())
    assert torch.equal(got[1:R + 1], clean[1:R + 1])
    assert bool(got[0].isnan().all())


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("R,C,F", [(3, 40, 56), (200, 72, 130)])
def test_guard_bytes_stay(dt, R, C, F):
    """Outputs, `saved` and the workspace are written inside their bounds only."""
    code = mec._binding._DTYPE[DT[dt]]
    x, wg, wu, wd, dy = (t.cuda() for t in make(R, C, F, dt))

    def guarded(nbytes):
        n = (nbytes + 15) // 16 * 16
        return torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda"), nbytes

    def view(buf, like):
        return buf[0][256:256 + buf[1]].view(like.dtype).view(like.shape)

    like = dict(y=x, dx=x, dwg=wg, dwu=wu, dwd=wd)
    bufs = {k: guarded(v.numel() * v.element_size()) for k, v in like.items()}
    raw = {k: guarded(mec.im2win_gated_ffn_size(b, R, C, F, code))
           for k, b in (("saved", mec.FFN_SAVED), ("train", mec.FFN_TRAIN), ("back", mec.FFN_BACKWARD))}
    part = {k: b[0][256:256 + b[1]] for k, b in raw.items()}
    mec.im2win_gated_ffn(x, wg, wu, wd, view(bufs["y"], x), part["saved"], part["train"])
    mec.im2win_gated_ffn_backward(dy, x, wg, wu, wd, part["saved"], view(bufs["dx"], x), view(bufs["dwg"], wg),
                                  view(bufs["dwu"], wu), view(bufs["dwd"], wd), part["back"])
    torch.cuda.synchronize()
    for name, (buf, n) in {**bufs, **raw}.items():
        assert bool((buf[:256] == 0xA5).all()) and bool((buf[256 + n:] == 0xA5).all()), name
    assert mec.im2win_device_status(part["back"]) == 0


def test_another_stream():
    """The work is queued on the caller's current stream."""
    x, wg, wu, wd, dy = (t.cuda() for t in make(300, 128, 256, "bf16"))
    want = mec.gated_ffn(x, wg, wu, wd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    late = torch.zeros_like(x)
    with torch.cuda.stream(s):
        late.copy_(x)
        got = mec.gated_ffn(late, wg, wu, wd)
    s.synchronize()
    assert torch.equal(got, want)


def test_in_a_graph():
    x, wg, wu, wd, _ = (t.cuda() for t in make(2, 128, 256, "bf16"))
    ws = torch.empty(mec.im2win_gated_ffn_size(mec.FFN_FORWARD, 2, 128, 256, mec.BF16), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    want = mec.gated_ffn(x, wg, wu, wd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mec.gated_ffn(x, wg, wu, wd, ws=ws, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """The fp32 gradients along a direction against central differences of the
    formula in 64 bits. A difference at step s errs by s^2 / 6 of the third
    derivative (relu: none away from its kink, and a kink crossed errs by at most
    s a crossing); the directional derivative is a sum of N terms, each held to
    about 1e-6 of its size."""
    x, wg, wu, wd, dy = make(20, 24, 40, "f32", seed=3)
    got = run_train(x, wg, wu, wd, dy, act)
    p = [t.double() for t in (x, wg, wu, wd)]
    g = torch.Generator().manual_seed(5)
    v = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in p]
    s = 1e-4
    f = lambda k: (ref.ffn(*[a + k * s * b for a, b in zip(p, v)], act) * dy.double()).sum()  # noqa: E731
    diff = (f(1) - f(-1)) / (2 * s)
    terms = [got[k].double().cpu() * b for k, b in zip(("dx", "dw_gate", "dw_up", "dw_down"), v)]
    dot, size = sum(t.sum() for t in terms), sum(t.abs().sum() for t in terms)
    assert abs(float(dot - diff)) <= 1e-5 * float(size)
