"""The gated feed-forward of few channels, whose inference runs as one kernel: sizes
at the edges of its tiles (256 rows, 64 hidden channels, 16 to 128 channels), several
tiles a pair of SMs, and what is not finite, against the 64-bit reference."""
import pytest
import torch

import block_ref as ref
import memory_efficient_cnn_gb300 as mec
from test_gpu_gated_ffn import ACTS, DT, make

pytestmark = pytest.mark.gpu


def without_h(R, C, F, dt):
    """Whether the call's workspace has no room for h beside copies of x and the weights."""
    copies = 2 * (R + 2 * F) * (C + 8) * (C % 8 != 0) + 2 * C * (F + 8) * (F % 8 != 0)
    return mec.im2win_gated_ffn_size(mec.FFN_FORWARD, R, C, F, {"f16": 1, "bf16": 2}[dt]) < copies + R * F


def check(R, C, F, dt, act, seed=0):
    x, wg, wu, wd, _ = make(R, C, F, dt, seed)
    want = ref.ffn_all(*(t.double() for t in (x, wg, wu, wd)), act, DT[dt])["y"]
    y = mec.gated_ffn(x.cuda(), wg.cuda(), wu.cuda(), wd.cuda(), act=act)
    ref.check(dict(y=y), {"y": want}, f"{dt} {act} {(R, C, F)}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("R,C,F", [(256, 16, 64), (257, 24, 65), (511, 32, 127), (512, 40, 128), (513, 64, 192), (700, 72, 200),
                                   (1000, 128, 512), (1023, 136, 130), (2000, 17, 300), (1300, 127, 70), (3000, 112, 333),
                                   (900, 121, 129), (1500, 128, 640)])
def test_sizes(dt, R, C, F):
    check(R, C, F, dt, "gelu", seed=R + C + F)


@pytest.mark.parametrize("act", ACTS)
def test_activations(act):
    check(800, 96, 320, "bf16", act)


@pytest.mark.parametrize("R,C,F", [(45000, 32, 64), (45001, 64, 128), (40000, 128, 200), (39001, 122, 100), (60000, 120, 64),
                                   (50001, 99, 191)])
def test_several_tiles(R, C, F):
    assert without_h(R, C, F, "f16")
    check(R, C, F, "f16", "silu", seed=3)


def test_same_bits_every_time_and_on_another_stream():
    args = [t.cuda() for t in make(50000, 128, 256, "bf16")[:4]]
    assert without_h(50000, 128, 256, "bf16")
    want = mec.gated_ffn(*args, act="gelu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mec.gated_ffn(*args, act="gelu")
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_a_row_that_is_not_finite_stays_alone():
    x, wg, wu, wd, _ = (t.cuda() for t in make(600, 64, 128, "bf16"))
    clean = mec.gated_ffn(x, wg, wu, wd)
    for value in (float("inf"), float("nan")):
        bad = x.clone()
        bad[300, 5] = value
        y = mec.gated_ffn(bad, wg, wu, wd)
        keep = torch.arange(600, device="cuda") != 300
        assert torch.equal(y[keep], clean[keep]) and not torch.isfinite(y[300]).all()
