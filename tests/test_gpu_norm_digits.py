"""What the group norm's statistics keep of values that stand apart or lie far away, held to bounds that follow the
kernels' sums."""
import pytest
import torch

import block_ref
import memory_efficient_cnn_gb300 as mec
import norm_bounds

pytestmark = pytest.mark.gpu

EPS = 1e-5


def statistics(x, G, what, run=256):
    """y and the statistics of fp32 maps against 64 bits."""
    want = norm_bounds.group_norm(x.double(), G, None, None, "none", EPS, torch.float32, run=run)
    y, stats = mec.group_norm_train(x.cuda(), G, eps=EPS)
    block_ref.check(dict(y=y, stats=stats), want, what)


def noise(N, P, C, seed, mean=0.0):
    return torch.randn(N, P, C, generator=torch.Generator().manual_seed(seed)) + mean


# 66000 positions of 64 channels (16.9 MB) are read twice, in 565 chunks of 117 positions
@pytest.mark.parametrize("shift", [10.0, 100.0, -3000.0])
@pytest.mark.parametrize("G", [1, 8])
def test_first_chunk_apart(shift, G):
    """The group's first values are far from all others: its sums must not be made of distances to them."""
    for positions, channels in ((117, 1), (66000, 1), (117, 64), (1, 1)):
        x = noise(1, 66000, 64, 3)
        x[0, :positions, :channels] += shift
        statistics(x, G, f"{positions} x {channels} by {shift} in {G}")


@pytest.mark.parametrize("shift", [100.0, 3000.0])
def test_first_channel_of_a_wide_group_apart(shift):
    """138 chunks of 8 positions: a lane of the statistics takes 1104 of a group's chunks and channels, or a quarter."""
    x = noise(2, 1100, 2048, 4)
    x[:, :, 0] += shift
    statistics(x, 1, f"wide, {shift}", run=1200)
    statistics(x, 4, f"wide in four, {shift}", run=300)
