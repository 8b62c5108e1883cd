"""What the group norm's statistics keep of values that stand apart or lie far away, held to bounds that follow the
kernels' sums."""
import pytest
import torch

import block_ref
import memory_efficient_cnn_gb300 as mec
import norm_bounds

pytestmark = pytest.mark.gpu

EPS = 1e-5


def statistics(x, G, what, run=256, roundings=2):
    """y and the statistics of fp32 maps against 64 bits."""
    want = norm_bounds.group_norm(x.double(), G, None, None, "none", EPS, torch.float32, run=run, roundings=roundings)
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


# ---- means far away, in each of the ways: single rows in registers and maps in the shared memory of one CTA (one part),
# maps in that of a cluster, maps that are read twice
ONE_PART = [(900, 1, 64, 4), (300, 1, 1024, 1), (70, 1, 1000, 1), (70, 1, 96, 12), (320, 40, 16, 4), (320, 200, 16, 16)]
FAR = ONE_PART + [(4, 1500, 16, 4), (1, 30000, 16, 2), (3, 30000, 32, 1), (1, 66000, 64, 8)]


@pytest.mark.parametrize("N,P,C,G", FAR)
@pytest.mark.parametrize("mean", [400.0, -4000.0])
def test_far_mean(N, P, C, G, mean):
    """What is left of the mean's error is its rounding."""
    statistics(noise(N, P, C, 7, mean), G, f"{(N, P, C, G)} at {mean}", roundings=1 if (N, P, C, G) in ONE_PART else 2)


@pytest.mark.parametrize("N,P,C,G", FAR)
@pytest.mark.parametrize("first", [300.0, 3000.0])
def test_first_value_apart(N, P, C, G, first):
    x = noise(N, P, C, 8, 3.0)
    x[:, 0, ::C // G] = first
    statistics(x, G, f"{(N, P, C, G)} after {first}")


@pytest.mark.parametrize("N,P,C,G", [(2, 1500, 24, 3), (320, 200, 32, 4), (1, 200000, 24, 3)])
def test_positions_with_means_of_their_own(N, P, C, G):
    """The parts of a cluster or of a map have means far from one another."""
    x = noise(N, P, C, 9) + 100.0 + torch.linspace(-5000.0, 5000.0, P).view(1, P, 1)
    statistics(x, G, f"{(N, P, C, G)}")
