"""The largest calls of the experts' feed-forward that the header allows, and bounds of the group norm's cut that its kernels
build on; answered on the host."""
import ctypes
import random

import pytest

import memory_efficient_cnn_gb300 as mec
from memory_efficient_cnn_gb300 import build as mbuild
from memory_efficient_cnn_gb300._binding import ERR_UNSUPPORTED, OK
from test_expert_plans import i64, plans  # noqa: F401

MOST = (1 << 31) - 1024


@pytest.mark.parametrize("dtype", [mec.F32, mec.F16, mec.BF16])
@pytest.mark.parametrize("k", [1, 2, 7, 32])
@pytest.mark.parametrize("E", [1, 64, 1024])
def test_most_pairs(dtype, k, E):
    """T k + 64 E goes up to 2^31 - 1024, whatever k is; the grouped rows stay in 32 bits."""
    mbuild.build()
    size, sz = mec.lib().im2win_expert_ffn_size, ctypes.c_size_t()
    T = (MOST - 64 * E) // k
    for kind in range(4):
        assert size(kind, T, k, E, 8, 8, dtype, ctypes.byref(sz)) == OK
        assert sz.value < 1 << 45
        assert size(kind, T + 1, k, E, 8, 8, dtype, ctypes.byref(sz)) == ERR_UNSUPPORTED
    # saved holds a place for each pair, and the rows with their padding
    size(mec.FFN_SAVED, T, k, E, 8, 8, dtype, ctypes.byref(sz))
    assert sz.value >= 4 * T * k + (T * k) * (4 + 8 * 4)


def test_groups_of_a_slab(plans):  # noqa: F811
    """A resident CTA's slab of channels has at most 64 groups, one for each of its first threads, and fewer than 2^24 positions."""
    rng, out, most = random.Random(4), (i64 * 8)(), 0
    for _ in range(6000):
        D = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 15, 16, 30, 33, 64, 127, 256, 1000])
        G = max(1, int(2 ** rng.uniform(0, 13)) // D)
        size, maps, N, P = rng.choice([2, 4]), rng.choice([1, 2]), int(2 ** rng.uniform(0, 12)), int(2 ** rng.uniform(1, 20))
        plans.group_norm_cut(N, P, D * G, G, size, maps, out)
        resident, slab = out[0], out[3]
        if resident == 1:
            most = max(most, slab // D)
            assert slab % D == 0 and slab // D <= 64 and P < 1 << 24
    assert most == 64
