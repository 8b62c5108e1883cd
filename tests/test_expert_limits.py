"""The largest calls of the experts' feed-forward that the header allows, answered on the host."""
import ctypes

import pytest

import memory_efficient_cnn_gb300 as mec
from memory_efficient_cnn_gb300 import build as mbuild
from memory_efficient_cnn_gb300._binding import ERR_UNSUPPORTED, OK

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
