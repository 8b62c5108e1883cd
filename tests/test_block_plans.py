"""Plans of the residual-block operators for shapes that no test would run: answered by
their host code, compiled here into a small library; no GPU is needed."""
import ctypes
import os
import subprocess

import pytest

import memory_efficient_cnn_gb300 as mec
from memory_efficient_cnn_gb300 import build as mbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("plans") / "libblock_plans.so")
    main = mbuild.build()
    subprocess.run([mbuild.nvcc(), *mbuild.ARCH, *mbuild.NVCC_FLAGS, "-shared", "-o", out,
                    os.path.join(HERE, "block_plans.cu"), main, "-Xlinker", "-rpath," + os.path.dirname(main)], check=True)
    return ctypes.CDLL(out)


def test_one_kernel_columns(plans):
    """A product of two CTAs with 256 rows has 32, 64, ... 256 columns."""
    plans.ffn_fused_columns.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int64]
    taken = 0
    for C in range(1, 300):
        n = plans.ffn_fused_columns(100000, C, 256)
        if n:
            taken += 1
            assert n % 32 == 0 and 32 <= n <= 256 and n >= C, C
    assert taken == 113  # 16 to 128 channels


@pytest.mark.parametrize("R,C,F", [(131072, 131072, 131072), (2 ** 31 - 1024, 512, 512), (512, 2 ** 31 - 1024, 512),
                                   (512, 512, 2 ** 31 - 1024), (2 ** 20, 2 ** 20, 2 ** 20), (1, 1, 1)])
def test_every_product_has_a_plan(plans, R, C, F):
    """Whatever im2win_gated_ffn_size accepts can be launched: its products have tiles."""
    streamed = ctypes.c_int()
    for f32 in (0, 1):
        mec.im2win_gated_ffn_size(mec.FFN_BACKWARD, R, C, F, mec.F32 if f32 else mec.BF16)
        for M, N, K, kind, two in ((R, F, C, 1, 0), (R, C, F, 0, 0), (R, F, C, 2, 0), (R, C, F, 0, 1), (F, C, R, 0, 2),
                                   (C, F, R, 0, 0)):
            assert plans.ffn_product_units(f32, M, N, K, kind, two, ctypes.byref(streamed)) > 0, (f32, M, N, K, kind)


def test_norm_backward_reads_once(plans):
    """Rows of up to 8192 elements stay in registers whatever a gate's extent; short groups are taken whole."""
    plans.norm_back_blocks.argtypes = [ctypes.c_int64] * 3 + [ctypes.POINTER(ctypes.c_int)]
    short = ctypes.c_int()
    for R in (1, 16, 600, 4096, 100000):
        for C in (1, 64, 4096, 4097, 5000, 6000, 8191, 8192):
            for per in (1, 2, 8, 64, 1000, R):
                assert plans.norm_back_blocks(R, C, min(per, R), ctypes.byref(short)) > 0, (R, C, per)
                if per == 1 and R > 1:
                    assert short.value, (R, C)
