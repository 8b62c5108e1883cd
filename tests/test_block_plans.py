"""Plans of the residual-block operators for shapes that no test would run: answered by
their host code, compiled here into a small library; no GPU is needed."""
import ctypes
import os
import subprocess

import pytest

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
