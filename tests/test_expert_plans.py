"""Plans of the group norm and of the experts' products, for shapes that no test would run as well:
answered by their host code, compiled here into a small library; no GPU is needed."""
import ctypes
import os
import random
import subprocess

import pytest

import memory_efficient_cnn_gb300 as mec
from memory_efficient_cnn_gb300 import build as mbuild

HERE = os.path.dirname(os.path.abspath(__file__))
i64 = ctypes.c_int64


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("plans") / "libexpert_plans.so")
    main = mbuild.build()
    subprocess.run([mbuild.nvcc(), *mbuild.ARCH, *mbuild.NVCC_FLAGS, "-shared", "-o", out,
                    os.path.join(HERE, "expert_plans.cu"), main, "-Xlinker", "-rpath," + os.path.dirname(main)], check=True)
    lib = ctypes.CDLL(out)
    lib.group_product_units.argtypes = [ctypes.c_int] * 6 + [i64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                                             ctypes.POINTER(i64)]
    lib.expert_grouped_rows.argtypes, lib.expert_grouped_rows.restype = [i64, i64], i64
    lib.group_norm_cut.argtypes = [i64, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(i64)]
    return lib


def products(plans, f32, T, k, E, C, F):
    """{name: (units, streamed, bytes of partial tiles)} of a training step's products."""
    rows, streamed, part = plans.expert_grouped_rows(T * k, E), ctypes.c_int(), i64()
    out = {}
    for name, summed, M, N, K, kind, two in (
            ("gated", 0, rows, F, C, 1, 0), ("down", 0, rows, C, F, 0, 0), ("dgated", 0, rows, F, C, 2, 0), ("dx", 0, rows, C, F, 0, 1),
            ("dw_in", 1, F, C, rows, 0, 2), ("dw_down", 1, C, F, rows, 0, 0)):
        units = plans.group_product_units(f32, summed, M, N, K, E, T * k, kind, two, ctypes.byref(streamed), ctypes.byref(part))
        out[name] = (units, bool(streamed.value), part.value)
    return out


@pytest.mark.parametrize("T,k,E,C,F", [(1, 1, 1, 1, 1), (1, 32, 1024, 8, 8), (1 << 25, 32, 1, 32, 32), (1000, 2, 1024, 1 << 15, 1 << 15),
                                       (1 << 20, 1, 64, 1 << 19, 64), (1 << 20, 1, 64, 64, 1 << 19), (100, 1, 1, 1 << 20, 1 << 20)])
def test_every_product_has_a_plan(plans, T, k, E, C, F):
    """Whatever im2win_expert_ffn_size accepts can be launched, with partial tiles of a bounded size."""
    for f32 in (0, 1):
        for kind in range(4):
            assert mec.im2win_expert_ffn_size(kind, T, k, E, C, F, mec.F32 if f32 else mec.BF16) >= 0
        for name, (units, streamed, part) in products(plans, f32, T, k, E, C, F).items():
            assert 1 <= units <= 152, (name, units)
            assert streamed == (part > 0) and part <= 2 * 76 * 256 * 256 * 4, (name, part)


def test_long_sums_over_few_tiles_are_dealt_out(plans):
    """The shapes of the GPU test of that name reach both kinds of streamed products in both kernels."""
    seen = set()
    for f32, T, k, E, C, F in ((0, 70, 2, 3, 2000, 1607), (0, 9000, 1, 5, 72, 104), (0, 4100, 2, 2, 33, 40), (1, 150, 2, 3, 700, 1101),
                               (1, 4000, 1, 4, 40, 65), (0, 66, 1, 1, 2304, 136)):
        seen |= {(f32, name.startswith("dw")) for name, (_, streamed, _) in products(plans, f32, T, k, E, C, F).items() if streamed}
    assert seen == {(0, False), (0, True), (1, False), (1, True)}
    # many tiles are dealt out whole
    assert not any(streamed for _, streamed, _ in products(plans, 0, 8192, 2, 16, 2048, 4096).values())


def test_grouped_rows_hold_every_split(plans):
    """However the pairs fall on the experts, their padded groups fit the bound."""
    rng = random.Random(1)
    for _ in range(500):
        pairs, E = rng.randint(1, 2000), rng.choice([1, 2, 7, 64, 1024])
        bound = plans.expert_grouped_rows(pairs, E)
        assert bound % 64 == 0
        counts = [0] * E
        for _ in range(pairs):
            counts[rng.randrange(E) if rng.random() < 0.7 else 0] += 1
        assert sum((c + 63) // 64 * 64 for c in counts) <= bound
        one_each = min(pairs, E)
        assert (one_each - 1) * 64 + (pairs - one_each + 1 + 63) // 64 * 64 <= bound


def test_group_norm_cuts(plans):
    """Chunks cover the positions; what stays on the chip fits a CTA, with whole groups and vectors a slab."""
    rng = random.Random(2)
    out = (i64 * 8)()
    kept = 0
    for _ in range(4000):
        D = rng.choice([1, 2, 3, 4, 5, 8, 15, 16, 30, 64, 127, 256, 1000, 4100])
        G = max(1, int(2 ** rng.uniform(0, 11)) // D)
        C, P, N = D * G, int(2 ** rng.uniform(0, 22)), int(2 ** rng.uniform(0, 9))
        size, maps = rng.choice([2, 4]), rng.choice([1, 2])
        plans.group_norm_cut(N, P, C, G, size, maps, out)
        resident, chunks, length, slab, tile, smem, v, slabs = out[:]
        if resident == 2:
            rows, cols, lanes = length, slab, tile
            assert P == 1 and lanes in (1, 2, 4, 8, 16, 32) and 4 * lanes * v >= D and D % v == 0 and 1 <= chunks <= N
            assert cols % lanes == 0 and cols * rows <= 256 and slabs * cols >= G * lanes
            continue
        assert chunks >= 1 and chunks * length >= P and slab % v == 0 and slabs * slab >= C
        if resident:
            kept += 1
            assert chunks in (1, 2, 4, 8) and slab % D == 0 and slab // v <= 256
            rows = 256 // (slab // v)
            assert tile >= maps * size * v * 256 * -(-length // rows) and tile % (32 * maps) == 0
            assert tile < smem <= 227 * 1024 and N * P * C * size * maps <= 16 << 20
        else:
            assert (chunks - 1) * length < P
    assert kept > 400
