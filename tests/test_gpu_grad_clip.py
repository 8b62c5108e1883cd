"""Gradient clipping against 64 bits: sizes from none to several chunks, mixed
types, views at any element, in place and out of place, non-finite gradients.

The norm errs by the fp32 sums of at most 8192 squares (over 256 threads: 32
terms each, 32 * 2^-24 at worst) and its own rounding; an output by the factor's
two roundings, the product's and the output's."""
import math

import pytest
import torch

import memory_efficient_cnn_gb300 as mec

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
NORM_TOL = 20 * 2.0 ** -24


def make(sizes, dts, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale * (0.1 + i % 3)).to(DT[d])
            for i, (n, d) in enumerate(zip(sizes, dts))]


def true_norm(grads):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in grads))


def check(grads, outs, norm, max_norm, eps=1e-6):
    want = true_norm(grads)
    assert abs(float(norm) - want) <= NORM_TOL * want
    f = min(1.0, max_norm / (want + eps))
    for t, o in zip(grads, outs):
        v = t.double() * f
        assert o.dtype == t.dtype and o.shape == t.shape
        e = v.abs() * (U[t.dtype] + NORM_TOL + 4 * 2.0 ** -24) + TINY[t.dtype]
        assert bool(((o.double().cpu() - v).abs() <= e).all())


SIZES = [[1], [7], [8192], [8193, 1, 0, 255], [100000, 3, 64, 8191], [1 << 20, 77], [0], [0, 5], [16] * 64, [33] * 65,
         [9] * 1000, [4096] * 2500]


@pytest.mark.parametrize("max_norm", [0.5, 1e6, 0.0])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_lists(sizes, max_norm):
    names = list(DT)
    grads = make(sizes, [names[i % 3] for i in range(len(sizes))])
    dev = [t.cuda() for t in grads]
    outs = [torch.full_like(t, float("nan")) for t in dev]
    norm = mec.clip_grad_norm(dev, max_norm, outs=outs)
    check(grads, outs, norm, max_norm)
    assert all(torch.equal(a, b.cuda()) for a, b in zip(dev, grads))
    assert torch.equal(mec.grad_norm(dev), norm)
    assert torch.equal(mec.clip_grad_norm(dev, max_norm), norm)  # in place
    assert all(torch.equal(a, b) for a, b in zip(dev, outs))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("off,n", [(1, 20000), (3, 9), (2, 8192), (5, 8200), (7, 40001)])
def test_views_of_a_flat_buffer(dt, off, n):
    """Pointers at any element; neighbours of the outputs stay as they were."""
    base = make([n + 32], [dt])[0]
    dev, out = base.cuda(), torch.full((n + 64,), 7.0, dtype=DT[dt], device="cuda")
    for shift in (off, 4):
        out.fill_(7.0)
        norm = mec.clip_grad_norm([dev[off:off + n]], 0.25, outs=[out[shift:shift + n]])
        check([base[off:off + n]], [out[shift:shift + n]], norm, 0.25)
        assert bool((out[:shift] == 7).all()) and bool((out[shift + n:] == 7).all())


def test_zero_and_nonfinite():
    z = [torch.zeros(100, device="cuda"), torch.zeros(3, device="cuda")]
    assert float(mec.clip_grad_norm(z, 1.0)) == 0.0 and not any(bool(t.any()) for t in z)
    g = [torch.ones(9000, device="cuda"), torch.ones(5, device="cuda", dtype=torch.bfloat16)]
    g[1][2] = float("nan")
    outs = [torch.empty_like(t) for t in g]
    assert math.isnan(float(mec.clip_grad_norm(g, 1.0, outs=outs))) and all(bool(t.isnan().all()) for t in outs)
    g[1][2] = float("inf")
    assert math.isinf(float(mec.clip_grad_norm(g, 1.0, outs=outs)))
    assert not bool(outs[0].any()) and bool(outs[1][2].isnan()) and float(outs[1][1]) == 0.0


def test_half_precision_squares_do_not_overflow():
    g = [torch.full((5000,), 6e4, dtype=torch.float16, device="cuda")]
    norm = mec.clip_grad_norm(g, 1.0)
    want = float(torch.tensor(6e4, dtype=torch.float16)) * math.sqrt(5000)
    assert abs(float(norm) - want) <= NORM_TOL * want


def test_same_bits_every_time():
    dev = [t.cuda() for t in make([300001, 17, 90000], ["bf16", "f32", "f16"])]
    a, b = mec.grad_norm(dev), mec.grad_norm(dev)
    assert torch.equal(a, b)


def test_beyond_32_bit_offsets():
    """One tensor of more than 2^32 bytes and elements past 2^31."""
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-1], g[0], g[1 << 31] = 3.0, 4.0, 12.0
    norm = mec.clip_grad_norm([g], 1.3)
    assert abs(float(norm) - 13.0) <= NORM_TOL * 13
    want = torch.tensor([0.4, 0.3, 1.2], dtype=torch.float64)
    got = torch.stack([g[0], g[-1], g[1 << 31]]).double().cpu()
    assert bool(((got - want).abs() <= want * 2.0 ** -7).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [5, 8192, 70001])
@pytest.mark.parametrize("power", [-140, -100, -74, -55, 60, 66, 110])
def test_squares_outside_of_fp32(dt, n, power):
    """Gradients whose squares pass fp32's range below or above, alone and beside ordinary ones;
    the norm itself is within the range."""
    g = (make([n], ["f32"])[0] * 2.0 ** 10).double().mul(2.0 ** power / 2 ** 10).to(DT[dt])
    for grads in ([g], [g, torch.full((9,), 3.0, dtype=DT[dt])]):
        dev = [t.cuda() for t in grads]
        norm = mec.grad_norm(dev)
        want = true_norm(grads)
        assert abs(float(norm) - want) <= NORM_TOL * want + 2.0 ** -149, (float(norm), want)
        if want == 0:  # (bf16 ends at 2^-133)
            continue
        outs = [torch.empty_like(t) for t in dev]
        limit = 0.25 * want
        assert torch.equal(mec.clip_grad_norm(dev, limit, outs=outs, eps=0.0), norm)
        factor = limit / want
        for t, o in zip(grads, outs):
            v = t.double() * factor
            # a norm or a limit below fp32's normal numbers is a multiple of 2^-149
            e = v.abs() * (U[t.dtype] + NORM_TOL + 4 * 2.0 ** -24 + 2.0 ** -147 / want) + TINY[t.dtype]
            assert bool(((o.double().cpu() - v).abs() <= e).all())


def test_infinities_among_squares_outside_of_fp32():
    for big in (1e30, 1e-30):
        g = torch.full((9000,), big, device="cuda")
        for bad in (float("inf"), float("-inf"), float("nan")):
            g[17] = bad
            norm = float(mec.grad_norm([g]))
            assert norm != norm if bad != bad else norm == float("inf")
