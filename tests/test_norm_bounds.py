"""The bounds that the group norm's gradients are held to show what they are for: sums that leave out a chunk of positions, a
row of partial sums or an image are out of them. On the host, at the inputs' sizes of the GPU tests."""
import pytest
import torch

import norm_bounds

EPS = 1e-5


def sums(dz, hat):
    return {"dw": (dz * hat).sum((0, 1)), "db": dz.sum((0, 1))}


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N,P,C,G", [(1, 100000, 16, 1), (2, 40000, 16, 4), (10, 14000, 33, 3)])
def test_a_part_left_out_is_out_of_bounds(N, P, C, G, dtype):
    g = torch.Generator().manual_seed(5)
    n = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g) * std + mean).to(dtype).double()  # noqa: E731
    x, dy, w, b = n(N, P, C, std=1.5, mean=0.7), n(N, P, C, std=0.5), n(C, std=0.2, mean=1.0), n(C, std=0.3)
    want = norm_bounds.group_norm(x, G, w, b, "none", EPS, dtype, dy, run=128, run_params=256)
    hat = (want["y"][0] - b) / w
    full = sums(dy, hat)
    for name, v in full.items():
        assert ((v - want[name][0]).abs() <= 1e-9 * P).all()
    # a chunk of 128 positions, the last 1000, every 64th (a row of a block): gone from an image
    for gone in (slice(0, 128), slice(P - 1000, P), slice(0, P, 64)):
        part = dy.clone()
        part[-1, gone] = 0
        for name, v in sums(part, hat).items():
            value, bound = want[name]
            out = (v - value).abs() > bound
            assert out.double().mean() > 0.5, (name, gone, float(out.double().mean()))
            assert ((torch.zeros_like(v) - value).abs() > bound).double().mean() > 0.8  # nor do zeros pass
