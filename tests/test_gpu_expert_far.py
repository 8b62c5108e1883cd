"""Rows and images whose offsets pass 32 bits, in the ways that maps and matrices of that size do not take: the router's rows,
single rows of the group norm, many small images. The last of them against a call with them alone."""
import pytest
import torch

import memory_efficient_cnn_gb300 as mec

pytestmark = pytest.mark.gpu


def normal(*s, seed=1, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(mean, std, generator=g)


@pytest.mark.parametrize("over", mec.ROUTES)
def test_router(over):
    """2.2e9 logits."""
    T, E, k, n = 34_000_000, 64, 2, 5001
    logits, dw = normal(T, E), normal(T, k, seed=2)
    weights, experts = mec.expert_route(logits, k, over=over)
    dl = mec.expert_route_backward(dw, logits, experts, over=over)
    part = logits[-n:].clone()
    w, e = mec.expert_route(part, k, over=over)
    assert torch.equal(weights[-n:], w) and torch.equal(experts[-n:], e)
    assert torch.equal(dl[-n:], mec.expert_route_backward(dw[-n:].clone(), part, e, over=over))


@pytest.mark.parametrize("N,P,C,G", [(1_048_000, 1, 2048, 8), (20_000_000, 2, 64, 4)])
def test_group_norm_of_rows_and_of_images(N, P, C, G):
    """2.15e9 elements (as many as single rows may have: N C is at most 2^31) and 2.6e9; dw and db of four channels in 64 bits too."""
    n = 3001
    x, dy, w, b = normal(N, P, C, std=1.5, mean=0.5), normal(N, P, C, seed=2, std=0.5), normal(C, seed=3, std=0.2, mean=1.0), normal(C, seed=4)
    y, stats = mec.group_norm_train(x, G, w, b, act="relu")
    dx, dw, db = mec.group_norm_backward(dy, x, stats, w, b, act="relu")
    part, dpart = x[-n:].clone(), dy[-n:].clone()
    y2, stats2 = mec.group_norm_train(part, G, w, b, act="relu")
    dx2, _, _ = mec.group_norm_backward(dpart, part, stats2, w, b, act="relu")
    # (another number of images may take another way, in fp32: a step of the output)
    assert torch.allclose(stats[-n:], stats2, rtol=1e-5, atol=1e-5)
    for a, c in ((y, y2), (dx, dx2)):
        a, c = a[-n:].double(), c.double()
        assert ((a - c).abs() <= 2.0 ** -7 * c.abs() + 1e-4).all()
    # the sums: each term is known to 1e-5 of itself from the statistics, and relu's step at 0 counts whole within 1e-4 of it; chains
    # of 912 rows by 8 and 1150 a thread, or of 4473 runs by 8 and 4472 rows by 8, err by 8 sqrt(K) 2^-24 < 2e-5 of the terms
    for c in (0, C // G - 1, C // 2, C - 1):
        s = stats[:, c // (C // G)].double()
        hat = (x[..., c].double() - s[:, :1]) * s[:, 1:]
        z = hat * float(w[c]) + float(b[c])
        d = dy[..., c].double()
        dz = d * (z > 0)
        near = (d.abs() * (z.abs() < 1e-4)).sum()
        for got, t in ((dw[c], dz * hat), (db[c], dz)):
            assert abs(float(got) - float(t.sum())) <= 2.0 ** -8 * abs(float(t.sum())) + 3e-5 * float(t.abs().sum()) + 3 * float(near)
