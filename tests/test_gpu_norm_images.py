"""Group norms of very many images of few positions: gradients of the parameters, whose sums go over every image."""
import pytest
import torch

import block_ref
import memory_efficient_cnn_gb300 as mec
import norm_bounds

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("N,P,C,G", [(2049, 2, 24, 3), (20000, 2, 32, 4), (30001, 3, 6, 2), (9000, 16, 40, 5), (4099, 4, 257, 1),
                                     (70000, 4, 64, 8), (50000, 5, 33, 11)])
def test_many_images(N, P, C, G, dt):
    """Images on the chip (up to 16 MB of maps) and read twice; more than 2048 rows of partial sums, which no chain of
    additions takes more of than an eighth of their root and eight, twice (and 16 positions): 100 for 70000 images."""
    g = torch.Generator().manual_seed(N + C)
    n = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g) * std + mean).to(DT[dt])  # noqa: E731
    x, dy, w, b = n(N, P, C, mean=0.7), n(N, P, C, std=0.5), n(C, std=0.2, mean=1.0), n(C, std=0.3)
    want = norm_bounds.group_norm(x.double(), G, w.double(), b.double(), "relu", EPS, DT[dt], dy.double(), run=64, run_params=128)
    want.pop("stats")
    xd, dyd, wd, bd = x.cuda(), dy.cuda(), w.cuda(), b.cuda()
    y, stats = mec.group_norm_train(xd, G, wd, bd, act="relu", eps=EPS)
    dx, dw, db = mec.group_norm_backward(dyd, xd, stats, wd, bd, act="relu")
    block_ref.check(dict(y=y, dx=dx, dw=dw, db=db), want, f"{dt} {(N, P, C, G)}")
    only = mec.group_norm_backward(dyd, xd, stats, wd, bd, act="relu", need_dx=False)
    assert only[0] is None and torch.equal(only[1], dw) and torch.equal(only[2], db)
    again = mec.group_norm_backward(dyd, xd, stats, wd, bd, act="relu")
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and torch.equal(again[2], db)
    assert torch.equal(mec.group_norm_backward(dyd, xd, stats, wd, bd, act="relu", need_dw=False)[0], dx)


@pytest.mark.parametrize("N,P", [(400000, 2), (1000000, 2)])
def test_equal_gradients_do_not_drift(N, P):
    """A sum of equal terms, where every rounding may go the same way. A million images are 1000 runs of 1000 rows: 124
    additions of a thread and 7 of its block, twice, and one of the two positions, each off by half a step at most; and
    the output's rounding."""
    x = torch.randn(N, P, 8, generator=torch.Generator().manual_seed(1)).cuda()
    one, dy = torch.ones(8, device="cuda"), torch.full((N, P, 8), 0.1, device="cuda")
    _, stats = mec.group_norm_train(x, 2, one, one, eps=EPS)
    dx, dw, db = mec.group_norm_backward(dy, x, stats, one, one)
    want = float(dy[0, 0, 0]) * N * P
    assert float((db.double() - want).abs().max()) <= 264 * 2.0 ** -24 * want


def test_captured():
    x = torch.randn(5000, 3, 16, device="cuda", dtype=torch.bfloat16)
    dy, w = torch.randn_like(x), torch.ones(16, device="cuda", dtype=torch.bfloat16)

    def step():
        y, stats = mec.group_norm_train(x, 4, w, w, act="silu")
        return (y, *mec.group_norm_backward(dy, x, stats, w, w, act="silu"))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.mul_(1.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))
