"""The router against the 64-bit reference: types, one expert to a thousand, every tie,
masked experts, spoiled rows, and what the contract says about its gradient."""
import pytest
import torch

import block_ref
import expert_ref as ref
import memory_efficient_cnn_gb300 as mec

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def check(logits, dweights, k, over, what):
    dt = logits.dtype
    experts, want = ref.route_all(logits.double(), k, over, dt, dweights.double())
    l, d = logits.cuda(), dweights.cuda()
    weights, got = mec.expert_route(l, k, over=over)
    assert got.dtype == torch.int32 and torch.equal(got.cpu().long(), experts), what
    dl = mec.expert_route_backward(d, l, got, over=over)
    block_ref.check(dict(weights=weights, dlogits=dl), want, what)


def make(T, E, k, dt, seed=0, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * std).to(DT[dt]), torch.randn(T, k, generator=g).to(DT[dt])


@pytest.mark.parametrize("over", mec.ROUTES)
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 2, 2), (100, 7, 3), (257, 8, 8), (33, 9, 1), (64, 16, 4),
                                   (50, 24, 5), (1000, 31, 31), (129, 32, 2), (77, 33, 6), (500, 64, 4), (10, 65, 32),
                                   (60, 128, 8), (31, 200, 7), (40, 256, 32), (9, 257, 3), (21, 1000, 32), (5, 1024, 32)])
def test_sizes(over, dt, T, E, k):
    check(*make(T, E, k, dt, T + E), k, over, f"{over} {dt} {(T, E, k)}")


@pytest.mark.parametrize("over", mec.ROUTES)
@pytest.mark.parametrize("E", [8, 24, 64, 300])
def test_ties_go_to_the_lower_index(over, E):
    g = torch.Generator().manual_seed(E)
    k = 6
    logits = torch.randint(-1, 2, (200, E), generator=g).float()
    logits[::3] = 0.0
    logits[::5, ::2] = -0.0  # (equal to 0)
    check(logits, torch.randn(200, k, generator=g), k, over, f"ties {E}")


@pytest.mark.parametrize("over", mec.ROUTES)
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("E", [5, 40, 256])
def test_masked_experts(over, dt, E):
    """Experts at -inf are never taken; a row may have fewer than k, or none; the type's lowest value is a number."""
    logits, dw = make(60, E, 4, dt, 7)
    low = torch.finfo(DT[dt]).min
    logits[0] = float("-inf")
    logits[1, 1:] = float("-inf")
    logits[2, 3:] = float("-inf")
    logits[3] = low
    logits[4, 2:] = low
    logits[5:30, ::2] = float("-inf")
    check(logits, dw, 4, over, f"masked {dt} {E}")
    weights, experts = mec.expert_route(logits.cuda(), 4, over=over)
    assert (experts[0] == -1).all() and not weights[0].any()
    assert experts[1].tolist() == [0, -1, -1, -1] and weights[1].tolist() == [1.0, 0.0, 0.0, 0.0]
    assert experts[3].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("E", [8, 100])
def test_spoiled_rows(E):
    logits, dw = make(6, E, 3, "f32", 2)
    logits[1, 5] = float("nan")
    logits[3, 2] = float("inf")
    weights, experts = mec.expert_route(logits.cuda(), 3)
    dl = mec.expert_route_backward(dw.cuda(), logits.cuda(), experts)
    assert experts[1, 0] == 5 and experts[3, 0] == 2
    assert weights[1].isnan().all() and weights[3, 0].isnan()
    clean = [0, 2, 4, 5]
    w, e = mec.expert_route(logits[clean].cuda(), 3)
    assert torch.equal(w, weights[clean]) and torch.equal(e, experts[clean])
    assert torch.equal(dl[clean], mec.expert_route_backward(dw[clean].cuda(), logits[clean].cuda(), e))


@pytest.mark.parametrize("over", mec.ROUTES)
def test_gradient_at_given_experts(over):
    """Places outside of the experts take no part, and an expert may be given twice."""
    logits, dw = make(4, 12, 3, "f32", 9)
    experts = torch.tensor([[3, -1, 7], [12, 4, 4], [-1, -1, -1], [2147483647, -2147483648, 0]], dtype=torch.int32)
    _, want = ref.route_all(logits.double(), 3, over, torch.float32, dw.double(), experts.long())
    dl = mec.expert_route_backward(dw.cuda(), logits.cuda(), experts.cuda(), over=over)
    block_ref.check(dict(dlogits=dl), {"dlogits": want["dlogits"]})
    assert not dl[2].any()


@pytest.mark.parametrize("over", mec.ROUTES)
def test_gradient_by_differences(over):
    logits, dw = (t.double() for t in make(3, 6, 2, "f32", 4))
    w, experts = mec.expert_route(logits.float().cuda(), 2, over=over)
    got = mec.expert_route_backward(dw.float().cuda(), logits.float().cuda(), experts, over=over)

    def value(l):
        return (ref.route_all(l, 2, over, torch.float32, None, experts.cpu().long())[1]["weights"][0] * dw).sum()

    h = 1e-5
    for at in range(logits.numel()):
        up, down = logits.clone(), logits.clone()
        up.view(-1)[at] += h
        down.view(-1)[at] -= h
        slope = float((value(up) - value(down)) / (2 * h))
        assert abs(float(got.view(-1)[at]) - slope) < 1e-5


def test_shapes_and_empty():
    logits, dw = make(30, 16, 2, "bf16")
    w, e = mec.expert_route(logits.cuda(), 2)
    w3, e3 = mec.expert_route(logits.cuda().view(2, 15, 16), 2)
    assert w3.shape == (2, 15, 2) and torch.equal(w3.view(30, 2), w) and torch.equal(e3.view(30, 2), e)
    w, e = mec.expert_route(torch.empty(0, 16, device="cuda"), 2)
    assert w.shape == e.shape == (0, 2)
    assert mec.expert_route_backward(w, torch.empty(0, 16, device="cuda"), e).shape == (0, 16)
