"""Choices that the caller drops after the routing, because their expert is full: the gradient of the logits through the
experts that are left, against automatic differentiation in 64 bits."""
import pytest
import torch

import expert_ref as ref
import memory_efficient_cnn_gb300 as mec

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("over", mec.ROUTES)
@pytest.mark.parametrize("T,k,E,C,F", [(40, 2, 4, 16, 24), (130, 3, 6, 40, 32)])
def test_dropped_after_routing(over, T, k, E, C, F):
    g = torch.Generator().manual_seed(T)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std  # noqa: E731
    logits, x, dy = n(T, E), n(T, C), n(T, C, std=0.5)
    ws = [n(E, F, C, std=C ** -0.5), n(E, F, C, std=C ** -0.5), n(E, C, F, std=F ** -0.5)]
    weights, experts = mec.expert_route(logits.cuda(), k, over=over)
    left = experts.clone()
    left[::3, 0] = -1  # the largest weight
    left[1::4, k - 1] = -1
    wd = [w.cuda() for w in ws]
    y, saved = mec.expert_ffn_train(x.cuda(), left, weights, *wd)
    _, dweights, *_ = mec.expert_ffn_backward(dy.cuda(), weights, *wd, saved)
    assert not dweights[left < 0].any()
    got = mec.expert_route_backward(dweights, logits.cuda(), experts, over=over)

    l = logits.double().requires_grad_()
    at = experts.cpu().long()
    p = torch.softmax(l.gather(-1, at), -1) if over == "top" else torch.softmax(l, -1).gather(-1, at)
    out = ref.expert_ffn(x.double(), left.cpu().long(), p, *[w.double() for w in ws], "silu")
    (out * dy.double()).sum().backward()
    # fp32 products of up to 40 terms, their sums over k places and the softmax: 1e-5 of the largest gradient is 160 roundings
    assert float((got.double().cpu() - l.grad).abs().max()) <= 1e-5 * float(l.grad.abs().max())
    # the shortened list is another softmax over "top"
    other = mec.expert_route_backward(dweights, logits.cuda(), left, over=over)
    assert torch.equal(other, got) == (over == "all")
