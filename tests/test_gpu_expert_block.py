"""The operators together, as examples/expert_block.py uses them: gradients of the whole block
against automatic differentiation of its formulas in 64 bits at the experts that were chosen,
inference beside training, a captured step, and a second stream."""
import importlib.util
import os

import pytest
import torch

import expert_ref as ref
import memory_efficient_cnn_gb300 as mec

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("expert_block_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(data, params, maps, experts, groups=8):
    """Loss and gradients in 64 bits from the convolution's output, at the given experts."""
    p = {k: v.double().requires_grad_() for k, v in params.items()}
    x = maps.double().reshape(maps.shape[0], -1, groups, maps.shape[-1] // groups)
    dev = x - x.mean((1, 3), keepdim=True)
    n = (dev / torch.sqrt((dev * dev).mean((1, 3), keepdim=True) + 1e-5)).reshape(-1, maps.shape[-1])
    n = torch.nn.functional.silu(n * p["w_norm"] + p["b_norm"])
    at = experts.long()
    weights = torch.softmax((n @ p["w_router"].t()).gather(-1, at), -1)
    y = ref.expert_ffn(n, at, weights, p["w_gate"], p["w_up"], p["w_down"], "silu")
    loss = ((maps.double().reshape(y.shape) + y - data["target"].double().reshape(y.shape)) ** 2).mean()
    loss.backward()
    return float(loss.detach()), {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 5e-5), (torch.float16, 2e-2), (torch.bfloat16, 1.2e-1)])
def test_gradients_of_the_block(example, dtype, tol):
    """Every 16-bit intermediate (n, the logits, the weights, y, out, d_out, the rows' and logits' gradients and
    the feed-forward's own four) is rounded once, about a dozen roundings of 2^-11 or 2^-8 that add up at
    random over a sum; the router's gradient is a difference of the choices' shares and keeps a third
    of their size. Forty (fp16) and thirty (bf16) times one rounding bound the error in the 2-norm; fp32 has
    the products' 2^-20 and the same factor."""
    data, params = example.make(dtype=dtype)
    loss, grads, experts = example.loss_and_gradients(data, params)
    assert (experts >= 0).all() and experts.unique().numel() > 1
    want_loss, want = reference(data, params, example.convolved(data), experts)
    assert abs(float(loss) - want_loss) <= tol * want_loss
    for k, g in grads.items():
        assert g.dtype == dtype and g.shape == params[k].shape
        err = (g.double() - want[k]).norm() / want[k].norm()
        assert float(err) <= tol, (k, float(err))


def test_the_example_trains(example):
    data, params = example.make(dtype=torch.bfloat16)
    before = {k: v.clone() for k, v in params.items()}
    seen = example.train(data, params, steps=3)
    assert len(seen) == 3 and all(a > 0 and b > 0 for a, b in seen)
    assert all(not torch.equal(before[k], params[k]) for k in params)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_inference_beside_training(example, dtype):
    """The same kernels but for the activation's value, which training takes from its pair with the slope: one
    fp32 rounding apart, so one of h's."""
    data, params = example.make(dtype=dtype)
    maps = example.convolved(data)
    n, _ = mec.group_norm_train(maps, 8, params["w_norm"], params["b_norm"], act="silu")
    rows = n.flatten(0, -2)
    weights, experts = mec.expert_route(rows @ params["w_router"].t(), 2)
    y, _ = mec.expert_ffn_train(rows, experts, weights, params["w_gate"], params["w_up"], params["w_down"])
    out = mec.residual_norm(maps, y.view_as(maps), pre="none")[0].float()
    got = example.infer(data, params).float()
    assert float((got - out).abs().max()) <= 4 * torch.finfo(dtype).eps * float(out.abs().max())


def test_a_captured_step(example):
    """A whole step in a graph, replayed on other images, beside one on a second stream."""
    data, params = example.make(dtype=torch.bfloat16)
    other, _ = example.make(dtype=torch.bfloat16, seed=5)
    want_loss, want, _ = example.loss_and_gradients(other, params)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        example.loss_and_gradients(data, params)  # torch's own products set themselves up outside of a capture
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        loss, grads, _ = example.loss_and_gradients(data, params)
    for k in ("images", "target", "filter"):
        data[k].copy_(other[k])
    graph.replay()
    with torch.cuda.stream(side):
        again_loss, again, _ = example.loss_and_gradients(other, params)
    torch.cuda.synchronize()
    assert torch.equal(loss, want_loss) and torch.equal(again_loss, want_loss)
    for k in want:
        assert torch.equal(grads[k], want[k]) and torch.equal(again[k], want[k]), k
