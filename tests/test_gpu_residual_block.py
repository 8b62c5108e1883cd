"""The operators together, as examples/residual_block.py uses them: gradients of the
whole block against automatic differentiation of its formulas in 64 bits, a loss that
falls, and the same output with and without what training keeps."""
import importlib.util
import os

import pytest
import torch

import block_ref as ref
import memory_efficient_cnn_gb300 as mec

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "residual_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("residual_block_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(example, data, params, maps):
    """Loss and gradients in 64 bits from the convolution's output."""
    p = {k: v.double().requires_grad_() for k, v in params.items()}
    rows = maps.double().reshape(-1, maps.shape[-1])
    none = dict(rows_per_gate=None, gate=None, res_scale=None, w_post=None, b_post=None, b_pre=None, eps=1e-6)
    first = dict(none, post="none", pre="layer", w_pre=p["w_first"], b_pre=p["b_first"])
    n = ref.residual_norm(rows, None, first)[1]
    y = ref.ffn(n, p["w_gate"], p["w_up"], p["w_down"], "silu")
    seam = dict(none, post="rms", pre="rms", w_post=p["w_post"], w_pre=p["w_pre"], gate=p["gate"],
                res_scale=p["res_scale"], rows_per_gate=maps.shape[1] * maps.shape[2])
    out = ref.residual_norm(rows, y, seam)[1]
    loss = ((out - data["target"].double().reshape(rows.shape)) ** 2).mean()
    loss.backward()
    return float(loss.detach()), {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 2e-5), (torch.float16, 2e-2), (torch.bfloat16, 8e-2)])
def test_gradients_of_the_block(example, dtype, tol):
    """Through the whole block every 16-bit intermediate (n, y, the output, d_out, d_n, dy)
    is rounded once: about ten roundings of 2^-11 or 2^-8 relative to its rows, which add
    up at random over a sum; twenty times that, or 2e-5 in fp32, bounds the gradient's
    error in the 2-norm with room."""
    data, params = example.make(dtype=dtype)
    loss, grads = example.loss_and_gradients(data, params)
    maps = mec.conv_fused_ex(data["images"], data["filter"], pad=(1, 1), layout=mec.NHWC)
    want_loss, want = reference(example, data, params, maps)
    assert abs(float(loss) - want_loss) <= tol * want_loss
    for k, g in grads.items():
        assert g.dtype == dtype and g.shape == params[k].shape
        err = (g.double() - want[k]).norm() / want[k].norm()
        assert float(err) <= tol, (k, float(err))


def test_training_lowers_the_loss(example):
    data, params = example.make(dtype=torch.bfloat16)
    seen = example.train(data, params, steps=6)
    assert all(b[0] < a[0] for a, b in zip(seen, seen[1:])), seen


def test_inference_equals_training_forward(example):
    data, params = example.make(dtype=torch.float16)
    maps = mec.conv_fused_ex(data["images"], data["filter"], pad=(1, 1), layout=mec.NHWC)
    _, n = mec.residual_norm(maps, **dict(example.FIRST, w_pre=params["w_first"], b_pre=params["b_first"]))
    y, _ = mec.gated_ffn_train(n, params["w_gate"], params["w_up"], params["w_down"])
    out = mec.residual_norm(maps, y, **example.seam_args(params, maps.shape[1] * maps.shape[2]))[1]
    assert out.shape == data["target"].shape
    # (the activation's value may come from its pair with the slope: one fp32 rounding apart)
    assert float((example.infer(data, params).float() - out.float()).abs().max()) <= 2.0 ** -9 * float(out.float().abs().max())
