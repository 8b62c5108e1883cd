"""A channels-last block of experts after an im2win convolution, trained for a few steps.

    maps = conv(images)                          fused im2win convolution, NHWC, "same" padding
    n    = silu(group norm(maps))                over each image's positions and groups of channels
    p, e = route(n Wr^T)                         each position's k experts and their weights
    y    = sum_j p_j ffn_(e_j)(n)                the chosen experts' gated feed-forwards
    out  = maps + y

with the mean over out against a target as the loss, the gradients of every parameter of
the block, their clipping by the global norm and a plain gradient step. The convolution's
filter stays as it is, and the router's product of a few columns is torch's.

    python examples/expert_block.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import memory_efficient_cnn_gb300 as mec  # noqa: E402


def make(images=4, height=14, width=14, c_in=8, channels=64, hidden=96, experts=6, dtype=torch.float32, seed=0, device="cuda"):
    """Inputs, filter and the block's parameters."""
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *s, std=1.0, mean=0.0: torch.empty(s, device=device, dtype=dtype).normal_(mean, std, generator=g)  # noqa: E731
    data = dict(images=rand(images, height, width, c_in), filter=rand(channels, c_in, 3, 3, std=(9 * c_in) ** -0.5),
                target=rand(images, height, width, channels))
    params = dict(w_norm=rand(channels, std=0.1, mean=1.0), b_norm=rand(channels, std=0.1),
                  w_router=rand(experts, channels, std=2 * channels ** -0.5),
                  w_gate=rand(experts, hidden, channels, std=channels ** -0.5),
                  w_up=rand(experts, hidden, channels, std=channels ** -0.5),
                  w_down=rand(experts, channels, hidden, std=hidden ** -0.5))
    return data, params


def convolved(data):
    return mec.conv_fused_ex(data["images"], data["filter"], pad=(1, 1), layout=mec.NHWC)


def loss_and_gradients(data, p, k=2, groups=8, act="silu"):
    """The loss, the gradient of each parameter by name, and the experts that were chosen."""
    maps = convolved(data)
    n, stats = mec.group_norm_train(maps, groups, p["w_norm"], p["b_norm"], act="silu")
    rows = n.flatten(0, -2)
    logits = rows @ p["w_router"].t()
    weights, experts = mec.expert_route(logits, k)
    y, saved = mec.expert_ffn_train(rows, experts, weights, p["w_gate"], p["w_up"], p["w_down"], act=act)
    out, _ = mec.residual_norm(maps, y.view_as(maps), pre="none")

    diff = out.float() - data["target"].float()
    loss = (diff * diff).mean()
    d_out = (2.0 / diff.numel() * diff).to(out.dtype)

    d_rows, d_weights, dwg, dwu, dwd = mec.expert_ffn_backward(d_out.flatten(0, -2), weights, p["w_gate"], p["w_up"],
                                                               p["w_down"], saved, act=act)
    d_logits = mec.expert_route_backward(d_weights, logits, experts)
    d_n = torch.addmm(d_rows, d_logits, p["w_router"]).view_as(n)
    # the block's input is the convolution's output, which is not trained: only the norm's parameters
    _, dw, db = mec.group_norm_backward(d_n, maps, stats, p["w_norm"], p["b_norm"], act="silu", need_dx=False)
    return loss, dict(w_norm=dw, b_norm=db, w_router=d_logits.t() @ rows, w_gate=dwg, w_up=dwu, w_down=dwd), experts


def train(data, params, steps=5, rate=1.0, max_norm=1.0):
    """[(loss, gradient norm before clipping)] of each step; the parameters are updated in place."""
    seen = []
    for _ in range(steps):
        loss, grads, _ = loss_and_gradients(data, params)
        norm = mec.clip_grad_norm(grads.values(), max_norm)
        for name, d in grads.items():
            params[name].sub_(rate * d)
        seen.append((loss, norm))
    return [(float(a), float(b)) for a, b in seen]


def infer(data, p, k=2, groups=8, act="silu"):
    """The block's output without what training keeps."""
    maps = convolved(data)
    rows = mec.group_norm(maps, groups, p["w_norm"], p["b_norm"], act="silu").flatten(0, -2)
    weights, experts = mec.expert_route(rows @ p["w_router"].t(), k)
    y = mec.expert_ffn(rows, experts, weights, p["w_gate"], p["w_up"], p["w_down"], act=act)
    return mec.residual_norm(maps, y.view_as(maps), pre="none")[0]


if __name__ == "__main__":
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 5
    for i, (loss, norm) in enumerate(train(*make(dtype=torch.bfloat16), steps=steps)):
        print(f"step {i}: loss {loss:.5f}, gradient norm {norm:.4f}")
