"""A channels-last residual block after an im2win convolution, trained for a few steps.

    maps  = conv(images)                       fused im2win convolution, NHWC, "same" padding
    n     = pre(maps)                          the first norm of the block
    y     = (act(n Wg^T) * (n Wu^T)) Wd^T      gated feed-forward over the channels
    r, n' = res_scale * maps + gate * post(y), pre'(r)

with a gate for each image and channel, the mean over n' against a target as the
loss, the gradients of every parameter of the block, their clipping by the global
norm and a plain gradient step. The convolution's filter stays as it is.

    python examples/residual_block.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import memory_efficient_cnn_gb300 as mec  # noqa: E402

FIRST = dict(pre="layer")                # maps -> n
SEAM = dict(post="rms", pre="rms")       # maps, y -> r, n'


def make(images=4, height=14, width=14, c_in=8, channels=64, hidden=160, dtype=torch.float32, seed=0, device="cuda"):
    """Inputs, filter and the block's parameters."""
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *s, std=1.0, mean=0.0: torch.empty(s, device=device, dtype=dtype).normal_(mean, std, generator=g)  # noqa: E731
    data = dict(images=rand(images, height, width, c_in), filter=rand(channels, c_in, 3, 3, std=(9 * c_in) ** -0.5),
                target=rand(images, height, width, channels))
    params = dict(w_first=rand(channels, std=0.1, mean=1.0), b_first=rand(channels, std=0.1),
                  w_gate=rand(hidden, channels, std=channels ** -0.5), w_up=rand(hidden, channels, std=channels ** -0.5),
                  w_down=rand(channels, hidden, std=hidden ** -0.5), w_post=rand(channels, std=0.1, mean=1.0),
                  gate=rand(images, channels, std=0.2, mean=0.5), res_scale=rand(channels, std=0.1, mean=1.0),
                  w_pre=rand(channels, std=0.1, mean=1.0))
    return data, params


def seam_args(p, rows_per_gate):
    return dict(SEAM, w_post=p["w_post"], gate=p["gate"], rows_per_gate=rows_per_gate, res_scale=p["res_scale"],
                w_pre=p["w_pre"])


def loss_and_gradients(data, p, act="silu"):
    """The loss, and the gradient of each parameter by name."""
    maps = mec.conv_fused_ex(data["images"], data["filter"], pad=(1, 1), layout=mec.NHWC)
    rows_per_gate = maps.shape[1] * maps.shape[2]
    first = dict(FIRST, w_pre=p["w_first"], b_pre=p["b_first"])
    seam = seam_args(p, rows_per_gate)
    _, n = mec.residual_norm(maps, **first)
    y, saved = mec.gated_ffn_train(n, p["w_gate"], p["w_up"], p["w_down"], act=act)
    _, out = mec.residual_norm(maps, y, **seam)

    diff = out.float() - data["target"].float()
    loss = (diff * diff).mean()
    d_out = (2.0 / diff.numel() * diff).to(out.dtype)

    g = mec.residual_norm_backward(None, d_out, maps, y, **seam)
    d_n, dwg, dwu, dwd = mec.gated_ffn_backward(g["dy"], n, p["w_gate"], p["w_up"], p["w_down"], saved, act=act)
    # the block's input is the convolution's output, which is not trained: only its norm's parameters
    f = mec.residual_norm_backward(None, d_n, maps, **first)
    return loss, dict(w_first=f["dw_pre"], b_first=f["db_pre"], w_gate=dwg, w_up=dwu, w_down=dwd, w_post=g["dw_post"],
                      gate=g["dgate"], res_scale=g["dres_scale"], w_pre=g["dw_pre"])


def train(data, params, steps=5, rate=1.0, max_norm=1.0):
    """[(loss, gradient norm before clipping)] of each step; the parameters are updated in place."""
    seen = []
    for _ in range(steps):
        loss, grads = loss_and_gradients(data, params)
        norm = mec.clip_grad_norm(grads.values(), max_norm)
        for name, d in grads.items():
            params[name].sub_(rate * d)
        seen.append((loss, norm))
    return [(float(a), float(b)) for a, b in seen]


def infer(data, params, act="silu"):
    """The block's output without what training keeps."""
    maps = mec.conv_fused_ex(data["images"], data["filter"], pad=(1, 1), layout=mec.NHWC)
    _, n = mec.residual_norm(maps, **dict(FIRST, w_pre=params["w_first"], b_pre=params["b_first"]))
    y = mec.gated_ffn(n, params["w_gate"], params["w_up"], params["w_down"], act=act)
    return mec.residual_norm(maps, y, **seam_args(params, maps.shape[1] * maps.shape[2]))[1]


if __name__ == "__main__":
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 5
    for i, (loss, norm) in enumerate(train(*make(dtype=torch.bfloat16), steps=steps)):
        print(f"step {i}: loss {loss:.5f}, gradient norm {norm:.4f}")
