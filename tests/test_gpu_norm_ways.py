"""Calls of the group norm that its documentation allows, in each of its three ways (single rows in registers, maps that
stay on the chip, maps that are read twice): parts of a batch, in place, right behind the launch that writes the inputs."""
import pytest
import torch

import memory_efficient_cnn_gb300 as mec

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def make(N, P, C, dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, std=1.0, mean=0.0: torch.empty(s, device="cuda", dtype=DT[dt]).normal_(mean, std, generator=g)  # noqa: E731
    return n(N, P, C, std=1.5, mean=0.7), n(C, std=0.2, mean=1.0), n(C, std=0.3), n(N, P, C, std=0.5)


@pytest.mark.parametrize("N,P,C,G", [(6, 1, 24, 3), (4, 50, 24, 3), (3, 180000, 24, 3)])
def test_gradients_of_a_part_of_a_batch(N, P, C, G):
    """The statistics of its later images begin anywhere on 8 bytes."""
    x, w, b, dy = make(N, P, C, "bf16")
    _, stats = mec.group_norm_train(x, G, w, b, act="silu")
    for first in range(1, N):
        part, own = stats[first:], stats[first:].clone()
        got = mec.group_norm_backward(dy[first:], x[first:], part, w, b, act="silu")
        want = mec.group_norm_backward(dy[first:], x[first:], own, w, b, act="silu")
        assert all(torch.equal(a, c) for a, c in zip(got, want))
