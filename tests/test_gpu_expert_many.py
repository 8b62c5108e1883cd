"""Many experts: decode batches of 9 to 512 pairs of rows with eight of up to 1024 experts, and training over them; and the values of
gradients whose sums and buffers pass 32 bits."""
import pytest
import torch

import block_ref
import expert_ref as ref
import memory_efficient_cnn_gb300 as mec
import norm_bounds
from test_gpu_expert_ffn import DT, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("choose", ["uneven", "one", "any"])
@pytest.mark.parametrize("T,k,E,C,F", [(2, 8, 64, 256, 192), (1, 8, 256, 512, 128), (8, 8, 128, 256, 128), (9, 8, 256, 128, 64),
                                       (17, 2, 96, 136, 264), (64, 8, 256, 128, 256), (33, 4, 1024, 64, 48), (50, 8, 70, 100, 66)])
def test_decode_batches(dt, choose, T, k, E, C, F):
    x, experts, weights, wg, wu, wd, _ = make(T, k, E, C, F, dt, T + E, choose)
    want = ref.experts_all(x.double(), experts, weights.double(), wg.double(), wu.double(), wd.double(), "silu", DT[dt])
    args = [t.cuda() for t in (x, experts, weights, wg, wu, wd)]
    y = mec.expert_ffn(*args, act="silu")
    block_ref.check(dict(y=y), want, f"{dt} {choose} {(T, k, E, C, F)}")
    assert torch.equal(mec.expert_ffn(*args, act="silu"), y)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,k,E,C,F", [(300, 8, 100, 136, 72), (64, 8, 256, 128, 96), (2000, 2, 300, 64, 40), (40, 3, 1024, 72, 24)])
def test_training_over_many_experts(dt, T, k, E, C, F):
    for choose in ("uneven", "any"):
        check(T, k, E, C, F, dt, "gelu", seed=E, choose=choose)


def test_unused_experts_of_many_stay_out():
    """Past 64 pairs too, in each way the matrices are read: in place, and copied to a pitch or to planes."""
    for dt, C, F in (("bf16", 128, 96), ("f16", 100, 66), ("f32", 64, 48)):
        x, experts, weights, wg, wu, wd, dy = (t.cuda() for t in make(90, 2, 200, C, F, dt))
        experts = experts % 7
        y, saved = mec.expert_ffn_train(x, experts, weights, wg, wu, wd)
        grads = mec.expert_ffn_backward(dy, weights, wg, wu, wd, saved)
        for w in (wg, wu, wd):
            w[7:] = float("nan")
        y2, saved = mec.expert_ffn_train(x, experts, weights, wg, wu, wd)
        grads2 = mec.expert_ffn_backward(dy, weights, wg, wu, wd, saved)
        assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(grads, grads2))
        assert all(not g[7:].any() for g in grads[2:])


def test_group_norm_gradients_past_32_bits():
    """2.4e9 elements: dw and db of the last group's channels. A thread adds 2831 positions, an eighth of 424 rows follow."""
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s, std=1.0, mean=0.0: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(mean, std, generator=g)  # noqa: E731
    x, dy, w, b = n(2, 600000, 2048, std=1.5, mean=0.5), n(2, 600000, 2048, std=0.5), n(2048, std=0.2, mean=1.0), n(2048, std=0.3)
    _, stats = mec.group_norm_train(x, 32, w, b, act="relu")
    dx, dw, db = mec.group_norm_backward(dy, x, stats, w, b, act="relu")
    last = slice(-64, None)
    want = norm_bounds.group_norm(x[..., last].double(), 1, w[last].double(), b[last].double(), "relu", 1e-5, torch.bfloat16,
                                  dy[..., last].double(), run=3200, run_params=3200)
    for name, got in (("dw", dw), ("db", db)):
        value, bound = want[name]
        assert ((got[last].double() - value).abs() <= bound).all(), name
        assert (value.abs() > 2 * bound).double().mean() > 0.8  # (zeros would not pass)
    value, bound = want["dx"]
    assert ((dx[..., last].double() - value).abs() <= bound).all()


def test_expert_gradients_past_32_bits_of_rows():
    """2.5e9 hidden values: the gradients of the last expert's matrices, 64 of its hidden channels, against 64 bits. Each output is off by
    its own rounding and by that of its operand (16-bit dg, du and weight * h), 2^-8 / sqrt(3) of the 2-norm each at most."""
    T, E, C, F = 300000, 3, 16, 8192
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s, std=1.0: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)  # noqa: E731
    x, dy = n(T, C), n(T, C, std=0.3)
    wg, wu, wd = n(E, F, C, std=0.25), n(E, F, C, std=0.25), n(E, C, F, std=F ** -0.5)
    experts = (torch.arange(T, device="cuda").view(T, 1) % E).int()
    p = torch.full((T, 1), 0.5, dtype=torch.bfloat16, device="cuda")
    _, saved = mec.expert_ffn_train(x, experts, p, wg, wu, wd)
    _, _, *got = mec.expert_ffn_backward(dy, p, wg, wu, wd, saved)
    for part in (slice(0, 64), slice(F - 64, F)):
        xe, de = x[E - 1::E].double(), dy[E - 1::E].double()
        a, slope = block_ref.act_pair("silu", xe @ wg[-1, part].double().T)
        u, dh = xe @ wu[-1, part].double().T, 0.5 * (de @ wd[-1][:, part].double())
        for have, want in ((got[0][-1, part], (dh * u * slope).T @ xe), (got[1][-1, part], (dh * a).T @ xe),
                           (got[2][-1][:, part], 0.5 * de.T @ (a * u))):
            assert float((have.double() - want).norm() / want.norm()) <= 2.0 ** -8
