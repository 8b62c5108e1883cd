"""Ways through the group norm, the router and the experts' feed-forward that their sizes alone do not take:
offsets past 32 bits, workspaces of the caller's shared by calls in a row, views into larger tensors."""
import pytest
import torch

import memory_efficient_cnn_gb300 as mec

pytestmark = pytest.mark.gpu


def test_group_norm_past_32_bits():
    """2.4e9 elements: the last image's last group, against the formula in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(2, 600000, 2048, dtype=torch.bfloat16, device="cuda").normal_(0.5, 1.5, generator=g)
    w = torch.empty(2048, dtype=torch.bfloat16, device="cuda").normal_(1.0, 0.2, generator=g)
    y, stats = mec.group_norm_train(x, 32, w, act="relu")
    v = x[1, :, -64:].double()
    mean, inv = v.mean(), 1 / torch.sqrt(v.var(correction=0) + 1e-5)
    assert abs(float(stats[1, 31, 0]) - float(mean)) < 1e-6 * 16 and abs(float(stats[1, 31, 1] / inv) - 1) < 1e-6 * 4
    z = ((v - mean) * inv * w[-64:].double()).clamp(min=0)
    assert ((y[1, :, -64:].double() - z).abs() <= 2.0 ** -8 * z + 1e-4).all()
    # (the gradient of sum(y dy) at dy = y: its sums go over 1.2e6 positions)
    dx, dw, _ = mec.group_norm_backward(y, x, stats, w, act="relu")
    hat = (v - mean) * inv
    dz = y[1, :, -64:].double() * (z > 0)
    e = dz * w[-64:].double()
    want = inv * (e - e.mean() - hat * (e * hat).mean())
    assert ((dx[1, :, -64:].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-3).all()
    assert bool(dw.isfinite().all())


def test_experts_past_32_bits_of_weights():
    """2.7e9 elements a matrix: the last expert's, by few rows and by many, against a call with the two used ones alone."""
    E, C, F = 40, 8192, 8192
    g = torch.Generator(device="cuda").manual_seed(2)
    ws = [torch.empty(E, *s, dtype=torch.bfloat16, device="cuda") for s in ((F, C), (F, C), (C, F))]
    for w in ws:
        for e in (0, E - 1):
            w[e].normal_(0, C ** -0.5, generator=g)
    few = [w[[0, E - 1]].contiguous() for w in ws]
    for T in (3, 70):
        x = torch.empty(T, C, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
        at = torch.arange(T, device="cuda").view(T, 1) % 2
        p = torch.full((T, 1), 0.5, dtype=torch.bfloat16, device="cuda")
        y = mec.expert_ffn(x, (at * (E - 1)).int(), p, *ws).float()
        want = mec.expert_ffn(x, at.int(), p, *few).float()
        # (the order of K alone may differ: a rounding of y, and of h on its way)
        assert float((y - want).norm() / want.norm()) <= 2.0 ** -8


def test_experts_past_32_bits_of_rows():
    """2.5e9 hidden values: the last rows against a call with them alone."""
    T, E, C, F = 300000, 3, 16, 8192
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s, std=1.0: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)  # noqa: E731
    x, dy = n(T, C), n(T, C, std=0.3)
    ws = [n(E, F, C, std=0.25), n(E, F, C, std=0.25), n(E, C, F, std=F ** -0.5)]
    experts = (torch.arange(T, device="cuda").view(T, 1) % E).int()
    p = torch.full((T, 1), 0.5, dtype=torch.bfloat16, device="cuda")
    y, saved = mec.expert_ffn_train(x, experts, p, *ws)
    dx, dp, *dws = mec.expert_ffn_backward(dy, p, *ws, saved)
    last = slice(T - 999, T)
    part = [t[last].clone() for t in (x, experts, p, dy)]
    y1, saved1 = mec.expert_ffn_train(*part[:3], *ws)
    dx1, dp1, *_ = mec.expert_ffn_backward(part[3], part[2], *ws, saved1)
    for a, b in ((y, y1), (dx, dx1), (dp, dp1)):
        a, b = a[last].float(), b.float()
        assert float((a - b).norm() / b.norm()) <= 2.0 ** -8
    assert all(bool(d.isfinite().all()) and bool(d.any()) for d in dws)


@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
def test_a_workspace_for_calls_in_a_row(dt):
    """One workspace for calls of other sizes one after another gives what each call's own gives."""
    g = torch.Generator(device="cuda").manual_seed(4)
    n = lambda *s, std=1.0: torch.empty(s, dtype=dt, device="cuda").normal_(0, std, generator=g)  # noqa: E731
    code = {torch.float32: mec.F32, torch.float16: mec.F16, torch.bfloat16: mec.BF16}[dt]
    ws = [n(6, 88, 72, std=0.1), n(6, 88, 72, std=0.1), n(6, 72, 88, std=0.1)]
    sizes = [(700, 2), (5, 3), (90, 1), (31, 2)]
    shared = torch.full((max(mec.im2win_expert_ffn_size(mec.FFN_FORWARD, T, k, 6, 72, 88, code) for T, k in sizes),), 0xff,
                        dtype=torch.uint8, device="cuda")
    cases = []
    for T, k in sizes:
        p, e = mec.expert_route(n(T, 6), k)
        x = n(T, 72)
        cases.append((x, e, p, mec.expert_ffn(x, e, p, *ws)))
    got = [mec.expert_ffn(x, e, p, *ws, ws=shared) for x, e, p, _ in cases + cases[::-1]]
    assert all(torch.equal(a, c[3]) for a, c in zip(got, cases + cases[::-1]))


def test_views_and_refusals_on_the_gpu():
    """Contiguous views that begin on 16 bytes are taken; others, and tensors that are not contiguous, are refused."""
    x = torch.randn(4, 30, 64, device="cuda", dtype=torch.bfloat16)
    assert torch.equal(mec.group_norm(x[1:3], 8), mec.group_norm(x[1:3].clone(), 8))
    with pytest.raises(ValueError, match="contiguous"):
        mec.group_norm(x.transpose(1, 2), 5)
    with pytest.raises(mec.Im2winError, match="align"):
        mec.group_norm(x.view(-1)[1:1 + 8 * 64].view(1, 8, 64), 8)
    # a part of a longer list of choices, which begins anywhere
    w = torch.randn(3, 16, 64, device="cuda", dtype=torch.bfloat16)
    ws = (w, w, w.transpose(1, 2).contiguous())
    p, e = mec.expert_route(torch.randn(120, 3, device="cuda", dtype=torch.bfloat16), 1)
    for T in (3, 100):
        rows = x.view(-1, 64)[:T]
        got = mec.expert_ffn(rows, e[7:7 + T], p[7:7 + T], *ws)
        assert torch.equal(got, mec.expert_ffn(rows, e[7:7 + T].clone(), p[7:7 + T].clone(), *ws))
    with pytest.raises(ValueError, match="contiguous"):
        mec.expert_route(x[..., ::2], 2)
    with pytest.raises(ValueError, match="contiguous"):
        mec.expert_route(x.transpose(0, 1), 2)
    rows, (p, e) = x.view(-1, 64), mec.expert_route(x.view(-1, 64)[:, :3].contiguous(), 2)
    with pytest.raises(ValueError, match="contiguous"):
        mec.expert_ffn(rows, e, p, w, w, w.transpose(1, 2))
    with pytest.raises(TypeError, match="int32"):
        mec.expert_ffn(rows, e.long(), p, w, w, w.transpose(1, 2).contiguous())
    with pytest.raises(ValueError, match="ws is too small"):
        mec.expert_ffn(rows, e, p, w, w, w.transpose(1, 2).contiguous(), ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
