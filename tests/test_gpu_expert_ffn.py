"""The experts' feed-forward against the 64-bit reference: types and activations, one row to
many tiles, experts without rows and with nearly all, dropped and repeated choices, odd and
ragged sizes, and what the contract says about empty calls, spoiled rows and repeatability."""
import pytest
import torch

import block_ref
import expert_ref as ref
import memory_efficient_cnn_gb300 as mec

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NAMES = ("dx", "dweights", "dw_gate", "dw_up", "dw_down")


def make(T, k, E, C, F, dt, seed=0, choose="uneven"):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(DT[dt])  # noqa: E731
    if choose == "one":  # everything to the last expert
        experts = torch.full((T, k), E - 1)
    elif choose == "any":  # also outside of the experts, and the same one twice
        experts = torch.randint(-2, E + 2, (T, k), generator=g)
    else:
        experts = (torch.rand(T, E, generator=g) * (1.0 + torch.arange(E) % 3)).topk(min(k, E), -1)[1]
        experts = experts.repeat(1, -(-k // experts.shape[1]))[:, :k]
    weights = torch.softmax(torch.randn(T, k, generator=g), -1).to(DT[dt])
    return (n(T, C), experts.to(torch.int32), weights, n(E, F, C, std=C ** -0.5), n(E, F, C, std=C ** -0.5),
            n(E, C, F, std=F ** -0.5), n(T, C, std=0.5))


def run(x, experts, weights, wg, wu, wd, dy, act):
    x, experts, weights, wg, wu, wd, dy = (t.cuda() for t in (x, experts, weights, wg, wu, wd, dy))
    y, saved = mec.expert_ffn_train(x, experts, weights, wg, wu, wd, act=act)
    grads = mec.expert_ffn_backward(dy, weights, wg, wu, wd, saved, act=act)
    plain = mec.expert_ffn(x, experts, weights, wg, wu, wd, act=act)
    torch.cuda.synchronize()
    return dict(y=y, **dict(zip(NAMES, grads))), plain


def check(T, k, E, C, F, dt, act="silu", seed=0, choose="uneven"):
    x, experts, weights, wg, wu, wd, dy = make(T, k, E, C, F, dt, seed, choose)
    want = ref.experts_all(x.double(), experts, weights.double(), wg.double(), wu.double(), wd.double(), act, DT[dt], dy.double())
    got, plain = run(x, experts, weights, wg, wu, wd, dy, act)
    what = f"{dt} {act} {(T, k, E, C, F)} {choose}"
    block_ref.check(got, want, what)
    block_ref.check(dict(y=plain), {"y": want["y"]}, "inference " + what)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("act", mec.ACTS)
def test_activations(dt, act):
    check(90, 2, 4, 48, 136, dt, act)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("choose", ["uneven", "one", "any"])
@pytest.mark.parametrize("T,k,E,C,F", [
    (1, 1, 1, 1, 1), (1, 2, 8, 64, 128), (2, 1, 3, 7, 9), (3, 4, 4, 130, 66), (9, 2, 5, 72, 200), (33, 3, 7, 64, 96),
    (64, 1, 1, 128, 128), (100, 2, 16, 40, 264), (129, 1, 2, 136, 120), (300, 2, 3, 257, 255), (700, 1, 5, 64, 72)])
def test_sizes(dt, choose, T, k, E, C, F):
    check(T, k, E, C, F, dt, seed=T + E + F, choose=choose)


@pytest.mark.parametrize("dt,T,k,E,C,F", [("bf16", 5000, 2, 8, 128, 256), ("f16", 1500, 2, 3, 520, 1000), ("bf16", 900, 4, 40, 200, 328),
                                          ("f32", 800, 2, 6, 136, 250), ("bf16", 70000, 1, 3, 16, 24), ("f16", 300, 2, 4, 1032, 2056)])
def test_large(dt, T, k, E, C, F):
    """Several tiles of an expert, and more pairs than one planning block takes."""
    check(T, k, E, C, F, dt, "gelu", seed=3)


@pytest.mark.parametrize("choose", ["uneven", "one", "any"])
@pytest.mark.parametrize("dt,T,k,E,C,F", [("bf16", 70, 2, 3, 2000, 1607), ("f16", 9000, 1, 5, 72, 104), ("bf16", 4100, 2, 2, 33, 40),
                                          ("f32", 150, 2, 3, 700, 1101), ("f32", 4000, 1, 4, 40, 65), ("f16", 66, 1, 1, 2304, 136)])
def test_long_sums_over_few_tiles(choose, dt, T, k, E, C, F):
    """Sums whose K blocks are dealt out over more CTAs than there are tiles, with experts that get none."""
    check(T, k, E, C, F, dt, seed=T, choose=choose)


@pytest.mark.parametrize("E", [300, 1024])
def test_many_experts(E):
    check(500, 3, E, 24, 40, "bf16", seed=E)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("choose", ["uneven", "one", "any"])
@pytest.mark.parametrize("T,k,E,C,F", [(1, 2, 8, 512, 1024), (32, 2, 6, 520, 264), (16, 4, 3, 1000, 366), (64, 1, 20, 64, 200), (16, 2, 6, 520, 264), (8, 1, 3, 2048, 4096),
                                       (2, 32, 9, 48, 33), (5, 3, 40, 1030, 514), (13, 5, 4, 72, 4100)])
def test_few_rows(dt, choose, T, k, E, C, F):
    """Inference of up to 8, 32 or 64 pairs, which has kernels of its own, and of 65."""
    x, experts, weights, wg, wu, wd, _ = make(T, k, E, C, F, dt, T + F, choose)
    want = ref.experts_all(x.double(), experts, weights.double(), wg.double(), wu.double(), wd.double(), "gelu", DT[dt])
    y = mec.expert_ffn(*(t.cuda() for t in (x, experts, weights, wg, wu, wd)), act="gelu")
    block_ref.check(dict(y=y), want, f"{dt} {choose} {(T, k, E, C, F)}")


def test_few_rows_touch_their_experts_alone():
    """The other experts' weights are not read into the result, whatever they hold."""
    for dt in DT:
        x, experts, weights, wg, wu, wd, _ = (t.cuda() for t in make(3, 2, 8, 264, 136, dt))
        want = mec.expert_ffn(x, experts, weights, wg, wu, wd)
        for e in set(range(8)) - set(experts.flatten().tolist()):
            wg[e] = wu[e] = wd[e] = float("nan")
        assert torch.equal(mec.expert_ffn(x, experts, weights, wg, wu, wd), want)


def test_no_choice_left():
    x, experts, weights, wg, wu, wd, dy = make(20, 2, 3, 40, 48, "bf16")
    experts[:] = -1
    got, plain = run(x, experts, weights, wg, wu, wd, dy, "silu")
    assert all(not t.any() for t in (*got.values(), plain))


def test_dropped_choices_do_not_spoil():
    """What a dropped place's weight holds does not matter."""
    x, experts, weights, wg, wu, wd, dy = make(70, 2, 3, 40, 48, "f16")
    experts[::3, 0] = -1
    want, plain = run(x, experts, weights, wg, wu, wd, dy, "silu")
    weights[::3, 0] = float("nan")
    got, plain2 = run(x, experts, weights, wg, wu, wd, dy, "silu")
    assert torch.equal(plain, plain2) and all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("dt", DT)
def test_spoiled_rows_and_experts(dt, T):
    """A row's NaN stays in its own outputs and its experts' gradients; an expert whose weights are
    infinite spoils no other expert and no row that did not choose it."""
    x, experts, weights, wg, wu, wd, dy = make(T, 1, 4, 72, 88, dt)
    experts[:, 0] = torch.arange(T) % 3  # (expert 3 has no rows)
    clean, plain = run(x, experts, weights, wg, wu, wd, dy, "silu")
    x2 = x.clone()
    x2[1] = float("nan")
    got, plain2 = run(x2, experts, weights, wg, wu, wd, dy, "silu")
    others = torch.arange(T) != 1
    assert torch.equal(plain2[others.cuda()], plain[others.cuda()]) and plain2[1].isnan().all()
    for n in ("dw_gate", "dw_up", "dw_down"):
        assert torch.equal(got[n][[0, 2, 3]], clean[n][[0, 2, 3]]) and got[n][1].isnan().any()
        assert not got[n][3].any()
    for w in (0, 1, 2):
        ws = [wg.clone(), wu.clone(), wd.clone()]
        ws[w][1] = float("inf")
        ws[w][3] = float("nan")
        got, plain2 = run(x, experts, weights, *ws, dy, "silu")
        keep = (experts[:, 0] != 1).cuda()
        assert torch.equal(plain2[keep], plain[keep])
        for n in ("y", "dx", "dweights"):
            assert torch.equal(got[n][keep], clean[n][keep])
        for n in ("dw_gate", "dw_up", "dw_down"):
            assert torch.equal(got[n][[0, 2, 3]], clean[n][[0, 2, 3]])


def test_empty():
    x, experts, weights, wg, wu, wd, dy = (t.cuda() for t in make(1, 2, 3, 16, 24, "bf16"))
    x, experts, weights, dy = x[:0], experts[:0], weights[:0], dy[:0]
    y, saved = mec.expert_ffn_train(x, experts, weights, wg, wu, wd)
    grads = mec.expert_ffn_backward(dy, weights, wg, wu, wd, saved)
    assert y.shape == (0, 16) and all(not g.any() for g in grads)


def test_leading_axes_and_out():
    x, experts, weights, wg, wu, wd, _ = (t.cuda() for t in make(30, 2, 4, 64, 80, "bf16"))
    want = mec.expert_ffn(x, experts, weights, wg, wu, wd)
    out = torch.full((2, 3, 5, 64), float("nan"), dtype=x.dtype, device="cuda")
    got = mec.expert_ffn(x.view(2, 3, 5, 64), experts.view(2, 3, 5, 2), weights.view(2, 3, 5, 2), wg, wu, wd, out=out)
    assert got is out and torch.equal(out.view(30, 64), want)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,k,E,C,F", [(1, 2, 8, 256, 512), (50, 2, 6, 130, 72), (3000, 2, 5, 64, 128)])
def test_same_bits_every_time(dt, T, k, E, C, F):
    args = make(T, k, E, C, F, dt)
    (a, p), (b, q) = run(*args, "silu"), run(*args, "silu")
    assert torch.equal(p, q) and all(torch.equal(a[n], b[n]) for n in a)


def test_gradients_asked_for_alone():
    x, experts, weights, wg, wu, wd, dy = (t.cuda() for t in make(80, 2, 4, 72, 40, "f16"))
    _, saved = mec.expert_ffn_train(x, experts, weights, wg, wu, wd)
    full = mec.expert_ffn_backward(dy, weights, wg, wu, wd, saved)
    for need in range(8):
        want = [bool(need & 1), bool(need & 2)] + [bool(need & 4)] * 3
        got = mec.expert_ffn_backward(dy, weights, wg, wu, wd, saved, need_dx=want[0], need_dweights=want[1], need_dw=want[2])
        for g, f, w in zip(got, full, want):
            assert (g is not None) == w and (g is None or torch.equal(g, f))


def test_gradient_by_differences():
    x, experts, weights, wg, wu, wd, dy = make(6, 2, 3, 5, 4, "f32", seed=2)
    got, _ = run(x, experts, weights, wg, wu, wd, dy, "silu")
    args = [t.double() for t in (x, weights, wg, wu, wd)]

    def value(x, weights, wg, wu, wd):
        return (ref.expert_ffn(x, experts, weights, wg, wu, wd, "silu") * dy.double()).sum()

    h = 1e-5
    for i, n in enumerate(NAMES):
        for at in range(0, args[i].numel(), 3):
            up, down = [t.clone() for t in args], [t.clone() for t in args]
            up[i].view(-1)[at] += h
            down[i].view(-1)[at] -= h
            slope = float((value(*up) - value(*down)) / (2 * h))
            assert abs(float(got[n].view(-1)[at]) - slope) < 2e-5 * (1 + abs(slope)), n


def test_graph_and_streams():
    x, experts, weights, wg, wu, wd, dy = (t.cuda() for t in make(300, 2, 4, 64, 96, "bf16"))
    other = (torch.roll(experts, 7, 0) + 1) % 4
    want, saved = mec.expert_ffn_train(x, experts, weights, wg, wu, wd)
    back = mec.expert_ffn_backward(dy, weights, wg, wu, wd, saved)
    want_other = mec.expert_ffn(x, other, weights, wg, wu, wd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mec.expert_ffn(x, other, weights, wg, wu, wd)
    again = mec.expert_ffn(x, experts, weights, wg, wu, wd)  # at the same time, on its own workspace
    torch.cuda.synchronize()
    assert torch.equal(got, want_other) and torch.equal(again, want)
    graph, chosen = torch.cuda.CUDAGraph(), experts.clone()
    with torch.cuda.graph(graph):
        y, s = mec.expert_ffn_train(x, chosen, weights, wg, wu, wd)
        grads = mec.expert_ffn_backward(dy, weights, wg, wu, wd, s)
    chosen.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want_other)
    chosen.copy_(experts)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and all(torch.equal(a, b) for a, b in zip(grads, back))


def test_workspaces_that_begin_as_nan():
    args = [t.cuda() for t in make(150, 2, 5, 100, 60, "f16")]
    x, experts, weights, wg, wu, wd, dy = args
    dims = (150, 2, 5, 100, 60, mec.F16)
    want, saved = mec.expert_ffn_train(x, experts, weights, wg, wu, wd)
    back = mec.expert_ffn_backward(dy, weights, wg, wu, wd, saved)
    fresh = lambda kind: torch.full((mec.im2win_expert_ffn_size(kind, *dims),), 0xff, dtype=torch.uint8, device="cuda")  # noqa: E731
    saved2 = fresh(mec.FFN_SAVED)
    y, _ = mec.expert_ffn_train(x, experts, weights, wg, wu, wd, ws=fresh(mec.FFN_TRAIN), saved=saved2)
    again = mec.expert_ffn_backward(dy, weights, wg, wu, wd, saved2, ws=fresh(mec.FFN_BACKWARD))
    plain = mec.expert_ffn(x, experts, weights, wg, wu, wd, ws=fresh(mec.FFN_FORWARD))
    assert torch.equal(y, want) and torch.equal(plain, mec.expert_ffn(x, experts, weights, wg, wu, wd))
    assert all(torch.equal(a, b) for a, b in zip(again, back))
