"""Refusals and sizes of the group norm, the router and the experts' feed-forward,
answered on the host: no GPU is needed, and nothing is launched."""
import ctypes

import pytest
import torch

import memory_efficient_cnn_gb300 as mec
from memory_efficient_cnn_gb300 import build as mbuild
from memory_efficient_cnn_gb300._binding import (
    BF16, ERR_INVALID_ARG, ERR_MISALIGNED, ERR_UNSUPPORTED, ERR_WORKSPACE, F16, F32, OK)


@pytest.fixture(scope="module", autouse=True)
def lib():
    mbuild.build()
    return mec.lib()


# ---------------------------------------------------------------- group norm
def norm_call(x=4096, w=4096, b=4096, y=8192, stats=None, ws=16384, ws_bytes=1 << 40, N=2, P=9, C=8, G=2, act=5, eps=1e-5,
              dtype=F16):
    return mec.lib().im2win_group_norm(x, w, b, y, stats, ws, ws_bytes, N, P, C, G, act, eps, dtype, None)


def test_group_norm_refusals():
    for kw in (dict(x=None), dict(y=None), dict(act=6), dict(act=-1), dict(dtype=3), dict(N=-1), dict(P=-1), dict(C=0),
               dict(G=0), dict(G=3), dict(G=16), dict(eps=-1.0), dict(eps=float("nan"))):
        assert norm_call(**kw) == ERR_INVALID_ARG, kw
    for kw in (dict(x=4098), dict(w=4104), dict(b=4100), dict(y=8200), dict(stats=8), dict(ws=16392)):
        assert norm_call(**kw) == ERR_MISALIGNED, kw
    for kw in (dict(C=1 << 21, G=1), dict(N=1 << 31), dict(P=1 << 31), dict(N=1 << 20, P=1 << 20), dict(N=1 << 12, C=1 << 20)):
        assert norm_call(**kw) == ERR_UNSUPPORTED, kw
    # maps that stay on the chip need no workspace, large ones do
    assert mec.im2win_group_norm_size(False, 2, 9, 8, 2, F16) == 0 < mec.im2win_group_norm_size(True, 2, 9, 8, 2, F16)
    large = dict(N=64, P=3136, C=128)
    assert norm_call(ws=None, **large) == ERR_WORKSPACE
    assert norm_call(ws_bytes=mec.im2win_group_norm_size(False, 64, 3136, 128, 2, F16) - 1, **large) == ERR_WORKSPACE
    for kw in (dict(N=0), dict(P=0)):
        assert norm_call(x=None, y=None, ws=None, ws_bytes=0, **kw) == OK
    sz = ctypes.c_size_t()
    assert mec.lib().im2win_group_norm_size(0, 2, 9, 8, 2, F16, None) == ERR_INVALID_ARG
    assert mec.lib().im2win_group_norm_size(0, 2, 9, 8, 3, F16, ctypes.byref(sz)) == ERR_INVALID_ARG


def test_group_norm_backward_refusals():
    def call(dy=4096, x=4096, stats=4096, w=4096, b=4096, dx=8192, dw=8192, db=8192, ws=16384, ws_bytes=1 << 40, P=9, act=0):
        return mec.lib().im2win_group_norm_backward(dy, x, stats, w, b, dx, dw, db, ws, ws_bytes, 2, P, 8, 2, act, F32, None)

    for kw in (dict(dy=None), dict(x=None), dict(stats=None), dict(w=None), dict(b=None), dict(act=6)):
        assert call(**kw) == ERR_INVALID_ARG, kw
    for kw in (dict(dy=8), dict(dx=8200), dict(dw=8), dict(db=4), dict(ws=8)):
        assert call(**kw) == ERR_MISALIGNED, kw
    assert call(ws=None) == ERR_WORKSPACE and call(ws_bytes=0) == ERR_WORKSPACE
    assert call(dx=None, dw=None, db=None, ws=None) == OK  # nothing asked for
    assert call(P=0, dy=None, x=None, stats=None, dw=None, db=None, ws=None) == OK


def test_group_norm_binding_refusals():
    x, w = torch.zeros(2, 9, 8), torch.zeros(8)
    stats = torch.zeros(2, 4, 2)
    with pytest.raises(ValueError, match="do not form 3 groups"):
        mec.group_norm(x, 3)
    with pytest.raises(ValueError, match="do not form 0 groups"):
        mec.group_norm(x, 0)
    with pytest.raises(ValueError, match=r"\[N, ..., C\]"):
        mec.group_norm(w, 2)
    with pytest.raises(ValueError, match="w has shape"):
        mec.group_norm(x, 2, torch.zeros(7))
    with pytest.raises(ValueError, match="out has shape"):
        mec.group_norm(x, 2, out=torch.zeros(2, 8, 8))
    with pytest.raises(TypeError, match="one dtype"):
        mec.group_norm(x, 2, w.half())
    with pytest.raises(ValueError, match="out is x"):
        mec.group_norm_train(x, 2, out=x)
    with pytest.raises(ValueError, match="requires grad"):
        mec.group_norm(x, 2, w.requires_grad_())
    w = w.detach()
    with pytest.raises(ValueError, match="dy has shape"):
        mec.group_norm_backward(torch.zeros(2, 9, 16), x, stats)
    with pytest.raises(ValueError, match=r"stats must be"):
        mec.group_norm_backward(x, x, stats[0])
    with pytest.raises(ValueError, match="CUDA"):
        mec.group_norm(x, 2, w, w)


# ---------------------------------------------------------------- router
def test_route_refusals():
    def call(logits=4096, weights=4096, experts=4096, T=3, E=8, k=2, over=0, dtype=BF16):
        return mec.lib().im2win_expert_route(logits, weights, experts, T, E, k, over, dtype, None)

    def back(dw=4096, logits=4096, experts=4096, dl=4096, T=3, E=8, k=2, over=0, dtype=BF16):
        return mec.lib().im2win_expert_route_backward(dw, logits, experts, dl, T, E, k, over, dtype, None)

    for fn, names in ((call, ("logits", "weights", "experts")), (back, ("dw", "logits", "experts", "dl"))):
        for name in names:
            assert fn(**{name: None}) == ERR_INVALID_ARG
            assert fn(**{name: 4097}) == ERR_MISALIGNED  # (lists of choices need their element's alignment alone)
            if name in ("logits", "dl"):
                assert fn(**{name: 4104}) == ERR_MISALIGNED
        for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(over=2), dict(over=-1), dict(dtype=4)):
            assert fn(**kw) == ERR_INVALID_ARG, kw
        for kw in (dict(E=1025), dict(E=64, k=33), dict(T=1 << 31)):
            assert fn(**kw) == ERR_UNSUPPORTED, kw
        assert fn(T=0, **{n: None for n in names}) == OK


def test_route_binding_refusals():
    logits, w, e = torch.zeros(4, 8), torch.zeros(4, 2), torch.zeros(4, 2, dtype=torch.int32)
    for k in (0, 9):
        with pytest.raises(ValueError, match="k must be between"):
            mec.expert_route(logits, k)
    with pytest.raises(ValueError, match="dweights has shape"):
        mec.expert_route_backward(torch.zeros(3, 2), logits, e)
    with pytest.raises(TypeError, match="one dtype"):
        mec.expert_route_backward(w.half(), logits, e)
    with pytest.raises(ValueError, match="requires grad"):
        mec.expert_route(logits.clone().requires_grad_(), 2)
    with pytest.raises(ValueError, match="CUDA"):
        mec.expert_route(logits, 2)


# ---------------------------------------------------------------- experts' feed-forward
def test_expert_ffn_sizes():
    for dt in (0, 1, 2):
        for T, k, E, C, F in ((0, 1, 1, 8, 8), (1, 2, 8, 512, 2048), (777, 2, 24, 1000, 1366), (5, 32, 3, 7, 9)):
            sizes = [mec.im2win_expert_ffn_size(b, T, k, E, C, F, dt) for b in range(4)]
            assert all(s % 256 == 0 and s >= 256 for s in sizes)
    sz = ctypes.c_size_t()
    q = mec.lib().im2win_expert_ffn_size
    for bad in ((0, -1, 1, 1, 8, 8, 0), (0, 1, 0, 1, 8, 8, 0), (0, 1, 1, 0, 8, 8, 0), (0, 1, 1, 1, 0, 8, 0), (0, 1, 1, 1, 8, 0, 0),
                (4, 1, 1, 1, 8, 8, 0), (0, 1, 1, 1, 8, 8, 3)):
        assert q(*bad, ctypes.byref(sz)) == ERR_INVALID_ARG
    assert q(0, 1, 1, 1, 8, 8, 0, None) == ERR_INVALID_ARG
    for big in ((0, 1, 33, 40, 8, 8, 0), (0, 1, 1, 1025, 8, 8, 0), (0, 1 << 31, 1, 1, 8, 8, 0), (0, 1 << 30, 2, 1, 8, 8, 0),
                (0, 1, 1, 1024, 1 << 21, 8, 0), (0, 1, 1, 1024, 8, 1 << 21, 0), (0, 1, 1, 1024, 1 << 16, 1 << 16, 0),
                (0, 1 << 24, 1, 1, 1 << 17, 8, 0)):
        assert q(*big, ctypes.byref(sz)) == ERR_UNSUPPORTED, big


def test_expert_ffn_refusals():
    def call(x=4096, experts=4096, weights=4096, wg=8192, wu=8192, wd=8192, y=4096, saved=None, ws=16384, ws_bytes=1 << 40, T=3,
             k=2, E=4, C=8, F=8, act=0, dtype=F16):
        return mec.lib().im2win_expert_ffn(x, experts, weights, wg, wu, wd, y, saved, ws, ws_bytes, T, k, E, C, F, act, dtype, None)

    for kw in (dict(x=None), dict(experts=None), dict(weights=None), dict(wg=None), dict(wu=None), dict(wd=None), dict(y=None),
               dict(act=5), dict(act=-1), dict(dtype=3), dict(T=-1), dict(k=0), dict(E=0), dict(C=0), dict(F=0)):
        assert call(**kw) == ERR_INVALID_ARG, kw
    for name in ("x", "wg", "wu", "wd", "y", "saved", "ws"):
        assert call(**{name: 4104}) == ERR_MISALIGNED, name
    assert call(experts=4098) == ERR_MISALIGNED and call(weights=4097) == ERR_MISALIGNED
    assert call(ws=None) == ERR_WORKSPACE
    assert call(ws_bytes=mec.im2win_expert_ffn_size(mec.FFN_FORWARD, 3, 2, 4, 8, 8, F16) - 1) == ERR_WORKSPACE
    assert call(E=1025) == ERR_UNSUPPORTED and call(k=33) == ERR_UNSUPPORTED
    assert call(T=0, x=None, y=None, ws=None) == OK

    def back(dy=4096, weights=4096, w=8192, saved=8192, dx=4096, dweights=4096, dw=(4096,) * 3, ws=16384, ws_bytes=1 << 40, T=3,
             act=0):
        return mec.lib().im2win_expert_ffn_backward(dy, weights, w, w, w, saved, dx, dweights, *dw, ws, ws_bytes, T, 2, 4, 8, 8, act,
                                                    F32, None)

    for kw in (dict(dy=None), dict(weights=None), dict(w=None), dict(saved=None), dict(act=5), dict(dw=(4096, None, 4096)),
               dict(dw=(None, 4096, 4096))):
        assert back(**kw) == ERR_INVALID_ARG, kw
    for kw in (dict(dy=8), dict(weights=2), dict(w=8), dict(saved=8), dict(dx=8), dict(dweights=2), dict(dw=(8,) * 3), dict(ws=8)):
        assert back(**kw) == ERR_MISALIGNED, kw
    assert back(ws=None) == ERR_WORKSPACE and back(ws_bytes=16) == ERR_WORKSPACE
    assert back(dx=None, dweights=None, dw=(None,) * 3, ws=None) == OK


def test_expert_ffn_binding_refusals():
    x, e, p = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    w, d = torch.zeros(3, 16, 8), torch.zeros(3, 8, 16)
    with pytest.raises(ValueError, match="w_up has shape"):
        mec.expert_ffn(x, e, p, w, w[:2], d)
    with pytest.raises(ValueError, match="w_down has shape"):
        mec.expert_ffn(x, e, p, w, w, w)
    with pytest.raises(ValueError, match="weights has shape"):
        mec.expert_ffn(x, e, p[:3], w, w, d)
    with pytest.raises(ValueError, match=r"w_gate \[E, F, C\]"):
        mec.expert_ffn(x, e, p, w[0], w[0], d[0])
    with pytest.raises(TypeError, match="one dtype"):
        mec.expert_ffn(x, e, p.half(), w, w, d)
    with pytest.raises(ValueError, match="CUDA"):
        mec.expert_ffn(x, e, p, w, w, d)
    with pytest.raises(ValueError, match="requires grad"):
        mec.expert_ffn(x, e, p, w, w, d.clone().requires_grad_())
    with pytest.raises(TypeError, match="int32"):
        mec.experts._experts("f", e.long(), x, (4, 2))
    with pytest.raises(ValueError, match="experts has shape"):
        mec.experts._experts("f", e[:3], x, (4, 2))
