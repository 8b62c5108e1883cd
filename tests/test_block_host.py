"""Refusals and sizes of the residual-block operators, answered on the host: no
GPU is needed, and nothing is launched."""
import ctypes

import pytest
import torch

import block_ref as ref
import memory_efficient_cnn_gb300 as mec
from memory_efficient_cnn_gb300 import build as mbuild
from memory_efficient_cnn_gb300._binding import (
    ERR_INVALID_ARG, ERR_MISALIGNED, ERR_UNSUPPORTED, ERR_WORKSPACE, F16, F32, OK)


@pytest.fixture(scope="module", autouse=True)
def lib():
    mbuild.build()
    return mec.lib()


# ---------------------------------------------------------------- gated feed-forward
def test_ffn_sizes():
    for dt in (0, 1, 2):
        for R, C, F in ((0, 8, 8), (1, 1, 1), (5, 7, 9), (1000, 256, 1024)):
            sizes = [mec.im2win_gated_ffn_size(b, R, C, F, dt) for b in range(4)]
            assert all(s % 256 == 0 for s in sizes) and all(s >= 256 for s in sizes[:3])
    sz = ctypes.c_size_t()
    q = mec.lib().im2win_gated_ffn_size
    for bad in ((0, -1, 8, 8, 0), (0, 1, 0, 8, 0), (0, 1, 8, 0, 0), (4, 1, 8, 8, 0), (0, 1, 8, 8, 3)):
        assert q(*bad, ctypes.byref(sz)) == ERR_INVALID_ARG
    assert q(0, 1, 8, 8, 0, None) == ERR_INVALID_ARG
    for big in ((0, 1 << 31, 8, 8, 0), (0, 1, 1 << 31, 8, 0), (0, 1 << 30, 1 << 11, 8, 0), (0, 1, 1 << 21, 1 << 20, 0)):
        assert q(*big, ctypes.byref(sz)) == ERR_UNSUPPORTED


def ffn_call(x=4096, wg=8192, wu=8192, wd=8192, y=4096, saved=None, ws=16384, ws_bytes=1 << 30, R=2, C=8, F=8, act=0,
             dtype=F16):
    return mec.lib().im2win_gated_ffn(x, wg, wu, wd, y, saved, ws, ws_bytes, R, C, F, act, dtype, None)


def test_ffn_refusals():
    for kw in (dict(x=None), dict(wg=None), dict(wu=None), dict(wd=None), dict(y=None), dict(act=5), dict(act=-1),
               dict(dtype=7), dict(R=-1), dict(C=0), dict(F=0)):
        assert ffn_call(**kw) == ERR_INVALID_ARG, kw
    for kw in (dict(x=4104), dict(wg=8200), dict(wu=8194), dict(wd=8193), dict(y=4100), dict(saved=40), dict(ws=16392)):
        assert ffn_call(**kw) == ERR_MISALIGNED, kw
    assert ffn_call(ws=None) == ERR_WORKSPACE
    assert ffn_call(ws_bytes=mec.im2win_gated_ffn_size(mec.FFN_FORWARD, 2, 8, 8, F16) - 1) == ERR_WORKSPACE
    assert ffn_call(R=1 << 32) == ERR_UNSUPPORTED
    assert ffn_call(R=0, x=None, y=None, ws=None, ws_bytes=0) == OK


def back_call(dw=(4096, 4096, 4096), dx=4096, saved=8192, ws=16384, ws_bytes=1 << 30, R=2, act=0, dtype=F16, dy=4096):
    return mec.lib().im2win_gated_ffn_backward(dy, 4096, 8192, 8192, 8192, saved, dx, *dw, ws, ws_bytes, R, 8, 8, act,
                                               dtype, None)


def test_ffn_backward_refusals():
    assert back_call(dw=(4096, None, 4096)) == ERR_INVALID_ARG
    assert back_call(dw=(None, 4096, 4096)) == ERR_INVALID_ARG
    assert back_call(saved=None) == ERR_INVALID_ARG
    assert back_call(dy=None) == ERR_INVALID_ARG
    assert back_call(act=9) == ERR_INVALID_ARG
    assert back_call(dx=4098) == ERR_MISALIGNED
    assert back_call(dw=(4096, 4104, 4096)) == ERR_MISALIGNED
    assert back_call(ws_bytes=16) == ERR_WORKSPACE
    assert back_call(dw=(None,) * 3, dx=None) == OK  # nothing asked for


def test_ffn_binding_refusals():
    x, w, d = torch.zeros(4, 8), torch.zeros(16, 8), torch.zeros(8, 16)
    with pytest.raises(ValueError, match="w_up has shape"):
        mec.gated_ffn(x, w, torch.zeros(15, 8), d)
    with pytest.raises(ValueError, match="w_down has shape"):
        mec.gated_ffn(x, w, w, w)
    with pytest.raises(TypeError, match="one dtype"):
        mec.gated_ffn(x, w, w.half(), d)
    with pytest.raises(ValueError, match="CUDA"):
        mec.gated_ffn(x, w, w, d)
    with pytest.raises(ValueError, match="at least 1"):
        mec.gated_ffn(torch.zeros(4, 0), torch.zeros(16, 0), torch.zeros(16, 0), torch.zeros(0, 16))


# ---------------------------------------------------------------- norms
def norm_call(x=4096, y=4096, gate=4096, per=1, rs=4096, post=1, wq=4096, bq=None, pre=2, wp=4096, bp=4096, eps=1e-6,
              r=8192, n=8192, R=2, C=8, dtype=F32):
    return mec.lib().im2win_residual_norm(x, y, gate, per, rs, post, wq, bq, pre, wp, bp, eps, r, n, R, C, dtype, None)


def test_norm_refusals():
    for kw in (dict(x=None), dict(y=None), dict(y=None, gate=None), dict(y=None, post=0, wq=None), dict(per=0),
               dict(post=3), dict(pre=-1), dict(bq=4096), dict(post=0), dict(pre=0, bp=None), dict(pre=1),
               dict(n=None), dict(pre=0, wp=None, bp=None), dict(pre=0, wp=None, bp=None, n=None, r=None),
               dict(eps=-1.0), dict(eps=float("nan")), dict(R=-1), dict(C=0), dict(dtype=5)):
        assert norm_call(**kw) == ERR_INVALID_ARG, kw
    for kw in (dict(x=4100), dict(y=4100), dict(gate=4100), dict(rs=4104), dict(wq=4104), dict(wp=4108), dict(bp=4100),
               dict(r=4100), dict(n=4100)):
        assert norm_call(**kw) == ERR_MISALIGNED, kw
    assert norm_call(C=(1 << 20) + 1) == ERR_UNSUPPORTED
    assert norm_call(R=1 << 31) == ERR_UNSUPPORTED
    assert norm_call(R=0, x=None, y=None, r=None, n=None) == OK


def norm_back(dr=4096, dn=4096, y=4096, gate=4096, per=1, rs=4096, post=1, wq=4096, pre=1, wp=4096, dx=8192, dy=8192,
              dgate=8192, drs=8192, dwq=8192, dbq=None, dwp=8192, dbp=None, ws=16384, ws_bytes=1 << 30, R=2, C=8):
    return mec.lib().im2win_residual_norm_backward(
        dr, dn, 4096, y, gate, per, rs, post, wq, None, pre, wp, None, 1e-6, dx, dy, dgate, drs, dwq, dbq, dwp, dbp, ws,
        ws_bytes, R, C, F32, None)


def test_norm_backward_refusals():
    for kw in (dict(gate=None), dict(rs=None), dict(wq=None), dict(dbq=8192), dict(wp=None), dict(dbp=8192),
               dict(y=None), dict(pre=0, wp=None, dwp=None), dict(per=0)):
        assert norm_back(**kw) == ERR_INVALID_ARG, kw
    assert norm_back(dgate=8200) == ERR_MISALIGNED
    assert norm_back(ws_bytes=mec.im2win_residual_norm_backward_size(2, 8, 1, F32) - 1) == ERR_WORKSPACE
    assert norm_back(ws=None) == ERR_WORKSPACE
    sz = ctypes.c_size_t()
    q = mec.lib().im2win_residual_norm_backward_size
    assert q(2, 8, 0, F32, ctypes.byref(sz)) == ERR_INVALID_ARG
    assert q(2, 8, 1, F32, None) == ERR_INVALID_ARG
    assert q(1 << 30, 1 << 20, 1, F32, ctypes.byref(sz)) == ERR_UNSUPPORTED


def test_norm_binding_refusals():
    x, w = torch.zeros(6, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="y has shape"):
        mec.residual_norm(x, torch.zeros(5, 8))
    with pytest.raises(ValueError, match="gate has shape"):
        mec.residual_norm(x, x, gate=torch.zeros(2, 8), rows_per_gate=4 + 2)
    with pytest.raises(ValueError, match="rows_per_gate"):
        mec.residual_norm(x, x, gate=torch.zeros(2, 8), rows_per_gate=0)
    with pytest.raises(ValueError, match="w_pre has shape"):
        mec.residual_norm(x, x, w_pre=torch.zeros(7))
    with pytest.raises(TypeError, match="one dtype"):
        mec.residual_norm(x, x, w_pre=w.half())
    with pytest.raises(ValueError, match="CUDA"):
        mec.residual_norm(x, x, w_pre=w)


# ---------------------------------------------------------------- clipping
def clip_call(ptrs=(4096,), outs=(4096,), sizes=(10,), dts=(0,), max_norm=1.0, eps=1e-6, norm=64, ws=256,
              ws_bytes=1 << 20):
    k = len(sizes)
    arr = lambda t, v: None if v is None else (t * k)(*v)  # noqa: E731
    return mec.lib().im2win_clip_grad_norm(arr(ctypes.c_void_p, ptrs), arr(ctypes.c_void_p, outs),
                                           arr(ctypes.c_int64, sizes), arr(ctypes.c_int, dts), k, max_norm, eps, norm,
                                           ws, ws_bytes, None)


def test_clip_refusals():
    for kw in (dict(ptrs=None), dict(dts=None), dict(ptrs=(None,)), dict(outs=(None,)), dict(sizes=(-1,)),
               dict(dts=(3,)), dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(eps=-1.0), dict(norm=None)):
        assert clip_call(**kw) == ERR_INVALID_ARG, kw
    assert clip_call(ptrs=(4098,)) == ERR_MISALIGNED
    assert clip_call(outs=(4097,), dts=(1,)) == ERR_MISALIGNED
    assert clip_call(norm=66) == ERR_MISALIGNED
    assert clip_call(ws=264) == ERR_MISALIGNED
    assert clip_call(ws_bytes=8) == ERR_WORKSPACE
    assert clip_call(ws=None) == ERR_WORKSPACE
    assert clip_call(sizes=((1 << 40) + 1,)) == ERR_UNSUPPORTED


def test_clip_binding_refusals():
    g = torch.zeros(4)
    with pytest.raises(ValueError, match="no gradients"):
        mec.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError, match="outputs for"):
        mec.clip_grad_norm([g], 1.0, outs=[])
    with pytest.raises(ValueError, match=r"outs\[0\] has shape"):
        mec.clip_grad_norm([g], 1.0, outs=[torch.zeros(5)])
    with pytest.raises(ValueError, match="CUDA"):
        mec.clip_grad_norm([g], 1.0)


# ---------------------------------------------------------------- autograd
@pytest.mark.parametrize("which", range(4))
def test_ffn_refuses_what_autograd_would_lose(which):
    ts = [torch.zeros(4, 8), torch.zeros(16, 8), torch.zeros(16, 8), torch.zeros(8, 16)]
    ts[which].requires_grad_()
    for call in (mec.gated_ffn, mec.gated_ffn_train):
        with pytest.raises(ValueError, match="requires grad"):
            call(*ts)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # as any tensor without a GPU
            call(*ts)


@pytest.mark.parametrize("name", ["x", "y", "gate", "res_scale", "w_post", "b_post", "w_pre", "b_pre"])
def test_norm_refuses_what_autograd_would_lose(name):
    ts = dict(x=torch.zeros(6, 8), y=torch.zeros(6, 8), gate=torch.zeros(1, 8),
              **{k: torch.zeros(8) for k in ("res_scale", "w_post", "b_post", "w_pre", "b_pre")})
    ts[name].requires_grad_()
    with pytest.raises(ValueError, match="requires grad"):
        mec.residual_norm(**ts, post="layer", pre="layer")
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        mec.residual_norm(**ts, post="layer", pre="layer")


# ---------------------------------------------------------------- the references themselves
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "sigmoid", "relu"])
def test_ffn_reference_gradients(act):
    """The reference's gradients are those of its forward formula."""
    g = torch.Generator().manual_seed(0)
    x, wg, wu, wd = (torch.randn(*s, generator=g, dtype=torch.float64).requires_grad_()
                     for s in ((5, 6), (7, 6), (7, 6), (6, 7)))
    dy = torch.randn(5, 6, generator=g, dtype=torch.float64)
    ref.ffn(x, wg, wu, wd, act).backward(dy)
    with torch.no_grad():
        want = ref.ffn_all(x, wg, wu, wd, act, torch.float32, dy)
    for k, t in (("dx", x), ("dw_gate", wg), ("dw_up", wu), ("dw_down", wd)):
        assert torch.allclose(want[k][0], t.grad, rtol=1e-10, atol=1e-12), k


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
def test_norm_reference_gradients(post, pre):
    g = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64).requires_grad_()  # noqa: E731
    x, y = n(7, 5), n(7, 5)
    p = dict(post=post, pre=pre, eps=1e-3, rows_per_gate=3, gate=n(3, 5), res_scale=n(5),
             w_post=n(5) if post != "none" else None, b_post=n(5) if post == "layer" else None,
             w_pre=n(5) if pre != "none" else None, b_pre=n(5) if pre == "layer" else None)
    dr, dn = (torch.randn(7, 5, generator=g, dtype=torch.float64) for _ in range(2))
    r, nn = ref.residual_norm(x, y, p)
    ((r * dr).sum() + (0 if nn is None else (nn * dn).sum())).backward()
    with torch.no_grad():
        want = ref.residual_norm_all(x, y, p, torch.float32, dr, None if nn is None else dn, backward=True)
    for k, t in dict(x=x, y=y, **{k: v for k, v in p.items() if isinstance(v, torch.Tensor)}).items():
        assert torch.allclose(want["d" + k][0], t.grad, rtol=1e-9, atol=1e-11), k
