"""The residual block around a convolution: ctypes marshalling of the gated
feed-forward, the norms with gate and residual scale, and gradient clipping.

As in the convolutions' binding, the im2win_* functions take caller-allocated
outputs and map one to one onto the C entry points, the names without the prefix
allocate through torch, and nothing is computed here.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as _b
from ._binding import _check, _cuda, _dtype_code, _same_device, _stream, lib

ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3, "sigmoid": 4}
NORMS = {"none": 0, "rms": 1, "layer": 2}
FFN_FORWARD, FFN_TRAIN, FFN_BACKWARD, FFN_SAVED = 0, 1, 2, 3


def _code(table, name, what):
    try:
        return table[name]
    except KeyError:
        raise ValueError(f"{what} must be one of {', '.join(table)}; got {name!r}") from None


def _ptr(t):
    return None if t is None else t.data_ptr()


def _bytes(t):
    return t.numel() * t.element_size()


def _same_dtype(fn, *ts):
    for t in ts[1:]:
        if t.dtype != ts[0].dtype:
            raise TypeError(f"{fn}: every tensor must have one dtype ({ts[0].dtype} and {t.dtype} given)")


def _shape(fn, name, t, want):
    if tuple(t.shape) != tuple(want):
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(want)}")


def _empty(nbytes, device):
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- gated feed-forward
def im2win_gated_ffn_size(buffer: int, R, C, F, dtype: int) -> int:
    out = ctypes.c_size_t(0)
    _check("im2win_gated_ffn_size", lib().im2win_gated_ffn_size(buffer, R, C, F, dtype, ctypes.byref(out)))
    return out.value


def _ffn_shapes(fn, x, w_gate, w_up, w_down):
    """(R, C, F) after the shape, type and device checks of the inputs; x is
    [..., C] with its leading axes as rows."""
    if x.dim() < 1 or w_gate.dim() != 2:
        raise ValueError(f"{fn}: x must be [..., C] and w_gate [F, C]")
    C, F = x.shape[-1], w_gate.shape[0]
    _shape(fn, "w_gate", w_gate, (F, C))
    _shape(fn, "w_up", w_up, (F, C))
    _shape(fn, "w_down", w_down, (C, F))
    if C < 1 or F < 1:
        raise ValueError(f"{fn}: C and F must be at least 1")
    _same_dtype(fn, x, w_gate, w_up, w_down)
    _same_device(fn, x, w_gate, w_up, w_down)
    _cuda(x, w_gate, w_up, w_down)
    return x.numel() // C, C, F


def im2win_gated_ffn(x, w_gate, w_up, w_down, y, saved, ws, act: str = "silu") -> None:
    """y = (act(x w_gate^T) * (x w_up^T)) w_down^T; saved None: inference."""
    fn = "im2win_gated_ffn"
    R, C, F = _ffn_shapes(fn, x, w_gate, w_up, w_down)
    _shape(fn, "y", y, x.shape)
    _same_dtype(fn, x, y)
    _same_device(fn, x, y, ws, *([] if saved is None else [saved]))
    _cuda(y, ws, *([] if saved is None else [saved]))
    code = _dtype_code(x)
    if saved is not None and _bytes(saved) < im2win_gated_ffn_size(FFN_SAVED, R, C, F, code):
        raise ValueError(f"{fn}: saved is too small")
    _check(fn, lib().im2win_gated_ffn(_ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(y), _ptr(saved), _ptr(ws),
                                      _bytes(ws), R, C, F, _code(ACTS, act, "act"), code, _stream(x)))


def im2win_gated_ffn_backward(dy, x, w_gate, w_up, w_down, saved, dx, dw_gate, dw_up, dw_down, ws,
                              act: str = "silu") -> None:
    """Gradients of im2win_gated_ffn; dx, or the three dw, may be None."""
    fn = "im2win_gated_ffn_backward"
    R, C, F = _ffn_shapes(fn, x, w_gate, w_up, w_down)
    _shape(fn, "dy", dy, x.shape)
    outs = [t for t in (dx, dw_gate, dw_up, dw_down) if t is not None]
    for name, t, like in (("dx", dx, x), ("dw_gate", dw_gate, w_gate), ("dw_up", dw_up, w_up), ("dw_down", dw_down, w_down)):
        if t is not None:
            _shape(fn, name, t, like.shape)
    _same_dtype(fn, x, dy, *outs)
    _same_device(fn, x, dy, saved, ws, *outs)
    _cuda(dy, saved, ws, *outs)
    code = _dtype_code(x)
    if _bytes(saved) < im2win_gated_ffn_size(FFN_SAVED, R, C, F, code):
        raise ValueError(f"{fn}: saved is too small")
    _check(fn, lib().im2win_gated_ffn_backward(
        _ptr(dy), _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(saved), _ptr(dx), _ptr(dw_gate), _ptr(dw_up),
        _ptr(dw_down), _ptr(ws), _bytes(ws), R, C, F, _code(ACTS, act, "act"), code, _stream(x)))


def _ffn_buffer(buffer, x, w_gate):
    C = x.shape[-1]
    return _empty(im2win_gated_ffn_size(buffer, x.numel() // max(C, 1), C, w_gate.shape[0], _dtype_code(x)), x.device)


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, act: str = "silu",
              ws: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Gated feed-forward block over the last axis of x[..., C]."""
    _ffn_shapes("gated_ffn", x, w_gate, w_up, w_down)
    if ws is None:
        ws = _ffn_buffer(FFN_FORWARD, x, w_gate)
    if out is None:
        out = torch.empty_like(x)
    im2win_gated_ffn(x, w_gate, w_up, w_down, out, None, ws, act)
    return out


def gated_ffn_train(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                    act: str = "silu", ws: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    saved: torch.Tensor | None = None):
    """gated_ffn() and the buffer its gated_ffn_backward() needs: (y, saved)."""
    _ffn_shapes("gated_ffn_train", x, w_gate, w_up, w_down)
    if ws is None:
        ws = _ffn_buffer(FFN_TRAIN, x, w_gate)
    if saved is None:
        saved = _ffn_buffer(FFN_SAVED, x, w_gate)
    if out is None:
        out = torch.empty_like(x)
    im2win_gated_ffn(x, w_gate, w_up, w_down, out, saved, ws, act)
    return out, saved


def gated_ffn_backward(dy: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                       w_down: torch.Tensor, saved: torch.Tensor, act: str = "silu", ws: torch.Tensor | None = None,
                       need_dx: bool = True, need_dw: bool = True):
    """(dx, dw_gate, dw_up, dw_down) of gated_ffn_train() at the same arguments;
    None for what is not needed."""
    _ffn_shapes("gated_ffn_backward", x, w_gate, w_up, w_down)
    if ws is None:
        ws = _ffn_buffer(FFN_BACKWARD, x, w_gate)
    dx = torch.empty_like(x) if need_dx else None
    dws = [torch.empty_like(w) if need_dw else None for w in (w_gate, w_up, w_down)]
    im2win_gated_ffn_backward(dy, x, w_gate, w_up, w_down, saved, dx, *dws, ws, act)
    return (dx, *dws)


# ---------------------------------------------------------------- norms, gate and residual scale
_NORM_PARAMS = ("res_scale", "w_post", "b_post", "w_pre", "b_pre")


def _norm_check(fn, x, y, gate, rows_per_gate, outs, params):
    """(R, C, rows a gate) after the checks of a call's tensors; outs are
    (name, tensor or None, shape)."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"{fn}: x must be [..., C]")
    C = x.shape[-1]
    R = x.numel() // C
    if y is not None:
        _shape(fn, "y", y, x.shape)
    if gate is not None:
        if rows_per_gate is None:
            rows_per_gate = max(R, 1)
        if rows_per_gate < 1:
            raise ValueError(f"{fn}: rows_per_gate must be at least 1")
        _shape(fn, "gate", gate, (-(-R // rows_per_gate), C))
    else:
        rows_per_gate = max(R, 1)
    for name, t in zip(_NORM_PARAMS, params):
        if t is not None:
            _shape(fn, name, t, (C,))
    for name, t, want in outs:
        if t is not None:
            _shape(fn, name, t, want)
    given = [t for t in (x, y, gate, *params, *(t for _, t, _ in outs)) if t is not None]
    _same_dtype(fn, *given)
    _same_device(fn, *given)
    _cuda(*given)
    return R, C, rows_per_gate


def im2win_residual_norm(x, y, gate, rows_per_gate, res_scale, post, w_post, b_post, pre, w_pre, b_pre, eps, r,
                         n) -> None:
    """r = res_scale * x + gate * post(y), n = pre(r); None: absent."""
    fn = "im2win_residual_norm"
    R, C, per = _norm_check(fn, x, y, gate, rows_per_gate, (("r", r, x.shape), ("n", n, x.shape)),
                            (res_scale, w_post, b_post, w_pre, b_pre))
    _check(fn, lib().im2win_residual_norm(
        _ptr(x), _ptr(y), _ptr(gate), per, _ptr(res_scale), _code(NORMS, post, "post"), _ptr(w_post), _ptr(b_post),
        _code(NORMS, pre, "pre"), _ptr(w_pre), _ptr(b_pre), eps, _ptr(r), _ptr(n), R, C, _dtype_code(x), _stream(x)))


def im2win_residual_norm_backward_size(R, C, rows_per_gate, dtype: int) -> int:
    out = ctypes.c_size_t(0)
    _check("im2win_residual_norm_backward_size",
           lib().im2win_residual_norm_backward_size(R, C, rows_per_gate, dtype, ctypes.byref(out)))
    return out.value


def im2win_residual_norm_backward(dr, dn, x, y, gate, rows_per_gate, res_scale, post, w_post, b_post, pre, w_pre,
                                  b_pre, eps, dx, dy, dgate, dres_scale, dw_post, db_post, dw_pre, db_pre, ws) -> None:
    """Gradients of im2win_residual_norm; None: an absent input, or a gradient not computed."""
    fn = "im2win_residual_norm_backward"
    outs = [("dr", dr, x.shape), ("dn", dn, x.shape), ("dx", dx, x.shape), ("dy", dy, x.shape)]
    if dgate is not None and gate is not None:
        outs.append(("dgate", dgate, gate.shape))
    outs += [(name, t, x.shape[-1:]) for name, t in (("dres_scale", dres_scale), ("dw_post", dw_post),
                                                     ("db_post", db_post), ("dw_pre", dw_pre), ("db_pre", db_pre))]
    R, C, per = _norm_check(fn, x, y, gate, rows_per_gate, outs, (res_scale, w_post, b_post, w_pre, b_pre))
    _same_device(fn, x, ws)
    _cuda(ws)
    _check(fn, lib().im2win_residual_norm_backward(
        _ptr(dr), _ptr(dn), _ptr(x), _ptr(y), _ptr(gate), per, _ptr(res_scale), _code(NORMS, post, "post"),
        _ptr(w_post), _ptr(b_post), _code(NORMS, pre, "pre"), _ptr(w_pre), _ptr(b_pre), eps, _ptr(dx), _ptr(dy),
        _ptr(dgate), _ptr(dres_scale), _ptr(dw_post), _ptr(db_post), _ptr(dw_pre), _ptr(db_pre), _ptr(ws), _bytes(ws),
        R, C, _dtype_code(x), _stream(x)))


def residual_norm(x: torch.Tensor, y: torch.Tensor | None = None, *, post: str = "none", w_post=None, b_post=None,
                  gate=None, rows_per_gate: int | None = None, res_scale=None, pre: str = "rms", w_pre=None,
                  b_pre=None, eps: float = 1e-6):
    """(r, n) of r = res_scale * x + gate * post(y), n = pre(r) over the last
    axis; n is None where pre is "none". gate[i] belongs to rows_per_gate
    consecutive rows (None: all rows). y None: r = res_scale * x."""
    r = torch.empty_like(x)
    n = torch.empty_like(x) if pre != "none" else None
    im2win_residual_norm(x, y, gate, rows_per_gate, res_scale, post, w_post, b_post, pre, w_pre, b_pre, eps, r, n)
    return r, n


def residual_norm_backward(dr, dn, x: torch.Tensor, y: torch.Tensor | None = None, *, post: str = "none",
                           w_post=None, b_post=None, gate=None, rows_per_gate: int | None = None, res_scale=None,
                           pre: str = "rms", w_pre=None, b_pre=None, eps: float = 1e-6,
                           ws: torch.Tensor | None = None) -> dict:
    """Gradients of residual_norm() at the same arguments, as a dict of dx, dy,
    dgate, dres_scale, dw_post, db_post, dw_pre, db_pre (None for an absent input)."""
    fn = "residual_norm_backward"
    R, C, per = _norm_check(fn, x, y, gate, rows_per_gate, (("dr", dr, x.shape), ("dn", dn, x.shape)),
                            (res_scale, w_post, b_post, w_pre, b_pre))
    if ws is None:
        ws = _empty(im2win_residual_norm_backward_size(R, C, per, _dtype_code(x)), x.device)
    like = dict(dx=x, dy=y, dgate=gate, dres_scale=res_scale, dw_post=w_post, db_post=b_post, dw_pre=w_pre,
                db_pre=b_pre)
    out = {k: None if v is None else torch.empty_like(v) for k, v in like.items()}
    im2win_residual_norm_backward(dr, dn, x, y, gate, rows_per_gate, res_scale, post, w_post, b_post, pre, w_pre,
                                  b_pre, eps, *out.values(), ws)
    return out


# ---------------------------------------------------------------- gradient clipping
def im2win_clip_grad_norm_size(sizes) -> int:
    out = ctypes.c_size_t(0)
    arr = (ctypes.c_int64 * len(sizes))(*sizes)
    _check("im2win_clip_grad_norm_size", lib().im2win_clip_grad_norm_size(arr, len(sizes), ctypes.byref(out)))
    return out.value


def im2win_clip_grad_norm(grads, outs, max_norm: float, eps: float, norm, ws) -> None:
    """*norm = the gradients' global 2-norm; outs[i] = grads[i] * min(1, max_norm / (norm + eps)); outs None: the
    norm alone."""
    fn = "im2win_clip_grad_norm"
    grads = list(grads)
    outs = None if outs is None else list(outs)
    if outs is not None:
        if len(outs) != len(grads):
            raise ValueError(f"{fn}: {len(outs)} outputs for {len(grads)} gradients")
        for i, (g, o) in enumerate(zip(grads, outs)):
            if o is not g:
                _shape(fn, f"outs[{i}]", o, g.shape)
                _same_dtype(fn, g, o)
    if norm.dtype != torch.float32 or norm.numel() != 1:
        raise ValueError(f"{fn}: norm must be one float32")
    given = grads + (outs or [])
    _same_device(fn, norm, ws, *given)
    _cuda(norm, ws, *given)
    k = len(grads)
    vps, i64s, ints = ctypes.c_void_p * k, ctypes.c_int64 * k, ctypes.c_int * k
    _check(fn, lib().im2win_clip_grad_norm(
        vps(*[g.data_ptr() for g in grads]), None if outs is None else vps(*[o.data_ptr() for o in outs]),
        i64s(*[g.numel() for g in grads]), ints(*[_dtype_code(g) for g in grads]), k, max_norm, eps, _ptr(norm), _ptr(ws),
        _bytes(ws), _stream(norm)))


def _clip(grads, outs, max_norm, eps, ws, device):
    if ws is None:
        ws = _empty(im2win_clip_grad_norm_size([g.numel() for g in grads]), device)
    norm = torch.empty((), dtype=torch.float32, device=device)
    im2win_clip_grad_norm(grads, outs, max_norm, eps, norm, ws)
    return norm


def clip_grad_norm(grads, max_norm: float, outs=None, eps: float = 1e-6, ws: torch.Tensor | None = None):
    """Scale the gradients by min(1, max_norm / (norm + eps)), in place or into
    `outs`, and return their global 2-norm (a float32 scalar on the device)."""
    grads = list(grads)
    if not grads:
        raise ValueError("clip_grad_norm: no gradients")
    return _clip(grads, grads if outs is None else list(outs), max_norm, eps, ws, grads[0].device)


def grad_norm(grads, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Global 2-norm of the gradients (a float32 scalar on the device)."""
    grads = list(grads)
    if not grads:
        raise ValueError("grad_norm: no gradients")
    return _clip(grads, None, 0.0, 0.0, ws, grads[0].device)
