"""The residual block around a convolution: ctypes marshalling of the gated
feed-forward, the norms with gate and residual scale, and gradient clipping.

As in the convolutions' binding, the im2win_* functions take caller-allocated
outputs and map one to one onto the C entry points, the names without the prefix
allocate through torch, and nothing is computed here.
"""
from __future__ import annotations

import ctypes
import functools
import operator
from array import array

import torch

from ._binding import _DTYPE, _check, _cuda, _dtype_code, _same_device, lib

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


def _stream(device: int):
    """The current stream of a device, as an integer (a call costs a tenth of building a Stream object)."""
    return torch._C._cuda_getCurrentRawStream(device)


def _alike(dtype, device: int, *ts) -> bool:
    """Whether every tensor is contiguous, of one dtype and on one CUDA device. The
    calls test this first and look for what is wrong only where it fails: a small
    call costs less on the GPU than a full set of checks on the host."""
    if device < 0:
        return False
    for t in ts:
        if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
            return False
    return True


def _bytes(t):
    return t.numel() * t.element_size()


def _same_dtype(fn, *ts):
    for t in ts[1:]:
        if t.dtype != ts[0].dtype:
            raise TypeError(f"{fn}: every tensor must have one dtype ({ts[0].dtype} and {t.dtype} given)")


def _shape(fn, name, t, want):
    if tuple(t.shape) != tuple(want):
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(want)}")


def _unrecorded(fn, *ts):
    """Refuses tensors whose gradients would silently go missing: nothing here is recorded
    by autograd, the gradients are calls of their own."""
    if torch.is_grad_enabled():
        for t in ts:
            if t is not None and t.requires_grad:
                raise ValueError(f"{fn}: a tensor requires grad, but autograd does not record this call; make it under "
                                 "torch.no_grad() (its gradients are a call of their own) or detach the tensor")


def _empty(nbytes, device):
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- gated feed-forward
@functools.lru_cache(maxsize=4096)
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
    if not (C >= 1 and F >= 1 and w_gate.shape == w_up.shape == (F, C) and w_down.shape == (C, F)
            and _alike(x.dtype, x.get_device(), x, w_gate, w_up, w_down)):
        _shape(fn, "w_gate", w_gate, (F, C))
        _shape(fn, "w_up", w_up, (F, C))
        _shape(fn, "w_down", w_down, (C, F))
        if C < 1 or F < 1:
            raise ValueError(f"{fn}: C and F must be at least 1")
        _same_dtype(fn, x, w_gate, w_up, w_down)
        _same_device(fn, x, w_gate, w_up, w_down)
        _cuda(x, w_gate, w_up, w_down)
    return x.numel() // C, C, F


def _ffn(fn, dims, x, w_gate, w_up, w_down, y, saved, ws, act):
    """The call itself, on checked tensors."""
    _check(fn, lib().im2win_gated_ffn(
        x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), y.data_ptr(), _ptr(saved), ws.data_ptr(),
        _bytes(ws), *dims, _code(ACTS, act, "act"), _dtype_code(x), _stream(x.get_device())))


def _ffn_outputs(fn, dims, x, y, saved, ws):
    if not (y.shape == x.shape and _alike(x.dtype, x.get_device(), y)):
        _shape(fn, "y", y, x.shape)
        _same_dtype(fn, x, y)
    others = [y, ws] if saved is None else [y, ws, saved]
    _same_device(fn, x, *others)
    _cuda(*others)
    if saved is not None and _bytes(saved) < im2win_gated_ffn_size(FFN_SAVED, *dims, _dtype_code(x)):
        raise ValueError(f"{fn}: saved is too small")


def im2win_gated_ffn(x, w_gate, w_up, w_down, y, saved, ws, act: str = "silu") -> None:
    """y = (act(x w_gate^T) * (x w_up^T)) w_down^T; saved None: inference."""
    fn = "im2win_gated_ffn"
    dims = _ffn_shapes(fn, x, w_gate, w_up, w_down)
    _ffn_outputs(fn, dims, x, y, saved, ws)
    _ffn(fn, dims, x, w_gate, w_up, w_down, y, saved, ws, act)


def _ffn_backward(fn, dims, dy, x, w_gate, w_up, w_down, saved, dx, dw_gate, dw_up, dw_down, ws, act):
    _check(fn, lib().im2win_gated_ffn_backward(
        dy.data_ptr(), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), saved.data_ptr(), _ptr(dx),
        _ptr(dw_gate), _ptr(dw_up), _ptr(dw_down), ws.data_ptr(), _bytes(ws), *dims, _code(ACTS, act, "act"),
        _dtype_code(x), _stream(x.get_device())))


def _ffn_backward_inputs(fn, dims, dy, x, saved, ws):
    device = x.get_device()
    if not (dy.shape == x.shape and _alike(x.dtype, device, dy) and saved.get_device() == ws.get_device() == device
            and saved.is_contiguous() and ws.is_contiguous()):
        _shape(fn, "dy", dy, x.shape)
        _same_dtype(fn, x, dy)
        _same_device(fn, x, dy, saved, ws)
        _cuda(dy, saved, ws)
    if _bytes(saved) < im2win_gated_ffn_size(FFN_SAVED, *dims, _dtype_code(x)):
        raise ValueError(f"{fn}: saved is too small")


def im2win_gated_ffn_backward(dy, x, w_gate, w_up, w_down, saved, dx, dw_gate, dw_up, dw_down, ws,
                              act: str = "silu") -> None:
    """Gradients of im2win_gated_ffn; dx, or the three dw, may be None."""
    fn = "im2win_gated_ffn_backward"
    dims = _ffn_shapes(fn, x, w_gate, w_up, w_down)
    _ffn_backward_inputs(fn, dims, dy, x, saved, ws)
    for name, t, like in (("dx", dx, x), ("dw_gate", dw_gate, w_gate), ("dw_up", dw_up, w_up), ("dw_down", dw_down, w_down)):
        if t is not None:
            _shape(fn, name, t, like.shape)
            _same_dtype(fn, x, t)
            _same_device(fn, x, t)
            _cuda(t)
    _ffn_backward(fn, dims, dy, x, w_gate, w_up, w_down, saved, dx, dw_gate, dw_up, dw_down, ws, act)


def _ffn_buffer(buffer, dims, x):
    return _empty(im2win_gated_ffn_size(buffer, *dims, _dtype_code(x)), x.device)


def _ffn_forward(fn, x, w_gate, w_up, w_down, act, ws, out, saved, train):
    _unrecorded(fn, x, w_gate, w_up, w_down)
    dims = _ffn_shapes(fn, x, w_gate, w_up, w_down)
    given = ws is not None or out is not None or saved is not None
    if ws is None:
        ws = _ffn_buffer(FFN_TRAIN if train else FFN_FORWARD, dims, x)
    if saved is None and train:
        saved = _ffn_buffer(FFN_SAVED, dims, x)
    if out is None:
        out = torch.empty_like(x)
    if given:
        _ffn_outputs(fn, dims, x, out, saved, ws)
    _ffn(fn, dims, x, w_gate, w_up, w_down, out, saved, ws, act)
    return out, saved


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, act: str = "silu",
              ws: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Gated feed-forward block over the last axis of x[..., C]. Autograd does not record it:
    tensors that require grad are refused outside of torch.no_grad()."""
    return _ffn_forward("gated_ffn", x, w_gate, w_up, w_down, act, ws, out, None, False)[0]


def gated_ffn_train(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                    act: str = "silu", ws: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    saved: torch.Tensor | None = None):
    """gated_ffn() and the buffer its gated_ffn_backward() needs: (y, saved)."""
    return _ffn_forward("gated_ffn_train", x, w_gate, w_up, w_down, act, ws, out, saved, True)


def gated_ffn_backward(dy: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                       w_down: torch.Tensor, saved: torch.Tensor, act: str = "silu", ws: torch.Tensor | None = None,
                       need_dx: bool = True, need_dw: bool = True):
    """(dx, dw_gate, dw_up, dw_down) of gated_ffn_train() at the same arguments;
    None for what is not needed."""
    fn = "gated_ffn_backward"
    dims = _ffn_shapes(fn, x, w_gate, w_up, w_down)
    if ws is None:
        ws = _ffn_buffer(FFN_BACKWARD, dims, x)
    _ffn_backward_inputs(fn, dims, dy, x, saved, ws)
    dx = torch.empty_like(x) if need_dx else None
    dws = [torch.empty_like(w) if need_dw else None for w in (w_gate, w_up, w_down)]
    _ffn_backward(fn, dims, dy, x, w_gate, w_up, w_down, saved, dx, *dws, ws, act)
    return (dx, *dws)


# ---------------------------------------------------------------- norms, gate and residual scale
_NORM_PARAMS = ("res_scale", "w_post", "b_post", "w_pre", "b_pre")


def _norm_check(fn, x, y, gate, rows_per_gate, rows, params):
    """(R, C, rows a gate) after the checks of a call's tensors; rows are (name,
    tensor or None) of x's shape, params the tensors of _NORM_PARAMS."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"{fn}: x must be [..., C]")
    shape = x.shape
    C = shape[-1]
    R = x.numel() // C
    if gate is None or rows_per_gate is None:
        rows_per_gate = max(R, 1)
    elif rows_per_gate < 1:
        raise ValueError(f"{fn}: rows_per_gate must be at least 1")
    if y is not None:
        rows = (("y", y), *rows)
    given = [t for _, t in rows if t is not None]
    for t in given:
        if t.shape != shape:
            for name, v in rows:
                if v is not None:
                    _shape(fn, name, v, shape)
    if gate is not None:
        _shape(fn, "gate", gate, (-(-R // rows_per_gate), C))
        given.append(gate)
    for name, t in zip(_NORM_PARAMS, params):
        if t is not None:
            _shape(fn, name, t, (C,))
            given.append(t)
    if not _alike(x.dtype, x.get_device(), x, *given):
        _same_dtype(fn, x, *given)
        _same_device(fn, x, *given)
        _cuda(x, *given)
    return R, C, rows_per_gate


def _norm_args(dims, x, y, gate, res_scale, post, w_post, b_post, pre, w_pre, b_pre, eps):
    return (x.data_ptr(), _ptr(y), _ptr(gate), dims[2], _ptr(res_scale), _code(NORMS, post, "post"), _ptr(w_post),
            _ptr(b_post), _code(NORMS, pre, "pre"), _ptr(w_pre), _ptr(b_pre), eps)


def _norm(fn, dims, args, x, r, n):
    _check(fn, lib().im2win_residual_norm(*args, _ptr(r), _ptr(n), dims[0], dims[1], _dtype_code(x),
                                          _stream(x.get_device())))


def im2win_residual_norm(x, y, gate, rows_per_gate, res_scale, post, w_post, b_post, pre, w_pre, b_pre, eps, r,
                         n) -> None:
    """r = res_scale * x + gate * post(y), n = pre(r); None: absent."""
    fn = "im2win_residual_norm"
    dims = _norm_check(fn, x, y, gate, rows_per_gate, (("r", r), ("n", n)), (res_scale, w_post, b_post, w_pre, b_pre))
    _norm(fn, dims, _norm_args(dims, x, y, gate, res_scale, post, w_post, b_post, pre, w_pre, b_pre, eps), x, r, n)


@functools.lru_cache(maxsize=4096)
def im2win_residual_norm_backward_size(R, C, rows_per_gate, dtype: int) -> int:
    out = ctypes.c_size_t(0)
    _check("im2win_residual_norm_backward_size",
           lib().im2win_residual_norm_backward_size(R, C, rows_per_gate, dtype, ctypes.byref(out)))
    return out.value


def _norm_backward(fn, dims, args, dr, dn, x, grads, ws):
    _check(fn, lib().im2win_residual_norm_backward(
        _ptr(dr), _ptr(dn), *args, *[_ptr(t) for t in grads], ws.data_ptr(), _bytes(ws), dims[0], dims[1],
        _dtype_code(x), _stream(x.get_device())))


def im2win_residual_norm_backward(dr, dn, x, y, gate, rows_per_gate, res_scale, post, w_post, b_post, pre, w_pre,
                                  b_pre, eps, dx, dy, dgate, dres_scale, dw_post, db_post, dw_pre, db_pre, ws) -> None:
    """Gradients of im2win_residual_norm; None: an absent input, or a gradient not computed."""
    fn = "im2win_residual_norm_backward"
    dims = _norm_check(fn, x, y, gate, rows_per_gate, (("dr", dr), ("dn", dn), ("dx", dx), ("dy", dy)),
                       (res_scale, w_post, b_post, w_pre, b_pre))
    grads = (dx, dy, dgate, dres_scale, dw_post, db_post, dw_pre, db_pre)
    for name, t, want in (("dgate", dgate, None if gate is None else gate.shape), ("dres_scale", dres_scale, dims[1:2]),
                          ("dw_post", dw_post, dims[1:2]), ("db_post", db_post, dims[1:2]),
                          ("dw_pre", dw_pre, dims[1:2]), ("db_pre", db_pre, dims[1:2])):
        if t is not None:
            if want is not None:
                _shape(fn, name, t, want)
            _same_dtype(fn, x, t)
            _same_device(fn, x, t)
            _cuda(t)
    _same_device(fn, x, ws)
    _cuda(ws)
    _norm_backward(fn, dims, _norm_args(dims, x, y, gate, res_scale, post, w_post, b_post, pre, w_pre, b_pre, eps), dr,
                   dn, x, grads, ws)


def residual_norm(x: torch.Tensor, y: torch.Tensor | None = None, *, post: str = "none", w_post=None, b_post=None,
                  gate=None, rows_per_gate: int | None = None, res_scale=None, pre: str = "rms", w_pre=None,
                  b_pre=None, eps: float = 1e-6):
    """(r, n) of r = res_scale * x + gate * post(y), n = pre(r) over the last
    axis; n is None where pre is "none". gate[i] belongs to rows_per_gate
    consecutive rows (None: all rows). y None: r = res_scale * x. Autograd does not
    record it: tensors that require grad are refused outside of torch.no_grad()."""
    fn = "residual_norm"
    _unrecorded(fn, x, y, gate, res_scale, w_post, b_post, w_pre, b_pre)
    dims = _norm_check(fn, x, y, gate, rows_per_gate, (), (res_scale, w_post, b_post, w_pre, b_pre))
    r = torch.empty_like(x)
    n = torch.empty_like(x) if pre != "none" else None
    _norm(fn, dims, _norm_args(dims, x, y, gate, res_scale, post, w_post, b_post, pre, w_pre, b_pre, eps), x, r, n)
    return r, n


def residual_norm_backward(dr, dn, x: torch.Tensor, y: torch.Tensor | None = None, *, post: str = "none",
                           w_post=None, b_post=None, gate=None, rows_per_gate: int | None = None, res_scale=None,
                           pre: str = "rms", w_pre=None, b_pre=None, eps: float = 1e-6,
                           ws: torch.Tensor | None = None) -> dict:
    """Gradients of residual_norm() at the same arguments, as a dict of dx, dy,
    dgate, dres_scale, dw_post, db_post, dw_pre, db_pre (None for an absent input)."""
    fn = "residual_norm_backward"
    dims = _norm_check(fn, x, y, gate, rows_per_gate, (("dr", dr), ("dn", dn)), (res_scale, w_post, b_post, w_pre, b_pre))
    if ws is None:
        ws = _empty(im2win_residual_norm_backward_size(*dims, _dtype_code(x)), x.device)
    else:
        _same_device(fn, x, ws)
        _cuda(ws)
    like = dict(dx=x, dy=y, dgate=gate, dres_scale=res_scale, dw_post=w_post, db_post=b_post, dw_pre=w_pre,
                db_pre=b_pre)
    out = {k: None if v is None else torch.empty_like(v) for k, v in like.items()}
    _norm_backward(fn, dims, _norm_args(dims, x, y, gate, res_scale, post, w_post, b_post, pre, w_pre, b_pre, eps), dr,
                   dn, x, out.values(), ws)
    return out


# ---------------------------------------------------------------- gradient clipping
# Lists go through map() and array: a list of hundreds costs more on the host than on the GPU.
_dtype_of, _shape_of = operator.attrgetter("dtype"), operator.attrgetter("shape")
_pointer, _device_of, _contiguous = torch.Tensor.data_ptr, torch.Tensor.get_device, torch.Tensor.is_contiguous


def _address(values):
    return values.buffer_info()[0]


def im2win_clip_grad_norm_size(sizes) -> int:
    out = ctypes.c_size_t(0)
    sizes = sizes if isinstance(sizes, array) else array("q", sizes)
    _check("im2win_clip_grad_norm_size",
           lib().im2win_clip_grad_norm_size(_address(sizes), len(sizes), ctypes.byref(out)))
    return out.value


def _clip_check(fn, grads, outs, device: int):
    """The gradients' dtype codes after the checks of the lists."""
    given, dtypes = grads, list(map(_dtype_of, grads))
    if outs is not None and outs is not grads:
        if len(outs) != len(grads):
            raise ValueError(f"{fn}: {len(outs)} outputs for {len(grads)} gradients")
        if list(map(_shape_of, outs)) != list(map(_shape_of, grads)) or list(map(_dtype_of, outs)) != dtypes:
            for i, (g, o) in enumerate(zip(grads, outs)):
                _shape(fn, f"outs[{i}]", o, g.shape)
                _same_dtype(fn, g, o)
        given = grads + outs
    if device < 0 or not all(map(_contiguous, given)) or any(map(device.__ne__, map(_device_of, given))):
        _cuda(*given)
        _same_device(fn, *given)
        raise ValueError(f"{fn}: every tensor must be on one device")
    try:
        return array("i", map(_DTYPE.__getitem__, dtypes))
    except KeyError:
        return [_dtype_code(t) for t in grads]  # raises


def _counts(grads):
    return array("q", map(torch.Tensor.numel, grads))


def _clip(fn, grads, outs, counts, codes, max_norm, eps, norm, ws):
    at = array("Q", map(_pointer, grads))
    to = None if outs is None else at if outs is grads else array("Q", map(_pointer, outs))
    _check(fn, lib().im2win_clip_grad_norm(
        _address(at), None if to is None else _address(to), _address(counts), _address(codes), len(grads), max_norm, eps,
        norm.data_ptr(), ws.data_ptr(), _bytes(ws), _stream(norm.get_device())))


def im2win_clip_grad_norm(grads, outs, max_norm: float, eps: float, norm, ws) -> None:
    """*norm = the gradients' global 2-norm; outs[i] = grads[i] * min(1, max_norm / (norm + eps)); outs None: the
    norm alone."""
    fn = "im2win_clip_grad_norm"
    grads = list(grads)
    outs = None if outs is None else list(outs)
    if norm.dtype != torch.float32 or norm.numel() != 1:
        raise ValueError(f"{fn}: norm must be one float32")
    _same_device(fn, norm, ws)
    _cuda(norm, ws)
    codes = _clip_check(fn, grads, outs, norm.get_device())
    _clip(fn, grads, outs, _counts(grads), codes, max_norm, eps, norm, ws)


def _clip_lists(fn, grads, outs, max_norm, eps, ws):
    if not grads:
        raise ValueError(f"{fn}: no gradients")
    codes = _clip_check(fn, grads, outs, grads[0].get_device())
    counts = _counts(grads)
    device = grads[0].device
    if ws is None:
        ws = _empty(im2win_clip_grad_norm_size(counts), device)
    else:
        _same_device(fn, grads[0], ws)
        _cuda(ws)
    norm = torch.empty((), dtype=torch.float32, device=device)
    _clip(fn, grads, outs, counts, codes, max_norm, eps, norm, ws)
    return norm


def clip_grad_norm(grads, max_norm: float, outs=None, eps: float = 1e-6, ws: torch.Tensor | None = None):
    """Scale the gradients by min(1, max_norm / (norm + eps)), in place or into
    `outs`, and return their global 2-norm (a float32 scalar on the device)."""
    grads = list(grads)
    return _clip_lists("clip_grad_norm", grads, grads if outs is None else list(outs), max_norm, eps, ws)


def grad_norm(grads, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Global 2-norm of the gradients (a float32 scalar on the device)."""
    return _clip_lists("grad_norm", list(grads), None, 0.0, 0.0, ws)
