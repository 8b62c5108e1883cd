"""A block of experts: ctypes marshalling of the router and of the gated feed-forward
grouped by expert.

As in block.py, the im2win_* functions take caller-allocated outputs and map one to
one onto the C entry points, the names without the prefix allocate through torch,
and nothing is computed here.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from ._binding import _check, _cuda, _dtype_code, _same_device, lib
from .block import (
    ACTS, FFN_BACKWARD, FFN_FORWARD, FFN_SAVED, FFN_TRAIN, _alike, _bytes, _code, _count, _ptr, _same_dtype, _shape,
    _stream, _unrecorded)

ROUTES = {"top": 0, "all": 1}


def _experts(fn, experts, like, shape):
    """Checks an index tensor of a call on like's device."""
    if experts.shape != shape:
        _shape(fn, "experts", experts, shape)
    if experts.dtype is not torch.int32:
        raise TypeError(f"{fn}: experts must be int32, got {experts.dtype}")
    if experts.get_device() != like.get_device() or not experts.is_contiguous() or not experts.is_cuda:
        _same_device(fn, like, experts)
        _cuda(experts)


def _same(fn, x, *ts):
    if not _alike(x.dtype, x.get_device(), x, *ts):
        _same_dtype(fn, x, *ts)
        _same_device(fn, x, *ts)
        _cuda(x, *ts)


# ---------------------------------------------------------------- router
# (2.0 hashes as 2, and an answer holds what it was asked with: callers pass ints alone)
@functools.lru_cache(maxsize=4096, typed=True)
def _route_plan(shape, k, over):
    """(T, E, the code of over, the choices' shape) of logits' shape; ValueError where they do not fit."""
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError("logits must be [..., E]")
    E = shape[-1]
    if not 1 <= k <= E:
        raise ValueError(f"k must be between 1 and {E}, the number of experts; got {k}")
    return math.prod(shape[:-1]), E, _code(ROUTES, over, "over"), (*shape[:-1], k)


def _route_dims(fn, logits, k, over):
    if type(k) is not int:
        k = _count(fn, "k", k)
    try:
        return _route_plan(logits.shape, k, over)
    except ValueError as e:
        raise ValueError(f"{fn}: {e}") from None


def im2win_expert_route(logits, weights, experts, over: str = "top") -> None:
    """experts = the indexes of the k largest logits of each row, weights = their softmax weights."""
    fn = "im2win_expert_route"
    k = weights.shape[-1] if weights.dim() else 0
    T, E, code, shape = _route_dims(fn, logits, k, over)
    _shape(fn, "weights", weights, shape)
    _same(fn, logits, weights)
    _experts(fn, experts, logits, shape)
    _route(fn, T, E, k, code, logits, weights, experts)


def im2win_expert_route_backward(dweights, logits, experts, dlogits, over: str = "top") -> None:
    """dlogits from dweights at the same logits and the experts chosen there."""
    fn = "im2win_expert_route_backward"
    _shape(fn, "dlogits", dlogits, logits.shape)
    _same(fn, logits, dlogits)
    _route_backward(fn, dweights, logits, experts, dlogits, over)


def _route(fn, T, E, k, code, logits, weights, experts):
    _check(fn, lib().im2win_expert_route(logits.data_ptr(), weights.data_ptr(), experts.data_ptr(), T, E, k, code,
                                         _dtype_code(logits), _stream(logits.get_device())))


def _route_backward(fn, dweights, logits, experts, dlogits, over):
    k = dweights.shape[-1] if dweights.dim() else 0
    T, E, code, shape = _route_dims(fn, logits, k, over)
    if dweights.shape != shape:
        _shape(fn, "dweights", dweights, shape)
    _same(fn, logits, dweights)
    _experts(fn, experts, logits, shape)
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    _check(fn, lib().im2win_expert_route_backward(
        dweights.data_ptr(), logits.data_ptr(), experts.data_ptr(), dlogits.data_ptr(), T, E, k, code, _dtype_code(logits),
        _stream(logits.get_device())))
    return dlogits


def expert_route(logits: torch.Tensor, k: int, over: str = "top"):
    """(weights, experts), [..., k] each, of logits[..., E]: the k largest of a row by falling value, equal
    ones by rising index (int32), and their softmax weights over the k choices ("top") or over all
    experts ("all"). A logit of -inf is an expert the row may not take; places left over have expert -1
    and weight 0. Autograd does not record it: tensors that require grad are refused outside of
    torch.no_grad()."""
    fn = "expert_route"
    if logits.requires_grad:
        _unrecorded(fn, logits)
    T, E, code, shape = _route_dims(fn, logits, k, over)
    if not (logits.is_cuda and logits.is_contiguous()):
        _cuda(logits)
    weights = torch.empty(shape, dtype=logits.dtype, device=logits.device)
    experts = torch.empty_like(weights, dtype=torch.int32)
    _route(fn, T, E, k, code, logits, weights, experts)
    return weights, experts


def expert_route_backward(dweights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, over: str = "top"):
    """dlogits of expert_route() at the same logits and over, and the experts it chose: its own list, also where
    places were dropped (-1) from a copy of it before expert_ffn(), whose dweights are zero there. A list with
    -1 in place of a chosen expert would make the other places' softmax over "top" another one."""
    return _route_backward("expert_route_backward", dweights, logits, experts, None, over)


# ---------------------------------------------------------------- feed-forward
@functools.lru_cache(maxsize=4096)
def im2win_expert_ffn_size(buffer: int, T, k, E, C, F, dtype: int) -> int:
    out = ctypes.c_size_t(0)
    _check("im2win_expert_ffn_size", lib().im2win_expert_ffn_size(buffer, T, k, E, C, F, dtype, ctypes.byref(out)))
    return out.value


@functools.lru_cache(maxsize=4096)
def _ffn_plan(x, weights, w_gate, w_up, w_down):
    """(T, k, E, C, F) of the tensors' shapes; ValueError where they do not fit."""
    if len(x) < 1 or len(weights) < 1 or len(w_gate) != 3:
        raise ValueError("x must be [..., C], weights [..., k] and w_gate [E, F, C]")
    C, k = x[-1], weights[-1]
    E, F = w_gate[:2]
    for name, shape, want in (("weights", weights, (*x[:-1], k)), ("w_gate", w_gate, (E, F, C)), ("w_up", w_up, (E, F, C)),
                              ("w_down", w_down, (E, C, F))):
        if shape != want:
            raise ValueError(f"{name} has shape {tuple(shape)}, expected {want}")
    if C < 1 or F < 1 or E < 1 or k < 1:
        raise ValueError("C, F, the experts and a row's choices must be at least 1")
    return math.prod(x[:-1]), k, E, C, F


def _ffn_dims(fn, x, weights, w_gate, w_up, w_down):
    """(T, k, E, C, F) after the shape, type and device checks; x is [..., C] and weights
    [..., k] with the same leading axes."""
    try:
        dims = _ffn_plan(x.shape, weights.shape, w_gate.shape, w_up.shape, w_down.shape)
    except ValueError as e:
        raise ValueError(f"{fn}: {e}") from None
    if not _alike(x.dtype, x.get_device(), x, weights, w_gate, w_up, w_down):
        _same(fn, x, weights, w_gate, w_up, w_down)
    return dims


def _buffer(fn, name, t, x, kind, dims):
    """A buffer of the call: the caller's, checked, or a new one."""
    size = im2win_expert_ffn_size(kind, *dims, _dtype_code(x))
    if t is None:
        return torch.empty(size, dtype=torch.uint8, device=x.device)
    _same_device(fn, x, t)
    _cuda(t)
    if _bytes(t) < size:
        raise ValueError(f"{fn}: {name} is too small")
    return t


def _ffn(fn, dims, x, experts, weights, w_gate, w_up, w_down, y, saved, ws, act):
    _check(fn, lib().im2win_expert_ffn(
        x.data_ptr(), experts.data_ptr(), weights.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
        y.data_ptr(), _ptr(saved), ws.data_ptr(), _bytes(ws), *dims, _code(ACTS, act, "act"), _dtype_code(x),
        _stream(x.get_device())))


def im2win_expert_ffn(x, experts, weights, w_gate, w_up, w_down, y, saved, ws, act: str = "silu") -> None:
    """y = the sum of the chosen experts' weighted outputs; saved None: inference."""
    fn = "im2win_expert_ffn"
    dims = _ffn_dims(fn, x, weights, w_gate, w_up, w_down)
    _experts(fn, experts, x, weights.shape)
    _shape(fn, "y", y, x.shape)
    _same(fn, x, y)
    if saved is not None:
        _buffer(fn, "saved", saved, x, FFN_SAVED, dims)
    _same_device(fn, x, ws)
    _cuda(ws)
    _ffn(fn, dims, x, experts, weights, w_gate, w_up, w_down, y, saved, ws, act)


def _ffn_backward(fn, dims, dy, weights, w_gate, w_up, w_down, saved, grads, ws, act):
    _check(fn, lib().im2win_expert_ffn_backward(
        dy.data_ptr(), weights.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), saved.data_ptr(),
        *[_ptr(t) for t in grads], ws.data_ptr(), _bytes(ws), *dims, _code(ACTS, act, "act"), _dtype_code(dy),
        _stream(dy.get_device())))


def im2win_expert_ffn_backward(dy, weights, w_gate, w_up, w_down, saved, dx, dweights, dw_gate, dw_up, dw_down, ws,
                               act: str = "silu") -> None:
    """Gradients of im2win_expert_ffn; dx, dweights, or the three dw, may be None."""
    fn = "im2win_expert_ffn_backward"
    dims = _ffn_dims(fn, dy, weights, w_gate, w_up, w_down)
    _buffer(fn, "saved", saved, dy, FFN_SAVED, dims)
    grads = (dx, dweights, dw_gate, dw_up, dw_down)
    for name, t, like in zip(("dx", "dweights", "dw_gate", "dw_up", "dw_down"), grads, (dy, weights, w_gate, w_up, w_down)):
        if t is not None:
            _shape(fn, name, t, like.shape)
            _same(fn, dy, t)
    _same_device(fn, dy, ws)
    _cuda(ws)
    _ffn_backward(fn, dims, dy, weights, w_gate, w_up, w_down, saved, grads, ws, act)


def _forward(fn, x, experts, weights, w_gate, w_up, w_down, act, ws, out, saved, train):
    _unrecorded(fn, x, weights, w_gate, w_up, w_down)
    dims = _ffn_dims(fn, x, weights, w_gate, w_up, w_down)
    _experts(fn, experts, x, weights.shape)
    ws = _buffer(fn, "ws", ws, x, FFN_TRAIN if train else FFN_FORWARD, dims)
    if train:
        saved = _buffer(fn, "saved", saved, x, FFN_SAVED, dims)
    if out is None:
        out = torch.empty_like(x)
    else:
        _shape(fn, "out", out, x.shape)
        _same(fn, x, out)
    _ffn(fn, dims, x, experts, weights, w_gate, w_up, w_down, out, saved, ws, act)
    return out, saved


def expert_ffn(x: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
               w_down: torch.Tensor, act: str = "silu", ws: torch.Tensor | None = None,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """Gated feed-forward of x[..., C] by experts: the sum over a row's choices, experts[..., k] (int32) and
    weights[..., k] as expert_route() gives them, of weight * gated_ffn(row) with that expert's w_gate[E, F, C],
    w_up[E, F, C] and w_down[E, C, F]. A choice outside of the experts (-1) takes no part. Autograd does not
    record it: tensors that require grad are refused outside of torch.no_grad()."""
    return _forward("expert_ffn", x, experts, weights, w_gate, w_up, w_down, act, ws, out, None, False)[0]


def expert_ffn_train(x: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor, w_gate: torch.Tensor,
                     w_up: torch.Tensor, w_down: torch.Tensor, act: str = "silu", ws: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, saved: torch.Tensor | None = None):
    """expert_ffn() and the buffer its expert_ffn_backward() needs: (y, saved)."""
    return _forward("expert_ffn_train", x, experts, weights, w_gate, w_up, w_down, act, ws, out, saved, True)


def expert_ffn_backward(dy: torch.Tensor, weights: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                        w_down: torch.Tensor, saved: torch.Tensor, act: str = "silu", ws: torch.Tensor | None = None,
                        need_dx: bool = True, need_dweights: bool = True, need_dw: bool = True):
    """(dx, dweights, dw_gate, dw_up, dw_down) of expert_ffn_train() at the same weights; None for
    what is not needed. x and the experts are in `saved`."""
    fn = "expert_ffn_backward"
    dims = _ffn_dims(fn, dy, weights, w_gate, w_up, w_down)
    _buffer(fn, "saved", saved, dy, FFN_SAVED, dims)
    ws = _buffer(fn, "ws", ws, dy, FFN_BACKWARD, dims)
    grads = [torch.empty_like(t) if need else None for t, need in (
        (dy, need_dx), (weights, need_dweights), (w_gate, need_dw), (w_up, need_dw), (w_down, need_dw))]
    _ffn_backward(fn, dims, dy, weights, w_gate, w_up, w_down, saved, grads, ws, act)
    return tuple(grads)
