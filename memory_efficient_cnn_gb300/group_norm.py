"""Group norm of channels-last maps with its activation: ctypes marshalling.

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
from .block import ACTS, _bytes, _code, _count, _ptr, _same_dtype, _shape, _stream, _unrecorded

NORM_ACTS = {**ACTS, "none": 5}


@functools.lru_cache(maxsize=4096)
def im2win_group_norm_size(backward: bool, N, P, C, G, dtype: int) -> int:
    out = ctypes.c_size_t(0)
    _check("im2win_group_norm_size", lib().im2win_group_norm_size(int(backward), N, P, C, G, dtype, ctypes.byref(out)))
    return out.value


# Shapes are looked up, not worked out again: a small call costs less on the GPU than on the host.
# (8.0 and True hash as 8 and 1, and an answer holds what it was asked with: callers pass ints alone)
@functools.lru_cache(maxsize=4096, typed=True)
def _plan(shape, groups):
    """((N, P, C, G), (C,)) of x's shape; ValueError where x or the groups do not fit."""
    if len(shape) < 2 or shape[-1] < 1:
        raise ValueError("x must be [N, ..., C]")
    N, C = shape[0], shape[-1]
    if groups < 1 or C % groups:
        raise ValueError(f"{C} channels do not form {groups} groups")
    return (N, math.prod(shape[1:-1]), C, groups), (C,)


def _dims(fn, x, groups, params, maps):
    """(N, P, C, G) after the checks of a call's tensors; maps are (name, tensor or
    None) of x's shape, params those of its channels."""
    if type(groups) is not int:
        groups = _count(fn, "groups", groups)
    try:
        dims, channels = _plan(x.shape, groups)
    except ValueError as e:
        raise ValueError(f"{fn}: {e}") from None
    dtype, device = x.dtype, x.get_device()
    fine = device >= 0 and x.is_contiguous()
    for want, named in ((channels, params), (x.shape, maps)):
        for name, t in named:
            if t is not None:
                if t.shape != want:
                    _shape(fn, name, t, want)
                fine = fine and t.dtype is dtype and t.get_device() == device and t.is_contiguous()
    if not fine:
        given = [x, *(t for _, t in (*params, *maps) if t is not None)]
        _same_dtype(fn, *given)
        _same_device(fn, *given)
        _cuda(*given)
    return dims


def _statistics(fn, stats, x, dims):
    if stats.shape != (dims[0], dims[3], 2):
        _shape(fn, "stats", stats, (dims[0], dims[3], 2))
    if stats.dtype is not torch.float32:
        raise TypeError(f"{fn}: stats must be float32, got {stats.dtype}")
    if stats.get_device() != x.get_device() or not stats.is_contiguous():
        _same_device(fn, x, stats)
        _cuda(stats)


def _workspace(fn, ws, x, dims, backward):
    """The address and size of the caller's workspace, or of a new one, and what keeps it alive."""
    if ws is None:
        size = im2win_group_norm_size(backward, *dims, _dtype_code(x))
        if size == 0:
            return None, 0, None
        ws = torch.empty(size, dtype=torch.uint8, device=x.device)
        return ws.data_ptr(), size, ws
    _same_device(fn, x, ws)
    _cuda(ws)
    return ws.data_ptr(), _bytes(ws), ws


def _forward(fn, dims, x, w, b, y, stats, ws, act, eps):
    ws, size, keep = _workspace(fn, ws, x, dims, False)
    _check(fn, lib().im2win_group_norm(
        x.data_ptr(), _ptr(w), _ptr(b), y.data_ptr(), _ptr(stats), ws, size, *dims, _code(NORM_ACTS, act, "act"), eps,
        _dtype_code(x), _stream(x.get_device())))


def im2win_group_norm(x, groups: int, w, b, y, stats, ws, act: str = "none", eps: float = 1e-5) -> None:
    """y = act(group norm of x); stats (None: not kept) receives each group's mean and inverse deviation;
    ws None: a new one."""
    fn = "im2win_group_norm"
    dims = _dims(fn, x, groups, (("w", w), ("b", b)), (("y", y),))
    if stats is not None:
        _statistics(fn, stats, x, dims)
    _forward(fn, dims, x, w, b, y, stats, ws, act, eps)


def _backward(fn, dims, dy, x, stats, w, b, dx, dw, db, ws, act):
    ws, size, keep = _workspace(fn, ws, x, dims, True)
    _check(fn, lib().im2win_group_norm_backward(
        dy.data_ptr(), x.data_ptr(), stats.data_ptr(), _ptr(w), _ptr(b), _ptr(dx), _ptr(dw), _ptr(db), ws, size, *dims,
        _code(NORM_ACTS, act, "act"), _dtype_code(x), _stream(x.get_device())))


def im2win_group_norm_backward(dy, x, stats, w, b, dx, dw, db, ws, act: str = "none") -> None:
    """Gradients of im2win_group_norm; dx, dw and db may be None; ws None: a new one."""
    fn = "im2win_group_norm_backward"
    if stats.dim() != 3:
        raise ValueError(f"{fn}: stats must be [N, groups, 2]")
    dims = _dims(fn, x, stats.shape[1], (("w", w), ("b", b), ("dw", dw), ("db", db)), (("dy", dy), ("dx", dx)))
    _statistics(fn, stats, x, dims)
    _backward(fn, dims, dy, x, stats, w, b, dx, dw, db, ws, act)


def _normed(fn, x, groups, w, b, act, eps, ws, out, train):
    _unrecorded(fn, x, w, b)
    dims = _dims(fn, x, groups, (("w", w), ("b", b)), (("out", out),))
    y = torch.empty_like(x) if out is None else out
    stats = torch.empty((dims[0], dims[3], 2), dtype=torch.float32, device=x.device) if train else None
    _forward(fn, dims, x, w, b, y, stats, ws, act, eps)
    return y, stats


def group_norm(x: torch.Tensor, groups: int, w: torch.Tensor | None = None, b: torch.Tensor | None = None,
               act: str = "none", eps: float = 1e-5, ws: torch.Tensor | None = None,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """act(norm(x) * w + b) of channels-last maps x[N, ..., C], normed over each image's
    positions and each group of C / groups neighbouring channels; out may be x. Autograd does
    not record it: tensors that require grad are refused outside of torch.no_grad()."""
    return _normed("group_norm", x, groups, w, b, act, eps, ws, out, False)[0]


def group_norm_train(x: torch.Tensor, groups: int, w: torch.Tensor | None = None, b: torch.Tensor | None = None,
                     act: str = "none", eps: float = 1e-5, ws: torch.Tensor | None = None,
                     out: torch.Tensor | None = None):
    """group_norm() and the statistics its group_norm_backward() needs: (y, stats), stats[N, groups, 2]
    the groups' means and inverse deviations in float32. The gradient needs x: out must not be x."""
    fn = "group_norm_train"
    if out is not None and out.data_ptr() == x.data_ptr() and x.numel():
        raise ValueError(f"{fn}: out is x, which the gradient needs")
    return _normed(fn, x, groups, w, b, act, eps, ws, out, True)


def group_norm_backward(dy: torch.Tensor, x: torch.Tensor, stats: torch.Tensor, w: torch.Tensor | None = None,
                        b: torch.Tensor | None = None, act: str = "none", ws: torch.Tensor | None = None,
                        need_dx: bool = True, need_dw: bool = True):
    """(dx, dw, db) of group_norm_train() at the same x, w, b and act; None for what is
    not needed or belongs to an absent parameter."""
    fn = "group_norm_backward"
    if stats.dim() != 3:
        raise ValueError(f"{fn}: stats must be [N, groups, 2]")
    dims = _dims(fn, x, stats.shape[1], (("w", w), ("b", b)), (("dy", dy),))
    _statistics(fn, stats, x, dims)
    dx = torch.empty_like(x) if need_dx else None
    dw = torch.empty_like(w) if need_dw and w is not None else None
    db = torch.empty_like(b) if need_dw and b is not None else None
    _backward(fn, dims, dy, x, stats, w, b, dx, dw, db, ws, act)
    return dx, dw, db
