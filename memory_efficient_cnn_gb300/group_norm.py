"""Group norm of channels-last maps with its activation: ctypes marshalling.

As in block.py, the im2win_* functions take caller-allocated outputs and map one to
one onto the C entry points, the names without the prefix allocate through torch,
and nothing is computed here.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._binding import _check, _cuda, _dtype_code, _same_device, lib
from .block import ACTS, _alike, _bytes, _code, _empty, _ptr, _same_dtype, _shape, _stream, _unrecorded

NORM_ACTS = {**ACTS, "none": 5}


@functools.lru_cache(maxsize=4096)
def im2win_group_norm_size(N, P, C, G, dtype: int) -> int:
    out = ctypes.c_size_t(0)
    _check("im2win_group_norm_size", lib().im2win_group_norm_size(N, P, C, G, dtype, ctypes.byref(out)))
    return out.value


def _dims(fn, x, groups, params, maps):
    """(N, P, C, G) after the checks of a call's tensors; maps are (name, tensor or
    None) of x's shape, params those of its channels."""
    if x.dim() < 2 or x.shape[-1] < 1:
        raise ValueError(f"{fn}: x must be [N, ..., C]")
    N, C = x.shape[0], x.shape[-1]
    if groups < 1 or C % groups:
        raise ValueError(f"{fn}: {C} channels do not form {groups} groups")
    P = 1
    for n in x.shape[1:-1]:
        P *= n
    given = []
    for name, t in maps:
        if t is not None:
            if t.shape != x.shape:
                _shape(fn, name, t, x.shape)
            given.append(t)
    for name, t in params:
        if t is not None:
            if t.shape != (C,):
                _shape(fn, name, t, (C,))
            given.append(t)
    if not _alike(x.dtype, x.get_device(), x, *given):
        _same_dtype(fn, x, *given)
        _same_device(fn, x, *given)
        _cuda(x, *given)
    return N, P, C, groups


def _statistics(fn, stats, x, dims):
    _shape(fn, "stats", stats, (dims[0], dims[3], 2))
    if stats.dtype != torch.float32:
        raise TypeError(f"{fn}: stats must be float32, got {stats.dtype}")
    _same_device(fn, x, stats)
    _cuda(stats)


def _workspace(fn, ws, x, dims):
    if ws is None:
        return _empty(im2win_group_norm_size(*dims, _dtype_code(x)), x.device)
    _same_device(fn, x, ws)
    _cuda(ws)
    return ws


def _forward(fn, dims, x, w, b, y, stats, ws, act, eps):
    _check(fn, lib().im2win_group_norm(
        x.data_ptr(), _ptr(w), _ptr(b), y.data_ptr(), _ptr(stats), ws.data_ptr(), _bytes(ws), *dims,
        _code(NORM_ACTS, act, "act"), eps, _dtype_code(x), _stream(x.get_device())))


def im2win_group_norm(x, groups: int, w, b, y, stats, ws, act: str = "none", eps: float = 1e-5) -> None:
    """y = act(group norm of x); stats (None: not kept) receives each group's mean and inverse deviation."""
    fn = "im2win_group_norm"
    dims = _dims(fn, x, groups, (("w", w), ("b", b)), (("y", y),))
    if stats is not None:
        _statistics(fn, stats, x, dims)
    _forward(fn, dims, x, w, b, y, stats, _workspace(fn, ws, x, dims), act, eps)


def im2win_group_norm_backward(dy, x, stats, w, b, dx, dw, db, ws, act: str = "none") -> None:
    """Gradients of im2win_group_norm; dx, dw and db may be None."""
    fn = "im2win_group_norm_backward"
    if stats.dim() != 3:
        raise ValueError(f"{fn}: stats must be [N, groups, 2]")
    dims = _dims(fn, x, stats.shape[1], (("w", w), ("b", b), ("dw", dw), ("db", db)), (("dy", dy), ("dx", dx)))
    _statistics(fn, stats, x, dims)
    ws = _workspace(fn, ws, x, dims)
    _check(fn, lib().im2win_group_norm_backward(
        dy.data_ptr(), x.data_ptr(), stats.data_ptr(), _ptr(w), _ptr(b), _ptr(dx), _ptr(dw), _ptr(db), ws.data_ptr(),
        _bytes(ws), *dims, _code(NORM_ACTS, act, "act"), _dtype_code(x), _stream(x.get_device())))


def _normed(fn, x, groups, w, b, act, eps, ws, out, train):
    _unrecorded(fn, x, w, b)
    dims = _dims(fn, x, groups, (("w", w), ("b", b)), (("out", out),))
    y = torch.empty_like(x) if out is None else out
    stats = torch.empty((dims[0], groups, 2), dtype=torch.float32, device=x.device) if train else None
    _forward(fn, dims, x, w, b, y, stats, _workspace(fn, ws, x, dims), act, eps)
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
    dx = torch.empty_like(x) if need_dx else None
    dw = torch.empty_like(w) if need_dw and w is not None else None
    db = torch.empty_like(b) if need_dw and b is not None else None
    im2win_group_norm_backward(dy, x, stats, w, b, dx, dw, db, ws, act)
    return dx, dw, db
