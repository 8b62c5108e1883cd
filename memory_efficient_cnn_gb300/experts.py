"""A block of experts: ctypes marshalling of the router and of the gated feed-forward
grouped by expert.

As in block.py, the im2win_* functions take caller-allocated outputs and map one to
one onto the C entry points, the names without the prefix allocate through torch,
and nothing is computed here.
"""
from __future__ import annotations

import torch

from ._binding import _check, _cuda, _dtype_code, _same_device, lib
from .block import _alike, _code, _same_dtype, _shape, _stream, _unrecorded

ROUTES = {"top": 0, "all": 1}


def _experts(fn, experts, like, shape):
    """Checks an index tensor of a call on like's device."""
    if tuple(experts.shape) != tuple(shape):
        _shape(fn, "experts", experts, shape)
    if experts.dtype != torch.int32:
        raise TypeError(f"{fn}: experts must be int32, got {experts.dtype}")
    if not _alike(torch.int32, like.get_device(), experts):
        _same_device(fn, like, experts)
        _cuda(experts)


def _same(fn, x, *ts):
    if not _alike(x.dtype, x.get_device(), x, *ts):
        _same_dtype(fn, x, *ts)
        _same_device(fn, x, *ts)
        _cuda(x, *ts)


# ---------------------------------------------------------------- router
def _route_dims(fn, logits, k):
    if logits.dim() < 1 or logits.shape[-1] < 1:
        raise ValueError(f"{fn}: logits must be [..., E]")
    E = logits.shape[-1]
    if not 1 <= k <= E:
        raise ValueError(f"{fn}: k must be between 1 and {E}, the number of experts; got {k}")
    return logits.numel() // E, E, k


def im2win_expert_route(logits, weights, experts, over: str = "top") -> None:
    """experts = the indexes of the k largest logits of each row, weights = their softmax weights."""
    fn = "im2win_expert_route"
    k = weights.shape[-1] if weights.dim() else 0
    dims = _route_dims(fn, logits, k)
    _shape(fn, "weights", weights, (*logits.shape[:-1], k))
    _same(fn, logits, weights)
    _experts(fn, experts, logits, weights.shape)
    _check(fn, lib().im2win_expert_route(logits.data_ptr(), weights.data_ptr(), experts.data_ptr(), *dims,
                                         _code(ROUTES, over, "over"), _dtype_code(logits), _stream(logits.get_device())))


def im2win_expert_route_backward(dweights, logits, experts, dlogits, over: str = "top") -> None:
    """dlogits from dweights at the same logits and the experts chosen there."""
    fn = "im2win_expert_route_backward"
    k = dweights.shape[-1] if dweights.dim() else 0
    dims = _route_dims(fn, logits, k)
    _shape(fn, "dweights", dweights, (*logits.shape[:-1], k))
    _shape(fn, "dlogits", dlogits, logits.shape)
    _same(fn, logits, dweights, dlogits)
    _experts(fn, experts, logits, dweights.shape)
    _check(fn, lib().im2win_expert_route_backward(
        dweights.data_ptr(), logits.data_ptr(), experts.data_ptr(), dlogits.data_ptr(), *dims, _code(ROUTES, over, "over"),
        _dtype_code(logits), _stream(logits.get_device())))


def expert_route(logits: torch.Tensor, k: int, over: str = "top"):
    """(weights, experts), [..., k] each, of logits[..., E]: the k largest of a row by falling value, equal
    ones by rising index (int32), and their softmax weights over the k choices ("top") or over all
    experts ("all"). A logit of -inf is an expert the row may not take; places left over have expert -1
    and weight 0. Autograd does not record it: tensors that require grad are refused outside of
    torch.no_grad()."""
    fn = "expert_route"
    _unrecorded(fn, logits)
    _route_dims(fn, logits, k)
    shape = (*logits.shape[:-1], k)
    weights = torch.empty(shape, dtype=logits.dtype, device=logits.device)
    experts = torch.empty(shape, dtype=torch.int32, device=logits.device)
    im2win_expert_route(logits, weights, experts, over)
    return weights, experts


def expert_route_backward(dweights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, over: str = "top"):
    """dlogits of expert_route() at the same logits and over, and the experts it chose."""
    dlogits = torch.empty_like(logits)
    im2win_expert_route_backward(dweights, logits, experts, dlogits, over)
    return dlogits
