"""Counts that callers pass to the group norm and the router: what is no whole number is refused, and a
refused call leaves the next right one of the same shape as it was. On the host; nothing is launched."""
import importlib

import numpy as np
import pytest
import torch

import memory_efficient_cnn_gb300 as mec
from memory_efficient_cnn_gb300 import experts

norm = importlib.import_module("memory_efficient_cnn_gb300.group_norm")  # (the name is the function's in the package)


def all_ints(v):
    return all(all_ints(i) for i in v) if isinstance(v, tuple) else type(v) is int


@pytest.mark.parametrize("wrong", [8.0, 64 / 8, "8", None])
def test_group_counts(wrong):
    x = torch.zeros(2, 5, 64)
    for call in (mec.group_norm, mec.group_norm_train):
        with pytest.raises(TypeError, match="groups must be a whole number"):
            call(x, wrong)
    dims, channels = norm._plan(x.shape, 8)
    assert dims == (2, 5, 64, 8) and all_ints(dims) and all_ints(tuple(channels))
    # whole numbers of other types become ints, and then the host tensors are what is wrong
    for groups in (np.int64(8), True, torch.tensor(8)):
        with pytest.raises(ValueError, match="CUDA"):
            mec.group_norm(x, groups)
    for groups in (8, 1):
        assert all_ints(norm._plan(x.shape, groups)[0])


@pytest.mark.parametrize("wrong", [2.0, 4 / 2, "2", None])
def test_choice_counts(wrong):
    logits = torch.zeros(5, 8)
    with pytest.raises(TypeError, match="k must be a whole number"):
        mec.expert_route(logits, wrong)
    T, E, code, shape = experts._route_plan(logits.shape, 2, "top")
    assert (T, E, code, shape) == (5, 8, 0, (5, 2)) and all_ints((T, E, code, tuple(shape)))
    for k in (np.int32(2), True):
        with pytest.raises(ValueError, match="CUDA"):
            mec.expert_route(logits, k)
    for k in (2, 1):
        assert all_ints(experts._route_plan(logits.shape, k, "top"))


def test_answers_by_shape_do_not_mix_types():
    """What is looked up by a shape holds the caller's own numbers."""
    norm._plan(torch.Size([3, 7, 32]), 4.0)
    assert all_ints(norm._plan(torch.Size([3, 7, 32]), 4)[0])
    experts._route_plan(torch.Size([3, 9]), 3.0, "all")
    assert all_ints(experts._route_plan(torch.Size([3, 9]), 3, "all"))
