"""Arguments of the group norm and the router that are no plain ones: counts that are no whole numbers are refused, and a
refused call leaves the next right one of the same shape as it was; statistics of a part of a batch. On the host;
nothing is launched."""
import importlib

import numpy as np
import pytest
import torch

import memory_efficient_cnn_gb300 as mec
from memory_efficient_cnn_gb300 import build as mbuild, experts
from memory_efficient_cnn_gb300._binding import ERR_MISALIGNED, ERR_WORKSPACE

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


def test_statistics_of_a_part_of_a_batch_may_begin_on_8_bytes():
    mbuild.build()

    def call(stats, ws=None):
        return mec.lib().im2win_group_norm_backward(4096, 4096, stats, 4096, 4096, 8192, 8192, 8192, ws, 0, 2, 9, 8, 2, 0, mec.F32, None)

    assert call(4104) == call(4096) == ERR_WORKSPACE  # (what is looked at next)
    assert call(4100) == call(4097) == ERR_MISALIGNED
