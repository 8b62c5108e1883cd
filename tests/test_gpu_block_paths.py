"""Paths of the residual-block operators that sizes of the other tests do not reach, or that
they reach one call at a time: calls in a row, in graphs and on two streams, buffers that begin
as NaN, blocks of several tiles."""
import pytest
import torch

import block_ref as ref
import memory_efficient_cnn_gb300 as mec
from test_gpu_gated_ffn import DT, make

pytestmark = pytest.mark.gpu

# sizes of each way through the feed-forward
FFN_PATHS = {
    "few": (5, 520, 1000), "one kernel": (40000, 128, 200), "single tiles": (300, 256, 640),
    "pairs": (8192, 1024, 2048), "pairs, streamed": (512, 4096, 1024), "odd": (777, 1001, 271)}


@pytest.mark.parametrize("path", FFN_PATHS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_calls_in_a_row(dt, path):
    """Launches that begin while the one before ends, fifty calls on: the same bits, and no wait
    of any that gave up."""
    R, C, F = FFN_PATHS[path]
    code = mec._binding._DTYPE[DT[dt]]
    x, wg, wu, wd, dy = (t.cuda() for t in make(R, C, F, dt))
    ws = torch.empty(mec.im2win_gated_ffn_size(mec.FFN_FORWARD, R, C, F, code), dtype=torch.uint8, device="cuda")
    wb = torch.empty(mec.im2win_gated_ffn_size(mec.FFN_BACKWARD, R, C, F, code), dtype=torch.uint8, device="cuda")
    want = mec.gated_ffn(x, wg, wu, wd, ws=ws)
    _, saved = mec.gated_ffn_train(x, wg, wu, wd)
    grads = mec.gated_ffn_backward(dy, x, wg, wu, wd, saved, ws=wb)
    got = [(mec.gated_ffn(x, wg, wu, wd, ws=ws), mec.gated_ffn_backward(dy, x, wg, wu, wd, saved, ws=wb)) for _ in range(50)]
    assert mec.im2win_device_status(ws) == 0 and mec.im2win_device_status(wb) == 0
    for y, g in got:
        assert torch.equal(y, want) and all(torch.equal(a, b) for a, b in zip(g, grads))
