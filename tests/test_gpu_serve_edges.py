"""The operators around a decode step on the GPU where one kernel, type or size gives way to another, and after other calls' errors."""
import numpy as np
import pytest
import torch

from test_gpu_serve import DEV, choices, dev, layer_rows, matrices, note, on_gpu

pytestmark = pytest.mark.gpu

lh = pytest.importorskip("nvfp4_scale_calibration_lh_amd")


@pytest.mark.parametrize("tokens", [3, 40])            # rows taken as they are, and made ready first
@pytest.mark.parametrize("x", ["bf16", "f32", "e4m3"])
def test_moe_after_an_older_error(tokens, x):
    """An error that an earlier runtime call of this thread has left is not the expert layer's."""
    note(f"moe after an older error, {tokens} tokens of {x}")
    gate_up, down = on_gpu(matrices(2, 288, 272, 1)), on_gpu(matrices(2, 272, 144, 2))
    xd, scale, _ = layer_rows(tokens, 272, x, 0, 3)
    ids, w = (torch.from_numpy(t).to(DEV) for t in choices(tokens, 2, 2, 4))
    want = lh.lh_moe(xd, ids, w, gate_up, down, x_scale=scale)
    y = torch.zeros_like(want)
    work = torch.empty(lh.lh_moe_workspace(xd.dtype, tokens, 272, 144, 2, 2), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    hip = lh.lib()                                     # (the runtime's functions are found through the library that needs it)
    assert hip.hipSetDevice(9999) != 0
    try:
        assert hip.hipPeekAtLastError() != 0
        lh.lh_moe(xd, ids, w, gate_up, down, y, x_scale=scale, workspace=work)
    finally:
        hip.hipGetLastError()
    assert torch.equal(y, want)
