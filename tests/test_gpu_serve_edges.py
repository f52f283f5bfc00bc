"""The operators around a decode step on the GPU where one kernel, type or size gives way to another, and after other calls' errors."""
import numpy as np
import pytest
import torch

from test_gpu_serve import DEV, check_extend, choices, layer_rows, matrices, note, on_gpu, requests

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


# ------------------------------------------------------------------------- growth of the cache's sequences
def one_workgroup(batch, max_tokens):
    """Whether the call is one kernel, which needs no workspace."""
    return lh.lh_cache_extend_workspace(batch, max_tokens) == 0


@pytest.mark.parametrize("batch,width,page,max_tokens,one", [(512, 3, 5, 512, True), (512, 3, 5, 513, False), (513, 3, 5, 512, False), (1, 90, 7, 512, True),
                                                             (1, 90, 7, 513, False), (66, 5, 16, 500, True), (200, 40, 64, 511, True), (511, 9, 1, 300, True),
                                                             (320, 4, 3, 0, True), (512, 6, 4, 1, True)])
@pytest.mark.parametrize("new", ["mixed", "one", "idle", "back"])
def test_extend_where_one_workgroup_ends(batch, width, page, max_tokens, one, new):
    note(f"extend {batch} requests, {width} pages of {page}, {max_tokens} rows, {new}")
    assert one_workgroup(batch, max_tokens) == one
    case = requests(batch, width, page, batch + max_tokens, new)
    check_extend(*case, page, max_tokens)
    check_extend(*case, page, max_tokens, in_place=True)
    check_extend(*case, page, max_tokens, calls=3)


@pytest.mark.parametrize("batch,max_tokens,one", [(60, 400, True), (300, 512, True), (512, 512, True), (512, 513, False), (513, 300, False)])
@pytest.mark.parametrize("free", [0, 1, 37])
def test_extend_pages_run_out_in_either_kernel(batch, max_tokens, one, free):
    assert one_workgroup(batch, max_tokens) == one
    for seed in range(4):
        note(f"extend {batch} requests, {max_tokens} rows, {free} free pages, seed {seed}")
        case = requests(batch, 6, 4, seed, free=free)
        if seed % 2:                                   # single tokens, so that rows are left when pages are not
            case = (*case[:2], np.where(case[2] > 0, 1, case[2]), *case[3:])
        check_extend(*case, 4, max_tokens)
        check_extend(*case, 4, max_tokens, in_place=True)


@pytest.mark.parametrize("batch,max_tokens,one", [(5, 300, True), (300, 512, True), (512, 512, True), (512, 513, False), (600, 200, False)])
def test_extend_numbers_out_of_range_in_either_kernel(batch, max_tokens, one):
    assert one_workgroup(batch, max_tokens) == one
    table, lengths, asked, stack, count = requests(batch, 5, 8, 11)
    lengths[0], lengths[1], lengths[2] = -5, 2 ** 31 - 1, -2 ** 31
    table[3] = -123
    for c in (-1, -2 ** 31, 10 ** 9, 3):
        note(f"extend {batch} requests, {max_tokens} rows, with a count of {c}")
        check_extend(table, lengths, asked, stack, np.array([c]), 8, max_tokens)
    note(f"extend {batch} requests, {max_tokens} rows, with a short stack")
    check_extend(table, lengths, asked, stack[:4].copy(), np.array([3]), 8, max_tokens)
