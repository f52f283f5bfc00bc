"""The operators around a decode step on the GPU where one kernel, type or size gives way to another, and after other calls' errors."""
import numpy as np
import pytest
import torch

from oracle import serve
from test_gpu_serve import DEV, check_extend, check_moe, choices, dev, heads_of, layer_rows, matrices, note, on_gpu, requests

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


# --------------------------------------------------------------------------------------- rotary positions
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_fast_angles(interleaved):
    """Frequencies up to 2^16, the largest documented, at the largest positions.  The angle is taken in turns with whole numbers; then as for any
    position: sine and cosine to 2^-23, one rounding with the scale, one of a product, of the sum and of the output."""
    note(f"rotary fast angles, interleaved {interleaved}")
    f = np.array([2 ** 16, 65535.99, 40961.37, -31415.926, 1.0 / 3, 7.25, 2 ** 16 - 1, 1e-3], np.float32)
    positions = np.array([2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30 + 12345, 1999999973, 1, 0, 65537])
    pi = 31415926535897932384626433832795028841971693993751058209749445923        # times 10^64
    turns = np.array([[int(p) * int(float(v) * 2 ** 60) for v in f] for p in positions], object)       # angles times 2^60; whole numbers
    whole = 2 * pi * 2 ** 60
    left = [[t * 10 ** 64 % whole for t in row] for row in turns]
    w = np.array([[float((v if 2 * v < whole else v - whole) // 2 ** 60) / 1e64 for v in row] for row in left])
    x, xv = heads_of(len(positions), 3, 32, "f32", 5)
    y, _ = lh.lh_rotary(x, None, dev(positions), torch.from_numpy(f).to(DEV), interleaved=interleaved, scale=1.25)
    at = (np.arange(8) * 2, np.arange(8) * 2 + 1) if interleaved else (np.arange(8), np.arange(8) + 8)
    a, b = xv[..., at[0]], xv[..., at[1]]
    c, s = 1.25 * np.cos(w)[:, None], 1.25 * np.sin(w)[:, None]
    want = xv.copy()
    want[..., at[0]], want[..., at[1]] = a * c - b * s, a * s + b * c
    bound = np.zeros_like(want)
    u = 2.0 ** -24
    bound[..., at[0]] = bound[..., at[1]] = 1.25 * (np.abs(a) + np.abs(b)) * (2 + 1 + 1 + 1) * u
    bound += u * (np.abs(want) + bound) * (bound > 0)
    err = np.abs(y.double().cpu().numpy() - want)
    assert np.all(err <= bound), float((err - bound).max())


# ------------------------------------------------------------------------------------------ the expert layer
def moe64(x, ids, weights, gate_up, down, norm=448.0):
    """oracle.serve.moe in 64 bits on the device, an expert at a time."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    grid = torch.cat((grid, -grid))

    def matrix(m, e):
        code, fp4 = (torch.from_numpy(t[e]).to(DEV) for t in m[:2])
        nib = torch.stack((fp4 & 15, fp4 >> 4), -1).flatten(-2).long()
        return grid[nib] * code.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * float(m[2][e] / np.float32(6.0 * norm))

    x = torch.from_numpy(x).to(DEV)
    y, terms = torch.zeros_like(x), torch.zeros_like(x)
    for e in np.unique(ids[(ids >= 0) & (ids < len(gate_up[2]))]):
        t, j = (torch.from_numpy(a).to(DEV) for a in np.nonzero(ids == e))
        wg, wd, v = matrix(gate_up, e), matrix(down, e), x[t]
        w = torch.from_numpy(np.asarray(weights, np.float64)).to(DEV)[t, j][:, None]
        gate, up = (v @ wg.t()).chunk(2, -1)
        ag, au = (v.abs() @ wg.abs().t()).chunk(2, -1)
        s = gate / (1 + torch.exp(-gate))
        h = s * up
        y.index_add_(0, t, w * (h @ wd.t()))
        terms.index_add_(0, t, w.abs() * ((h.abs() + 1.1 * ag * up.abs() + s.abs() * au) @ wd.abs().t()))
    return y.cpu().numpy(), terms.cpu().numpy()


def test_moe64_is_the_oracle():
    note("the expert layer in 64 bits on the device")
    gate_up, down = matrices(9, 128, 256, 5), matrices(9, 256, 64, 6)
    x = np.random.default_rng(7).standard_normal((30, 256))
    ids, w = choices(30, 9, 3, 8)
    ids[3], ids[4, 1], ids[5] = -1, 9, 4
    for got, want in zip(moe64(x, ids, w, gate_up, down, 256.0), serve.moe(x, ids, w.astype(np.float64), gate_up, down, 256.0)):
        assert np.all(np.abs(got - want) <= 1e-12 * np.abs(want).max(1, keepdims=True))


# The first expert has every token, so more rows than one pass takes.  Rows as they are, held in several panels of LDS (of the first product,
# of the second) that several groups of channels go through, each wave with all of k: over half the chip's wave slots have channels of
# their own.  Few tokens, likewise and with k shared by eight waves.  Rows made ready first, several panels, k not shared and shared.
@pytest.mark.parametrize("tokens,experts,topk,hidden,inner", [(40, 104, 10, 1040, 640), (40, 104, 10, 640, 1296), (32, 130, 10, 2560, 640), (16, 16, 3, 2576, 784),
                                                              (16, 5, 2, 4112, 272), (70, 12, 2, 2064, 1040), (70, 12, 2, 1040, 5504)])
@pytest.mark.parametrize("x,group", [("bf16", 0), ("f32", 0), ("e4m3", 0), ("e4m3", 128)])
def test_moe_of_many_channels(tokens, experts, topk, hidden, inner, x, group, monkeypatch):
    note(f"moe {tokens} tokens top {topk} of {experts}, {hidden} x {inner}, {x} group {group}")
    monkeypatch.setattr(serve, "moe", moe64)
    gate_up, down = matrices(experts, 2 * inner, hidden, 1), matrices(experts, hidden, inner, 2)
    xd, scale, xv = layer_rows(tokens, hidden, x, group, 3)
    ids, w = choices(tokens, experts - 1, topk, 4)
    ids += 1
    ids[:, topk // 2] = 0
    check_moe(xd, scale, xv, x, group, ids, w, gate_up, down)


@pytest.mark.parametrize("x", ["bf16", "f32", "e4m3"])
def test_moe_gates_past_the_range_of_exp(x):
    """Gates of -87 to -140, where exp(-g) ends fp32 at 88.7, beside ups that make their products ordinary numbers.
    A gate has one term, so three roundings (the factor, the weights' two scales), which exp passes on times the gate; exp and the division
    take 8 more.  h is held to 2^-11 or 2^-23 of itself, an up has three roundings, the sum of 128 terms one a term (three times for fp32)."""
    note(f"moe with gates past the range of exp, {x}")
    hidden, inner = 256, 128
    r = np.random.default_rng(1)
    code, fp4, amax = matrices(1, 2 * inner, hidden, 2)
    fp4[:] = 0
    fp4[0, :inner, 0], fp4[0, inner:, hidden // 4] = 2, 2                   # 1 at element 0 of the gates, at element 128 of the ups
    code[0, :inner] = np.array([0x53, 0x54, 0x55], np.uint8)[r.integers(0, 3, inner)][:, None]         # scales of 11, 12 and 13
    amax[:] = 2688.0                                                        # a global scale of 1
    down = matrices(1, hidden, inner, 3)
    v = np.zeros((2, hidden))
    v[:, 0], v[:, 128] = [-7.92, -10.8], [1e25, -3e37]
    v[:, 1:128] = r.standard_normal((2, 127))                               # (their weights are 0)
    if x == "e4m3":
        s = np.array([[7.92 / 448, 1e25 / 448], [10.8 / 448, 3e37 / 448]], np.float32)
        q = torch.from_numpy(v / np.repeat(s.astype(np.float64), 128, 1)).float().clamp(-448, 448).to(torch.float8_e4m3fn)
        xd, scale, xv = q.to(DEV), torch.from_numpy(s).to(DEV), q.double().numpy() * np.repeat(s.astype(np.float64), 128, 1)
    else:
        t = torch.from_numpy(v).to(torch.bfloat16 if x == "bf16" else torch.float32)
        xd, scale, xv = t.to(DEV), None, t.double().numpy()
    ids, w = np.zeros((2, 1), np.int32), np.ones((2, 1), np.float32)
    y = lh.lh_moe(xd, torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), on_gpu((code, fp4, amax)), on_gpu(down), x_scale=scale,
                  x_group=128 if x == "e4m3" else 0).double().cpu().numpy()
    want, _ = serve.moe(xv, ids, w, (code, fp4, amax), down)
    wg, wd = (serve.decode.weights(m[0][0], m[1][0], m[2][0], 448.0) for m in ((code, fp4, amax), down))
    gate, up = np.split(xv @ wg.T, 2, 1)
    assert np.all((gate > -150) & (gate < -80)) and len(np.unique(gate)) >= 6
    terms = np.abs(serve.silu(gate) * up) @ np.abs(wd).T
    u = 2.0 ** -24
    rel = (150 * 3 + 8 + 3 + (3 if x == "f32" else 1) * (inner + 8)) * u + (2.0 ** -23 if x == "f32" else 2.0 ** -11)
    bound = rel * terms
    bound += (u if x == "f32" else 2.0 ** -8) * (np.abs(want) + bound)
    assert np.all(np.abs(y - want) <= bound), float((np.abs(y - want) / bound).max())
    assert np.abs(want).min() > 0
