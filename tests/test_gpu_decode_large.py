"""Products at sizes whose kernels small shapes do not reach, against the float64 oracle: several channel tiles a
workgroup, several channel tiles at a time, several steps along k, and groups whose runs of tiles end in part of a set."""
import functools

import numpy as np
import pytest
import torch

from oracle import decode
from test_gpu_decode import DEV, U, f64, lh, note, rows_of, weights

pytestmark = pytest.mark.gpu

KINDS = [("bf16", 0), ("f32", 0), ("e4m3", 0), ("e4m3", 128)]


@functools.lru_cache(maxsize=1)
def layer(cout, cin):
    """(codes, nibbles and amax on the GPU, the weights in float64)."""
    code, fp4, amax = weights(1, cout, cin, cout + cin)
    return [torch.from_numpy(a).to(DEV) for a in (code, fp4, amax)], decode.weights(code[0], fp4[0], amax[0])


def check(y, x, w):
    """The tolerance of test_gpu_decode.check_product."""
    want, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    tol = 2 * (x.shape[1] + 8) * U * mag + (np.abs(want) * 2.0 ** -8 if y.dtype == torch.bfloat16 else 0)
    bad = ~(np.abs(f64(y) - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outputs, channels {np.unique(np.nonzero(bad)[1])[:8]}"


# cout, cin: rows
#   12301 x 4112: 4 tiles a workgroup, the last set of them partial, 16 channels past whole chunks; from 17 rows on
#     2 or 3 tiles at a time
#   300 x 12304: several steps along k, rows loaded a step ahead
#   4333 x 2576: 3 chunks a wave from 9 rows on, several tiles a workgroup; 2 tiles at a time from 17 on
#   8229 x 2064: 2 chunks a wave, several tiles a workgroup
#   57400 x 1040: one chunk a wave, 8 tiles a workgroup
DENSE = ([(12301, 4112, r) for r in (1, 4, 5, 8, 9, 16, 17, 20, 32, 33, 64, 65)] + [(300, 12304, r) for r in (1, 4, 5, 8, 16, 17, 40)]
         + [(4333, 2576, r) for r in (1, 6, 9, 16, 20)] + [(8229, 2064, r) for r in (1, 8, 9, 16)] + [(57400, 1040, r) for r in (2, 16)])


@pytest.mark.parametrize("cout,cin,rows,x,group", [(*d, *k) for d in DENSE for k in KINDS])
def test_matvec_of_large_layers(cout, cin, rows, x, group):
    note(f"matvec {rows}x{cin} -> {cout} {x} group {group}")
    gpu, w = layer(cout, cin)
    t, s, v = rows_of(rows, cin, x, group, rows)
    y = lh.lh_matvec(t.to(DEV), *gpu, x_scale=None if s is None else s.to(DEV), x_group=group)
    check(y, v, w)
    again = lh.lh_matvec(t.to(DEV), *gpu, x_scale=None if s is None else s.to(DEV), x_group=group)
    assert torch.equal(y, again)


# 82 or 85 tiles of a matrix in runs of whole sets of 4, the last one partial; groups of every size around 4, 16 and 17
MIXED = [0, 1, 4, 5, 0, 16, 17, 3, 33, 0, 8, 1, 2, 0, 0, 40, 1, 15, 2, 1, 0, 7, 1, 1, 9, 0, 2, 1, 1, 1, 0, 3, 1, 1, 5, 0]
FEW = [0, 1, 0, 0, 2, 0, 0, 0, 0, 0, 0, 0, 0] * 60                  # few rows a group: pieces of 4 rows for every type


@pytest.mark.parametrize("counts,cout,cin", [(MIXED, 1300, 2576), (MIXED, 1345, 2064), (MIXED, 1300, 4112), (MIXED, 1300, 784),
                                             (FEW, 200, 2064), (FEW, 200, 2576)], ids=lambda v: f"{len(v)}groups" if isinstance(v, list) else str(v))
@pytest.mark.parametrize("x,group", KINDS)
def test_matvec_of_many_experts(counts, cout, cin, x, group):
    note(f"matvec {len(counts)} groups, {sum(counts)} rows of {cin} -> {cout} {x} group {group}")
    code, fp4, amax = weights(len(counts), cout, cin, 11)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    t, s, v = rows_of(int(off[-1]), cin, x, group, 5)
    y = lh.lh_matvec(t.to(DEV), *(torch.from_numpy(a).to(DEV) for a in (code, fp4, amax)), x_scale=None if s is None else s.to(DEV),
                     x_group=group, offsets=torch.from_numpy(off).to(DEV))
    hit = np.flatnonzero(counts)
    for g in hit if len(hit) < 40 else hit[[0, 1, len(hit) // 3, len(hit) // 2, -2, -1]]:
        check(y[off[g]:off[g + 1]], v[off[g]:off[g + 1]], decode.weights(code[g], fp4[g], amax[g]))
    assert torch.isfinite(y).all()
