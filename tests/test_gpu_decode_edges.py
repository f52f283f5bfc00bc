"""Edges of the decode-step operators on the GPU, against the float64 oracle: scales under fp32's normal numbers,
infinities and NaN."""
import numpy as np
import pytest
import torch

from oracle import decode

pytestmark = pytest.mark.gpu

lh = pytest.importorskip("nvfp4_scale_calibration_lh_amd")
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24                       # fp32 unit roundoff
TINY = 2.0 ** -149                   # the smallest fp32 number


def note(msg):
    print(f"[case] {msg}", flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(t):
    return t.detach().cpu().double().numpy()


# ----------------------------------------------------------------------------------------- the norm
# a wave a row, a workgroup a row, the long rows' kernel
@pytest.mark.parametrize("cin", [256, 2064, 16400])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_of_rows_with_subnormal_scales(cin, dtype, group):
    """Rows whose largest |y| goes from 2^-149 to 2^-128 in steps of a quarter of a binade: an outlier in channel 0, whose gamma
    is 0, sets the root mean square, and the other channels' gamma is the smallest of the type (fp32: 2^-133, too).

    scale and y are within an ulp of the smallest fp32 number and the sum's rounding; scale may be rounded far down, so
    q saturates at 448, and it is within half a step of y / scale."""
    note(f"norm with subnormal scales, {cin} {dtype} group {group}")
    rows, t = 85, TYPES[dtype]
    g = gen(cin)
    h = torch.rand(rows, cin, generator=g) * 0.875 + 0.125
    h[:, 5::7] *= -1
    top = torch.exp2(-149 + torch.arange(rows, dtype=torch.float64) / 4)
    h[:, 0] = (2.0 ** -133 / top * cin ** 0.5).float()             # root mean square about 2^-133 / top
    h = h.to(t)
    gamma = torch.full((cin,), 2.0 ** -133)
    gamma[0] = 0
    gamma = gamma.to(t)
    assert float(gamma[1]) > 0
    q, scale, _ = lh.lh_rms_norm_quant(h.to(DEV), gamma.to(DEV), eps=0.0, group=group)
    y, want = decode.rms_norm(f64(h), f64(gamma), 0.0, group)
    rel = (cin / 64 + 16) / 2 * U + 8 * U
    s = f64(scale)
    assert np.all(np.abs(s - want) <= rel * want + TINY)
    got = f64(q.float())
    assert np.isfinite(got).all()
    wide = np.repeat(s, group or cin, axis=1)[:, :cin]
    held = np.clip(y, -448 * wide, 448 * wide)
    tol = np.maximum(np.abs(y) * 2.0 ** -4, wide * 2.0 ** -10) * (1 + 2 ** -10) + 2 * rel * np.abs(y) + TINY
    assert np.all(np.abs(got * wide - held) <= tol)


@pytest.mark.parametrize("cin", [256, 2064, 16400])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_shows_infinities_and_nan(cin, dtype, group, residual):
    """h / sqrt(mean h^2 + eps) is NaN everywhere for a row with a NaN, and for one with an infinity NaN there and 0
    elsewhere.  The other rows are those of a call without them, and gamma's NaN or infinity stays in its run."""
    note(f"norm with infinities and NaN, {cin} {dtype} group {group} residual {residual}")
    t, g, rows, at = TYPES[dtype], gen(cin + 1), 9, cin - 70
    x = torch.randn(rows, cin, generator=g).to(t)
    r = torch.randn(rows, cin, generator=g).to(t) if residual else None
    gamma = (1 + 0.2 * torch.randn(cin, generator=g)).to(t)

    def call(x, gamma):
        q, s, h = lh.lh_rms_norm_quant(x.to(DEV), gamma.to(DEV), None if r is None else r.to(DEV), group=group)
        return f64(q.float()), f64(s), h

    good_q, good_s, _ = call(x, gamma)
    bad = x.clone()
    bad[1, at], bad[3, at], bad[6, at] = float("nan"), float("inf"), -float("inf")
    q, s, h = call(bad, gamma)
    run = at // 128 if group else 0
    others = [i for i in range(rows) if i not in (1, 3, 6)]
    assert np.array_equal(q[others], good_q[others]) and np.array_equal(s[others], good_s[others])
    assert np.isnan(s[1]).all() and (q[[1, 3, 6]] == 0).all()
    for i in (3, 6):
        assert np.isnan(s[i, run]) and (np.delete(s[i], run) == 0).all()
    if residual:
        assert torch.isnan(h[1, at]) and h[3, at] == float("inf") and h[6, at] == -float("inf")

    for value in (float("nan"), float("inf")):
        gm = gamma.clone()
        gm[at] = value
        q, s, _ = call(x, gm)
        keep = np.arange(cin) // 128 != run if group else np.zeros(cin, bool)
        assert not np.isfinite(s[:, run]).any() and np.array_equal(np.delete(s, run, 1), np.delete(good_s, run, 1))
        assert np.array_equal(q[:, keep], good_q[:, keep]) and (q[:, ~keep] == 0).all()
