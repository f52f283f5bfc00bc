"""Edges of the decode-step operators on the GPU, against the float64 oracle: scales under fp32's normal numbers,
infinities and NaN, and decisions at midpoints."""
import numpy as np
import pytest
import torch

from oracle import decode
from test_gpu_decode import DEV, TYPES, U, attention_case, f64, gen, lh, make_cache, note, weights

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -149                   # the smallest fp32 number


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


@pytest.mark.parametrize("dtype,cin", [("bf16", 256), ("bf16", 2048), ("bf16", 32768), ("f32", 256), ("f32", 2048), ("f32", 16384)])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_writes_the_code_nearest_to_the_quotient(dtype, cin, group):
    """Rows of +-2^k have a reciprocal root mean square of 2^-k and y = +-gamma without a rounding, so scale and the exact
    quotient are known: gamma holds every midpoint of the E4M3 grid times the scale, with its neighbours in fp32."""
    note(f"norm, midpoints, {cin} {dtype} group {group}")
    t, width = TYPES[dtype], group or cin
    vals = decode.e4m3_values(np.arange(127))
    mids = (vals[1:] + vals[:-1]) / 2
    r = np.random.default_rng(cin + group)
    gamma, at = np.zeros(cin, np.float32), 0
    exponents = [0, -3, -97, -105, -120, 60, 105, 115, 5, -20] if group else [(-112 if cin == 2048 else 1)]
    for k, c in enumerate(range(0, cin, width)):
        top = float(torch.tensor(r.uniform(1, 2) * 2.0 ** exponents[k % len(exponents)]).to(t))
        s = np.float32(np.float32(top) * np.float32(1 / 448.0))
        m = np.resize(np.roll(mids, -at), width // 3).astype(np.float64) * np.float64(s)
        at += width // 3
        m = m.astype(np.float32)
        run = np.concatenate([[np.float32(top)], m, np.nextafter(m, np.float32(0)), np.nextafter(m, np.float32(np.inf))])
        gamma[c:c + width] = np.minimum(np.resize(run, width), np.float32(top))
    gamma = torch.from_numpy(gamma).to(t)
    g = gen(cin)
    h = torch.where(torch.rand(5, cin, generator=g) < 0.5, -1.0, 1.0) * torch.tensor([[1.0], [0.25], [64.0], [2.0 ** -9], [2.0 ** 20]])
    q, scale, _ = lh.lh_rms_norm_quant(h.to(t).to(DEV), gamma.to(DEV), eps=0.0, group=group)
    y = np.sign(f64(h)) * f64(gamma)
    want = (np.abs(gamma.float().numpy()).reshape(-1, width).max(1) * np.float32(1 / 448.0)).astype(np.float32)
    assert np.array_equal(scale.cpu().numpy(), np.tile(want, (5, 1)))
    codes = decode.e4m3_codes(y / np.repeat(want.astype(np.float64), width))
    got = q.view(torch.uint8).cpu().numpy()
    assert np.array_equal(got, codes), f"{(got != codes).sum()} of {got.size} codes differ"


# -------------------------------------------------------------------------------------- the products
def on_gpu(*arrays):
    return [torch.from_numpy(a).to(DEV) for a in arrays]


@pytest.mark.parametrize("rows", [1, 5, 9, 17, 33])
@pytest.mark.parametrize("cin", [48, 144, 2064, 4112])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_matvec_of_infinities_and_nan(rows, cin, x):
    """A row with an infinity gives plus or minus infinity by the weight's sign, NaN where the weight is 0; with two of them
    or a NaN, what their sum is.  The other rows are those of a call without."""
    note(f"matvec with infinities and NaN, {rows}x{cin} {x}")
    cout = 40
    code, fp4, amax = weights(1, cout, cin, cin)
    w = decode.weights(code[0], fp4[0], amax[0])
    t = torch.randn(rows, cin, generator=gen(rows)).to(TYPES[x])
    args = on_gpu(code, fp4, amax)
    good = lh.lh_matvec(t.to(DEV), *args).cpu()
    for row, put in ((0, {3: "inf"}), (rows - 1, {cin - 1: "-inf"}), (rows // 2, {1: "inf", cin - 2: "inf"}),
                     (0, {5: "nan"}), (rows - 1, {0: "inf", 17: "-inf"})):
        bad = t.clone()
        for at, v in put.items():
            bad[row, at] = float(v)
        got = lh.lh_matvec(bad.to(DEV), *args).cpu()
        with np.errstate(invalid="ignore"):
            want = np.stack([f64(bad[row, list(put)]) * w[c, list(put)] for c in range(cout)]).sum(1)
        others = [r for r in range(rows) if r != row]
        assert torch.equal(got[others], good[others])
        assert np.array_equal(f64(got[row]), want, equal_nan=True), put


def test_matvec_keeps_a_nan_of_any_payload():
    note("matvec, NaN payloads")
    code, fp4, amax = on_gpu(*weights(1, 24, 160, 2))
    for bits in (0x7F800001, 0x7FC00000, -1, -0x7FFFFF):            # the last: 0xFF800001
        t = torch.randn(3, 160, generator=gen(4))
        t.view(torch.int32)[1, 40] = bits
        y = lh.lh_matvec(t.to(DEV), code, fp4, amax).cpu()
        assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2]]).all()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("cin", [144, 2064, 4112])
def test_matvec_of_nan_codes_and_scales(group, cin):
    """A NaN code or a NaN scale of an E4M3 row, as the norm writes it, makes the row NaN and no other."""
    note(f"matvec with NaN codes, cin {cin} group {group}")
    rows = 6
    args = on_gpu(*weights(1, 40, cin, 1))
    q = (torch.randn(rows, cin, generator=gen(cin)) * 20).to(torch.float8_e4m3fn)
    s = torch.rand(rows, -(-cin // 128) if group else 1, generator=gen(3)) + 0.5
    good = lh.lh_matvec(q.to(DEV), *args, x_scale=s.to(DEV), x_group=group).cpu()
    bq, bs = q.clone(), s.clone()
    bq.view(torch.uint8)[1, cin - 3], bs[4, -1] = 0xFF, float("nan")
    bq.view(torch.uint8)[4] = 0                                    # the codes under it are 0
    got = lh.lh_matvec(bq.to(DEV), *args, x_scale=bs.to(DEV), x_group=group).cpu()
    assert torch.isnan(got[[1, 4]]).all() and torch.equal(got[[0, 2, 3, 5]], good[[0, 2, 3, 5]])


def test_matvec_of_the_smallest_fp32_rows():
    """The three bf16 pieces of an fp32 element hold it to within 2^-133, the smallest bf16 number, and exactly from 2^-110 on."""
    rows, cin, cout = 6, 272, 24
    note("matvec of fp32 rows from 2^-149 to 2^-100")
    code, fp4, _ = weights(1, cout, cin, 8)
    amax = np.array([2.0 ** 110], np.float32)
    x = torch.randn(rows, cin, generator=gen(8)) * torch.tensor([2.0 ** -e for e in (100, 111, 118, 126, 133, 145)])[:, None]
    y = f64(lh.lh_matvec(x.to(DEV), *on_gpu(code, fp4, amax)))
    w = decode.weights(code[0], fp4[0], amax[0])
    held = np.where(np.abs(f64(x)) >= 2.0 ** -110, 0.0, 2.0 ** -133)
    tol = 2 * (cin + 8) * U * (np.abs(f64(x)) @ np.abs(w).T) + held @ np.abs(w).T
    # a sum of products under fp32's normal numbers is itself held to 2^-149 a term, times the matrix' scale
    tol = tol + cin * TINY * float(amax[0] / np.float32(2688.0))
    assert np.all(np.abs(y - f64(x) @ w.T) <= tol)


# ----------------------------------------------------------------------------------------- the cache
@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("amax", [3.0, 1e-34])
def test_cache_holds_nan_and_saturates_infinities(four, dtype, amax):
    """A NaN reads back as NaN, alone in E4M3 and with its 16 elements in NVFP4; an infinity is written as the largest finite
    number would be; everything else is as without them.  Attention over a held NaN gives NaN to the heads that read it."""
    note(f"cache of NaN and infinities, four {four} {dtype} amax {amax}")
    tokens, heads, dim, t = 37, 2, 64, TYPES[dtype]
    x = (torch.randn(2, tokens, heads, dim, generator=gen(6)) * amax / 3).to(t)
    plain = x.clone()
    big = torch.finfo(t).max
    put = [(0, 3, 0, 5, "nan"), (0, 3, 0, 40, "-nan"), (1, 20, 1, 63, "nan"), (0, 9, 1, 0, "inf"), (1, 9, 1, 17, "-inf"), (1, 36, 0, 2, "nan")]
    for i, tok, h, d, v in put:
        x[i, tok, h, d] = float("nan") if "nan" in v else float(v)
        if "nan" not in v:
            plain[i, tok, h, d] = big if v == "inf" else -big
    a = (torch.full((heads,), amax), torch.full((heads,), amax))
    slots = torch.randperm(48, generator=gen(1))[:tokens].to(DEV)
    back, caches = [], []
    for data in (x, plain):
        cache = make_cache(3, 16, heads, dim, four, a)
        lh.lh_cache_write(cache, data[0].to(DEV), data[1].to(DEV), slots)
        back.append(torch.stack(lh.lh_cache_read(cache, slots, dtype=torch.float32)).cpu())
        caches.append(cache)
    nan = torch.zeros(x.shape, dtype=torch.bool)
    for i, tok, h, d, v in put:
        if "nan" in v:
            nan[i, tok, h, slice(d // 16 * 16, d // 16 * 16 + 16) if four else d] = True
    assert torch.equal(torch.isnan(back[0]), nan)
    assert torch.equal(back[0][~nan], back[1][~nan])
    assert torch.isfinite(back[1]).all()

    # tokens 0..36 in order, by pages of one token: head 0 meets the NaN of K, or of V past it; head 1 that of V
    pages = {n: getattr(caches[0], n) for n in ("k", "v", "k_scale", "v_scale")}
    def by_token(p):                     # noqa: E306
        return None if p is None else p.permute(0, 2, 1, 3).reshape(48, heads, 1, -1).contiguous()
    one = lh.Cache(by_token(pages["k"]), by_token(pages["v"]), caches[0].k_amax, caches[0].v_amax, by_token(pages["k_scale"]), by_token(pages["v_scale"]))
    q = torch.randn(3, 2 * heads, dim, generator=gen(2)).to(t).to(DEV)
    table = slots.to(torch.int32).expand(3, tokens).contiguous()
    o = lh.lh_paged_attention(q, one, table, torch.tensor([3, 20, 37], dtype=torch.int32, device=DEV), scale=0.125).float().cpu()
    assert torch.isfinite(o[0]).all() and torch.isfinite(o[1, 2:]).all()
    assert torch.isnan(o[1, :2]).all() and torch.isnan(o[2, :2]).all()
    assert torch.isnan(o[2, 2:]).any(-1).all()


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("dim", [96, 128, 272])
def test_cache_slots_named_twice_disturb_no_other(four, dim):
    """Tokens 3, 40 and 77 share a slot, whose contents are unspecified; every other one holds its token."""
    note(f"cache, a slot named three times, dim {dim} four {four}")
    heads, tokens = 3, 90
    x = torch.randn(2, tokens, heads, dim, generator=gen(dim)).to(DEV)
    a = (torch.full((heads,), 4.0), torch.full((heads,), 4.0))
    slots = torch.randperm(7 * 16, generator=gen(9))[:tokens].to(DEV)
    apart = make_cache(7, 16, heads, dim, four, a)
    lh.lh_cache_write(apart, x[0], x[1], slots)
    shared = slots.clone()
    shared[40] = shared[77] = shared[3]
    cache = make_cache(7, 16, heads, dim, four, a)
    lh.lh_cache_write(cache, x[0], x[1], shared)
    keep = torch.ones(tokens, dtype=torch.bool)
    keep[[3, 40, 77]] = False
    for got, want in zip(lh.lh_cache_read(cache, slots[keep.to(DEV)]), lh.lh_cache_read(apart, slots[keep.to(DEV)])):
        assert torch.equal(got, want)
    for got in lh.lh_cache_read(cache, slots[[40, 77]]):
        assert torch.count_nonzero(got) == 0                       # not named any more: as they were


def test_cache_attributes_are_fixed():
    """The kernels read the tensors that the Cache was made with; another one is refused, its values can be copied."""
    note("cache, attributes assigned")
    cache = make_cache(2, 16, 1, 64, True, (torch.ones(1), torch.ones(1)))
    kept = {n: getattr(cache, n) for n in ("k", "v", "k_amax", "v_amax", "k_scale", "v_scale", "n_pages", "n_heads", "page_size", "head_dim")}
    for name, value in kept.items():
        with pytest.raises(AttributeError, match=name):
            setattr(cache, name, value.clone() if torch.is_tensor(value) else value + 1)
        with pytest.raises(AttributeError, match=name):
            delattr(cache, name)
        assert getattr(cache, name) is value
    cache.label = "layer 3"                                        # the caller's own are not in the way
    x, slots = torch.full((1, 1, 64), 8.0, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    for amax, held in ((1.0, 1.0), (4.0, 4.0)):                    # every element saturates
        cache.k_amax.copy_(torch.tensor([amax]))
        lh.lh_cache_write(cache, x, x, slots)
        assert abs(float(lh.lh_cache_read(cache, slots, dtype=torch.float32)[0].max()) - held) <= 2 ** -22 * held


# ----------------------------------------------------------------------------------- launches' limits
def test_norm_of_as_many_rows_as_a_launch_takes():
    rows, cin = 2 ** 26, 16
    note(f"norm of {rows} rows, refused, and of 4 fewer")
    x = torch.empty(rows, cin, dtype=torch.bfloat16, device=DEV)
    gamma = torch.ones(cin, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(lh.LHError) as e:
        lh.lh_rms_norm_quant(x, gamma)
    assert e.value.code == lh.LH_ERR_INVALID_ARGUMENT and "too large" in e.value.message
    x[-5:] = torch.randn(5, cin, generator=gen(3)).bfloat16()
    x[:5] = x[-5:]
    q, s, _ = lh.lh_rms_norm_quant(x[:-4], gamma)
    assert torch.equal(s[-1], s[0]) and torch.equal(q[-1].view(torch.uint8), q[0].view(torch.uint8)) and float(s[0]) > 0


def test_attention_of_more_sequences_than_a_launch_takes():
    batch, heads = 2 ** 21, 8
    note(f"attention of {batch} sequences of {heads} heads, refused, and of one fewer, all but one empty")
    cache = make_cache(2, 16, heads, 64, True, (torch.ones(heads), torch.ones(heads)))
    cache.v.fill_(0x22)                                            # 1.0
    cache.v_scale.fill_(0x38)                                      # 1.0
    q = torch.empty(batch, heads, 64, dtype=torch.bfloat16, device=DEV)
    table, lengths = torch.ones(batch, 1, dtype=torch.int32, device=DEV), torch.zeros(batch, dtype=torch.int32, device=DEV)
    with pytest.raises(lh.LHError) as e:
        lh.lh_paged_attention(q, cache, table, lengths, scale=0.125)
    assert e.value.code == lh.LH_ERR_INVALID_ARGUMENT and "too large" in e.value.message
    q[-2] = 0
    lengths[-2] = 11
    o = lh.lh_paged_attention(q[:-1], cache, table[:-1], lengths[:-1], scale=0.125)
    assert torch.count_nonzero(o[:-1]) == 0 and bool((o[-1] == torch.tensor(1 / 2688.0).bfloat16().to(DEV)).all())


# ----------------------------------------------------------------------------------------- attention
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("four", [True, False])
def test_attention_holds_q_to_a_part_of_its_largest_element(dtype, four):
    """Two tokens, equal but for element 1 of K, which is 1 and 0; V is 1 and 0, so o is the logistic function of scale * q1 and
    gives q1 back as it was held.  q's largest element meets zeros of K.  The bound is 2^-39 of it, and nothing at all (for
    fp32 2^-22 of q1) for elements from 2^-31 of it on."""
    note(f"attention, q far apart, four {four} {dtype}")
    t, one = TYPES[dtype], 0x38                                    # E4M3's 1, also a scale's
    amax = 2688.0 if four else 448.0
    cache = make_cache(1, 2, 1, 64, four, (torch.tensor([amax]), torch.tensor([amax])))
    for tensor, scales, at in ((cache.k, cache.k_scale, 1), (cache.v, cache.v_scale, slice(0, 64))):
        values = torch.zeros(64, dtype=torch.uint8)
        values[at] = 2 if four else one
        tensor[0, 0, 0] = (values[0::2] | (values[1::2] << 4) if four else values).to(DEV)
        if four:
            scales.fill_(one)
    table, lengths = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.tensor([2], dtype=torch.int32, device=DEV)
    for top in (2.0 ** 14, 1.99 * 2.0 ** 14, 2.0 ** 40, 3e-20):
        for e in (-10, -22, -29, -31, -33, -35, -37, -38):
            for f in (1.0, 1.296875, 1.5, 1.703125, -1.9921875):
                q = torch.zeros(1, 1, 64, dtype=torch.float64)
                q[0, 0, 0], q[0, 0, 1] = top, f * 2.0 ** e * top
                q = q.to(t)
                q0, q1 = float(q[0, 0, 0]), float(q[0, 0, 1])
                scale = float(np.float32(1.0 / abs(q1)))
                o = float(lh.lh_paged_attention(q.to(DEV), cache, table, lengths, scale=scale)[0, 0, 0])
                held = np.log(o / (1 - o)) / scale
                # o is off by its type's rounding and a few fp32 ones; d log(o / (1 - o)) = do / (o (1 - o))
                off = ((2.0 ** -9 if dtype == "bf16" else 0) + (2.0 ** -11 if dtype == "bf16" else 2.0 ** -21) + 16 * U) * o / (o * (1 - o)) / scale
                bound = 0.0 if abs(q1) >= 2.0 ** -31 * q0 else 2.0 ** -39 * q0
                if dtype == "f32":
                    bound = max(2.0 ** -39 * q0, 2.0 ** -22 * abs(q1))
                assert abs(held - q1) <= bound + off, (top, e, f, held / q1, bound / abs(q1), off / abs(q1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("four", [True, False])
def test_attention_of_queries_with_nan_and_infinities(dtype, four):
    """Such a head gives NaN, the others what they give without it; an empty sequence gives 0 all the same."""
    note(f"attention, NaN and infinite q, four {four} {dtype}")
    cache, table, lengths, q, _ = attention_case([700, 0, 33], 2, 4, 64, 16, four, dtype, 12)
    good = lh.lh_paged_attention(q.to(DEV), cache, table, lengths, scale=0.125)
    bad = q.clone()
    bad[0, 1, 5], bad[0, 6, 63], bad[1, 0, 0], bad[2, 3, 9] = float("nan"), float("inf"), float("nan"), -float("inf")
    o = lh.lh_paged_attention(bad.to(DEV), cache, table, lengths, scale=0.125)
    nan = torch.zeros(3, 8, dtype=torch.bool, device=DEV)
    nan[0, 1] = nan[0, 6] = nan[2, 3] = True
    assert torch.isnan(o[nan]).all() and torch.equal(o[~nan], good[~nan])
    assert torch.count_nonzero(o[1]) == 0
