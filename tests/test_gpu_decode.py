"""The decode-step operators on the GPU against the float64 oracle, with tolerances derived from their
arithmetic, and their behaviour at empty, odd, strided, out-of-range and very long inputs."""
import numpy as np
import pytest
import torch

from oracle import decode

pytestmark = pytest.mark.gpu

lh = pytest.importorskip("nvfp4_scale_calibration_lh_amd")
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24                       # fp32 unit roundoff


def note(msg):
    print(f"[case] {msg}", flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(t):
    return t.detach().cpu().double().numpy()


# ----------------------------------------------------------------------------------------- the norm
@pytest.mark.parametrize("rows,cin", [(1, 16), (3, 128), (5, 144), (1, 2048), (2, 4096), (7, 2560), (2, 12288),
                                      (1, 16384), (3, 16400), (1, 40016), (300, 1008)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("residual", [True, False])
def test_norm(rows, cin, dtype, group, residual):
    note(f"norm {rows}x{cin} {dtype} group {group} residual {residual}")
    t, g = TYPES[dtype], gen(rows * cin)
    x = torch.randn(rows, cin, generator=g).to(t)
    r = (torch.randn(rows, cin, generator=g) * 3).to(t) if residual else None
    gamma = (1 + 0.3 * torch.randn(cin, generator=g)).to(t)
    if rows > 2:
        x[1] = 0
        if residual:
            r[1] = 0
    h = x if r is None else (x.float() + r.float()).to(t)
    q, scale, summed = lh.lh_rms_norm_quant(x.to(DEV), gamma.to(DEV), None if r is None else r.to(DEV), eps=1e-5, group=group)
    assert (summed is None) == (r is None)
    if r is not None:
        assert torch.equal(summed.cpu(), h)
    check_norm(q, scale, f64(h), f64(gamma), 1e-5, group)


def check_norm(q, scale, h, gamma, eps, group):
    """scale within the sum's rounding, q within half a step of y / scale.  The sum of squares adds at most cin / 64
    terms in a chain and a tree after it; its square root halves the relative error, and seven further roundings
    lead to scale.  q rounds to 4 significant bits (2^-4 of itself) or to 2^-10 below 2^-6."""
    y, s = decode.rms_norm(h, gamma, eps, group)
    rel = (h.shape[1] / 64 + 16) / 2 * U + 8 * U
    got = f64(scale)
    assert got.shape == s.shape
    assert np.all(np.abs(got - s) <= rel * s)
    width = group or h.shape[1]
    wide = np.repeat(got, width, axis=1)[:, :h.shape[1]]
    v = f64(q) * wide
    assert np.isfinite(v).all()
    assert np.all(np.abs(v - y) <= np.maximum(np.abs(y) * 2.0 ** -4, wide * 2.0 ** -10) * (1 + 2 ** -10) + 2 * rel * np.abs(y))


def test_norm_in_place_and_tiny_scales():
    g = gen(5)
    x, r = torch.randn(4, 640, generator=g).bfloat16(), torch.randn(4, 640, generator=g).bfloat16()
    gamma = torch.ones(640, dtype=torch.bfloat16)
    h = (x.float() + r.float()).bfloat16()
    for which in ("x", "residual"):
        note(f"norm in place of {which}")
        xd, rd = x.to(DEV), r.to(DEV)
        q, s, summed = lh.lh_rms_norm_quant(xd, gamma.to(DEV), rd, summed=xd if which == "x" else rd)
        assert torch.equal(summed.cpu(), h) and summed.data_ptr() == (xd if which == "x" else rd).data_ptr()
        check_norm(q, s, f64(h), f64(gamma), 1e-6, 0)
    note("norm with scales under 2^-100 and eps 0")
    x = torch.randn(3, 256, generator=g)
    x[1] = 0
    gamma = torch.full((256,), 1e-35)
    q, s, _ = lh.lh_rms_norm_quant(x.to(DEV), gamma.to(DEV), eps=0.0)
    assert torch.count_nonzero(q[1].float()) == 0 and float(s[1]) == 0.0
    y, want = decode.rms_norm(f64(x), f64(gamma), 1e-300, 0)
    keep = [0, 2]
    assert np.all(np.abs(f64(s) - want)[keep] <= 1e-5 * want[keep])
    assert np.all(np.abs(f64(q) * f64(s) - y)[keep] <= np.maximum(np.abs(y) * 2.0 ** -4, f64(s) * 2.0 ** -10)[keep] * (1 + 1e-4))


def test_norm_no_rows():
    q, s, summed = lh.lh_rms_norm_quant(torch.empty(0, 32, device=DEV), torch.ones(32, device=DEV))
    assert q.shape == (0, 32) and s.shape == (0, 1) and summed is None


# -------------------------------------------------------------------------------------- the products
def weights(groups, cout, cin, seed):
    r = np.random.default_rng(seed)
    code = r.integers(1, 127, (groups, cout, cin // 16)).astype(np.uint8)
    fp4 = r.integers(0, 256, (groups, cout, cin // 2)).astype(np.uint8)
    amax = (0.1 + r.random(groups)).astype(np.float32)
    return code, fp4, amax


def rows_of(rows, cin, x, group, seed):
    """(tensor, x_scale tensor or None, values in float64)"""
    g = gen(seed)
    v = torch.randn(rows, cin, generator=g) * torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g).float())
    if x != "e4m3":
        t = v.to(TYPES[x])
        return t, None, f64(t)
    n = -(-cin // group) if group else 1
    s = torch.exp2(torch.randn(rows, n, generator=g))
    q = (v * 10).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q, s, f64(q.float()) * np.repeat(f64(s), group or cin, axis=1)[:, :cin]


def check_product(y, x, code, fp4, amax, offsets, norm=448.0):
    """Products are exact; a row's sum of cin + a few terms in fp32 is within (cin + 8) U of the sum of magnitudes;
    a factor 2 for matrix instructions that truncate.  bf16 rounds the result by at most 2^-9 of it."""
    got = f64(y)
    for g in range(len(offsets) - 1):
        a, b = offsets[g], offsets[g + 1]
        if a == b:
            continue
        w = decode.weights(code[g], fp4[g], amax[g], norm)
        want, mag = x[a:b] @ w.T, np.abs(x[a:b]) @ np.abs(w).T
        tol = 2 * (x.shape[1] + 8) * U * mag + (np.abs(want) * 2.0 ** -8 if y.dtype == torch.bfloat16 else 0)
        bad = np.abs(got[a:b] - want) > tol
        assert not bad.any(), f"group {g}: {bad.sum()} of {bad.size}; worst {np.nanmax(np.abs(got[a:b] - want) / tol)}"


@pytest.mark.parametrize("rows", [1, 2, 4, 5, 8, 9, 16, 17, 33, 64, 65, 130])
@pytest.mark.parametrize("cout,cin", [(1, 16), (16, 128), (33, 144), (70, 1040), (100, 2064), (257, 4096)])
@pytest.mark.parametrize("x,group", [("bf16", 0), ("f32", 0), ("e4m3", 0), ("e4m3", 128)])
def test_matvec(rows, cout, cin, x, group):
    note(f"matvec {rows}x{cin} -> {cout} {x} group {group}")
    code, fp4, amax = weights(1, cout, cin, rows + cin)
    t, s, v = rows_of(rows, cin, x, group, rows)
    y = lh.lh_matvec(t.to(DEV), torch.from_numpy(code).to(DEV), torch.from_numpy(fp4).to(DEV), torch.from_numpy(amax).to(DEV),
                     x_scale=None if s is None else s.to(DEV), x_group=group)
    assert y.dtype == (torch.float32 if x == "f32" else torch.bfloat16)
    check_product(y, v, code, fp4, amax, [0, rows])


@pytest.mark.parametrize("x,group", [("bf16", 0), ("f32", 0), ("e4m3", 128)])
@pytest.mark.parametrize("counts", [[1, 0, 3], [0, 0, 0, 17, 0, 40, 1], [0] * 299 + [2] + [0] * 300 + [5, 1, 0], [0, 0, 7], [7, 0]])
def test_matvec_experts(x, group, counts):
    cout, cin = 90, 272
    note(f"matvec experts {len(counts)} groups, {sum(counts)} rows, {x}")
    code, fp4, amax = weights(len(counts), cout, cin, 7)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    t, s, v = rows_of(int(off[-1]), cin, x, group, 3)
    y = lh.lh_matvec(t.to(DEV), torch.from_numpy(code).to(DEV), torch.from_numpy(fp4).to(DEV), torch.from_numpy(amax).to(DEV),
                     x_scale=None if s is None else s.to(DEV), x_group=group, offsets=torch.from_numpy(off).to(DEV), norm=256.0)
    check_product(y, v, code, fp4, amax, off, 256.0)


def test_matvec_agrees_with_dequantized_weights():
    note("matvec on a sweep's result")
    W = torch.randn(1, 96, 256, generator=gen(1)).mul(0.02).bfloat16().to(DEV)
    amax = lh.lh_absmax(W)
    code, fp4, _ = lh.lh_scale_sweep_mse(W, amax)
    Wq, _ = lh.lh_dequantize(code, fp4, amax, dtype=torch.float32)
    x = torch.randn(6, 256, generator=gen(2)).to(DEV)
    y = lh.lh_matvec(x, code, fp4, amax)
    want, mag = f64(x) @ f64(Wq[0]).T, np.abs(f64(x)) @ np.abs(f64(Wq[0])).T
    assert np.all(np.abs(f64(y) - want) <= 2 * (256 + 10) * U * mag)


def test_matvec_no_rows_no_channels():
    code, fp4, amax = (torch.from_numpy(a).to(DEV) for a in weights(2, 4, 32, 0))
    off = torch.zeros(3, dtype=torch.int64, device=DEV)
    assert lh.lh_matvec(torch.empty(0, 32, device=DEV), code, fp4, amax, offsets=off).shape == (0, 4)
    assert lh.lh_matvec(torch.ones(3, 32, device=DEV), code[:1, :0].contiguous(), fp4[:1, :0].contiguous(), amax[:1]).shape == (3, 0)


def test_matvec_weights_past_four_gigabytes():
    note("matvec, last expert past 2^32 bytes of nibbles")
    G, cout, cin = 2100, 1024, 4096
    code = torch.zeros(G, cout, cin // 16, dtype=torch.uint8, device=DEV)
    fp4 = torch.zeros(G, cout, cin // 2, dtype=torch.uint8, device=DEV)
    assert fp4.numel() > 2 ** 32
    c, f, a = weights(1, cout, cin, 9)
    code[-1], fp4[-1] = torch.from_numpy(c[0]).to(DEV), torch.from_numpy(f[0]).to(DEV)
    amax = torch.full((G,), float(a[0]), device=DEV)
    off = torch.zeros(G + 1, dtype=torch.int64, device=DEV)
    off[-1] = 3
    t, _, v = rows_of(3, cin, "bf16", 0, 4)
    y = lh.lh_matvec(t.to(DEV), code, fp4, amax, offsets=off)
    check_product(y, v, c, f, a, [0, 3])


# ----------------------------------------------------------------------------------------- the cache
def make_cache(pages, page, heads, dim, four, amax, fill=None):
    c = lh.Cache.empty(pages, page, heads, dim, amax[0].to(DEV), amax[1].to(DEV), four_bit=four)
    if fill is not None:
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            if t is not None:
                t.fill_(fill)
    return c


def paged(t, slots, page):
    """Rows [tokens, heads, n] of a cache tensor at the slots, as numpy."""
    a = t.cpu().numpy()
    return a[slots // page, :, slots % page]


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,heads,dim,page", [(1, 1, 16, 1), (5, 3, 96, 7), (33, 2, 64, 24), (70, 8, 128, 16), (9, 1, 272, 5)])
def test_cache_write_and_read(four, dtype, tokens, heads, dim, page):
    note(f"cache {tokens}x{heads}x{dim} page {page} four {four} {dtype}")
    g, t = gen(tokens + dim), TYPES[dtype]
    pages = -(-tokens // page) + 2
    qkv = torch.randn(tokens, 3 * heads, dim, generator=g)
    qkv[:, :, ::5] *= 20
    qkv[0, :, :16] = 0
    qkv = qkv.to(t)
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    amax = (k.float().abs().amax((0, 2)).clamp(min=1e-3), v.float().abs().amax((0, 2)) * 0.7)     # v saturates
    amax[1][0] = 0.0
    cache = make_cache(pages, page, heads, dim, four, amax, fill=0x5A)
    slots = np.random.default_rng(dim).permutation(pages * page)[:tokens].astype(np.int64)
    sd = slots.copy()
    if tokens > 4:
        sd[2], sd[3] = -1, pages * page                  # skipped
    keep = (sd >= 0) & (sd < pages * page)
    d = qkv.to(DEV)
    lh.lh_cache_write(cache, d[:, heads:2 * heads], d[:, 2 * heads:], torch.from_numpy(sd).to(DEV))
    K, V = lh.lh_cache_read(cache, torch.from_numpy(sd).to(DEV), dtype=t)
    for name, x, a, back in (("k", k, amax[0], K), ("v", v, amax[1], V)):
        codes, scales = decode.cache_codes(f64(x), a.numpy(), four)
        held = getattr(cache, name)
        assert np.array_equal(paged(held, slots[keep], page), codes[keep])
        others = np.setdiff1d(np.arange(pages * page), slots[keep])
        assert (paged(held, others, page) == 0x5A).all()
        if four:
            s = getattr(cache, name + "_scale")
            assert np.array_equal(paged(s, slots[keep], page), scales[keep])
            assert (paged(s, others, page) == 0x5A).all()
        want = torch.from_numpy(decode.cache_values(codes, scales, a.numpy(), four).astype(np.float32)).to(t)
        want[torch.from_numpy(~keep)] = 0
        assert torch.equal(back.cpu(), want)


@pytest.mark.parametrize("four", [True, False])
def test_cache_rounds_ties_and_neighbours_exactly(four):
    """Every midpoint of the E4M3 or E2M1 grid times the scale and its fp32 neighbours; amax from 1e-38 to 1e38."""
    for amax in (1.0, 2.3, 0.0071, 3e-31, 1e-33, 1e-37, 4e30, 1e37):
        note(f"cache ties, four {four}, amax {amax}")
        a = torch.tensor([amax], dtype=torch.float32)
        unit = decode.cache_unit(a.numpy(), four)[0]
        if four:
            mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * np.float64(np.float32(448.0 * unit))
            rows = []
            for m in mids.astype(np.float32):
                for x in (np.nextafter(m, np.float32(0)), m, np.nextafter(m, np.float32(np.inf))):
                    row = np.zeros(16, np.float32)
                    row[0], row[1], row[2] = 6 * 448.0 * unit, x, -x
                    rows.append(row)
            vals = decode.e4m3_values(np.arange(127))
            for m in ((vals[1:] + vals[:-1]) / 2 * 6 * unit).astype(np.float32):      # block scales at midpoints
                for x in (np.nextafter(m, np.float32(0)), m, np.nextafter(m, np.float32(np.inf))):
                    row = np.full(16, x / 3, np.float32)
                    row[3] = x
                    rows.append(row)
        else:
            vals = decode.e4m3_values(np.arange(127))
            m = ((vals[1:] + vals[:-1]) / 2 * unit).astype(np.float32)
            x = np.concatenate([np.nextafter(m, np.float32(0)), m, np.nextafter(m, np.float32(np.inf))])
            x = np.concatenate([x, -x])
            rows = np.resize(x, (-(-x.size // 16), 16))
        x = torch.from_numpy(np.stack(rows).astype(np.float32)).reshape(-1, 1, 16)
        n = x.shape[0]
        cache = make_cache(n, 1, 1, 16, four, (a, a))
        lh.lh_cache_write(cache, x.to(DEV), x.to(DEV), torch.arange(n, device=DEV))
        codes, scales = decode.cache_codes(f64(x), a.numpy(), four)
        for name in ("k", "v"):
            assert np.array_equal(getattr(cache, name).cpu().numpy()[:, :, 0], codes)
            if four:
                assert np.array_equal(getattr(cache, name + "_scale").cpu().numpy()[:, :, 0], scales)


def test_cache_no_tokens():
    cache = make_cache(2, 4, 1, 64, True, (torch.ones(1), torch.ones(1)))
    e = torch.empty(0, 1, 64, device=DEV)
    slots = torch.empty(0, dtype=torch.int64, device=DEV)
    lh.lh_cache_write(cache, e, e, slots)
    assert lh.lh_cache_read(cache, slots)[0].shape == (0, 1, 64)


# ----------------------------------------------------------------------------------------- attention
def attention_case(lens, heads, share, dim, page, four, dtype, seed, pad_pages=3, spread=1.0):
    """A cache with random codes; unused slots and pages hold NaN codes and the table's unused entries -1."""
    r = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + pad_pages
    amax = [torch.from_numpy((0.5 + r.random(heads)).astype(np.float32) * 4) for _ in range(2)]
    cache = make_cache(pages, page, heads, dim, four, amax, fill=0xFF if not four else 0x7F)
    table = np.full((len(lens), max(need + [1]) + 2), -1, np.int32)
    order = r.permutation(pages)
    host = {n: (None if getattr(cache, n) is None else getattr(cache, n).cpu().numpy()) for n in ("k", "v", "k_scale", "v_scale")}
    values = []
    for b, n in enumerate(lens):
        mine = order[sum(need[:b]):sum(need[:b]) + need[b]]
        table[b, :need[b]] = mine
        t = np.arange(n)
        per = []
        for i, name in enumerate(("k", "v")):
            x = r.standard_normal((n, heads, dim)) * spread
            codes, scales = decode.cache_codes(x.astype(np.float32), amax[i].numpy(), four)
            if n:
                host[name][mine[t // page], :, t % page] = codes
                if four:
                    host[name + "_scale"][mine[t // page], :, t % page] = scales
            unit = decode.cache_unit(amax[i].numpy(), four)[:, None]
            if four:      # the values attention uses: E2M1 * v * g, unrounded
                per.append(decode.e2m1_values(codes) * np.repeat(decode.e4m3_values(scales), 16, -1) * unit)
            else:
                per.append(decode.e4m3_values(codes) * unit)
        values.append(per)
    for n, a in host.items():
        if a is not None:
            getattr(cache, n).copy_(torch.from_numpy(a))
    q = torch.from_numpy(r.standard_normal((len(lens), heads * share, dim)) * 1.3).to(TYPES[dtype])
    return cache, torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), q, values


def check_attention(o, q, values, heads, share, dim, scale):
    """The error of o against sum p |v|: a score's error ds gives p a relative error ds in p and in the sum of p.  ds is at
    most D + 4 roundings of sum |q k| scale (twice for matrix instructions that truncate; an fp32 q is held to 2^-22),
    and in base 2 two roundings of numbers under 2^7 + 2^7 (times ln 2).  p is rounded to fp16 (2^-11), or to two pieces (2^-21);
    each sum of up to n / 4 terms in a chain adds n U.  bf16 rounds the result by 2^-9 of it."""
    got, x = f64(o), f64(q)
    worst = 0.0
    for b, (k, v) in enumerate(values):
        n = k.shape[0]
        for h in range(heads * share):
            want, mag, qk = decode.attention(x[b, h], k[:, h // share], v[:, h // share], scale)
            f32 = q.dtype == torch.float32
            ds = (2 * (dim + 4) * U + (2.0 ** -22 if f32 else 0)) * qk * abs(scale) + 2.0 ** -15
            tol = (2 * ds + (2.0 ** -21 if f32 else 2.0 ** -11) + 2 * (n + 16) * U) * mag
            tol = tol + (0 if f32 else np.abs(want) * 2.0 ** -8) + 1e-30
            err = np.abs(got[b, h] - want)
            assert np.all(err <= tol), f"sequence {b} ({n} tokens) head {h}: {(err / tol).max()}"
            worst = max(worst, float((err / tol).max()))
    return worst


LENS = [[1], [0], [31, 0, 32, 33], [16, 17, 15, 1], [127, 128, 129, 255, 256, 257], [700, 3, 0, 1100]]


@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v)))
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("four,dtype", [(True, "bf16"), (False, "bf16"), (True, "f32"), (False, "f32")])
@pytest.mark.parametrize("page", [16, 24, 1])
def test_attention(lens, dim, four, dtype, page):
    note(f"attention lens {lens} dim {dim} four {four} {dtype} page {page}")
    heads, share = (2, 4) if dim != 128 else (1, 7)
    cache, table, lengths, q, values = attention_case(lens, heads, share, dim, page, four, dtype, dim + page)
    o = lh.lh_paged_attention(q.to(DEV), cache, table, lengths, scale=dim ** -0.5)
    check_attention(o, q, values, heads, share, dim, dim ** -0.5)


@pytest.mark.parametrize("share", [1, 16, 17, 40])
@pytest.mark.parametrize("page", [16, 48, 64, 7])
def test_attention_head_layouts(share, page):
    note(f"attention share {share} page {page}")
    cache, table, lengths, q, values = attention_case([5, 400, 90], 2, share, 64, page, True, "bf16", share)
    o = lh.lh_paged_attention(q.to(DEV), cache, table, lengths, scale=0.2)
    check_attention(o, q, values, 2, share, 64, 0.2)


def test_attention_strided_queries_and_sharp_scores():
    """q as a part of a wider projection; scores tens apart, so the running maximum moves and most p vanish."""
    note("attention strided, sharp")
    for dtype in ("bf16", "f32"):
        cache, table, lengths, q, values = attention_case([600, 41], 2, 4, 128, 16, True, dtype, 3)
        wide = torch.zeros(2, 12, 128, dtype=TYPES[dtype])
        wide[:, :8] = q
        o = lh.lh_paged_attention(wide.to(DEV)[:, :8], cache, table, lengths, scale=1.0)
        check_attention(o, q, values, 2, 4, 128, 1.0)
        note("attention with a negative and a zero scale")
        for scale in (-0.3, 0.0):
            o = lh.lh_paged_attention(q.to(DEV), cache, table, lengths, scale=scale)
            check_attention(o, q, values, 2, 4, 128, scale)


@pytest.mark.parametrize("size", [1e-30, 1e-3, 1e6, 1e30])
def test_attention_queries_of_any_size(size):
    """q far from 1 is brought to fp16's range by a power of two per head; the scale undoes it."""
    note(f"attention q of size {size}")
    for dtype in ("bf16", "f32"):
        cache, table, lengths, q, values = attention_case([300], 1, 3, 64, 16, True, dtype, 8)
        q = (q.double() * torch.tensor([size, 0.0, size * 2.0 ** -12]).double()[None, :, None]).to(TYPES[dtype])
        scale = float(np.float32(0.125 / size))
        o = lh.lh_paged_attention(q.to(DEV), cache, table, lengths, scale=scale)
        check_attention(o, q, values, 1, 3, 64, scale)


def test_attention_one_long_sequence():
    note("attention, 40001 tokens")
    cache, table, lengths, q, values = attention_case([40001, 9], 1, 2, 64, 16, True, "f32", 4)
    o = lh.lh_paged_attention(q.to(DEV), cache, table, lengths, scale=0.125)
    check_attention(o, q, values, 1, 2, 64, 0.125)


def uneven(n, most, seed):
    """n lengths up to `most`, a few of them empty and one longer than all others together would suggest."""
    r = np.random.default_rng(seed)
    lens = (most * r.random(n) ** 3).astype(int)
    lens[r.permutation(n)[:n // 8]] = 0
    lens[n // 3] = 4 * most
    return lens.tolist()


# (lengths, heads, share): up to 64 sequences cut to one length, by what is resident or by twice that; more
# than 64 with equal counts; enough to fill the card uncut; key-value heads in more than one tile
CUTS = [(uneven(64, 1200, 1), 1, 2), (uneven(63, 700, 2), 3, 1), (uneven(65, 600, 3), 1, 2), (uneven(200, 500, 4), 1, 1),
        (uneven(5, 2000, 5), 40, 1), ([2111], 96, 1), ([1300, 0, 2700], 3, 17), ([513, 0], 1, 1), (uneven(130, 300, 6), 8, 1)]


@pytest.mark.parametrize("lens,heads,share", CUTS, ids=lambda v: f"{len(v)}x{max(v)}" if isinstance(v, list) else str(v))
@pytest.mark.parametrize("four", [True, False])
def test_attention_cuts_of_uneven_sequences(lens, heads, share, four):
    note(f"attention cuts {len(lens)} sequences up to {max(lens)} heads {heads} share {share} four {four}")
    cache, table, lengths, q, values = attention_case(lens, heads, share, 64, 16, four, "bf16", len(lens) + heads)
    o = lh.lh_paged_attention(q.to(DEV), cache, table, lengths, scale=0.125)
    check_attention(o, q, values, heads, share, 64, 0.125)
    again = lh.lh_paged_attention(q.to(DEV), cache, table, lengths, scale=0.125)
    assert torch.equal(o, again)


def test_attention_all_empty_under_a_wide_table():
    note("attention 64 empty sequences, table of 3 pages of 512")
    cache, table, lengths, q, _ = attention_case([0] * 64, 2, 1, 64, 512, True, "bf16", 9)
    for lens in (lengths, lengths - 7):
        o = lh.lh_paged_attention(q.to(DEV), cache, table, lens, scale=0.125)
        assert torch.equal(o, torch.zeros_like(o))


def test_attention_lengths_outside_the_table():
    """A negative length is 0 and one past the table ends with it; a page outside the cache reads page 0."""
    note("attention, lengths and pages out of range")
    cache, table, lengths, q, values = attention_case([64, 48], 1, 2, 64, 16, False, "f32", 6, pad_pages=0)
    t = table[:, :3].contiguous()
    t[1] = torch.tensor([cache.n_pages, -7, int(t[1, 2])], dtype=torch.int32)
    o = lh.lh_paged_attention(q.to(DEV), cache, t, torch.tensor([1 << 30, 48], dtype=torch.int32, device=DEV), scale=0.1)
    assert torch.isfinite(o).all()
    first = [[a[:48] for a in values[0]]]
    check_attention(o[:1], q[:1], first, 1, 2, 64, 0.1)
    o = lh.lh_paged_attention(q.to(DEV), cache, t, torch.tensor([-5, 0], dtype=torch.int32, device=DEV), scale=0.1)
    assert torch.count_nonzero(o) == 0
    o = lh.lh_paged_attention(q.to(DEV), cache, table[:, :0].contiguous(), lengths, scale=0.1)
    assert torch.count_nonzero(o) == 0
    assert lh.lh_paged_attention(q[:0].to(DEV), cache, table[:0], lengths[:0], scale=0.1).shape == (0, 2, 64)


@pytest.mark.parametrize("four", [True, False])
def test_cache_and_attention_past_four_gigabytes(four):
    note(f"cache past 2^32 bytes, four {four}")
    page, dim = 4096, 128
    pages = 2 ** 32 // (page * (dim // 2 if four else dim)) + 3
    a = torch.tensor([4.0])
    cache = make_cache(pages, page, 1, dim, four, (a, a))
    assert cache.k.numel() > 2 ** 32
    n = 300
    r = np.random.default_rng(1)
    x = r.standard_normal((2, n, 1, dim)).astype(np.float32)
    slots = (pages - 1) * page + np.arange(n, dtype=np.int64)
    xd, sd = torch.from_numpy(x).to(DEV), torch.from_numpy(slots).to(DEV)
    lh.lh_cache_write(cache, xd[0], xd[1], sd)
    values = []
    for i, back in enumerate(lh.lh_cache_read(cache, sd, dtype=torch.float32)):
        codes, scales = decode.cache_codes(x[i], a.numpy(), four)
        want = decode.cache_values(codes, scales, a.numpy(), four)
        assert np.array_equal(f64(back), want)
        values.append(want)
    q = torch.from_numpy(r.standard_normal((1, 4, dim)).astype(np.float32))
    o = lh.lh_paged_attention(q.to(DEV), cache, torch.tensor([[pages - 1]], dtype=torch.int32, device=DEV),
                              torch.tensor([n], dtype=torch.int32, device=DEV), scale=0.1)
    check_attention(o, q, [values], 1, 4, dim, 0.1)


# ------------------------------------------------------------------------------- streams and graphs
def decode_step(cache, s):
    q, scale, h = lh.lh_rms_norm_quant(s["x"], s["gamma"], s["r"], group=128)
    y = lh.lh_matvec(q, s["code"], s["fp4"], s["amax"], x_scale=scale, x_group=128).view(s["x"].shape[0], 8, 64)
    lh.lh_cache_write(cache, y[:, 4:6], y[:, 6:], s["slots"])
    return lh.lh_paged_attention(y[:, :4], cache, s["table"], s["lengths"], scale=0.125), h


def step_state(seed):
    g = gen(seed)
    rows, cin = 3, 256
    code, fp4, amax = (torch.from_numpy(a).to(DEV) for a in weights(1, 512, cin, seed))
    cache, table, lengths, _, _ = attention_case([40, 700, 17], 2, 2, 64, 16, True, "bf16", seed)
    at = (lengths.long() - 1)
    slots = table[torch.arange(rows, device=DEV), at // 16].long() * 16 + at % 16
    return cache, dict(x=torch.randn(rows, cin, generator=g).bfloat16().to(DEV), r=torch.randn(rows, cin, generator=g).bfloat16().to(DEV),
                       gamma=torch.ones(cin, dtype=torch.bfloat16, device=DEV), code=code, fp4=fp4, amax=amax * 1e-4, slots=slots,
                       table=table, lengths=lengths)


def test_step_on_another_stream_and_twice():
    note("decode step on a side stream")
    cache, s = step_state(1)
    want = decode_step(cache, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = decode_step(cache, s)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)                         # fixed orders: the same bits


def test_step_in_a_graph():
    note("decode step captured and replayed")
    cache, s = step_state(2)
    decode_step(cache, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = decode_step(cache, s)
    for k in range(4):
        s["x"].copy_(torch.randn(3, 256, generator=gen(50 + k)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        held = [t.clone() for t in got]
        eager = decode_step(cache, s)
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b)


# ------------------------------------------------------------------------------------------ refusals
def test_refusals():
    cache = make_cache(2, 16, 2, 64, True, (torch.ones(2), torch.ones(2)))
    x = torch.ones(2, 64, device=DEV)
    code, fp4, amax = (torch.from_numpy(a).to(DEV) for a in weights(1, 8, 64, 0))
    q = torch.ones(1, 4, 64, device=DEV)
    table, lengths = torch.zeros(1, 200, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    heads = torch.ones(3, 2, 64, device=DEV)
    slots = torch.zeros(3, dtype=torch.int64, device=DEV)
    for fn in (lambda: lh.lh_rms_norm_quant(x, torch.ones(64, device=DEV), group=64),
               lambda: lh.lh_rms_norm_quant(x, torch.ones(63, device=DEV)),
               lambda: lh.lh_rms_norm_quant(x, torch.ones(64, device=DEV), x.bfloat16()),
               lambda: lh.lh_rms_norm_quant(x.t(), torch.ones(2, device=DEV)),
               lambda: lh.lh_matvec(x, code, fp4[:, :, :16].contiguous(), amax),
               lambda: lh.lh_matvec(x.to(torch.float8_e4m3fn), code, fp4, amax),
               lambda: lh.lh_matvec(x, code, fp4, amax, x_scale=torch.ones(2, 1, device=DEV)),
               lambda: lh.lh_matvec(x, code, fp4, amax, x_group=64),
               lambda: lh.lh_cache_write(cache, heads, heads.bfloat16(), slots),
               lambda: lh.lh_cache_write(cache, heads[:, :1], heads, slots),
               lambda: lh.lh_cache_write(cache, heads.transpose(1, 2), heads, slots),
               lambda: lh.lh_cache_write(cache, heads, heads, slots[:2]),
               lambda: lh.lh_cache_read(cache, slots, dtype=torch.float16),
               lambda: lh.lh_paged_attention(q, cache, table.long(), lengths, scale=1.0),
               lambda: lh.lh_paged_attention(q, cache, table, lengths[:0], scale=1.0),
               lambda: lh.lh_paged_attention(q[:, :, :32], cache, table, lengths, scale=1.0),
               lambda: lh.Cache(cache.k, cache.v, cache.k_amax, cache.v_amax, cache.k_scale, None),
               lambda: lh.Cache(cache.k, cache.v, cache.k_amax[:1], cache.v_amax, cache.k_scale, cache.v_scale)):
        with pytest.raises(ValueError):
            fn()
    for fn, code_, word in ((lambda: lh.lh_rms_norm_quant(x[:, :40].contiguous(), torch.ones(40, device=DEV)), 1, "cin"),
                            (lambda: lh.lh_rms_norm_quant(x, torch.ones(64, device=DEV), eps=-1.0), 1, "eps"),
                            (lambda: lh.lh_matvec(x, code, fp4, amax, norm=300.0), 1, "scale_norm"),
                            (lambda: lh.lh_paged_attention(q[:, :3], cache, table, lengths, scale=1.0), 1, "multiple"),
                            (lambda: lh.lh_paged_attention(q, cache, table, lengths, scale=float("nan")), 1, "scale"),
                            (lambda: lh.lh_paged_attention(q, cache, table, lengths, scale=1.0,
                                                           workspace=torch.empty(16, dtype=torch.uint8, device=DEV)), 1, "workspace"),
                            (lambda: lh.lh_paged_attention(torch.ones(1, 4, 96, device=DEV), make_cache(2, 16, 2, 96, True, (torch.ones(2), torch.ones(2))),
                                                           table, lengths, scale=1.0), 2, "head_dim")):
        with pytest.raises(lh.LHError) as e:
            fn()
        assert e.value.code == code_ and word in e.value.message
    with pytest.raises(TypeError):
        lh.lh_matvec(x.half(), code, fp4, amax)
