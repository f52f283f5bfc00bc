"""The operators around a decode step on the GPU against their definitions in oracle/serve.py: growth of the cache's
sequences (whole numbers, equal), rotary positions and the choice of experts, with tolerances derived from their arithmetic."""
import numpy as np
import pytest
import torch

from oracle import serve

pytestmark = pytest.mark.gpu

lh = pytest.importorskip("nvfp4_scale_calibration_lh_amd")
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24                       # fp32 unit roundoff
HALF = {"bf16": 2.0 ** -8, "f32": U}  # half a step of the output's type, relative


def note(msg):
    print(f"[case] {msg}", flush=True)


def dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).to(DEV)


# ------------------------------------------------------------------------- growth of the cache's sequences
def requests(batch, width, page, seed, new="mixed", free=None):
    """(table, lengths, asked, stack, count): requests that hold distinct pages, and free ones on a stack with room for all."""
    r = np.random.default_rng(seed)
    most = width * page
    lengths = r.integers(0, most + 1, batch)
    lengths[r.random(batch) < 0.2] = 0
    lengths[r.random(batch) < 0.1] = most
    held = -(-lengths // page)
    total = int(held.sum())
    free = batch + 3 if free is None else free
    order = r.permutation(total + free)
    table = np.full((batch, width), -7)
    table[np.arange(width)[None, :] < held[:, None]] = order[free:]
    stack = np.full(total + free, -9)
    stack[:free] = order[:free]
    kind = r.random(batch)
    asked = np.where(kind < 0.4, 1, np.where(kind < 0.6, r.integers(0, 3 * page + 2, batch), np.where(kind < 0.8, -r.integers(0, 2 * page + 2, batch), 0)))
    asked[kind > 0.95] = -2 ** 31
    asked[(kind > 0.92) & (kind < 0.95)] = 2 ** 31 - 1
    return table, lengths, {"mixed": asked, "one": None, "idle": 0 * asked, "back": -abs(asked.clip(-2 ** 30, 2 ** 30))}[new], stack, np.array([free])


def check_extend(table, lengths, asked, stack, count, page, max_tokens, in_place=False, calls=1):
    t, n, s, c = dev(table), dev(lengths), dev(stack), dev(count)
    a = None if asked is None else dev(asked)
    kw = dict(new_lengths=n, new_count=c) if in_place else {}
    for _ in range(calls):
        got = lh.lh_cache_extend(t, n, a, s, c, page_size=page, max_tokens=max_tokens, **kw)
    wt, ws = table.copy(), stack.copy()
    slots, positions, sequence, offsets, new, left = serve.extend(wt, lengths, asked, ws, int(count[0]), page, max_tokens)
    for name, g, w in zip(("slots", "positions", "sequence", "offsets", "lengths", "count"), got, (slots, positions, sequence, offsets, new, [left])):
        np.testing.assert_array_equal(g.cpu().numpy(), np.array(w).astype(g.cpu().numpy().dtype), err_msg=name)
    np.testing.assert_array_equal(t.cpu().numpy(), wt, err_msg="table")
    np.testing.assert_array_equal(s.cpu().numpy(), ws, err_msg="stack")
    if not in_place:
        np.testing.assert_array_equal(n.cpu().numpy(), lengths)
        np.testing.assert_array_equal(c.cpu().numpy(), count)
    return got


# one workgroup and two kernels (up to 512 requests and rows, and over), waves that are not full
@pytest.mark.parametrize("batch,width,page,max_tokens", [(1, 1, 1, 1), (1, 4, 16, 64), (3, 5, 16, 40), (63, 7, 3, 300), (64, 9, 16, 64), (65, 9, 16, 200),
                                                         (256, 4, 24, 2048), (256, 4, 24, 2049), (512, 3, 5, 2048), (513, 3, 5, 2048), (1024, 3, 5, 2048), (1025, 3, 5, 2048),
                                                         (2500, 6, 7, 9001), (300, 40, 64, 70000)])
@pytest.mark.parametrize("new", ["mixed", "one", "idle", "back"])
def test_extend(batch, width, page, max_tokens, new):
    note(f"extend {batch} requests, {width} pages of {page}, {max_tokens} rows, {new}")
    case = requests(batch, width, page, batch + max_tokens, new)
    check_extend(*case, page, max_tokens)
    check_extend(*case, page, max_tokens, in_place=True)
    check_extend(*case, page, max_tokens, calls=3)          # not in place, so each call does the same


@pytest.mark.parametrize("batch,max_tokens", [(200, 900), (1500, 30000)])
@pytest.mark.parametrize("free", [0, 1, 37])
def test_extend_pages_run_out(batch, max_tokens, free):
    """Few free pages: requests take what others give back in the same step, and the later ones are not granted."""
    for seed in range(4):
        note(f"extend {batch} requests, {free} free pages, seed {seed}")
        check_extend(*requests(batch, 6, 4, seed, free=free), 4, max_tokens)


@pytest.mark.parametrize("batch", [5, 1200])
def test_extend_numbers_out_of_range(batch):
    """Lengths and counts below 0 and over what there is, page numbers that are none, a stack without room for what comes back."""
    table, lengths, asked, stack, count = requests(batch, 5, 8, 11)
    lengths[0], lengths[1], lengths[2] = -5, 2 ** 31 - 1, -2 ** 31
    table[3] = -123
    for c in (-1, -2 ** 31, 10 ** 9, 3):
        note(f"extend with a count of {c}")
        check_extend(table, lengths, asked, stack, np.array([c]), 8, 1000)
    note("extend with a short stack")
    check_extend(table, lengths, asked, stack[:4].copy(), np.array([3]), 8, 1000)


def test_extend_nothing():
    one = np.array([0])
    note("no requests")
    check_extend(np.zeros((0, 4), int), np.zeros(0, int), np.zeros(0, int), np.arange(6), np.array([6]), 16, 5)
    note("no requests and many rows")
    check_extend(np.zeros((0, 4), int), np.zeros(0, int), None, np.arange(6), np.array([6]), 16, 5000)
    note("no rows")
    check_extend(np.zeros((2, 4), int), np.array([3, 16]), np.array([1, -1]), np.arange(6), np.array([2]), 16, 0)
    note("tables of no page")
    check_extend(np.zeros((2, 0), int), np.array([3, 0]), np.array([1, 2]), np.arange(6), np.array([2]), 16, 8)
    note("a stack of no page")
    check_extend(np.full((2, 3), -1), np.array([0, 0]), np.array([1, 2]), np.zeros(0, int), one, 16, 8)


def test_extend_leaves_no_page_twice():
    """Fifty steps of admissions, decodes and releases: every page is held once or free once."""
    r = np.random.default_rng(3)
    batch, width, page, pages = 40, 9, 4, 200
    t, n, s, c = (dev(a) for a in (np.full((batch, width), -1), np.zeros(batch), r.permutation(pages), [pages]))
    work = torch.empty(lh.lh_cache_extend_workspace(batch, 4000), dtype=torch.uint8, device=DEV)
    assert work.numel() > 0
    for step in range(50):
        asked = np.where(r.random(batch) < 0.1, -2 ** 31, np.where(r.random(batch) < 0.2, r.integers(0, 20, batch), r.integers(-3, 3, batch)))
        lh.lh_cache_extend(t, n, dev(asked), s, c, page_size=page, max_tokens=60 if step % 2 else 4000, new_lengths=n, new_count=c,
                           workspace=work if step % 2 == 0 else None)
        table, lengths, free = t.cpu().numpy(), n.cpu().numpy(), s.cpu().numpy()[:int(c)]
        held = np.concatenate([table[b, :-(-lengths[b] // page)] for b in range(batch)] + [free])
        assert sorted(held) == list(range(pages)), step


# --------------------------------------------------------------------------------------- rotary positions
def heads_of(tokens, heads, dim, dtype, seed, extra=0):
    """A [tokens, heads, dim] part of wider rows (by `extra` heads)."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(tokens, heads + extra, dim, generator=g) * torch.exp2(torch.randint(-8, 9, (tokens, 1, 1), generator=g).float())).to(TYPES[dtype])
    return x.to(DEV)[:, :heads], x[:, :heads].double().numpy()


def check_rotary(got, x, positions, f, dtype, half, interleaved, inverse=False, scale=1.0):
    """sine and cosine to 2^-23 and one rounding with the scale (2^-24), a rounding of one product and one of the sum, then the type's."""
    want = serve.rotary(x, positions, f, interleaved, inverse, scale)
    pairs = x[..., :2 * half].reshape(*x.shape[:2], half, 2) if interleaved else np.stack([x[..., :half], x[..., half:2 * half]], -1)
    size = np.abs(pairs).sum(-1)
    size = np.repeat(size, 2, -1) if interleaved else np.concatenate([size, size], -1)
    bound = np.zeros_like(want)
    bound[..., :2 * half] = abs(scale) * size * (2 + 1 + 1 + 1) * U + 2.0 ** -149
    bound[np.asarray(positions) < 0] = 0
    bound += (bound > 0) * HALF[dtype] * (np.abs(want) + bound)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= bound), (float((err - bound).max()), float(err.max()))


@pytest.mark.parametrize("tokens,heads,kv,dim,rot", [(1, 32, 8, 128, 128), (1, 1, 0, 16, 2), (3, 7, 1, 64, 64), (65, 5, 5, 96, 48), (17, 8, 2, 256, 64),
                                                     (2, 3, 3, 80, 80), (40, 4, 2, 64, 20), (5, 2, 1, 112, 6), (3001, 8, 2, 64, 32),
                                                     (7, 3, 2, 64, 40), (9, 2, 1, 48, 8), (33001, 6, 1, 64, 64)])      # the last: several heads a thread
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary(tokens, heads, kv, dim, rot, dtype, interleaved):
    note(f"rotary {tokens} tokens {heads}+{kv} heads of {dim}, {rot} turned, {dtype} interleaved {interleaved}")
    q, qx = heads_of(tokens, heads, dim, dtype, 1, extra=kv)
    k, kx = heads_of(tokens, kv, dim, dtype, 2) if kv else (None, None)
    f, scale = lh.lh_rotary_frequencies(rot, device=DEV)
    assert scale == 1.0
    r = np.random.default_rng(tokens)
    positions = r.integers(0, 200000, tokens)
    if tokens > 2:
        positions[1] = -1
        positions[2] = 0
    args = (dev(positions), f)
    for inverse, scale in ((False, 1.0), (True, 1.3465735912322998)):
        oq, ok = lh.lh_rotary(q, k, *args, interleaved=interleaved, inverse=inverse, scale=scale)
        check_rotary(oq, qx, positions, f.cpu().numpy(), dtype, rot // 2, interleaved, inverse, scale)
        assert (ok is None) == (k is None)
        if k is not None:
            check_rotary(ok, kx, positions, f.cpu().numpy(), dtype, rot // 2, interleaved, inverse, scale)
    # in place, and into parts of wider rows, the same bits; nothing else of those rows changes
    wide = torch.full((tokens, heads + 3, dim), 7.0, dtype=q.dtype, device=DEV)
    out = wide[:, 1:1 + heads] if dim * (2 if dtype == "bf16" else 4) % 16 == 0 else wide[:, :heads]
    lh.lh_rotary(q, k, *args, interleaved=interleaved, inverse=inverse, scale=scale, out_q=out)
    assert torch.equal(out, oq) and bool((wide[:, 0] == 7).all()) and bool((wide[:, 1 + heads:] == 7).all())
    rest = q.as_strided((tokens, heads + kv, dim), (q.stride(0), dim, 1))[:, heads:].clone() if tokens > 1 else None
    lh.lh_rotary(q, k, *args, interleaved=interleaved, inverse=inverse, scale=scale, out_q=q, out_k=k)
    assert torch.equal(q, oq) and (k is None or torch.equal(k, ok))
    if rest is not None:
        assert torch.equal(q.as_strided((tokens, heads + kv, dim), (q.stride(0), dim, 1))[:, heads:], rest)


@pytest.mark.parametrize("scaling", ["plain", "linear", "base", "parts"])
def test_rotary_far_positions(scaling):
    """The angle loses nothing up to the largest position."""
    note(f"rotary far {scaling}")
    f, scale = lh.lh_rotary_frequencies(64, theta=500000.0, scaling=scaling, factor=8.0, original_context=8192, device=DEV)
    positions = np.array([0, 1, 2, 3, 4095, 131071, 1000003, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1, -1, -2 ** 31] + list(range(5, 400)))
    x, v = heads_of(len(positions), 2, 64, "f32", 3)
    y, _ = lh.lh_rotary(x, None, dev(positions), f, scale=scale)
    check_rotary(y, v, positions, f.cpu().numpy(), "f32", 32, False, scale=scale)
    quarter = torch.tensor([np.pi / 4], dtype=torch.float32, device=DEV)        # angles next to the borders of the reduction
    positions = np.arange(64)
    x, v = heads_of(64, 1, 16, "f32", 4)
    y, _ = lh.lh_rotary(x, None, dev(positions), quarter)
    check_rotary(y, v, positions, quarter.cpu().numpy(), "f32", 1, False)


def test_rotary_gradient():
    """The inverse is the transpose: <g, R x> = <R' g, x>, and differences of R give the same."""
    note("rotary gradient")
    f, scale = lh.lh_rotary_frequencies(32, scaling="parts", factor=4.0, original_context=64, device=DEV)
    x, xv = heads_of(9, 3, 64, "f32", 5)
    g, gv = heads_of(9, 3, 64, "f32", 6)
    p = dev(np.arange(9) * 37)
    y, _ = lh.lh_rotary(x, None, p, f, scale=scale)
    back, _ = lh.lh_rotary(g, None, p, f, scale=scale, inverse=True)
    a, b = (gv * y.double().cpu().numpy()).sum((1, 2)), (back.double().cpu().numpy() * xv).sum((1, 2))
    size = 2 * scale * np.abs(gv).sum((1, 2)) * np.abs(xv).max((1, 2))
    assert np.all(np.abs(a - b) <= 8 * U * size + 8 * U * 2 * scale * np.abs(xv).sum((1, 2)) * np.abs(gv).max((1, 2)))
    step = torch.zeros_like(x)
    step[4, 1, 3] = 1.0
    moved, _ = lh.lh_rotary(x + step, None, p, f, scale=scale)
    rounding = 16 * U * scale * float((x.abs() + 1).max())
    assert abs(float(((moved - y) * g).sum()) - float(back[4, 1, 3])) <= rounding * float(g[4, 1].abs().sum()) + 8 * U * scale * float(g.abs().max()) * 2


def test_rotary_nothing_and_nan():
    f, _ = lh.lh_rotary_frequencies(16, device=DEV)
    q, k = lh.lh_rotary(torch.empty(0, 4, 32, device=DEV), torch.empty(0, 2, 32, device=DEV), dev(np.zeros(0)), f)
    assert q.shape == (0, 4, 32) and k.shape == (0, 2, 32)
    x = torch.ones(2, 2, 32, device=DEV)
    x[0, 0, 3] = float("nan")
    x[1, 1, 20] = float("inf")
    y, _ = lh.lh_rotary(x, None, dev([5, 6]), f)
    bad = ~torch.isfinite(y).cpu()
    assert bad.nonzero().tolist() == [[0, 0, 3], [0, 0, 11], [1, 1, 20]]        # its pair, and an element past the turned ones


# ------------------------------------------------------------------------------------- the choice of experts
def check_route(x, topk, renormalize=True, scale=1.0):
    """Weights: the difference to the largest logit rounds once (2^-24 of it, at most 104 before exp underflows), exp to 2
    steps, the sum adds at most 64 in a lane and 6 in a tree, a division and a product."""
    ids, w = lh.lh_route(x, topk, renormalize=renormalize, scale=scale)
    want_ids, want = serve.route(x.double().cpu().numpy(), topk, renormalize, scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    rel = (2 * 104 + 2 * 4 + 70 + 2) * U
    assert np.all(np.abs(w.double().cpu().numpy() - want) <= rel * np.abs(want) + 2.0 ** -126)
    return ids, w


@pytest.mark.parametrize("tokens,experts,topk", [(1, 1, 1), (1, 2, 2), (5, 8, 2), (3, 63, 5), (9, 64, 64), (2, 65, 6), (33, 128, 8), (7, 200, 10), (32, 512, 10),
                                                 (4, 513, 1), (6, 1024, 16), (2, 2000, 64), (3, 2049, 9), (2, 4096, 64), (3000, 60, 6)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route(tokens, experts, topk, dtype, renormalize):
    note(f"route {tokens} of {experts} top {topk} {dtype} renormalize {renormalize}")
    g = torch.Generator().manual_seed(experts)
    x = (torch.randn(tokens, experts, generator=g) * 3).to(TYPES[dtype]).to(DEV)
    check_route(x, topk, renormalize, 2.5)
    check_route((x / 4).round(), topk, renormalize)               # many equal ones


def test_route_masks_and_infinities():
    inf, nan = float("inf"), float("nan")
    x = torch.randn(12, 40, generator=torch.Generator().manual_seed(1))
    x[0] = -inf
    x[1, 3:] = -inf                                               # fewer than asked for
    x[2, ::2] = nan
    x[3] = nan
    x[4, 7] = inf
    x[5, [5, 9]] = inf
    x[6] = torch.finfo(torch.float32).min                         # the type's lowest value is no mask
    x[7] = torch.where(torch.arange(40) % 2 == 0, 0.0, -0.0)      # equal
    x[8] = -200.0
    x[8, 39] = 5.0                                                # the others' weights are next to nothing
    x[9] = torch.finfo(torch.float32).max
    x[10, :39] = -inf
    for dtype in ("f32", "bf16"):
        for renormalize in (True, False):
            note(f"route masks {dtype} renormalize {renormalize}")
            t = x.to(TYPES[dtype]).to(DEV)
            if dtype == "bf16":
                t[6], t[9] = torch.finfo(torch.bfloat16).min, torch.finfo(torch.bfloat16).max
            ids, w = check_route(t, 6, renormalize)
            assert ids[0].tolist() == [-1] * 6 and ids[3].tolist() == [-1] * 6 and float(w[0].abs().sum()) == 0
            assert ids[7].tolist() == [0, 1, 2, 3, 4, 5] and ids[10].tolist() == [39] + [-1] * 5


def test_route_nothing():
    ids, w = lh.lh_route(torch.empty(0, 16, device=DEV), 3)
    assert ids.shape == (0, 3) and w.shape == (0, 3)


# ------------------------------------------------------------------------------------------ the expert layer
def matrices(experts, cout, cin, seed):
    """NVFP4 weights whose values are near 1 / sqrt(cin): random nibbles, scale codes over a few binades."""
    r = np.random.default_rng(seed)
    code = r.integers(0x28, 0x48, (experts, cout, cin // 16)).astype(np.uint8)
    fp4 = r.integers(0, 256, (experts, cout, cin // 2)).astype(np.uint8)
    amax = ((0.5 + r.random(experts)) * 700 * cin ** -0.5).astype(np.float32)
    return code, fp4, amax


def on_gpu(m):
    return tuple(torch.from_numpy(t).to(DEV) for t in m)


def layer_rows(rows, cin, x, group, seed):
    """(tensor, x_scale tensor or None, values in float64)"""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(rows, cin, generator=g)
    if x != "e4m3":
        t = v.to(TYPES[x])
        return t.to(DEV), None, t.double().numpy()
    width = group or cin
    q = (v * 100).to(torch.float8_e4m3fn)
    s = 0.01 * (0.5 + torch.rand(rows, -(-cin // width), generator=g))
    return q.to(DEV), s.to(DEV), q.double().numpy() * np.repeat(s.double().numpy(), width, 1)[:, :cin]


def check_moe(xd, scale, xv, x, group, ids, w, gate_up, down, **kw):
    """Products are exact and sums fp32: a sum of n terms is off by at most (n + 8) roundings of its terms' magnitudes (every element of
    fp32 rows is three terms), which the two products pass on; between them exp, the division and three products.  h is one fp16 number
    with a factor: 11 bits, half a step is up to 2^-11 of it.  fp32 rows and their h are two: what the first leaves is at most 2^-11 of
    the power of two under the number, so its own half step is at most 2^-23 of that power, and never under 2^-25, where the largest of
    128 is at least 2^14: 2^-39 of that one."""
    y = lh.lh_moe(xd, torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), on_gpu(gate_up), on_gpu(down), x_scale=scale, x_group=group, **kw)
    want, terms = serve.moe(xv, ids, w.astype(np.float64), gate_up, down, kw.get("norm", 448.0))
    hidden, inner = xv.shape[1], down[0].shape[2] * 16
    pieces = 3 if x == "f32" else 1
    rel = (pieces * hidden + 8) * U + (3 * inner + 8) * U + 32 * U + (2 * 2.0 ** -23 if x == "f32" else 2.0 ** -11) + ids.shape[1] * U
    bound = rel * terms + 2.0 ** -38 * terms.max(1, keepdims=True) + 2.0 ** -120
    bound += HALF["f32" if x == "f32" else "bf16"] * (np.abs(want) + bound)
    got, none = y.double().cpu().numpy(), np.isnan(want)        # a NaN in a row (8 bits of what is over 464) is one in its outputs
    np.testing.assert_array_equal(np.isnan(got), none)
    err, bound, want = np.where(none, 0, np.abs(got - want)), np.where(none, 0, bound), np.where(none, 0, want)
    assert y.dtype == (torch.float32 if x == "f32" else torch.bfloat16)
    assert np.all(err <= bound), (float((err / bound).max()), float(err.max()))
    # and near the plain rounding of the right value in the mean, far under the bound above
    rms = np.sqrt((err ** 2).mean()) / max(np.sqrt((want ** 2).mean()), 1e-30)
    assert rms <= (2.0 ** -18 if x == "f32" else 2.0 ** -8), rms
    return y


def choices(tokens, experts, topk, seed):
    r = np.random.default_rng(seed)
    ids = np.argsort(r.random((tokens, experts)), 1)[:, :topk].astype(np.int32)
    w = r.random((tokens, topk)).astype(np.float32)
    return ids, w / w.sum(1, keepdims=True)


# whole and short chunks of 128, less than a chunk, several panels of LDS where rows are made ready first, shares of k, one tile of rows and more
@pytest.mark.parametrize("tokens,experts,topk,hidden,inner", [(1, 1, 1, 16, 16), (1, 4, 2, 128, 64), (2, 8, 3, 144, 80), (5, 16, 4, 272, 144), (17, 3, 2, 256, 128),
                                                              (64, 2, 1, 384, 48), (65, 5, 2, 640, 272), (33, 40, 10, 512, 32), (130, 6, 3, 112, 208),
                                                              (3, 7, 2, 2560, 640), (40, 2, 2, 2064, 1040), (1, 3, 3, 5136, 96), (20, 300, 6, 64, 16)])
@pytest.mark.parametrize("x,group", [("bf16", 0), ("f32", 0), ("e4m3", 0), ("e4m3", 128)])
def test_moe(tokens, experts, topk, hidden, inner, x, group):
    note(f"moe {tokens} tokens top {topk} of {experts}, {hidden} x {inner}, {x} group {group}")
    gate_up, down = matrices(experts, 2 * inner, hidden, 1), matrices(experts, hidden, inner, 2)
    xd, scale, xv = layer_rows(tokens, hidden, x, group, 3)
    ids, w = choices(tokens, experts, topk, 4)
    check_moe(xd, scale, xv, x, group, ids, w, gate_up, down)


def test_moe_choices():
    """Skipped and repeated choices, tokens without any, every token at one expert, weights of either sign, the other normalization."""
    gate_up, down = matrices(9, 128, 256, 5), matrices(9, 256, 64, 6)
    xd, scale, xv = layer_rows(70, 256, "bf16", 0, 7)
    r = np.random.default_rng(8)
    ids = r.integers(-2, 11, (70, 6)).astype(np.int32)             # repeats, and some outside
    ids[3], ids[69], ids[10] = -1, 2 ** 31 - 1, 4
    w = r.standard_normal((70, 6)).astype(np.float32)
    note("moe with repeats and choices outside")
    y = check_moe(xd, scale, xv, "bf16", 0, ids, w, gate_up, down, norm=256.0)
    assert torch.count_nonzero(y[[3, 69]]) == 0
    note("moe with every token at one expert")
    check_moe(xd, scale, xv, "bf16", 0, np.full((70, 2), 8, np.int32), np.full((70, 2), 0.5, np.float32), gate_up, down)
    note("moe with no choice at all")
    y = check_moe(xd, scale, xv, "bf16", 0, np.full((70, 2), -1, np.int32), np.ones((70, 2), np.float32), gate_up, down)
    assert torch.count_nonzero(y) == 0


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_moe_infinities_stay_in_their_rows(x):
    note(f"moe infinities {x}")
    gate_up, down = matrices(4, 96, 160, 9), matrices(4, 160, 48, 10)
    xd, _, _ = layer_rows(6, 160, x, 0, 11)
    ids, w = choices(6, 4, 2, 12)
    args = [torch.from_numpy(t).to(DEV) for t in (ids, w)]
    clean = lh.lh_moe(xd, *args, on_gpu(gate_up), on_gpu(down))
    bad = xd.clone()
    bad[1, 5], bad[4, 159] = float("nan"), float("inf")
    y = lh.lh_moe(bad, *args, on_gpu(gate_up), on_gpu(down))
    keep = [0, 2, 3, 5]
    assert torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[4]).all())


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_moe_infinities_where_experts_have_many_rows(x):
    note(f"moe infinities, many rows, {x}")
    gate_up, down = matrices(2, 288, 272, 17), matrices(2, 272, 144, 18)
    xd, _, _ = layer_rows(40, 272, x, 0, 19)
    ids, w = choices(40, 2, 2, 20)
    args = [torch.from_numpy(t).to(DEV) for t in (ids, w)]
    clean = lh.lh_moe(xd, *args, on_gpu(gate_up), on_gpu(down))
    bad = xd.clone()
    bad[1, 5], bad[38, 271] = float("nan"), float("-inf")
    y = lh.lh_moe(bad, *args, on_gpu(gate_up), on_gpu(down))
    keep = [t for t in range(40) if t not in (1, 38)]
    assert torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[38]).all())


def test_moe_most_experts():
    note("moe 64 of 4096 experts")
    gate_up, down = matrices(4096, 32, 16, 21), matrices(4096, 16, 16, 22)
    xd, scale, xv = layer_rows(3, 16, "bf16", 0, 23)
    ids, w = choices(3, 4096, 64, 24)
    ids[1, 7], ids[2, 63] = 4095, 0
    check_moe(xd, scale, xv, "bf16", 0, ids, w, gate_up, down)


def test_moe_large_activations():
    """silu far from 0: gates where exp overflows or the weight of the up product is next to nothing."""
    note("moe large activations")
    gate_up, down = matrices(2, 64, 64, 13), matrices(2, 64, 32, 14)
    xd, _, _ = layer_rows(4, 64, "f32", 0, 15)
    xd = xd * torch.tensor([1e3, 1e-3, 1e6, 30.0], device=DEV)[:, None]
    ids, w = choices(4, 2, 2, 16)
    check_moe(xd.contiguous(), None, xd.double().cpu().numpy(), "f32", 0, ids, w, gate_up, down)


def test_moe_nothing():
    y = lh.lh_moe(torch.empty(0, 32, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV),
                  on_gpu(matrices(2, 32, 32, 1)), on_gpu(matrices(2, 32, 16, 1)))
    assert y.shape == (0, 32)


# ------------------------------------------------------------------------------------------------- adapters
def adapter_case(rows, cin, cout, n, rank, x, group, weights, seed, ragged=True):
    """Arguments on the GPU and in float64; what lies past an adapter's rank is NaN."""
    g, r = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    xd, scale, xv = layer_rows(rows, cin, x, group, seed)
    base = torch.randn(rows, cout, generator=g).to(torch.float32 if x == "f32" else torch.bfloat16)
    a = (torch.randn(n, rank, cin, generator=g) * cin ** -0.5).to(TYPES[weights])
    b = torch.randn(n, cout, rank, generator=g).to(TYPES[weights])
    index = r.integers(0, n, rows)
    index[r.random(rows) < 0.2] = r.choice([-1, n, 2 ** 31 - 1, -2 ** 31])
    ranks = r.integers(0, rank + 1, n) if ragged else None
    if ragged:
        for k, m in enumerate(ranks):
            a[k, m:], b[k, :, m:] = float("nan"), float("nan")
    scaling = (r.random(n) * 2 - 0.5).astype(np.float32)
    return xd, scale, xv, base.to(DEV), a.to(DEV), b.to(DEV), index.astype(np.int32), ranks, scaling


def check_adapter(case, x, group, weights, **kw):
    """Sums of n terms are off by at most (n + 8) roundings of their terms' magnitudes (fp32 elements are three terms each, fp32
    weights round their products, too), u by its pieces and its scaling, and Y once more by its type.  Of two pieces of 8 bits the first, cut off,
    leaves under 2^-7 of the power of two under u, and the second is off by half a step of that, 2^-8 of 2^-8: 2^-16."""
    xd, scale, xv, base, a, b, index, ranks, scaling = case
    args = dict(scaling=torch.from_numpy(scaling).to(DEV), ranks=None if ranks is None else dev(ranks), x_scale=scale, x_group=group)
    y = lh.lh_adapter(xd, base, a, b, dev(index), **args, **kw)
    want, terms = serve.adapter(xv, base.double().cpu().numpy(), a.double().cpu().numpy(), b.double().cpu().numpy(), index, scaling, ranks)
    held = 2.0 ** -24 if x == "f32" or weights == "f32" else 2.0 ** -16
    rel = (3 * a.shape[2] + 8) * U + (3 * a.shape[1] + 8) * U + 8 * U + held
    none = np.isnan(want)
    np.testing.assert_array_equal(np.isnan(y.double().cpu().numpy()), none)
    want, terms = np.where(none, 0, want), np.where(none, 0, terms)
    bound = rel * terms
    bound += HALF["f32" if x == "f32" else "bf16"] * (np.abs(want) + bound)
    err = np.where(none, 0, np.abs(y.double().cpu().numpy() - want))
    assert y.dtype == base.dtype and np.all(err <= bound), (float((err / bound).max()), float(err.max()))
    # in the mean far under that: a bf16 rounding, or a few fp32 ones
    assert np.sqrt((err ** 2).mean()) <= (2.0 ** -19 if x == "f32" else 2.0 ** -8) * np.sqrt((want ** 2).mean())
    out = (index < 0) | (index >= len(a))
    assert torch.equal(y[torch.from_numpy(out).to(DEV)], base[torch.from_numpy(out).to(DEV)])
    return y


@pytest.mark.parametrize("rows,cin,cout,n,rank", [(1, 16, 1, 1, 8), (1, 4096, 512, 3, 16), (5, 144, 30, 2, 8), (17, 256, 257, 1, 24), (64, 528, 100, 7, 64),
                                                  (65, 640, 1000, 70, 40), (130, 272, 260, 3, 72), (33, 2064, 68, 4, 128), (20, 1040, 52, 2, 136),
                                                  (9, 384, 2049, 5, 256), (40, 12288, 130, 40, 16)])
@pytest.mark.parametrize("x,group", [("bf16", 0), ("f32", 0), ("e4m3", 0), ("e4m3", 128)])
@pytest.mark.parametrize("weights", ["bf16", "f32"])
def test_adapter(rows, cin, cout, n, rank, x, group, weights):
    note(f"adapter {rows} rows {cin} to {cout}, {n} of rank {rank} {weights}, {x} group {group}")
    case = adapter_case(rows, cin, cout, n, rank, x, group, weights, rows + rank)
    y = check_adapter(case, x, group, weights)
    xd, scale, _, base, a, b, index, ranks, scaling = case
    again = base.clone()
    lh.lh_adapter(xd, again, a, b, dev(index), again, scaling=torch.from_numpy(scaling).to(DEV), ranks=dev(ranks), x_scale=scale, x_group=group)
    assert torch.equal(again.view(torch.uint8), y.view(torch.uint8))          # in place, the same bits


def test_adapter_full_ranks_and_no_scaling():
    note("adapter without ranks, one request for all rows")
    case = adapter_case(70, 256, 192, 2, 32, "bf16", 0, "bf16", 4, ragged=False)
    case[6][:] = 1
    check_adapter(case, "bf16", 0, "bf16")
    xd, _, _, base, a, b, index, _, scaling = case
    y = lh.lh_adapter(xd, base, a, b, dev(index))
    one = lh.lh_adapter(xd, base, a, b, dev(index), scaling=torch.ones(2, device=DEV), ranks=dev([32, 32]))
    assert torch.equal(y, one)
    note("adapter with no row that has one")
    y = lh.lh_adapter(xd, base, a, b, dev(np.full(70, -1)))
    assert torch.equal(y, base)


def test_adapter_infinities_stay_in_their_rows():
    note("adapter infinities")
    xd, _, _, base, a, b, index, _, _ = adapter_case(6, 144, 64, 2, 16, "bf16", 0, "bf16", 5, ragged=False)
    index[:] = [0, 0, 1, 1, 0, -1]
    clean = lh.lh_adapter(xd, base, a, b, dev(index))
    bad = xd.clone()
    bad[0, 3], bad[2, 143], bad[5, 0] = float("nan"), float("inf"), float("nan")
    y = lh.lh_adapter(bad, base, a, b, dev(index))
    assert torch.equal(y[[1, 3, 4, 5]], clean[[1, 3, 4, 5]])
    assert bool(torch.isnan(y[0]).all()) and not bool(torch.isfinite(y[2]).all())


def test_adapter_nothing():
    a, b = torch.zeros(2, 8, 32, device=DEV), torch.zeros(2, 40, 8, device=DEV)
    y = lh.lh_adapter(torch.empty(0, 32, device=DEV), torch.empty(0, 40, device=DEV), a, b, dev([]))
    assert y.shape == (0, 40)
    y = lh.lh_adapter(torch.ones(3, 32, device=DEV), torch.empty(3, 0, device=DEV), a, torch.zeros(2, 0, 8, device=DEV), dev([0, 1, 0]))
    assert y.shape == (3, 0)


def test_adapter_many_rows():
    """More than 64 times 64 rows, whose adapters are shared out over workgroups 4096 rows at a time."""
    note("adapter 4300 rows")
    case = adapter_case(4300, 64, 100, 5, 8, "bf16", 0, "bf16", 6)
    check_adapter(case, "bf16", 0, "bf16")
