"""Cases for the decode-step operators: RMS norm with 8-bit output, matrix-vector products with NVFP4
weights, the quantised key-value cache, and attention of one new token over it.

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU from a seed, ``run``
makes one pass (elementary torch operations in 32 bits, or the library's entry points where ``own``
is true), ``exact`` gives the same outputs from the definitions in 64 bits, and ``work`` the bytes
and operations of one pass.

Formats.  NVFP4 holds 16 consecutive values as E2M1 nibbles (element 2j in the low half of byte j)
and one E4M3 scale byte v; a value is E2M1 * v * g with g = fp32(amax / (6 * 448)) of its weight
matrix or key-value head.  E4M3 holds a value as one byte, times fp32(amax / 448) of its head or
times a scale of its row (or of 128 channels of its row).
"""
import math

import numpy as np
import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token's hidden vector between two layers of a single-user decode: all latency
        dict(name="norm-one-token", op="norm", rows=1, cin=4096, group=0, dtype="bf16", residual=True),
        # the prompt's rows of the 12288x4096 layer, a scale for every 128 channels: all bandwidth
        dict(name="norm-prompt", op="norm", rows=8192, cin=4096, group=128, dtype="bf16", residual=True),
        # one token through the 2048x2048 layer: the smallest product, latency counts
        dict(name="matvec-one-token", op="matvec", cout=2048, cin=2048, rows=1, x="bf16", group=0),
        # sixteen sequences' tokens, already in 8 bits, through the 12288x4096 up projection
        dict(name="matvec-sixteen-8bit", op="matvec", cout=12288, cin=4096, rows=16, x="e4m3", group=128),
        # five fp32 rows (an evaluation in full precision) through the 4096x12288 down projection
        dict(name="matvec-five-fp32", op="matvec", cout=4096, cin=12288, rows=5, x="f32", group=0),
        # a decode batch of 32 tokens, ten of 512 experts each: few rows for each expert that is hit
        dict(name="matvec-experts", op="experts", experts=512, cout=1280, cin=2560, tokens=32, topk=10, x="bf16", group=0),
        # the cache's write of one decode step of 64 sequences, and its read back
        dict(name="cache-step", op="cache", fmt="nvfp4", tokens=64, heads=8, dim=128, page=16, dtype="bf16"),
        # a prompt of odd length written to scattered pages in 4 bits
        dict(name="cache-prompt-4bit", op="cache", fmt="nvfp4", tokens=8191, heads=8, dim=128, page=16, dtype="bf16"),
        # a longer one in 8 bits, narrow heads, pages of 24 tokens
        dict(name="cache-prompt-8bit", op="cache", fmt="e4m3", tokens=30011, heads=4, dim=64, page=24, dtype="bf16"),
        # one user's short conversation
        dict(name="attention-short", op="attention", fmt="e4m3", batch=1, longest=301, heads=8, share=4, dim=128, page=16, dtype="bf16", ragged=False),
        # a serving batch of mixed lengths, one of them empty
        dict(name="attention-batch", op="attention", fmt="nvfp4", batch=48, longest=8191, heads=8, share=4, dim=128, page=16, dtype="bf16", ragged=True),
        # four long documents
        dict(name="attention-long", op="attention", fmt="nvfp4", batch=4, longest=131001, heads=8, share=8, dim=128, page=64, dtype="bf16", ragged=False),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))

    op = rng.choice(["norm", "matvec", "matvec", "experts", "cache", "attention", "attention"])
    if op == "norm":
        cin = 16 * log(8, 768)
        return dict(op=op, rows=log(1, min(8192, 8192 * 4096 // cin)), cin=cin, group=rng.choice([0, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.75)
    if op == "matvec":
        return dict(op=op, cout=log(64, 12288), cin=16 * log(8, 768), rows=log(1, 64),
                    x=rng.choice(["bf16", "e4m3", "f32"]), group=rng.choice([0, 128]))
    if op == "experts":
        experts = log(8, 512)
        return dict(op=op, experts=experts, cout=log(64, 1280), cin=16 * log(8, 160), tokens=log(1, 32),
                    topk=rng.randint(1, min(10, experts)), x=rng.choice(["bf16", "e4m3", "f32"]), group=rng.choice([0, 128]))
    if op == "cache":
        heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 256])
        return dict(op=op, fmt=rng.choice(["nvfp4", "e4m3"]), tokens=log(1, 8191 * 8 * 128 // (heads * dim)), heads=heads,
                    dim=dim, page=rng.choice([16, 24, 64]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
    batch = log(1, 64)
    return dict(op=op, fmt=rng.choice(["nvfp4", "e4m3"]), batch=batch,
                longest=log(1, min(131001, 2 * 131001 * 8 * 128 // (heads * dim * batch))), heads=heads,
                share=rng.choice([1, 4, 7, 8, 16]), dim=dim, page=rng.choice([16, 32, 64, 24]),
                dtype=rng.choice(["bf16", "bf16", "f32"]), ragged=rng.random() < 0.6)


def _lengths(case):
    """Tokens in the cache for each sequence; ragged batches spread them evenly and hold an empty one."""
    n, most = case["batch"], case["longest"]
    if not case["ragged"]:
        return [most] * n
    lens = [max(1, int(most * (1.0 - (i * 0.6180339887498949) % 1.0))) for i in range(n)]
    if n >= 4:
        lens[n // 2] = 0
    return lens


def _routing(case, seed):
    """Row offsets of each expert and the token of each row: top-k of Zipf-weighted Gumbel scores."""
    r = np.random.default_rng([seed, 3])
    logits = -1.1 * np.log(r.permutation(case["experts"]) + 1.0)
    top = np.argsort(-(logits + r.gumbel(size=(case["tokens"], case["experts"]))), axis=1)[:, :case["topk"]]
    expert, token = top.reshape(-1), np.repeat(np.arange(case["tokens"]), case["topk"])
    order = np.argsort(expert, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(expert, minlength=case["experts"]))])
    return offsets.astype(np.int64), token[order].astype(np.int64)


def work(case):
    op = case["op"]
    if op == "norm":
        n, size = case["rows"] * case["cin"], 2 if case["dtype"] == "bf16" else 4
        scales = case["rows"] * (math.ceil(case["cin"] / case["group"]) if case["group"] else 1)
        return {"bytes": n * (size * (3 if case["residual"] else 1) + 1) + case["cin"] * size + 4 * scales, "flops": 7 * n}
    if op in ("matvec", "experts"):
        rows, matrices = case.get("rows", 0), 1
        if op == "experts":
            rows, matrices = case["tokens"] * case["topk"], int(np.count_nonzero(np.diff(_routing(case, 0)[0])))
        x, y = {"bf16": (2, 2), "f32": (4, 4), "e4m3": (1, 2)}[case["x"]]
        return {"bytes": matrices * case["cout"] * (case["cin"] // 2 + case["cin"] // 16) + rows * (case["cin"] * x + case["cout"] * y),
                "flops": 2 * rows * case["cin"] * case["cout"]}
    if op == "cache":
        n, size = 2 * case["tokens"] * case["heads"] * case["dim"], 2 if case["dtype"] == "bf16" else 4
        held = n if case["fmt"] == "e4m3" else n // 2 + n // 16
        return {"bytes": 2 * n * size + 2 * held + 16 * case["tokens"], "flops": 4 * n}
    n = sum(_lengths(case)) * case["heads"] * case["dim"]
    held = 2 * n if case["fmt"] == "e4m3" else 2 * (n // 2 + n // 16)
    q = case["batch"] * case["heads"] * case["share"] * case["dim"] * (2 if case["dtype"] == "bf16" else 4)
    return {"bytes": held + 2 * q, "flops": 4 * n * case["share"]}


# ------------------------------------------------------------------------------------- the inputs
def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _grid(dev="cuda"):
    return torch.tensor(GRID + tuple(-v for v in GRID), device=dev)


def _nearest(a, unit, factor, values, guess):
    """Indices into `values` of the one nearest to a / (factor * unit), ties to the even index.  `guess` is at most one
    off; a is compared with the midpoints times factor * unit in two exact halves of the product, so ties are decided
    exactly."""
    ends = torch.tensor([-math.inf, math.inf], device=a.device)
    mid = factor * torch.cat((ends[:1], (values[1:] + values[:-1]) / 2, ends[1:])).clamp(-1e30, 1e30)
    high = (unit.view(torch.int32) & -4096).view(torch.float32)
    low, odd = unit - high, guess % 2 == 1
    up, down = mid[guess + 1], mid[guess]
    over, under = a - up * high, a - down * high
    c = guess + ((over > up * low) | ((over == up * low) & odd)) - ((under < down * low) | ((under == down * low) & odd)).int()
    return torch.where(unit > 0, c, 0)


def _e4m3(a, unit, factor=1.0):
    """E4M3 bytes of the values nearest to a / (factor * unit), a >= 0, at most 448."""
    r = torch.where(unit > 0, a / (factor * unit), 0.0).clamp(max=448.0)
    values = torch.arange(127, dtype=torch.uint8, device=a.device).view(F8).float()
    return _nearest(a, unit, factor, values, r.to(F8).view(torch.uint8).int()).to(torch.uint8)


def _nvfp4(x, g):
    """(scale bytes [..., n/16], nibble bytes [..., n/2]) of x [..., n] with global scale g (broadcast over blocks)."""
    b = x.reshape(*x.shape[:-1], -1, 16)
    a, grid = b.abs(), torch.tensor(GRID, device=x.device)
    code = _e4m3(a.amax(-1), g, 6.0)
    s = (code.view(F8).float() * g)[..., None]
    r = torch.where(s > 0, a / s, 0.0)
    idx = _nearest(a, s, 1.0, grid, torch.bucketize(r, (grid[1:] + grid[:-1]) / 2).int()).to(torch.uint8)
    idx |= torch.signbit(b).to(torch.uint8) << 3
    idx = idx.reshape(*x.shape[:-1], -1, 2)
    return code, idx[..., 0] | (idx[..., 1] << 4)


def _activations(gen, rows, cin):
    """Rows of a residual stream: normal values, one channel in two hundred twenty times as large."""
    x = _rand(gen, rows, cin)
    out = torch.randperm(cin, generator=gen, device="cuda")[:max(1, cin // 200)]
    x[:, out] *= 20.0
    return x


def _eight_bit(x, group):
    """(E4M3 values, scales) of x [rows, cin], a scale for each row or each 128 channels of it."""
    rows, cin = x.shape
    width = group or cin
    n = math.ceil(cin / width)
    padded = torch.nn.functional.pad(x, (0, n * width - cin)).reshape(rows, n, width)
    s = padded.abs().amax(-1) / 448.0
    q = torch.where(s[..., None] > 0, padded / s[..., None], 0.0).clamp(-448.0, 448.0).to(F8)
    return q.reshape(rows, n * width)[:, :cin].contiguous(), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state, op = {"case": case}, case["op"]
    if op == "norm":
        t = TYPES[case["dtype"]]
        state["x"] = _rand(gen, case["rows"], case["cin"]).to(t)
        state["r"] = _activations(gen, case["rows"], case["cin"]).to(t) if case["residual"] else None
        state["gamma"] = (1.0 + 0.2 * _rand(gen, case["cin"])).to(t)
    elif op in ("matvec", "experts"):
        experts, cout, cin = case.get("experts", 1), case["cout"], case["cin"]
        code = torch.empty(experts, cout, cin // 16, dtype=torch.uint8, device="cuda")
        fp4 = torch.empty(experts, cout, cin // 2, dtype=torch.uint8, device="cuda")
        amax = torch.empty(experts, device="cuda")
        for e in range(0, experts, 32):
            w = 0.02 * _rand(gen, min(32, experts - e), cout, cin)
            amax[e:e + 32] = w.abs().amax((1, 2))
            code[e:e + 32], fp4[e:e + 32] = _nvfp4(w, (amax[e:e + 32] / 2688.0)[:, None, None])
        code.clamp_(1, 126)
        x = _activations(gen, case.get("rows") or case["tokens"], cin)
        state["offsets"] = None
        if op == "experts":
            offsets, token = _routing(case, seed)
            state["offsets"] = torch.from_numpy(offsets).cuda()
            x = x[torch.from_numpy(token).cuda()]
        if case["x"] == "e4m3":
            state["x"], state["x_scale"] = _eight_bit(x, case["group"])
        else:
            state["x"], state["x_scale"] = x.to(TYPES[case["x"]]), None
        state.update(code=code, fp4=fp4, amax=amax)
    elif op == "cache":
        pages = -(-case["tokens"] // case["page"]) + 3
        state.update(_pages(case, pages))
        # a projection's output [tokens, q | k | v heads], of which the cache takes the key and value parts
        t = TYPES[case["dtype"]]
        heads, dim = case["heads"], case["dim"]
        qkv = _rand(gen, case["tokens"], 3 * heads, dim)
        qkv[:, heads:2 * heads, ::31] *= 8.0
        state["qkv"] = qkv.to(t)
        state["k_amax"] = state["qkv"][:, heads:2 * heads].abs().amax((0, 2)).float()
        state["v_amax"] = state["qkv"][:, 2 * heads:].abs().amax((0, 2)).float()
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(case["tokens"], device="cuda")
        state["slots"] = order[at // case["page"]] * case["page"] + at % case["page"]
    else:
        lens = _lengths(case)
        need = [-(-n // case["page"]) for n in lens]
        pages, heads, dim = sum(need) + 1, case["heads"], case["dim"]
        state.update(_pages(case, pages))
        for name in ("k", "v"):
            state[name + "_amax"] = 4.0 + torch.rand(heads, generator=gen, device="cuda")
            g = state[name + "_amax"][None, :, None, None]
            for p in range(0, pages, 4096):
                x = _rand(gen, min(4096, pages - p), heads, case["page"], dim)
                if name == "k":
                    x[..., ::31] *= 3.0
                if case["fmt"] == "nvfp4":
                    state[name + "_scale"][p:p + 4096], state[name][p:p + 4096] = _nvfp4(x, g / 2688.0)
                else:
                    state[name][p:p + 4096] = (x / (g / 448.0)).clamp(-448.0, 448.0).to(F8).view(torch.uint8)
        table = np.full((case["batch"], max(need + [1])), -1, dtype=np.int32)
        order = np.random.default_rng([seed, 5]).permutation(pages)
        for b, n in enumerate(need):
            table[b, :n] = order[sum(need[:b]):sum(need[:b]) + n]
        state["table"] = torch.from_numpy(table).cuda()
        state["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        state["q"] = (1.5 * _rand(gen, case["batch"], heads * case["share"], dim)).to(TYPES[case["dtype"]])
    return state


def _pages(case, pages):
    shape = (pages, case["heads"], case["page"])
    four = case["fmt"] == "nvfp4"
    new = lambda n: torch.zeros(*shape, n, dtype=torch.uint8, device="cuda")  # noqa: E731
    d = {k: new(case["dim"] // 2 if four else case["dim"]) for k in ("k", "v")}
    d.update({k: new(case["dim"] // 16) if four else None for k in ("k_scale", "v_scale")})
    return d


# ------------------------------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return {"norm": _norm, "matvec": _matvec, "experts": _experts, "cache": _cache, "attention": _attention}[case["op"]](case, state)


def _own(case, s):
    import nvfp4_scale_calibration_lh_amd as lh
    op = case["op"]
    if op == "norm":
        q, scale, summed = lh.lh_rms_norm_quant(s["x"], s["gamma"], s["r"], eps=1e-6, group=case["group"])
        return {"q": q, "scale": scale, "summed": summed}
    if op in ("matvec", "experts"):
        return lh.lh_matvec(s["x"], s["code"], s["fp4"], s["amax"], x_scale=s["x_scale"], x_group=case["group"], offsets=s["offsets"])
    cache = lh.Cache(s["k"], s["v"], s["k_amax"], s["v_amax"], s["k_scale"], s["v_scale"])
    if op == "cache":
        h = case["heads"]
        lh.lh_cache_write(cache, s["qkv"][:, h:2 * h], s["qkv"][:, 2 * h:], s["slots"])
        return lh.lh_cache_read(cache, s["slots"])
    return lh.lh_paged_attention(s["q"], cache, s["table"], s["lengths"], scale=case["dim"] ** -0.5)


def _norm(case, s):
    x, t = s["x"], s["x"].dtype
    summed = (x.float() + s["r"].float()).to(t) if s["r"] is not None else None
    h = (x if summed is None else summed).float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["gamma"].float()
    q, scale = _eight_bit(y, case["group"])
    return {"q": q, "scale": scale, "summed": summed}


def _weights(code, fp4, amax):
    """Weight values [..., cout, cin] in 32 bits."""
    nibbles = torch.stack((fp4 & 15, fp4 >> 4), -1).flatten(-2)
    w = _grid()[nibbles.int()].unflatten(-1, (-1, 16))
    return (w * (code.view(F8).float() * (amax / 2688.0)[..., None, None])[..., None]).flatten(-2)


def _rows(case, s):
    x = s["x"].float()
    if s["x_scale"] is None:
        return x
    width = case["group"] or case["cin"]
    return x * s["x_scale"].repeat_interleave(width, 1)[:, :case["cin"]]


def _matvec(case, s):
    y = _rows(case, s) @ _weights(s["code"], s["fp4"], s["amax"])[0].t()
    return y.to(torch.float32 if case["x"] == "f32" else torch.bfloat16)


def _experts(case, s):
    x = _rows(case, s)
    e = torch.searchsorted(s["offsets"], torch.arange(x.shape[0], device=x.device), right=True) - 1
    y = (_weights(s["code"][e], s["fp4"][e], s["amax"][e]) * x[:, None, :]).sum(-1)
    return y.to(torch.float32 if case["x"] == "f32" else torch.bfloat16)


def _held(case, codes, scales, amax):
    """Values [..., heads, dim] in 32 bits of gathered cache rows (heads next to last)."""
    if case["fmt"] == "e4m3":
        return codes.view(F8).float() * (amax / 448.0)[:, None]
    nibbles = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    w = _grid()[nibbles.int()].unflatten(-1, (-1, 16))
    return (w * (scales.view(F8).float() * (amax / 2688.0)[:, None])[..., None]).flatten(-2)


def _cache(case, s):
    h, page, back = case["heads"], s["slots"] // case["page"], []
    at = s["slots"] % case["page"]
    for name, x in (("k", s["qkv"][:, h:2 * h]), ("v", s["qkv"][:, 2 * h:])):
        amax, scales = s[name + "_amax"], None
        if case["fmt"] == "nvfp4":
            s[name + "_scale"][page, :, at], s[name][page, :, at] = _nvfp4(x.float(), (amax / 2688.0)[:, None])
            scales = s[name + "_scale"][page, :, at]
        else:
            g = (amax / 448.0)[:, None]
            s[name][page, :, at] = _e4m3(x.float().abs(), g) | (torch.signbit(x).to(torch.uint8) << 7)
        back.append(_held(case, s[name][page, :, at], scales, amax).to(torch.bfloat16))
    return tuple(back)


def _attention(case, s):
    at = torch.arange(s["table"].shape[1] * case["page"], device="cuda")
    live = at[None, :] < s["lengths"][:, None]
    page, off = s["table"][:, at // case["page"]].clamp(min=0).long(), at % case["page"]
    held = lambda n: _held(case, s[n][page, :, off], None if s[n + "_scale"] is None else s[n + "_scale"][page, :, off], s[n + "_amax"])  # noqa: E731
    k, v = held("k").permute(0, 2, 3, 1).contiguous(), held("v").transpose(1, 2).contiguous()
    q = s["q"].float().unflatten(1, (case["heads"], case["share"]))
    scores = torch.matmul(q, k) * case["dim"] ** -0.5
    scores = torch.where(live[:, None, None, :], scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return o.flatten(1, 2).to(s["q"].dtype)


# ------------------------------------------------------------------------------------- in 64 bits
def _e4m3_64(byte):
    b = byte.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * torch.exp2(e.double() - 7.0))
    return torch.where(b >= 128, -mag, mag)


def _e2m1_64(byte):
    """Both values of each byte, low half first, on a new last axis flattened into the last."""
    def half(n):
        n = n.to(torch.int64)
        e, m = (n >> 1) & 3, (n & 1).double()
        mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2(e.double() - 1.0))
        return torch.where(n >= 8, -mag, mag)
    return torch.stack((half(byte & 15), half(byte >> 4)), -1).flatten(-2)


def _values_64(codes, scales, amax, four):
    """Values [..., n] of codes whose amax broadcasts over the last axis; the global scale is fp32 by definition."""
    if not four:
        return _e4m3_64(codes) * (amax / 448.0).double()
    v = _e4m3_64(scales) * (amax / 2688.0).double()
    return _e2m1_64(codes) * v.repeat_interleave(16, -1)


def _quantised_64(x, amax, four):
    """The values that x [..., n] is held as, by the definition; decisions on exact 64-bit numbers."""
    a = x.abs()
    if not four:
        g = (amax / 448.0).double()
        r = (a / g).clamp(max=448.0)
        step = torch.exp2(torch.floor(torch.log2(r.clamp(min=2.0 ** -6))) - 3.0)
        return torch.copysign(torch.round(r / step) * step * g, x)
    g = (amax / 2688.0).double()
    b = a.unflatten(-1, (-1, 16))
    r = (b.amax(-1) / (6.0 * g)).clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(r.clamp(min=2.0 ** -6))) - 3.0)
    s = ((torch.round(r / step) * step * g).float().double())[..., None]
    t = torch.where(s > 0, b / s, 0.0)
    step = torch.exp2(torch.floor(torch.log2(t.clamp(1.0, 4.0))) - 1.0)
    return torch.copysign(((torch.round(t / step) * step).clamp(max=6.0) * s).flatten(-2), x)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        total = s["x"].double() + s["r"].double() if s["r"] is not None else None
        h = s["x"].double() if total is None else total.to(s["x"].dtype).double()   # the norm is of the rounded sum
        y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["gamma"].double()
        width = case["group"] or case["cin"]
        parts = y.split(width, 1)
        scale = torch.stack([p.abs().amax(1) for p in parts], 1) / 448.0
        # q as the number that the 8 bits stand for before their rounding
        return {"q": torch.cat([p / scale[:, i:i + 1] for i, p in enumerate(parts)], 1), "scale": scale, "summed": total}
    if op in ("matvec", "experts"):
        x = s["x"].double() if case["x"] != "e4m3" else _e4m3_64(s["x"].view(torch.uint8))
        if s["x_scale"] is not None:
            width = case["group"] or case["cin"]
            x = torch.cat([p * s["x_scale"][:, i:i + 1].double() for i, p in enumerate(x.split(width, 1))], 1)
        offsets = [0, x.shape[0]] if s["offsets"] is None else s["offsets"].tolist()
        y = torch.zeros(x.shape[0], case["cout"], dtype=torch.float64, device="cuda")
        for e in range(len(offsets) - 1):
            a, b = offsets[e], offsets[e + 1]
            if b > a:
                y[a:b] = x[a:b] @ _values_64(s["fp4"][e], s["code"][e], s["amax"][e], True).t().contiguous()
        return y
    four = case["fmt"] == "nvfp4"
    if op == "cache":
        h = case["heads"]
        return tuple(_quantised_64(x.double(), s[n + "_amax"][:, None], four)
                     for n, x in (("k", s["qkv"][:, h:2 * h]), ("v", s["qkv"][:, 2 * h:])))
    out = torch.zeros(case["batch"], case["heads"] * case["share"], case["dim"], dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // case["page"])].long()
        for h in range(case["heads"]):
            k, v = (_values_64(s[i][pages, h].flatten(0, 1)[:n], None if not four else s[i + "_scale"][pages, h].flatten(0, 1)[:n],
                               s[i + "_amax"][h], four) for i in ("k", "v"))
            mine = slice(h * case["share"], (h + 1) * case["share"])
            p = torch.softmax(s["q"][b, mine].double() @ k.t().contiguous() * case["dim"] ** -0.5, -1)
            out[b, mine] = p @ v
    return out
