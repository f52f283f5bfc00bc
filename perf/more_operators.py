"""Cases for further operators of a serving step: growing the paged cache's block tables, rotary positions,
the choice of experts, a whole mixture-of-experts layer on NVFP4 weights, and low-rank adapters beside a
projection.

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU from a seed, ``run`` makes one pass
(elementary torch operations, or the library's entry points where ``own`` is true), ``exact`` gives the same
outputs from the definitions in 64 bits, and ``work`` the bytes and operations of one pass.

NVFP4 weights are E2M1 nibbles (element 2j in the low half of byte j) times an E4M3 scale byte per 16 of them
times g = fp32(amax / (6 * 448)) of their matrix.  E4M3 rows are bytes times a scale of their row or of 128 channels of it.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 64 conversations: a token each, a new page for some; all latency
        dict(name="extend-decode", op="extend", batch=64, longest=8191, page=16, rows=64, mixed=False),
        # a scheduler's step over many requests: prompts, decodes, idle and finished ones, drafted tokens taken back
        dict(name="extend-mixed", op="extend", batch=1024, longest=16411, page=24, rows=900000, mixed=True),
        # one user's next token, queries and keys as parts of the projection's row; all latency
        dict(name="rotary-one-token", op="rotary", tokens=1, heads=32, kv_heads=8, dim=128, rot=128, interleaved=False,
             parts=False, far=8191, dtype="bf16", inverse=False),
        # a prompt of odd length
        dict(name="rotary-prompt", op="rotary", tokens=8191, heads=32, kv_heads=8, dim=128, rot=128, interleaved=False,
             parts=False, far=8191, dtype="bf16", inverse=False),
        # a part of each head, neighbours paired, frequencies scaled for a long context, in full precision
        dict(name="rotary-far", op="rotary", tokens=3001, heads=8, kv_heads=2, dim=256, rot=64, interleaved=True,
             parts=True, far=131001, dtype="f32", inverse=False),
        # the choice of ten of 512 experts for a decode batch
        dict(name="route-step", op="route", tokens=32, experts=512, topk=10, dtype="bf16", renormalize=True, masked=1),
        # for a prompt
        dict(name="route-prompt", op="route", tokens=8192, experts=512, topk=10, dtype="f32", renormalize=True, masked=0),
        # one token through the 512-expert layer: its ten experts' weights, latency counts
        dict(name="moe-one-token", op="moe", experts=512, hidden=2560, inner=640, tokens=1, topk=10, x="bf16", group=0, padded=0),
        # a decode batch in 8 bits, its last rows padding
        dict(name="moe-batch-8bit", op="moe", experts=512, hidden=2560, inner=640, tokens=32, topk=10, x="e4m3", group=128, padded=3),
        # eight wide experts of the 12288x4096 projection's size, all of them hit several times
        dict(name="moe-wide", op="moe", experts=8, hidden=4096, inner=12288, tokens=61, topk=2, x="bf16", group=0, padded=0),
        # one request's adapter beside the 12288x4096 projection
        dict(name="adapter-one", op="adapter", rows=1, cin=4096, cout=12288, adapters=4, rank=16, x="bf16", group=0, weights="bf16", ragged=False),
        # a batch whose requests bring adapters of their own, of several ranks, some none
        dict(name="adapter-many", op="adapter", rows=96, cin=4096, cout=12288, adapters=64, rank=64, x="e4m3", group=128, weights="bf16", ragged=True),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))

    op = rng.choice(["extend", "rotary", "route", "moe", "moe", "adapter", "adapter"])
    if op == "extend":
        batch, mixed = log(1, 1024), rng.random() < 0.6
        longest = log(16, 16411)
        return dict(op=op, batch=batch, longest=longest, page=rng.choice([1, 16, 24, 64]),
                    rows=min(900000, batch * max(16, longest // 16)) if mixed else batch + rng.randint(0, 7), mixed=mixed)
    if op == "rotary":
        dim, kv = rng.choice([64, 96, 128, 256]), rng.choice([0, 1, 2, 8])
        heads = max(kv, 1) * rng.choice([1, 4, 7, 8])
        return dict(op=op, tokens=log(1, min(30000, 8191 * 40 * 128 // ((heads + kv) * dim))), heads=heads, kv_heads=kv, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, dim // 4, 20]), interleaved=rng.random() < 0.5, parts=rng.random() < 0.4,
                    far=rng.choice([100, 8191, 131001, 1000003]), dtype=rng.choice(["bf16", "bf16", "f32"]), inverse=rng.random() < 0.25)
    if op == "route":
        experts = log(4, 1024)
        return dict(op=op, tokens=log(1, min(8192, 8192 * 512 // experts)), experts=experts, topk=rng.randint(1, min(16, experts)),
                    dtype=rng.choice(["bf16", "f32"]), renormalize=rng.random() < 0.7, masked=rng.choice([0, 1, 3]))
    x, group = rng.choice(["bf16", "bf16", "e4m3", "f32"]), rng.choice([0, 128])
    if op == "moe":
        experts, hidden = log(4, 512), 16 * log(8, 256)
        inner = 16 * log(4, max(4, min(768, 1500000000 // (48 * experts * hidden))))
        tokens = log(1, 64)
        return dict(op=op, experts=experts, hidden=hidden, inner=inner, tokens=tokens, topk=rng.randint(1, min(10, experts)),
                    x=x, group=group, padded=rng.choice([0, 0, min(3, tokens - 1)]))
    rank, cin, cout = rng.choice([8, 16, 32, 64]), 16 * log(8, 768), log(64, 12288)
    adapters = log(1, max(1, min(128, 64 * 64 * 16384 // (rank * (cin + cout)))))
    return dict(op=op, rows=log(1, 128), cin=cin, cout=cout, adapters=adapters, rank=rank, x=x, group=group,
                weights=rng.choice(["bf16", "bf16", "f32"]), ragged=rng.random() < 0.5)


def _lengths(case):
    """Tokens that each request has in the cache: spread evenly up to the longest, an empty one among them."""
    lens = [max(1, int(case["longest"] * (1.0 - (i * 0.6180339887498949) % 1.0))) for i in range(case["batch"])]
    if case["batch"] > 2:
        lens[case["batch"] // 2] = 0
    return np.array(lens, dtype=np.int64)


def _most(case):
    """Tokens of a prompt are fewer than this."""
    return max(2, min(case["longest"], 12 * case["rows"] // case["batch"]))


def _asked(case, seed):
    """New tokens of each request: one, or a mix of prompts (0.1), decodes, idle ones, drafts taken back and finished ones."""
    batch = case["batch"]
    if not case["mixed"]:
        return np.ones(batch, dtype=np.int64)
    r = np.random.default_rng([seed, 7])
    kind = r.random(batch)
    asked = np.where(kind < 0.1, r.integers(1, _most(case), batch), 1)
    asked = np.where((kind > 0.8) & (kind < 0.88), 0, asked)
    asked = np.where((kind >= 0.88) & (kind < 0.94), -r.integers(1, 8, batch), asked)
    return np.where(kind >= 0.94, -(2 ** 31 - 1), asked)


def _choices(case, seed):
    """The experts [tokens, topk] of each token: top-k of Zipf-weighted Gumbel scores; -1 for padding rows."""
    r = np.random.default_rng([seed, 3])
    logits = -1.1 * np.log(r.permutation(case["experts"]) + 1.0)
    ids = np.argsort(-(logits + r.gumbel(size=(case["tokens"], case["experts"]))), axis=1)[:, :case["topk"]]
    ids[case["tokens"] - case["padded"]:] = -1
    return ids.astype(np.int32)


def _index(case, seed):
    """The adapter of each row, one row in eight without."""
    r = np.random.default_rng([seed, 11])
    index = r.integers(0, case["adapters"], case["rows"])
    if case["rows"] > 3:
        index[r.random(case["rows"]) < 0.125] = -1
    return index.astype(np.int32)


def _ranks(case, seed):
    r = np.random.default_rng([seed, 13])
    return r.integers(4, case["rank"] + 1, case["adapters"]).astype(np.int32) if case["ragged"] else np.full(case["adapters"], case["rank"], np.int32)


def work(case):
    op = case["op"]
    if op == "extend":
        new = np.maximum(_asked(case, 0), 0)
        pages = int(new.sum()) // case["page"] + case["batch"]
        return {"bytes": 16 * case["rows"] + 16 * case["batch"] + 8 * pages, "flops": 4 * case["rows"]}
    if op == "rotary":
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * (case["heads"] + case["kv_heads"])
        return {"bytes": 2 * n * case["dim"] * size + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    if op == "route":
        n = case["tokens"] * case["experts"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + 8 * case["tokens"] * case["topk"], "flops": 4 * n}
    x, y = {"bf16": (2, 2), "f32": (4, 4), "e4m3": (1, 2)}[case["x"]]
    if op == "moe":
        ids = _choices(case, 0)
        ids = ids[ids >= 0]
        weights = 3 * case["hidden"] * case["inner"]
        return {"bytes": len(np.unique(ids)) * weights * 9 // 16 + case["tokens"] * case["hidden"] * (x + y) + 8 * ids.size,
                "flops": 2 * ids.size * weights}
    index, ranks = _index(case, 0), _ranks(case, 0)
    both = case["cin"] + case["cout"]
    held = int(ranks[np.unique(index[index >= 0])].sum()) * both * (2 if case["weights"] == "bf16" else 4)
    return {"bytes": held + case["rows"] * (case["cin"] * x + 2 * case["cout"] * y), "flops": 2 * both * int(ranks[index[index >= 0]].sum())}


# ------------------------------------------------------------------------------------- the inputs
def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _nvfp4(w):
    """(scale bytes, nibble bytes, amax) of weights [n, cout, cin], block scales by their largest element."""
    amax = w.abs().amax((1, 2))
    g = (amax / 2688.0)[:, None, None]
    b = w.unflatten(-1, (-1, 16))
    code = (b.abs().amax(-1) / (6.0 * g)).clamp(2.0 ** -9, 448.0).to(F8)
    grid = torch.tensor(GRID, device=w.device)
    nib = torch.bucketize(b.abs() / (code.float() * g)[..., None], (grid[1:] + grid[:-1]) / 2, out_int32=True).to(torch.uint8)
    nib |= (b < 0).to(torch.uint8) << 3
    nib = nib.flatten(-2).unflatten(-1, (-1, 2))
    return code.view(torch.uint8), nib[..., 0] | (nib[..., 1] << 4), amax


def _matrices(gen, n, cout, cin):
    code = torch.empty(n, cout, cin // 16, dtype=torch.uint8, device="cuda")
    fp4 = torch.empty(n, cout, cin // 2, dtype=torch.uint8, device="cuda")
    amax = torch.empty(n, device="cuda")
    step = max(1, 200000000 // (cout * cin))
    for e in range(0, n, step):
        code[e:e + step], fp4[e:e + step], amax[e:e + step] = _nvfp4(0.02 * _rand(gen, min(step, n - e), cout, cin))
    return code, fp4, amax


def _activations(gen, case, rows, cin):
    """(rows of a normed stream with a few large channels, their scales or None), in the case's type."""
    x = _rand(gen, rows, cin)
    x[:, torch.randperm(cin, generator=gen, device="cuda")[:max(1, cin // 200)]] *= 20.0
    if case["x"] != "e4m3":
        return x.to(TYPES[case["x"]]), None
    width = case["group"] or cin
    n = math.ceil(cin / width)
    padded = torch.nn.functional.pad(x, (0, n * width - cin)).reshape(rows, n, width)
    s = padded.abs().amax(-1) / 448.0
    q = (padded / s[..., None].clamp(min=1e-30)).clamp(-448.0, 448.0).to(F8)
    return q.reshape(rows, n * width)[:, :cin].contiguous(), s


def _frequencies(case):
    """Angles per position, fp32; `parts` stretches those that turn fewer than 32 times in 4096 positions, by up to 32."""
    f = 10000.0 ** (-np.arange(0, case["rot"], 2) / case["rot"])
    if case["parts"]:
        keep = np.clip((4096 * f / (2 * np.pi) - 1.0) / 31.0, 0.0, 1.0)
        f = f * (keep + (1.0 - keep) / 32.0)
    return f.astype(np.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state, op = {"case": case}, case["op"]
    if op == "extend":
        lens, asked, page = _lengths(case), _asked(case, seed), case["page"]
        held = -(-lens // page)
        width = -(-(case["longest"] + _most(case)) // page)
        need, pool = int((-(-(lens + np.maximum(asked, 0)) // page) - held).sum()), case["rows"] // page + case["batch"]
        free = max(1, min(need - need // 16, pool))      # the last requests may find no page
        order = np.random.default_rng([seed, 5]).permutation(int(held.sum()) + pool).astype(np.int32)
        table = np.full((case["batch"], width), -1, dtype=np.int32)
        table[np.arange(width)[None, :] < held[:, None]] = order[pool:]
        stack = np.full(len(order), -1, dtype=np.int32)
        stack[:free] = order[:free]
        for name, a in (("table", table), ("lengths", lens.astype(np.int32)), ("asked", asked.astype(np.int32)), ("stack", stack),
                        ("count", np.array([free], dtype=np.int32))):
            state[name] = torch.from_numpy(a).cuda()
    elif op == "rotary":
        # parts of a projection's rows [tokens, q | k | v heads]
        qkv = _rand(gen, case["tokens"], case["heads"] + 2 * case["kv_heads"], case["dim"]).to(TYPES[case["dtype"]])
        state["q"] = qkv[:, :case["heads"]]
        state["k"] = qkv[:, case["heads"]:case["heads"] + case["kv_heads"]] if case["kv_heads"] else None
        at = torch.arange(case["tokens"], device="cuda") + max(0, case["far"] - case["tokens"])
        if case["tokens"] > 64:
            at[7::61] = -1                               # padding rows
        state["positions"] = at.to(torch.int32)
        state["frequencies"] = torch.from_numpy(_frequencies(case)).cuda()
        state["scale"] = 0.1 * math.log(32.0) + 1.0 if case["parts"] else 1.0
    elif op == "route":
        logits = 2.0 * _rand(gen, case["tokens"], case["experts"])
        if case["masked"]:                               # experts that are not to be chosen, and a row of none
            off = torch.randperm(case["experts"], generator=gen, device="cuda")[:case["experts"] // 4]
            logits[:, off] = -math.inf
            if case["tokens"] > case["masked"]:
                logits[case["tokens"] - case["masked"]:] = -math.inf
        state["logits"] = logits.to(TYPES[case["dtype"]])
    elif op == "moe":
        state["gate_up"] = _matrices(gen, case["experts"], 2 * case["inner"], case["hidden"])
        state["down"] = _matrices(gen, case["experts"], case["hidden"], case["inner"])
        state["x"], state["x_scale"] = _activations(gen, case, case["tokens"], case["hidden"])
        state["ids"] = torch.from_numpy(_choices(case, seed)).cuda()
        state["weights"] = torch.softmax(_rand(gen, case["tokens"], case["topk"]), -1)
    else:
        t = TYPES[case["weights"]]
        state["x"], state["x_scale"] = _activations(gen, case, case["rows"], case["cin"])
        state["base"] = _rand(gen, case["rows"], case["cout"]).to(TYPES["f32" if case["x"] == "f32" else "bf16"])
        state["a"] = (case["cin"] ** -0.5 * _rand(gen, case["adapters"], case["rank"], case["cin"])).to(t)
        state["b"] = (0.1 * _rand(gen, case["adapters"], case["cout"], case["rank"])).to(t)
        state["index"] = torch.from_numpy(_index(case, seed)).cuda()
        state["ranks"] = torch.from_numpy(_ranks(case, seed)).cuda()
        state["scaling"] = 16.0 / state["ranks"].float()
    return state


# ------------------------------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return {"extend": _extend, "rotary": _rotary, "route": _route, "moe": _moe, "adapter": _adapter}[case["op"]](case, state)


def _own(case, s):
    import nvfp4_scale_calibration_lh_amd as lh
    op = case["op"]
    if op == "extend":
        slots, positions, sequence, offsets, lengths, count = lh.lh_cache_extend(
            s["table"], s["lengths"], s["asked"] if case["mixed"] else None, s["stack"], s["count"], page_size=case["page"], max_tokens=case["rows"])
        return {"slots": slots, "positions": positions, "sequence": sequence, "offsets": offsets, "lengths": lengths, "count": count,
                "table": s["table"], "stack": s["stack"]}
    if op == "rotary":
        return lh.lh_rotary(s["q"], s["k"], s["positions"], s["frequencies"], interleaved=case["interleaved"], inverse=case["inverse"],
                            scale=s["scale"])
    if op == "route":
        return lh.lh_route(s["logits"], case["topk"], renormalize=case["renormalize"])
    if op == "moe":
        return lh.lh_moe(s["x"], s["ids"], s["weights"], s["gate_up"], s["down"], x_scale=s["x_scale"], x_group=case["group"])
    return lh.lh_adapter(s["x"], s["base"], s["a"], s["b"], s["index"], scaling=s["scaling"], ranks=s["ranks"] if case["ragged"] else None,
                         x_scale=s["x_scale"], x_group=case["group"])


def _extend(case, s):
    table, stack, page, rows = s["table"], s["stack"], case["page"], case["rows"]
    most = table.shape[1] * page
    lens, asked = s["lengths"].long().clamp(0, most), s["asked"].long()
    up = lambda n: (n + page - 1) // page  # noqa: E731
    # pages given back go on top of the stack, in the order of the requests
    cut = (lens + asked.clamp(max=0)).clamp(min=0)
    freed = up(lens) - up(cut)
    held = torch.arange(table.shape[1], device="cuda")[None, :]
    back = table[(held >= up(cut)[:, None]) & (held < up(lens)[:, None])]
    count = s["count"].long()
    at = count + torch.arange(back.shape[0], device="cuda")
    stack[at[at < stack.shape[0]]] = back[at < stack.shape[0]]
    avail = (count + freed.sum()).clamp(max=stack.shape[0])
    # first come, first served; a request gets all its rows or none
    new = asked.clamp(min=0)
    ends = new.cumsum(0)
    fits = (lens + new <= most) & (ends <= rows)
    need = torch.where(fits, up(lens + new) - up(lens), 0)
    upto = need.cumsum(0)
    granted = fits & ((need == 0) | (upto <= avail))
    lengths = torch.where(granted, cut + new, cut)
    taken = torch.where(upto <= avail, upto, 0).amax()
    offsets = torch.cat((ends.new_zeros(1), ends)).clamp(max=rows)
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(offsets, row, right=True) - 1
    live = seq < case["batch"]
    b = seq.clamp(max=case["batch"] - 1)
    position = lens[b] + row - offsets[b]
    good = live & granted[b]
    p = (position // page).clamp(max=table.shape[1] - 1)
    fresh = p - up(lens)[b]
    pop = (avail - 1 - (upto - need)[b] - fresh).clamp(0, stack.shape[0] - 1)
    which = torch.where(fresh >= 0, stack[pop], table[b, p]).long()
    opens = good & (fresh >= 0) & (position % page == 0)
    table[b[opens], p[opens]] = which[opens].int()
    return {"slots": torch.where(good, which * page + position % page, -1), "positions": torch.where(good, position, -1).int(),
            "sequence": torch.where(live, seq, -1).int(), "offsets": offsets.int(), "lengths": lengths.int(), "count": (avail - taken).int(),
            "table": table, "stack": stack}


def _rotary(case, s):
    angle = s["positions"].double()[:, None] * s["frequencies"].double()
    # as 32-bit numbers, with the sine of a negative angle for the inverse
    c, d = (s["scale"] * angle.cos()).float()[:, None], (s["scale"] * angle.sin()).float()[:, None] * (-1.0 if case["inverse"] else 1.0)
    pad, out = (s["positions"] < 0)[:, None, None], []
    for x in (s["q"], s["k"]):
        if x is None:
            out.append(None)
            continue
        part = x[..., :case["rot"]].float()
        a, b = (part[..., ::2], part[..., 1::2]) if case["interleaved"] else part.chunk(2, -1)
        y = (a * c - b * d, a * d + b * c)
        y = torch.stack(y, -1).flatten(-2) if case["interleaved"] else torch.cat(y, -1)
        y = torch.cat((y.to(x.dtype), x[..., case["rot"]:]), -1)
        out.append(torch.where(pad, x, y))
    return tuple(out)


def _route(case, s):
    x = s["logits"].float()
    x = torch.where(torch.isnan(x), -math.inf, x)
    top, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    high = top[:, :1]
    high = torch.where(high == -math.inf, 0.0, high)
    e = torch.exp(top - high)
    chosen, k = e[:, :case["topk"]], case["topk"]
    total = (chosen if case["renormalize"] else e).sum(-1, keepdim=True)
    return torch.where(top[:, :k] == -math.inf, -1, ids[:, :k]).int(), chosen / torch.where(total > 0, total, 1.0)


def _dequantized(code, fp4, amax):
    """Weight values [n, cout, cin] in 32 bits."""
    pairs = torch.tensor(GRID + tuple(-v for v in GRID), device="cuda")
    w = pairs[torch.stack((fp4 & 15, fp4 >> 4), -1).flatten(-2).int()].unflatten(-1, (-1, 16))
    return (w * (code.view(F8).float() * (amax / 2688.0)[:, None, None])[..., None]).flatten(-2)


def _x32(case, s):
    x = s["x"].float()
    if s["x_scale"] is None:
        return x
    return x * s["x_scale"].repeat_interleave(case["group"] or x.shape[1], 1)[:, :x.shape[1]]


def _moe(case, s):
    x, ids, n = _x32(case, s), s["ids"].long(), case["inner"]
    w = torch.where(ids >= 0, s["weights"], 0.0)
    if ids.numel() < case["experts"]:                    # the matrices of each choice
        e = ids.clamp(min=0).flatten()
        rows = x.repeat_interleave(case["topk"], 0)[:, :, None]
        h = torch.bmm(_dequantized(*(t[e] for t in s["gate_up"])), rows)[..., 0]
        h = h[:, :n] / (1.0 + torch.exp(-h[:, :n])) * h[:, n:]
        y = torch.bmm(_dequantized(*(t[e] for t in s["down"])), h[:, :, None])[..., 0]
        y = (y.unflatten(0, ids.shape) * w[..., None]).sum(1)
    else:                                                # every expert for every token, weighted by 0 where not chosen
        share = torch.zeros(x.shape[0], case["experts"], device="cuda").scatter_add_(1, ids.clamp(min=0), w)
        y, step = 0.0, max(1, 800000000 // (n * x.shape[1]))
        for e in range(0, case["experts"], step):
            h = torch.matmul(x[None], _dequantized(*(t[e:e + step] for t in s["gate_up"])).transpose(1, 2).contiguous())
            h = h[..., :n] / (1.0 + torch.exp(-h[..., :n])) * h[..., n:]
            h = torch.matmul(h, _dequantized(*(t[e:e + step] for t in s["down"])).transpose(1, 2).contiguous())
            y = y + (h * share[:, e:e + step].t()[..., None]).sum(0)
    return y.to(torch.float32 if case["x"] == "f32" else torch.bfloat16)


def _adapter(case, s):
    i = s["index"].long().clamp(min=0)
    u = torch.bmm(s["a"][i].float(), _x32(case, s)[:, :, None])[..., 0]
    u = torch.where(torch.arange(case["rank"], device="cuda") < s["ranks"][i][:, None], u, 0.0) * s["scaling"][i][:, None]
    y = torch.bmm(s["b"][i].float(), u[:, :, None])[..., 0]
    return (s["base"].float() + torch.where(s["index"][:, None] >= 0, y, 0.0)).to(s["base"].dtype)


# ------------------------------------------------------------------------------------- in 64 bits
def _e4m3_64(byte):
    b = byte.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2(e.double() - 10.0))
    return torch.where(b >= 128, -mag, mag)


def _weights_64(code, fp4, amax):
    """[cout, cin] of one matrix; its global scale is an fp32 number by definition."""
    def half(n):
        n = n.long()
        e, m = (n >> 1) & 3, (n & 1).double()
        mag = torch.where(e == 0, 0.5 * m, (2.0 + m) * torch.exp2(e.double() - 2.0))
        return torch.where(n >= 8, -mag, mag)
    w = torch.stack((half(fp4 & 15), half(fp4 >> 4)), -1).flatten(-2)
    return w * (_e4m3_64(code) * (amax / 2688.0).double()).repeat_interleave(16, -1)


def _rows_64(case, s):
    if s["x_scale"] is None:
        return s["x"].double()
    x, width = _e4m3_64(s["x"].view(torch.uint8)), case["group"] or s["x"].shape[1]
    return torch.cat([p * s["x_scale"][:, i:i + 1].double() for i, p in enumerate(x.split(width, 1))], 1)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    return {"extend": _exact_extend, "rotary": _exact_rotary, "route": _exact_route, "moe": _exact_moe, "adapter": _exact_adapter}[op](case, s)


def _exact_extend(case, s):
    """Request by request."""
    table, stack, lens, asked = (s[n].cpu().numpy().astype(np.int64) for n in ("table", "stack", "lengths", "asked"))
    page, rows, top = case["page"], case["rows"], int(s["count"])
    pages = lambda n: -(-n // page)  # noqa: E731
    out = lens.copy()
    for b, n in enumerate(asked):
        if n < 0:
            out[b] = max(0, lens[b] + n)
            for i in range(pages(out[b]), pages(lens[b])):
                if top < len(stack):
                    stack[top] = table[b, i]
                    top += 1
    slots, positions, sequence = (np.full(rows, -1, dtype=np.int64) for _ in range(3))
    offsets, wanted, start, left = [0], 0, 0, top
    for b, n in enumerate(asked):
        n = max(int(n), 0)
        sequence[start:start + n] = b
        if n and lens[b] + n <= table.shape[1] * page and start + n <= rows:
            have = pages(lens[b])
            need = pages(lens[b] + n) - have
            wanted += need
            if need == 0 or wanted <= top:
                table[b, have:have + need] = stack[left - need:left][::-1]
                left -= need
                at = lens[b] + np.arange(n)
                slots[start:start + n], positions[start:start + n] = table[b, at // page] * page + at % page, at
                out[b] += n
        start += n
        offsets.append(min(start, rows))
    return {"slots": slots, "positions": positions, "sequence": sequence, "offsets": np.array(offsets), "lengths": out, "count": np.array([left]),
            "table": table, "stack": stack}


def _exact_rotary(case, s):
    angle = s["positions"].cpu().numpy().astype(np.float64)[:, None] * _frequencies(case).astype(np.float64)
    turn = torch.from_numpy(s["scale"] * np.exp((-1j if case["inverse"] else 1j) * angle)).cuda()[:, None]
    live, half, out = (s["positions"] >= 0)[:, None, None], case["rot"] // 2, []
    for x in (s["q"], s["k"]):
        if x is None:
            out.append(None)
            continue
        y = x.double()
        a, b = (slice(0, case["rot"], 2), slice(1, case["rot"], 2)) if case["interleaved"] else (slice(0, half), slice(half, case["rot"]))
        z = torch.where(live, torch.complex(y[..., a], y[..., b]) * turn, torch.complex(y[..., a], y[..., b]))
        y[..., a], y[..., b] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_route(case, s):
    x = s["logits"].double().cpu().numpy()
    x = np.where(np.isnan(x), -np.inf, x)
    ids = np.argsort(-x, axis=1, kind="stable")[:, :case["topk"]]
    e = np.exp(x - np.where(np.isinf(x.max(1)), 0.0, x.max(1))[:, None])
    w = np.take_along_axis(e, ids, 1)
    total = (w if case["renormalize"] else e).sum(1, keepdims=True)
    none = np.isinf(np.take_along_axis(x, ids, 1))
    return np.where(none, -1, ids).astype(np.int32), w / np.where(total > 0, total, 1.0)


def _exact_moe(case, s):
    x, ids, y = _rows_64(case, s), s["ids"].cpu().numpy(), torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
    for e in np.unique(ids[ids >= 0]):
        t, j = (torch.from_numpy(i).cuda() for i in np.nonzero(ids == e))
        h = x[t] @ _weights_64(*(m[e] for m in s["gate_up"])).t().contiguous()
        gate, up = h.chunk(2, 1)
        h = gate * torch.sigmoid(gate) * up
        y.index_add_(0, t, s["weights"][t, j].double()[:, None] * (h @ _weights_64(*(m[e] for m in s["down"])).t().contiguous()))
    return y


def _exact_adapter(case, s):
    x, y, index = _rows_64(case, s), s["base"].double(), s["index"].cpu().numpy()
    for i in np.unique(index[index >= 0]):
        t, r = torch.from_numpy(np.nonzero(index == i)[0]).cuda(), int(s["ranks"][i])
        u = x[t] @ s["a"][i, :r].double().t().contiguous()
        y[t] += s["scaling"][i].double() * (u @ s["b"][i, :, :r].double().t().contiguous())
    return y
