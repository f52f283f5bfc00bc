"""A mixture-of-experts layer served to requests that come and go, prompts and single tokens in one batch.

    python examples/serve_layer.py [--rows 64]

Random bf16 weights are calibrated to NVFP4.  Each step then takes new tokens of some requests, takes drafts back from others and
lets finished ones go, with everything on the device:

    growth of the sequences | norm -> 8 bits | qkv product + adapters | rotary positions | cache write | attention over the cache |
    output product | norm + residual -> 8 bits | choice of experts | expert layer

A row of a prompt attends as a sequence of its own, of the length that its position gives.  The steps run eagerly and as one
replayed graph, and each row is compared with the same layer in float32 torch on the dequantized weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_scale_calibration_lh_amd as lh  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, EXPERTS, TOPK, INNER, PAGE, LONGEST, EPS = 512, 8, 2, 64, 16, 4, 256, 16, 96, 1e-6
ADAPTERS, RANK, CONTEXT = 3, 16, 4096
# new tokens of each of five requests, step by step: prompts, single tokens, idle ones, drafts taken back, one that ends and the next in its place
SCRIPT = [(13, 1, 30, 0, 7), (1, 1, 1, 5, 1), (1, 0, 4, 1, 1), (1, 1, -3, 1, 1), (1, -2 ** 31, 1, 1, 0), (1, 9, 1, 1, 1), (20, 1, 1, 1, -1), (1, 1, 1, 1, 1)]


def calibrated(W):
    """(code, fp4, amax) of W [G, cout, cin]."""
    amax = lh.lh_absmax(W)
    code, fp4, _ = lh.lh_scale_sweep_mse(W, amax, want_loss=False)
    return code, fp4, amax


class Layer:
    def __init__(self, rows, four_bit, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
        weight = lambda e, o, i: (rand(e, o, i) * i ** -0.5).bfloat16()  # noqa: E731
        self.rows, self.batch = rows, len(SCRIPT[0])
        self.gamma = [(1 + 0.1 * rand(HIDDEN)).bfloat16() for _ in range(2)]
        out = (HEADS + 2 * KV_HEADS) * DIM
        qkv = weight(1, out, HIDDEN)
        self.w = {"qkv": calibrated(qkv), "out": calibrated(weight(1, HIDDEN, HEADS * DIM)), "gate_up": calibrated(weight(EXPERTS, 2 * INNER, HIDDEN)),
                  "down": calibrated(weight(EXPERTS, HIDDEN, INNER))}
        self.router = rand(EXPERTS, HIDDEN).bfloat16() * HIDDEN ** -0.5
        self.a, self.b = weight(ADAPTERS, RANK, HIDDEN), (0.3 * rand(ADAPTERS, out, RANK)).bfloat16()
        self.ranks = torch.tensor([16, 5, 8], dtype=torch.int32, device="cuda")
        self.scaling = 2.0 / self.ranks.float()
        self.adapter_of = torch.tensor([0, 2, -1, 1, 0, -1], dtype=torch.int32, device="cuda")     # of each request; the last is for rows of none
        self.frequencies, self.scale = lh.lh_rotary_frequencies(DIM, scaling="parts", factor=4.0, original_context=CONTEXT)
        x = torch.nn.functional.rms_norm(rand(1024, HIDDEN), (HIDDEN,))
        amax = 1.6 * lh.lh_absmax((x @ qkv[0].float().t()).unflatten(1, (-1, DIM))[:, HEADS:].transpose(0, 1).contiguous())
        self.pages = self.batch * -(-LONGEST // PAGE)
        self.cache = lh.Cache.empty(self.pages, PAGE, KV_HEADS, DIM, amax[:KV_HEADS].contiguous(), amax[KV_HEADS:].contiguous(), four_bit=four_bit)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.order = torch.randperm(self.pages, generator=g, device="cuda").to(torch.int32)
        self.table = torch.empty(self.batch, -(-LONGEST // PAGE), **i32)
        self.lengths, self.stack, self.count, self.asked = torch.empty(self.batch, **i32), self.order.clone(), torch.empty(1, **i32), torch.zeros(self.batch, **i32)
        self.reset()

    def reset(self):
        self.table.fill_(-1)
        self.lengths.zero_()
        self.stack.copy_(self.order)
        self.count.fill_(self.pages)

    def step(self, tokens):
        """The new tokens asked for, tokens [batch, LONGEST, HIDDEN] bf16 by request and position: (rows' outputs, their inputs, the experts
        chosen, their weights, each row's request and position)."""
        slots, positions, sequence, _, _, _ = lh.lh_cache_extend(self.table, self.lengths, self.asked, self.stack, self.count, page_size=PAGE,
                                                                 max_tokens=self.rows, new_lengths=self.lengths, new_count=self.count)
        seq, pos = sequence.long(), positions.long()
        x = torch.where(pos[:, None] >= 0, tokens[seq, pos.clamp(min=0)], 0)           # (a sequence of -1 is the last)
        q, s, _ = lh.lh_rms_norm_quant(x, self.gamma[0], eps=EPS, group=128)
        qkv = lh.lh_matvec(q, *self.w["qkv"], x_scale=s, x_group=128)
        lh.lh_adapter(q, qkv, self.a, self.b, self.adapter_of[seq], qkv, scaling=self.scaling, ranks=self.ranks, x_scale=s, x_group=128)
        qkv = qkv.view(self.rows, -1, DIM)
        queries, keys = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS]
        lh.lh_rotary(queries, keys, positions, self.frequencies, scale=self.scale, out_q=queries, out_k=keys)
        lh.lh_cache_write(self.cache, keys, qkv[:, HEADS + KV_HEADS:], slots)
        o = lh.lh_paged_attention(queries, self.cache, self.table[seq], positions + 1, scale=DIM ** -0.5)
        y = lh.lh_matvec(o.view(self.rows, -1), *self.w["out"])
        q, s, y = lh.lh_rms_norm_quant(y, self.gamma[1], x, eps=EPS, group=128)
        normed = torch.nn.functional.rms_norm(y.float(), (HIDDEN,), self.gamma[1].float(), EPS)
        ids, weights = lh.lh_route(normed @ self.router.float().t(), TOPK)
        return y + lh.lh_moe(q, ids, weights, self.w["gate_up"], self.w["down"], x_scale=s, x_group=128), x, ids, weights, sequence, positions


class Plain:
    """The same layer in float32 torch on the dequantized weights, one row at a time, with the experts that were chosen."""

    def __init__(self, layer):
        self.l = layer
        self.w = {n: lh.lh_dequantize(*m, dtype=torch.float32, want_block_amax=False)[0] for n, m in layer.w.items()}
        self.keys, self.values = ([[] for _ in range(layer.batch)] for _ in range(2))
        self.a, self.b = layer.a.float(), layer.b.float()

    def cut(self, b, length):
        del self.keys[b][length:], self.values[b][length:]

    def row(self, x, b, position, ids, weights):
        layer = self.l
        h = torch.nn.functional.rms_norm(x, (HIDDEN,), layer.gamma[0].float(), EPS)
        qkv, a = self.w["qkv"][0] @ h, int(layer.adapter_of[b])
        if a >= 0:
            r = int(layer.ranks[a])
            qkv = qkv + layer.scaling[a] * (self.b[a][:, :r] @ (self.a[a][:r] @ h))
        qkv = qkv.view(-1, DIM)
        w = position * layer.frequencies.double()
        c, s = (layer.scale * w.cos()).float(), (layer.scale * w.sin()).float()
        first, second = qkv[:HEADS + KV_HEADS].chunk(2, -1)
        turned = torch.cat((first * c - second * s, first * s + second * c), -1)
        self.keys[b].append(turned[HEADS:])
        self.values[b].append(qkv[HEADS + KV_HEADS:])
        k, v = (torch.stack(t, 1).repeat_interleave(HEADS // KV_HEADS, 0) for t in (self.keys[b], self.values[b]))
        p = torch.softmax((turned[:HEADS, None] * k).sum(-1) * DIM ** -0.5, -1)
        y = x + self.w["out"][0] @ (p[..., None] * v).sum(1).flatten()
        h = torch.nn.functional.rms_norm(y, (HIDDEN,), layer.gamma[1].float(), EPS)
        for e, weight in zip(ids.tolist(), weights):
            gate, up = (self.w["gate_up"][e] @ h).chunk(2)
            y = y + weight * (self.w["down"][e] @ (torch.nn.functional.silu(gate) * up))
        return y


def run(rows=64, four_bit=False, seed=0):
    """(relative error of all rows against the plain layer, whether the graph's replays give the eager bits, rows)."""
    layer = Layer(rows, four_bit, seed)
    plain = Plain(layer)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    tokens = [torch.randn(layer.batch, LONGEST, HIDDEN, generator=g, device="cuda").bfloat16() for _ in SCRIPT]
    got, want, eager = [], [], []
    for asked, t in zip(SCRIPT, tokens):
        layer.asked.copy_(torch.tensor([max(n, -2 ** 31) for n in asked], dtype=torch.int32))
        out = layer.step(t)
        eager.append(out)
        y, x, ids, weights, sequence, positions = (o.cpu() for o in out)
        for b, n in enumerate(asked):
            if n < 0:
                plain.cut(b, max(len(plain.keys[b]) + n, 0))
        for r in range(sum(max(n, 0) for n in asked)):
            b = int(sequence[r])
            assert int(positions[r]) == len(plain.keys[b]), "a row's position is not the next of its request"
            got.append(y[r].float())
            want.append(plain.row(x[r].float().cuda(), b, int(positions[r]), ids[r], weights[r].cuda()).cpu())
    got, want = torch.stack(got), torch.stack(want)
    error = float((got - want).norm() / want.norm())

    x = tokens[0].clone()
    layer.reset()
    layer.step(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(x)
    layer.reset()
    same = True
    for asked, t, one in zip(SCRIPT, tokens, eager):
        layer.asked.copy_(torch.tensor(asked, dtype=torch.int32))
        x.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        same = same and all(torch.equal(p, q) for p, q in zip(out, one))
    return error, same, len(got)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--rows", type=int, default=64)
    a = p.parse_args()
    bad = False
    for four_bit in (False, True):
        error, same, n = run(a.rows, four_bit)
        print(f"{'NVFP4' if four_bit else 'E4M3'} cache, {n} rows in {len(SCRIPT)} steps: relative error {error:.4f}, graph {'equal' if same else 'DIFFERS'}")
        bad |= not same or not error < 0.15
    return int(bad)


if __name__ == "__main__":
    sys.exit(main())
