"""A transformer layer calibrated to NVFP4 and decoded token by token with the library's operators.

    python examples/decode_layer.py [--steps 64] [--batch 4]

Random bf16 weights are calibrated on random activations (max calibration, local Hessian, scale sweep); the
key-value cache gets its amax per head from the same activations.  Each step then runs

    norm + residual -> 8 bits | qkv product | cache write | attention over the cache | output product |
    norm + residual -> 8 bits | gate and up product | (SiLU in torch) | down product

once eagerly and once as a replayed graph, and the last hidden states are compared with the same layer in
float32 torch on the dequantized weights.  Exits with an error if they are far apart.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_scale_calibration_lh_amd as lh  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, FFN, PAGE, EPS = 512, 8, 2, 64, 1024, 16, 1e-6


def calibrated(W, X):
    """(code, fp4, amax) of W [cout, cin] against calibration rows X [rows, cin]."""
    amax = lh.lh_absmax(W)
    H, _ = lh.lh_accumulate(X)
    code, fp4, _ = lh.lh_scale_sweep(W, amax, H, want_loss=False)
    return code, fp4, amax


class Layer:
    def __init__(self, batch, max_tokens, four_bit, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
        weight = lambda o, i: (rand(o, i) * i ** -0.5).bfloat16()  # noqa: E731
        self.gamma = [(1 + 0.1 * rand(HIDDEN)).bfloat16() for _ in range(2)]
        x = rand(1024, HIDDEN).bfloat16()
        qkv = weight((HEADS + 2 * KV_HEADS) * DIM, HIDDEN)
        self.w = {"qkv": calibrated(qkv, x), "out": calibrated(weight(HIDDEN, HEADS * DIM), x),
                  "gate_up": calibrated(weight(2 * FFN, HIDDEN), x),
                  "down": calibrated(weight(HIDDEN, FFN), rand(1024, FFN).bfloat16())}
        # the cache's amax: the largest key and value of each head over normed calibration rows
        kv = (torch.nn.functional.rms_norm(x.float(), (HIDDEN,)) @ qkv.float().t()).unflatten(1, (-1, DIM))[:, HEADS:]
        amax = lh.lh_absmax(kv.transpose(0, 1).contiguous())
        pages = -(-max_tokens // PAGE)
        self.cache = lh.Cache.empty(batch * pages, PAGE, KV_HEADS, DIM, amax[:KV_HEADS].contiguous(), amax[KV_HEADS:].contiguous(),
                                    four_bit=four_bit)
        self.table = torch.randperm(batch * pages, generator=g, device="cuda").to(torch.int32).view(batch, pages)
        self.lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.rows = torch.arange(batch, device="cuda")

    def step(self, x, residual):
        """One token of every sequence: (layer output, residual stream), x and residual [batch, HIDDEN] bf16."""
        batch = x.shape[0]
        slots = self.table[self.rows, (self.lengths // PAGE).long()].long() * PAGE + self.lengths.long() % PAGE
        self.lengths += 1
        q, s, residual = lh.lh_rms_norm_quant(x, self.gamma[0], residual, eps=EPS, group=128)
        qkv = lh.lh_matvec(q, *self.w["qkv"], x_scale=s, x_group=128).view(batch, -1, DIM)
        lh.lh_cache_write(self.cache, qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:], slots)
        o = lh.lh_paged_attention(qkv[:, :HEADS], self.cache, self.table, self.lengths, scale=DIM ** -0.5)
        x = lh.lh_matvec(o.view(batch, -1), *self.w["out"])
        q, s, residual = lh.lh_rms_norm_quant(x, self.gamma[1], residual, eps=EPS, group=128)
        gate, up = lh.lh_matvec(q, *self.w["gate_up"], x_scale=s, x_group=128).chunk(2, 1)
        return lh.lh_matvec(torch.nn.functional.silu(gate) * up, *self.w["down"]), residual


class Plain:
    """The same layer in float32 torch on the dequantized weights, nothing else rounded."""

    def __init__(self, layer):
        self.gamma = [g.float() for g in layer.gamma]
        self.w = {n: lh.lh_dequantize(c, f, a, dtype=torch.float32, want_block_amax=False)[0][0] for n, (c, f, a) in layer.w.items()}
        self.k, self.v = [], []

    def step(self, x, residual):
        residual = residual + x
        h = torch.nn.functional.rms_norm(residual, (HIDDEN,), self.gamma[0], EPS)
        qkv = (h @ self.w["qkv"].t()).unflatten(1, (-1, DIM))
        self.k.append(qkv[:, HEADS:HEADS + KV_HEADS])
        self.v.append(qkv[:, HEADS + KV_HEADS:])
        k, v = (torch.stack(t, 2).repeat_interleave(HEADS // KV_HEADS, 1) for t in (self.k, self.v))
        p = torch.softmax((qkv[:, :HEADS, None] * k).sum(-1) * DIM ** -0.5, -1)
        x = (p[..., None] * v).sum(2).flatten(1) @ self.w["out"].t()
        residual = residual + x
        h = torch.nn.functional.rms_norm(residual, (HIDDEN,), self.gamma[1], EPS)
        gate, up = (h @ self.w["gate_up"].t()).chunk(2, 1)
        return (torch.nn.functional.silu(gate) * up) @ self.w["down"].t(), residual


def run(steps=64, batch=4, four_bit=True, seed=0):
    """(relative error of the last residual stream against the plain layer, whether a replayed graph gives the
    eager bits, microseconds of an eager and of a replayed step)."""
    layer = Layer(batch, steps, four_bit, seed)
    plain = Plain(layer)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    tokens = torch.randn(steps, batch, HIDDEN, generator=g, device="cuda").bfloat16()
    zero = torch.zeros(batch, HIDDEN, dtype=torch.bfloat16, device="cuda")
    eager = []
    for t in tokens:
        want = plain.step(t.float(), zero.float())
        eager.append(layer.step(t, zero))
    got, ref = (a[0].float() + a[1].float() for a in (eager[-1], want))
    error = float((got - ref).norm() / ref.norm())

    layer.lengths.zero_()                           # once more, as a graph that each step replays
    x = tokens[0].clone()
    layer.step(x, zero)
    layer.lengths.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(x, zero)
    same = True
    for t, want in zip(tokens, eager):
        x.copy_(t)
        graph.replay()
        same = same and all(torch.equal(a, b) for a, b in zip(out, want))

    def timed(f, n=20):
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            layer.lengths.fill_(steps - 1)
            f()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / n * 1e6
    return error, same, timed(lambda: layer.step(x, zero)), timed(graph.replay)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--batch", type=int, default=4)
    a = p.parse_args()
    bad = False
    for four_bit in (False, True):
        error, same, eager, replayed = run(a.steps, a.batch, four_bit)
        print(f"{'NVFP4' if four_bit else 'E4M3'} cache, {a.batch} sequences of {a.steps} tokens: relative error {error:.4f}, "
              f"graph {'equal' if same else 'DIFFERS'}, step {eager:.0f} us eager, {replayed:.0f} us replayed")
        bad |= not same or not error < 0.1
    return int(bad)


if __name__ == "__main__":
    sys.exit(main())
