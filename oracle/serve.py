"""Float64 (and whole-number) definitions of the operators around a decode step: growth of the cache's
sequences, rotary positions, the choice of experts, the expert layer, and low-rank adapters."""
import numpy as np

from . import decode


def extend(table, lengths, asked, stack, count, page, max_tokens):
    """(slots, positions, sequence, offsets, new lengths, new count) of the requests, one after another; table
    [batch, max_pages] and stack are changed."""
    batch, width = table.shape
    most, capacity = width * page, len(stack)
    lens = [min(max(int(n), 0), most) for n in lengths]
    asked = [1] * batch if asked is None else [int(n) for n in asked]
    held = min(max(int(count), 0), capacity)
    out = list(lens)
    for b in range(batch):
        if asked[b] < 0:
            out[b] = max(lens[b] + asked[b], 0)
            for i in range((out[b] + page - 1) // page, (lens[b] + page - 1) // page):
                if held < capacity:
                    stack[held] = table[b, i]
                    held += 1
    slots, positions, sequence = ([-1] * max_tokens for _ in range(3))
    offsets, row, demand, top = [], 0, 0, held
    for b in range(batch):
        offsets.append(min(row, max_tokens))
        n = max(asked[b], 0)
        for r in range(row, min(row + n, max_tokens)):
            sequence[r] = b
        if n > 0 and lens[b] + n <= most and row + n <= max_tokens:
            first, last = (lens[b] + page - 1) // page, (lens[b] + n + page - 1) // page
            demand += last - first
            if first == last or demand <= held:
                for i in range(first, last):
                    top -= 1
                    table[b, i] = stack[top]
                for j in range(n):
                    at = lens[b] + j
                    positions[row + j] = at
                    slots[row + j] = int(table[b, at // page]) * page + at % page
                out[b] = lens[b] + n
        row += n
    offsets.append(min(row, max_tokens))
    return slots, positions, sequence, offsets, out, top


def rotary(x, positions, frequencies, interleaved=False, inverse=False, scale=1.0):
    """x [tokens, heads, dim] turned; rows of negative position as they are."""
    x = np.asarray(x, np.float64)
    half = len(frequencies)
    if interleaved:
        first, second = np.arange(half) * 2, np.arange(half) * 2 + 1
    else:
        first, second = np.arange(half), np.arange(half) + half
    out = x.copy()
    for t, p in enumerate(positions):
        if p < 0:
            continue
        # whole turns are taken off the exact product (31 and 24 bits) in extended precision
        w = np.longdouble(int(p)) * np.asarray(frequencies, np.float32).astype(np.longdouble)
        two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
        w = (w - two_pi * np.rint(w / two_pi)).astype(np.float64) * (-1 if inverse else 1)
        c, s = scale * np.cos(w), scale * np.sin(w)
        a, b = x[t][:, first], x[t][:, second]
        out[t][:, first], out[t][:, second] = a * c - b * s, a * s + b * c
    return out


def route(logits, topk, renormalize=True, scale=1.0):
    """(ids, weights) [tokens, topk]."""
    logits = np.asarray(logits, np.float64)
    tokens, experts = logits.shape
    ids, weights = np.full((tokens, topk), -1), np.zeros((tokens, topk))
    for t in range(tokens):
        live = [e for e in range(experts) if logits[t, e] > -np.inf]        # not NaN either
        order = sorted(live, key=lambda e: (-logits[t, e], e))
        if not order:
            continue
        m = logits[t, order[0]]
        p = {e: 1.0 if logits[t, e] == m else np.exp(logits[t, e] - m) for e in live}
        chosen = order[:topk]
        total = sum(p[e] for e in (chosen if renormalize else live))
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = [p[e] / total * scale for e in chosen]
    return ids, weights


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def moe(x, ids, weights, gate_up, down, norm=448.0):
    """(y, terms) [tokens, hidden]: the expert layer on x [tokens, hidden] (float64 values of the rows), gate_up = (code, fp4,
    amax) [E, 2 * inner, hidden], down = (code, fp4, amax) [E, hidden, inner], and the sums of the magnitudes of what y adds up."""
    tokens, hidden = x.shape
    y, terms = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    made = {}
    for t in range(tokens):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < len(gate_up[2]):
                continue
            if e not in made:
                made[e] = [decode.weights(m[0][e], m[1][e], m[2][e], norm) for m in (gate_up, down)]
            wg, wd = made[e]
            inner = wg.shape[0] // 2
            gate, up = wg[:inner] @ x[t], wg[inner:] @ x[t]
            h = silu(gate) * up
            y[t] += weights[t, j] * (wd @ h)
            # every rounding is relative to a sum of magnitudes: of gate (silu's slope is at most 1.1), up and the products of h
            ag, au = np.abs(wg[:inner]) @ np.abs(x[t]), np.abs(wg[inner:]) @ np.abs(x[t])
            spread = np.abs(h) + 1.1 * ag * np.abs(up) + np.abs(silu(gate)) * au
            terms[t] += abs(weights[t, j]) * (np.abs(wd) @ spread)
    return y, terms


def adapter(x, base, a, b, index, scaling=None, ranks=None):
    """(y, terms) [rows, cout]: base + scaling * B (A x) for each row's adapter, and the sums of magnitudes behind it."""
    y, terms = np.array(base, np.float64), np.abs(np.asarray(base, np.float64))
    for t, i in enumerate(index):
        if not 0 <= i < len(a):
            continue
        r = a.shape[1] if ranks is None else min(max(int(ranks[i]), 0), a.shape[1])
        s = 1.0 if scaling is None else float(scaling[i])
        y[t] += s * (b[i][:, :r] @ (a[i][:r] @ x[t]))
        terms[t] += abs(s) * (np.abs(b[i][:, :r]) @ (np.abs(a[i][:r]) @ np.abs(x[t])))
    return y, terms
