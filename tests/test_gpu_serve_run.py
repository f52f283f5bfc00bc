"""The operators around a decode step run together, in graphs, on other streams, and where offsets pass 32 bits."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import serve
from test_gpu_serve import DEV, TYPES, U, adapter_case, check_rotary, choices, dev, layer_rows, matrices, note, on_gpu, requests

pytestmark = pytest.mark.gpu

lh = pytest.importorskip("nvfp4_scale_calibration_lh_amd")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("four_bit,bound", [(False, 0.06), (True, 0.1)])
def test_serve_layer(four_bit, bound):
    """Roundings to 8 bits are off by 2.6% of their vector, an NVFP4 cache by about 10% of each value, averaged over the tokens of the
    softmax; both branches (attention of norm about 0.5 of the input's, the experts' about 0.3) pass one such error each, the
    expert layer a second one of its input, on to a sum with the exact input.  The choice of experts is taken over."""
    spec = importlib.util.spec_from_file_location("serve_layer", os.path.join(ROOT, "examples", "serve_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    note(f"serving example, four_bit {four_bit}")
    error, same, rows = m.run(rows=64, four_bit=four_bit)
    assert rows == sum(max(n, 0) for step in m.SCRIPT for n in step)
    assert same, "a replayed graph differs from the eager steps"
    assert error < bound, error


class Calls:
    """One call of each operator at sizes that take their workspaces and both of their kernels, into outputs of its own."""

    def __init__(self):
        table, lengths, asked, stack, count = requests(1100, 4, 8, 1)
        self.extend = [dev(a) for a in (table, lengths, asked, stack, count)]
        self.q, _ = layer_rows(40, 512, "bf16", 0, 2)[:2]
        self.positions = dev(np.arange(40) * 100)
        self.frequencies, _ = lh.lh_rotary_frequencies(64, device=DEV)
        self.logits = torch.randn(40, 24, generator=torch.Generator().manual_seed(3)).to(DEV)
        self.gate_up, self.down = on_gpu(matrices(24, 256, 512, 4)), on_gpu(matrices(24, 512, 128, 5))
        xd, scale, _, base, a, b, index, ranks, scaling = adapter_case(40, 512, 300, 6, 24, "bf16", 0, "bf16", 6)
        self.adapter = (base, torch.nan_to_num(a), torch.nan_to_num(b), dev(index))
        self.ranks, self.scaling = dev(ranks), torch.from_numpy(scaling).to(DEV)

    def __call__(self):
        t, n, a, s, c = self.extend
        out = list(lh.lh_cache_extend(t, n, a, s, c, page_size=8, max_tokens=5000))
        out += lh.lh_rotary(self.q.view(40, 8, 64), None, self.positions, self.frequencies)[:1]
        ids, w = lh.lh_route(self.logits, 6)
        out += [ids, w, lh.lh_moe(self.q, ids, w, self.gate_up, self.down), lh.lh_moe(self.q[:3], ids[:3], w[:3], self.gate_up, self.down)]
        out.append(lh.lh_adapter(self.q, *self.adapter, scaling=self.scaling, ranks=self.ranks))
        return out


def equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_same_bits_twice_and_on_another_stream():
    note("all calls twice and on a side stream")
    calls = Calls()
    first = calls()
    assert equal(first, calls())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = calls()
    here = calls()                            # at once, each with a workspace of its own
    torch.cuda.synchronize()
    assert equal(first, other) and equal(first, here)


def test_graphs():
    """Two captured graphs, replayed in turn with eager work and changed inputs between, one of them in the other's memory pool."""
    note("all calls in graphs")
    calls, more = Calls(), Calls()
    calls()
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        out = calls()
    with torch.cuda.graph(second, pool=first.pool()):
        out2 = more()
    for seed in range(4):
        calls.logits.copy_(torch.randn(40, 24, generator=torch.Generator().manual_seed(seed)))
        calls.q.mul_(-0.75)
        first.replay()
        want = calls()
        torch.cuda.synchronize()
        assert equal(out, want), seed
        second.replay()
        want = more()
        torch.cuda.synchronize()
        assert equal(out2, want), seed


def test_callers_outputs_and_workspaces():
    """Outputs and workspaces that the caller holds, the workspaces full of other numbers before."""
    note("outputs and workspaces given")
    calls = Calls()
    want = calls()
    t, n, a, s, c = calls.extend
    work = torch.full((lh.lh_cache_extend_workspace(1100, 5000),), 255, dtype=torch.uint8, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    given = dict(slots=torch.empty(5000, dtype=torch.int64, device=DEV), positions=torch.empty(5000, **i32), sequence=torch.empty(5000, **i32),
                 offsets=torch.empty(1101, **i32), new_lengths=torch.empty(1100, **i32), new_count=torch.empty(1, **i32))
    got = lh.lh_cache_extend(t, n, a, s, c, page_size=8, max_tokens=5000, workspace=work, **given)
    assert equal(got, want[:6]) and all(g is h for g, h in zip(got, given.values()))
    ids, w = torch.empty(40, 6, **i32), torch.empty(40, 6, device=DEV)
    assert lh.lh_route(calls.logits, 6, ids=ids, weights=w)[0] is ids and equal((ids, w), want[7:9])
    work = torch.full((lh.lh_moe_workspace(torch.bfloat16, 40, 512, 128, 24, 6),), 255, dtype=torch.uint8, device=DEV)
    y = torch.empty(40, 512, dtype=torch.bfloat16, device=DEV)
    assert lh.lh_moe(calls.q, ids, w, calls.gate_up, calls.down, y, workspace=work) is y and torch.equal(y, want[9])
    work = torch.full((lh.lh_adapter_workspace(40, 512, 6, 24),), 255, dtype=torch.uint8, device=DEV)
    y = torch.empty(40, 300, dtype=torch.bfloat16, device=DEV)
    assert lh.lh_adapter(calls.q, *calls.adapter, y, scaling=calls.scaling, ranks=calls.ranks, workspace=work) is y and torch.equal(y, want[11])
    with pytest.raises(lh.LHError, match="workspace"):
        lh.lh_adapter(calls.q, *calls.adapter, workspace=work[:16])
    with pytest.raises(lh.LHError, match="workspace"):
        lh.lh_moe(calls.q, ids, w, calls.gate_up, calls.down, workspace=work[:16])


def test_refusals_on_the_device():
    note("refusals on the device")
    q = torch.zeros(4, 2, 64, device=DEV)
    f = torch.ones(32, device=DEV)
    p = dev([0, 1, 2, 3])
    with pytest.raises(ValueError, match="positions"):
        lh.lh_rotary(q, None, p.long(), f)
    with pytest.raises(ValueError, match="out_k"):
        lh.lh_rotary(q, None, p, f, out_k=q)
    with pytest.raises(lh.LHError, match="rot_dim"):
        lh.lh_rotary(q, None, p, torch.ones(40, device=DEV))
    with pytest.raises(TypeError):
        lh.lh_rotary(q.half(), None, p, f)
    with pytest.raises(lh.LHError, match="topk"):
        lh.lh_route(torch.zeros(2, 8, device=DEV), 9)
    with pytest.raises(lh.LHError, match="n_experts"):
        lh.lh_route(torch.zeros(2, 5000, device=DEV), 2)
    x, ids, w = torch.zeros(3, 64, device=DEV), dev(np.zeros((3, 2))), torch.zeros(3, 2, device=DEV)
    gate_up, down = on_gpu(matrices(4, 64, 64, 1)), on_gpu(matrices(4, 64, 32, 1))
    with pytest.raises(ValueError, match="gate_up"):
        lh.lh_moe(x, ids, w, on_gpu(matrices(4, 32, 64, 1)), down)
    with pytest.raises(ValueError, match="weights"):
        lh.lh_moe(x, ids, w[:, :1].contiguous(), gate_up, down)
    with pytest.raises(ValueError, match="x_scale"):
        lh.lh_moe(x, ids, w, gate_up, down, x_scale=torch.ones(3, 1, device=DEV))
    with pytest.raises(lh.LHError, match="scale_norm"):
        lh.lh_moe(x, ids, w, gate_up, down, norm=300.0)
    a, b = torch.zeros(2, 8, 64, device=DEV), torch.zeros(2, 40, 8, device=DEV)
    with pytest.raises(ValueError, match="base"):
        lh.lh_adapter(x, torch.zeros(3, 40, dtype=torch.bfloat16, device=DEV), a, b, dev([0, 0, 0]))
    with pytest.raises(ValueError, match="B has dtype"):
        lh.lh_adapter(x, torch.zeros(3, 40, device=DEV), a, b.bfloat16(), dev([0, 0, 0]))
    with pytest.raises(lh.LHError, match="rank"):
        lh.lh_adapter(x, torch.zeros(3, 40, device=DEV), torch.zeros(2, 4, 64, device=DEV), torch.zeros(2, 40, 4, device=DEV), dev([0, 0, 0]))
    with pytest.raises(ValueError, match="free_count"):
        lh.lh_cache_extend(dev(np.zeros((2, 3))), dev([0, 0]), None, dev([1, 2]), dev([1, 2]), page_size=16, max_tokens=2)


# --------------------------------------------------------------------------------------- offsets past 32 bits
def test_rotary_past_32_bits():
    tokens, heads, dim = 70001, 512, 128
    note(f"rotary of {tokens * heads * dim} elements")
    x = torch.zeros(tokens, heads, dim, dtype=torch.bfloat16, device=DEV)
    at = [0, 32767, 32768, 65536, 70000]
    x[at] = torch.randn(len(at), heads, dim, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    before = x[at].double().cpu().numpy()
    f, _ = lh.lh_rotary_frequencies(128, device=DEV)
    lh.lh_rotary(x, None, torch.arange(tokens, dtype=torch.int32, device=DEV), f, out_q=x)
    check_rotary(x[at], before, np.array(at), f.cpu().numpy(), "bf16", 64, False)


def test_moe_past_32_bits():
    """Matrices of 4.3e9 bytes together, of which the last experts are chosen."""
    experts, hidden, inner = 3300, 2048, 640
    note(f"moe with {experts * 2 * inner * hidden // 2} bytes of gate and up nibbles")
    small = matrices(4, 2 * inner, hidden, 1), matrices(4, hidden, inner, 2)
    big = []
    for (code, fp4, amax), cout, cin in ((small[0], 2 * inner, hidden), (small[1], hidden, inner)):
        c = torch.full((experts, cout, cin // 16), 0x38, dtype=torch.uint8, device=DEV)
        n = torch.zeros(experts, cout, cin // 2, dtype=torch.uint8, device=DEV)
        m = torch.ones(experts, device=DEV)
        c[-4:], n[-4:], m[-4:] = on_gpu((code, fp4, amax))
        big.append((c, n, m))
    assert big[0][1].numel() > 2 ** 32
    xd, _, _ = layer_rows(5, hidden, "bf16", 0, 3)
    ids, w = choices(5, 4, 2, 4)
    want = lh.lh_moe(xd, dev(ids), torch.from_numpy(w).to(DEV), *(on_gpu(m) for m in small))
    y = lh.lh_moe(xd, dev(ids + experts - 4), torch.from_numpy(w).to(DEV), *big)
    # (which waves share k depends on the number of experts, and with it the order of the sums)
    assert float((y.float() - want.float()).abs().max()) <= 2.0 ** -7 * float(want.float().abs().max())


def test_adapter_past_32_bits():
    n, rank, cin, cout = 520, 64, 65536, 96
    note(f"adapters of {n * rank * cin * 2} bytes")
    g = torch.Generator().manual_seed(1)
    a = torch.zeros(n, rank, cin, dtype=torch.bfloat16, device=DEV)
    last = torch.randn(rank, cin, generator=g).bfloat16() * 2.0 ** -8
    a[-1] = last.to(DEV)
    b = torch.randn(n, cout, rank, generator=g).bfloat16().to(DEV)
    x = torch.randn(2, cin, generator=g).bfloat16()
    base = torch.zeros(2, cout, dtype=torch.bfloat16, device=DEV)
    y = lh.lh_adapter(x.to(DEV), base, a, b, dev([n - 1, 0]))
    want, terms = serve.adapter(x.double().numpy(), np.zeros((2, cout)), last[None].double().numpy(), b[-1:].double().cpu().numpy(), [0, -1])
    err = np.abs(y.double().cpu().numpy() - want)
    assert np.all(err <= ((3 * cin + 3 * rank + 24) * U + 2.0 ** -17) * terms + 2.0 ** -8 * np.abs(want)) and torch.count_nonzero(y[1]) == 0
