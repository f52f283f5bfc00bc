"""Argument checks of the operators around a decode step: the host code built with AddressSanitizer and
UndefinedBehaviorSanitizer and driven through every check that needs no GPU, and the binding's own checks."""
import concurrent.futures as cf
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

import test_host_sanitize as base
from oracle import serve

lh = pytest.importorskip("nvfp4_scale_calibration_lh_amd")
KERNELS = ["extend.hip", "rotary.hip", "route.hip", "moe.hip", "adapter.hip"]


@pytest.mark.skipif(not os.path.exists(base.HIPCC), reason="hipcc is not installed")
def test_host_code_under_address_and_undefined_behavior_sanitizers():
    with tempfile.TemporaryDirectory() as d:
        def made(src, flags, folder=base.CSRC):
            o = os.path.join(d, src + ".o")
            base._run([base.HIPCC, *base.COMMON, *flags, "-c", os.path.join(folder, src), "-o", o])
            return o
        with cf.ThreadPoolExecutor(4) as pool:
            jobs = [pool.submit(made, src, []) for src in KERNELS]
            jobs.append(pool.submit(made, "lh_serve.cpp", [*base.SAN, "-x", "hip"]))
            jobs.append(pool.submit(made, "serve_checks.cpp", [*base.SAN, "-x", "hip"], os.path.join(base.ROOT, "tests", "host")))
            objs = [j.result() for j in jobs]
        exe = os.path.join(d, "serve_checks")
        base._run([base.HIPCC, "--offload-arch=gfx950", *base.SAN, *objs, "-o", exe])
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
        p = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
        assert p.returncode == 0, f"{p.stdout[-3000:]}\n{p.stderr[-5000:]}"
        assert "ok: 0 failures" in p.stdout
        assert "runtime error" not in p.stderr and "AddressSanitizer" not in p.stderr


def test_binding_refuses_cpu_tensors_and_shapes():
    z = torch.zeros
    i32 = torch.int32
    with pytest.raises(ValueError, match="GPU"):
        lh.lh_cache_extend(z(2, 3, dtype=i32), z(2, dtype=i32), None, z(4, dtype=i32), z(1, dtype=i32), page_size=16, max_tokens=2)
    with pytest.raises(ValueError, match="block_table"):
        lh.lh_cache_extend(z(2, dtype=i32), z(2, dtype=i32), None, z(4, dtype=i32), z(1, dtype=i32), page_size=16, max_tokens=2)
    with pytest.raises(ValueError, match="GPU"):
        lh.lh_rotary(z(2, 3, 16), None, z(2, dtype=i32), z(8))
    with pytest.raises(ValueError, match="Q must"):
        lh.lh_rotary(z(2, 48), None, z(2, dtype=i32), z(8))
    with pytest.raises(ValueError, match="scaling"):
        lh.lh_rotary_frequencies(16, scaling="other", device="cpu")
    with pytest.raises(lh.LHError, match="rot_dim"):
        lh.lh_rotary_frequencies(15, device="cpu")
    with pytest.raises(lh.LHError, match="rot_dim"):
        lh.lh_rotary_frequencies(-2, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        lh.lh_route(z(2, 8), 2)
    with pytest.raises(ValueError, match="logits"):
        lh.lh_route(z(8), 2)
    u8 = torch.uint8
    layer = [(z(2, 32, 1, dtype=u8), z(2, 32, 8, dtype=u8), z(2)), (z(2, 16, 1, dtype=u8), z(2, 16, 8, dtype=u8), z(2))]
    with pytest.raises(ValueError, match="GPU"):
        lh.lh_moe(z(3, 16), z(3, 2, dtype=i32), z(3, 2), *layer)
    with pytest.raises(ValueError, match="GPU"):
        lh.lh_adapter(z(3, 16), z(3, 8), z(2, 8, 16), z(2, 8, 8), z(3, dtype=i32))


def test_frequencies():
    """Against their definitions in 64 bits, rounded once."""
    j = np.arange(0, 64, 2) / 64
    f = 10000.0 ** -j
    for kind, factor, want, scale in (("plain", 1.0, f, 1.0), ("linear", 4.0, f / 4.0, 1.0), ("base", 4.0, (10000.0 * 4.0 ** (64 / 62)) ** -j, 1.0)):
        got, s = lh.lh_rotary_frequencies(64, scaling=kind, factor=factor, device="cpu")
        assert np.all(np.abs(got.double().numpy() - want) <= want * (2.0 ** -24 + 2.0 ** -48)) and s == scale
    got, s = lh.lh_rotary_frequencies(64, scaling="parts", factor=16.0, original_context=2048, low_turns=2.0, high_turns=20.0, device="cpu")
    turns = 2048 * f / (2 * np.pi)
    keep = np.clip((turns - 2) / 18, 0, 1)
    want = f * (keep + (1 - keep) / 16)
    assert np.all(np.abs(got.double().numpy() - want) <= want * (2.0 ** -24 + 2.0 ** -45)) and abs(s - (0.1 * np.log(16) + 1)) < 1e-7
    assert got[0] == 1.0 and keep[-1] == 0 and 0 < keep[12] < 1


def test_oracle_by_hand():
    """The definitions at sizes that can be followed by hand."""
    table, stack = np.array([[5, -1, -1], [6, 7, -1]]), np.array([3, 4, -1, -1])
    got = serve.extend(table, [3, 8], [2, -5], stack, 2, 4, 3)
    # the second gives page 7 back (3 of 8 tokens stay), which the first then takes for its fifth token
    assert got == ([23, 28, -1], [3, 4, -1], [0, 0, -1], [0, 2, 2], [5, 3], 2)
    assert table.tolist() == [[5, 7, -1], [6, 7, -1]] and stack.tolist() == [3, 4, 7, -1]
    x = np.array([[[1.0, 0.0, 0.0, 2.0, 9.0]]])
    y = serve.rotary(x, [1], np.array([np.pi / 2, 0.0], np.float32))
    np.testing.assert_allclose(y[0, 0], [0, 0, 1, 2, 9], atol=1e-7)
    y = serve.rotary(x, [1], np.array([np.pi / 2, 0.0], np.float32), interleaved=True, inverse=True, scale=2.0)
    np.testing.assert_allclose(y[0, 0], [0, -2, 0, 4, 9], atol=1e-6)
    ids, w = serve.route([[0.0, np.log(3.0), -np.inf, 0.0]], 2, renormalize=False)
    assert ids.tolist() == [[1, 0]]
    np.testing.assert_allclose(w, [[0.6, 0.2]])
    ids, w = serve.route([[np.nan, 1.0]], 2, scale=3.0)
    assert ids.tolist() == [[1, -1]] and w.tolist() == [[3.0, 0.0]]
    y, _ = serve.adapter(np.array([[2.0, 1.0]]), [[10.0]], np.array([[[1.0, 1.0], [0.0, 5.0]]]), np.array([[[4.0, 7.0]]]), [0], [0.5], [1])
    assert y.tolist() == [[16.0]]
    one = (np.full((1, 32, 1), 0x38, np.uint8), np.full((1, 32, 8), 0x22, np.uint8), np.array([2688.0], np.float32))     # weights of 1
    y, _ = serve.moe(np.ones((1, 16)), [[0, 3]], np.array([[2.0, 9.0]]), one, tuple(t[:, :16] if t.ndim == 3 else t for t in one))
    np.testing.assert_allclose(y, 2.0 * 16 * 16 * 16 / (1 + np.exp(-16.0)))
