"""Argument checks of the decode-step entry points: the host code built with AddressSanitizer and
UndefinedBehaviorSanitizer and driven through every check that needs no GPU, and the binding's own
checks that need none."""
import os
import subprocess
import tempfile

import pytest
import torch

import test_host_sanitize as base

lh = pytest.importorskip("nvfp4_scale_calibration_lh_amd")
KERNELS = ["rms_norm.hip", "matvec.hip", "cache.hip", "attention.hip", "absmax.hip", "accumulate.hip", "sweep.hip", "dequant.hip"]


@pytest.mark.skipif(not os.path.exists(base.HIPCC), reason="hipcc is not installed")
def test_host_code_under_address_and_undefined_behavior_sanitizers():
    with tempfile.TemporaryDirectory() as d:
        objs = []
        for src in KERNELS:
            o = os.path.join(d, src + ".o")
            base._run([base.HIPCC, *base.COMMON, "-c", os.path.join(base.CSRC, src), "-o", o])
            objs.append(o)
        for src in ("lh_abi.cpp", "lh_decode.cpp"):
            o = os.path.join(d, src + ".o")
            base._run([base.HIPCC, *base.COMMON, *base.SAN, "-x", "hip", "-c", os.path.join(base.CSRC, src), "-o", o])
            objs.append(o)
        drv = os.path.join(d, "decode_checks.o")
        base._run([base.HIPCC, *base.COMMON, *base.SAN, "-c", os.path.join(base.ROOT, "tests", "host", "decode_checks.cpp"), "-o", drv])
        exe = os.path.join(d, "decode_checks")
        base._run([base.HIPCC, "--offload-arch=gfx950", *base.SAN, drv, *objs, "-o", exe])
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
        p = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
        assert p.returncode == 0, f"{p.stdout[-3000:]}\n{p.stderr[-5000:]}"
        assert "ok: 0 failures" in p.stdout
        assert "runtime error" not in p.stderr and "AddressSanitizer" not in p.stderr


def test_binding_refuses_cpu_tensors():
    x = torch.ones(2, 64)
    for fn in (lambda: lh.lh_rms_norm_quant(x, torch.ones(64)),
               lambda: lh.lh_matvec(x, torch.ones(1, 4, 4, dtype=torch.uint8), torch.ones(1, 4, 32, dtype=torch.uint8), torch.ones(1)),
               lambda: lh.Cache.empty(2, 4, 1, 64, torch.ones(1), torch.ones(1), four_bit=True)):
        with pytest.raises(ValueError):
            fn()


def test_scale_norm_is_any_positive_e4m3_value_and_nothing_else():
    def status(norm):                            # no rows: the checks alone
        return lh.lib().lh_matvec(None, lh.LH_DTYPE_BF16, None, 0, 0, 64, None, 1, 16, None, None, None, norm, None, None)
    values = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    inf = torch.tensor(float("inf"))
    for v in values.tolist():
        assert status(v) == lh.LH_OK, v
        for other in (torch.nextafter(torch.tensor(v), inf), torch.nextafter(torch.tensor(v), -inf)):
            assert status(float(other)) == lh.LH_ERR_INVALID_ARGUMENT, float(other)
    for v in (0.0, -0.0, -448.0, 2.0 ** -10, 3 * 2.0 ** -10, 480.0, 512.0, 1e-45, 3e38, float("inf"), -float("inf"), float("nan")):
        assert status(v) == lh.LH_ERR_INVALID_ARGUMENT, v
