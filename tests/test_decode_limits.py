"""Limits of the decode-step entry points and host arithmetic at them, without a GPU."""
import ctypes
import os
import subprocess
import tempfile

import pytest

import test_host_sanitize as base

lh = pytest.importorskip("nvfp4_scale_calibration_lh_amd")

BYTES = (ctypes.c_uint8 * 4096)()                     # host memory: never a valid device pointer
HOST = (ctypes.addressof(BYTES) + 255) // 256 * 256


def cache(page_size, heads=2, dim=64):
    return lh.CacheStruct(lh.LH_CACHE_FP4, 4, page_size, heads, dim, HOST, HOST, HOST, HOST, HOST, HOST)


@pytest.mark.parametrize("page", [1, 16, 24, 4096, 1 << 20])
def test_attention_leaves_room_past_the_last_position(page):
    """Positions are 32-bit and a wave looks a step past a sequence's end, so a table may hold 2^31 - 4096 tokens, no more."""
    most = (2 ** 31 - 4096) // page
    for pages, fits in ((most, True), (most + 1, False), ((2 ** 31 - 1) // page + 1, False), (2 ** 62, False)):
        c = cache(page)
        nbytes = lh.lib().lh_paged_attention_workspace(ctypes.byref(c), 2, 8, pages)
        assert (nbytes > 0) == fits, (page, pages)
        status = lh.lib().lh_paged_attention(ctypes.byref(c), HOST, 512, lh.LH_DTYPE_BF16, 2, 8, HOST, pages, HOST, 1.0, HOST, HOST, 1 << 40, None)
        message = lh.lib().lh_last_error().decode()
        assert status == lh.LH_ERR_INVALID_ARGUMENT
        assert ("device" if fits else "max_pages") in message, message


@pytest.mark.skipif(not os.path.exists(base.HIPCC), reason="hipcc is not installed")
def test_parts_of_a_sequence_cover_it_and_pages_are_in_the_cache():
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "cut")
        base._run([base.HIPCC, *base.COMMON, *base.SAN, "-x", "hip", os.path.join(base.ROOT, "tests", "host", "attention_cut_checks.cpp"), "-o", exe])
        p = subprocess.run([exe], capture_output=True, text=True, timeout=60, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
        assert p.returncode == 0 and "ok: 0 failures" in p.stdout, p.stdout + p.stderr
