"""The waves of the expert layer's products pass the weights' scale bytes between their lanes through LDS, without a barrier of the
workgroup: each lane stores 8 bytes (ds_write_b64) and reads pairs that other lanes have stored (ds_read_u16).  The hardware carries a
wave's LDS accesses out in their order; that the compiler keeps this order has to be asked for.  This test compiles moe.hip for
gfx950 to assembly with the library's own flags and checks that a wave barrier (which is no instruction, but a comment of the listing)
or a workgroup's stands between every such store and the reads after it, and between those and the next store; a listing without
them must fail the same check."""
import os
import subprocess
import tempfile

import pytest

from test_partial_sum_ordering import HIPCC, ROOT


def functions(asm):
    """name -> the kinds of the lines that matter, in order, of every product kernel of a listing."""
    out, name = {}, None
    for line in asm.splitlines():
        if line.startswith("_ZN2lh") and "k_experts" in line and "k_experts_sum" not in line and ":" in line:
            name = line.split(":")[0]
            out[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name:
            t = line.strip()
            if t == "; wave barrier" or t.startswith("s_barrier"):
                out[name].append("turn")
            elif t.startswith("ds_write_b64"):
                out[name].append("store")
            elif t.startswith(("ds_read_u16", "ds_read_i16")):
                out[name].append("read")
    return out


def faults(kinds):
    """Stores and reads with no turn between them."""
    found, since = [], set()
    for at, kind in enumerate(kinds):
        if kind == "turn":
            since = set()
            continue
        if (kind == "read" and "store" in since) or (kind == "store" and "read" in since):
            found.append((at, kind))
        since.add(kind)
    return found


@pytest.fixture(scope="module")
def listing():
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is not installed")
    from nvfp4_scale_calibration_lh_amd.build import FLAGS
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "moe.s")
        src = os.path.join(ROOT, "nvfp4_scale_calibration_lh_amd", "csrc", "moe.hip")
        p = subprocess.run([HIPCC, *(f for f in FLAGS if f != "-fPIC"), "--cuda-device-only", "-S", src, "-o", out], capture_output=True, text=True)
        assert p.returncode == 0, p.stderr[-3000:]
        return open(out).read()


def test_scale_bytes_are_read_after_they_are_stored(listing):
    kernels = functions(listing)
    assert len(kernels) >= 20
    for name, kinds in kernels.items():
        assert kinds.count("store") >= 1 and kinds.count("read") >= 1, name
        assert not faults(kinds), f"{name}: {faults(kinds)[:3]}"


def test_the_check_sees_a_missing_barrier(listing):
    kernels = functions(listing.replace("; wave barrier", ""))
    assert all(faults(kinds) for kinds in kernels.values())
