"""The second kernel of the adapters shares its work out over as many workgroups as it takes to be resident at once.  Its launch bounds
name that number; where registers or LDS allow fewer, the compiler says so."""
import os
import subprocess
import tempfile

import pytest

from test_partial_sum_ordering import HIPCC, ROOT


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is not installed")
def test_the_workgroups_that_are_meant_to_be_resident_are():
    from nvfp4_scale_calibration_lh_amd.build import FLAGS
    src = os.path.join(ROOT, "nvfp4_scale_calibration_lh_amd", "csrc", "adapter.hip")
    with tempfile.TemporaryDirectory() as d:
        p = subprocess.run([HIPCC, *(f for f in FLAGS if f != "-fPIC"), "--cuda-device-only", "-S", src, "-o", os.path.join(d, "adapter.s"),
                            "-Wpass-failed", "-Rpass-analysis=kernel-resource-usage"], capture_output=True, text=True)
    assert p.returncode == 0, p.stderr[-3000:]
    assert p.stderr.count("k_adapter_out") >= 16 and "Occupancy" in p.stderr          # the compiler's remarks are there
    missed = [line for line in p.stderr.splitlines() if "failed to meet occupancy" in line]
    assert not missed, missed
