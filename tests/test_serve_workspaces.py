"""The workspace queries of the operators around a decode step: host computations that need no GPU."""
import pytest
import torch

lh = pytest.importorskip("nvfp4_scale_calibration_lh_amd")


def test_expert_layer_of_an_unknown_type_needs_none():
    query = lh.lib().lh_moe_workspace
    known = [query(t, 40, 256, 128, 8, 2) for t in (lh.LH_DTYPE_F32, lh.LH_DTYPE_BF16, lh.LH_DTYPE_E4M3)]
    assert all(n > 0 for n in known) and lh.lh_last_error() == ""
    for t in (3, 9, -1, 2 ** 31 - 1):
        assert query(t, 40, 256, 128, 8, 2) == 0 and "dtype" in lh.lh_last_error()
    assert [lh.lh_moe_workspace(t, 40, 256, 128, 8, 2) for t in (torch.float32, torch.bfloat16, torch.float8_e4m3fn)] == known
    for t in (torch.float16, torch.float64, torch.int8):
        with pytest.raises(TypeError, match="dtype"):
            lh.lh_moe_workspace(t, 40, 256, 128, 8, 2)
