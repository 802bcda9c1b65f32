"""CPU-only checks of the layer operators' Python entry points."""
import pytest
import torch

import state_space_sequence_exp_amd as m3


def test_scan_workspace_size_of_other_types():
    """Only the two storage types have a size; another one's would be a wrong
    one."""
    for dtype in (torch.float16, torch.float64, torch.int32, 2, -1):
        with pytest.raises(TypeError):
            m3.gated_scan_workspace_size(2, 300, 64, dtype)
    for code, dtype in ((m3.M3_F32, torch.float32), (m3.M3_BF16, torch.bfloat16)):
        assert m3.gated_scan_workspace_size(2, 300, 64, code) == m3.gated_scan_workspace_size(2, 300, 64, dtype) > 0
