"""More GPU tests of the short causal convolution and the selective scan."""
import pytest
import torch

from test_gpu_selective import TYPES, check_scan, oracle_scan, run_scan, scan_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,T,D,N", [(1, 3000, 16, 16), (1, 2000, 130, 64), (1, 1100, 20, 33), (2, 1300, 40, 20),
                                     (3, 1500, 40, 5)])
def test_scan_cut_in_both_types(dtype, B, T, D, N):
    """Segments of sequences with one, two and four states a lane: the oracle's values, the
    same bits from a workspace of any content."""
    import state_space_sequence_exp_amd as m3
    r, t = scan_inputs([31, B, T, D], B, T, D, N, dtype)
    need = m3.selective_scan_workspace_size(B, T, D, N, t["x"].dtype)
    assert need > 0
    y, h = run_scan(t)
    check_scan(y, h, oracle_scan(r), dtype)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")      # NaN
    y2, h2 = run_scan(t, workspace=ws)
    assert torch.equal(y, y2) and torch.equal(h, h2) and (ws[need:] == 255).all()
