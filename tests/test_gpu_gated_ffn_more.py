"""More GPU tests of the gated feed-forward projections and their gradients."""
import pytest
import torch

from test_gpu_gated_ffn import inputs

pytestmark = pytest.mark.gpu


def test_ffn_many_leading_axes():
    """Ten dimensions, rows of slices among them: the results of two."""
    import state_space_sequence_exp_amd as m3
    M, K, F = 2 ** 6 * 3, 40, 48
    _, t = inputs(21, M, K, F, "bf16")
    lead = (2, 2, 2, 1, 2, 3, 1, 2, 2)
    h, g, u = m3.gated_ffn(t["x"], t["wg"], t["wu"], want_pre=True)
    wide = torch.empty(lead + (K + 9,), dtype=torch.bfloat16, device="cuda")
    x = wide[..., 3:3 + K]
    x.copy_(t["x"].view(lead + (K,)))
    got = m3.gated_ffn(x, t["wg"], t["wu"], want_pre=True)
    assert all(a.shape == lead + (F,) and torch.equal(a.view(M, F), b) for a, b in zip(got, (h, g, u)))
    d = m3.gated_ffn_backward(t["dh"], t["x"], t["wg"], t["wu"], g, u)
    e = m3.gated_ffn_backward(t["dh"].view(lead + (F,)), x, t["wg"], t["wu"], got[1], got[2])
    assert e["x"].shape == lead + (K,) and torch.equal(e["x"].view(M, K), d["x"])
    assert all(torch.equal(e[k], d[k]) for k in ("w_gate", "w_up"))
