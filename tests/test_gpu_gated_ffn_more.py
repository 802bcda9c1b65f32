"""More GPU tests of the gated feed-forward projections and their gradients."""
import numpy as np
import pytest
import torch

from gpu_util import from_gpu, rel_l2
from layer_util import HALF_STEP, close
from oracle import selective as O
from state_space_sequence_exp_amd import inputs as I
from test_gpu_gated_ffn import TYPES, check, inputs
from test_gpu_selective import sliced

pytestmark = pytest.mark.gpu


def stored_as(v, dtype):
    """float64 values rounded to a storage type."""
    return I._store(np.ascontiguousarray(v, dtype=np.float32), dtype)[0].astype(np.float64)


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


@pytest.mark.parametrize("dtype", TYPES)
def test_ffn_many_more_rows(dtype):
    """More than 2^22 rows, forward and backward.  dh is zeros but for some rows, the last
    ones among them, so that the gradients are those of these rows alone."""
    import state_space_sequence_exp_amd as m3
    M, K, F = 2 ** 22 + 4099, 16, 12
    _, t = inputs([22], 64, K, F, dtype)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(M, K, device="cuda", generator=gen).to(t["x"].dtype)
    rows = torch.cat([torch.arange(0, 20), torch.randint(20, M - 50, (30,)), torch.arange(M - 50, M)]).unique().cuda()
    dh = torch.zeros(M, F, dtype=x.dtype, device="cuda")
    dh[rows] = torch.randn(len(rows), F, device="cuda", generator=gen).to(x.dtype)
    h, g, u = m3.gated_ffn(x, t["wg"], t["wu"], want_pre=True)
    d = m3.gated_ffn_backward(dh, x, t["wg"], t["wu"], g, u)
    r = [from_gpu(a) for a in (dh[rows], x[rows], t["wg"], t["wu"])]
    o = O.gated_ffn(*r[1:])
    for got, k, kind in ((h, "h", dtype), (g, "g", "f32"), (u, "u", "f32")):
        close(got[rows], o[k], o["e_" + k], kind, k)
    w = O.gated_ffn_backward(*r, HALF_STEP[dtype] if dtype == "bf16" else 0.0)
    close(d["x"][rows], w["dx"], w["e_dx"], dtype, "dx")
    for k in ("w_gate", "w_up"):
        close(d[k], w["d" + k], w["e_d" + k], dtype, "d" + k)
    d["x"][rows] = 0
    assert not d["x"].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [5, 90])
@pytest.mark.parametrize("odd", [("x",), ("wg",), ("wu",), ("x", "wg", "wu")])
def test_ffn_rows_at_odd_elements(dtype, M, odd):
    """Rows an even number of elements apart that start at odd ones, of one array alone or
    of all: the results of dense ones, backward in a workspace for dense ones too."""
    import state_space_sequence_exp_amd as m3
    K, F = 72, 136
    _, t = inputs([23, M], M, K, F, dtype)
    h, g, u = m3.gated_ffn(t["x"], t["wg"], t["wu"], want_pre=True)
    d = m3.gated_ffn_backward(t["dh"], t["x"], t["wg"], t["wu"], g, u)
    s = {k: sliced(v, 1, 1) if k in odd else v for k, v in t.items()}
    assert all(s[k].stride(0) == K + 2 and s[k].data_ptr() % 8 == s[k].element_size() for k in odd)
    got = m3.gated_ffn(s["x"], s["wg"], s["wu"], want_pre=True)
    assert all(torch.equal(a, b) for a, b in zip(got, (h, g, u)))
    need = m3.gated_ffn_backward_workspace_size(M, K, F, t["x"].dtype)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")      # NaN
    e = m3.gated_ffn_backward(s["dh"], s["x"], s["wg"], s["wu"], g, u, workspace=ws)
    assert all(torch.equal(e[k], d[k]) for k in d) and (ws[need:] == 255).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,F", [(157, 530, 2796), (333, 433, 2806), (687, 185, 3801), (5719, 134, 4503),
                                   (8301, 136, 2814), (1909, 67, 2233), (1268, 1452, 67), (16830, 70, 33)])
def test_ffn_other_kernels(dtype, M, K, F):
    """Sizes that take the kernels that no other size of these tests does: the smallest tile
    straight into the LDS and through registers, the second one through registers, k cut
    over the largest tile and, in float, over larger ones, and the second one whole."""
    r, t = inputs([24, M, K, F], M, K, F, dtype)
    check(r, t, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,F", [(3, 64, 40), (100, 130, 70), (300, 520, 200), (4090, 72, 4090), (4090, 71, 4090),
                                   (4090, 4090, 70), (70, 4090, 2040), (20, 48, 3000), (5001, 48, 40),
                                   (5719, 134, 4503), (8301, 136, 2814), (157, 530, 2796), (16830, 70, 33)])
def test_ffn_gradients_of_stored_slopes(dtype, M, K, F):
    """Every gradient, element by element, from a g and u that are given: with dg and du
    rounded by the oracle as by the kernels, the bound has no half step of theirs in it
    and shows a sum that loses a term.  And over each gradient: errors even within half a
    step are 3^-0.5 of it in the mean square, half a step being 2^-8 of the power of two
    below a value and less of the value (0.0017 is usual); the float sums' are far below."""
    import state_space_sequence_exp_amd as m3
    r, t = inputs([25, M, K, F], M, K, F, dtype)
    rng = np.random.default_rng([26, M, K, F])
    g, u = (rng.standard_normal((M, F)).astype(np.float32) for _ in range(2))
    d = m3.gated_ffn_backward(t["dh"], t["x"], t["wg"], t["wu"], torch.from_numpy(g).cuda(), torch.from_numpy(u).cuda())
    store = (lambda v: stored_as(v, dtype)) if dtype == "bf16" else (lambda v: v)
    w = O.gated_ffn_backward_stored(r["dh"], r["x"], r["wg"], r["wu"], g.astype(np.float64), u.astype(np.float64), store)
    for k in ("dx", "dw_gate", "dw_up"):
        got = d[k[1:]]
        close(got, w[k], w["e_" + k], dtype, k)
        if dtype == "bf16":
            assert rel_l2(from_gpu(got), w[k]) <= 2.0 ** -8 / 3 ** 0.5
