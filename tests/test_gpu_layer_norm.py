"""GPU parity of layer norm and its gradients against the fp64 oracle, element
by element within the oracle's error bounds plus one storage rounding."""
import numpy as np
import pytest

from layer_util import close, put, stored, torch_type
from gpu_util import from_gpu, log

pytestmark = pytest.mark.gpu


def run_case(M, D, dtype, residual, bias, seed, x=None, eps=1e-5):
    import state_space_sequence_exp_amd as m3
    from oracle import layer as O
    rng = np.random.default_rng(seed)
    vx, tx = stored(rng, (M, D), dtype, 0.3, 1.0) if x is None else put(x, dtype)
    vr, tr = stored(rng, (M, D), dtype, -0.2, 2.0) if residual else (0.0, None)
    vw, tw = put(rng.standard_normal(D) * 0.3 + 1, "f32")
    vb, tb = put(rng.standard_normal(D), "f32") if bias else (np.zeros(D), None)
    vdy, tdy = stored(rng, (M, D), dtype)
    vds, tds = stored(rng, (M, D), dtype) if residual else (None, None)
    y, s, mean, rstd = m3.layer_norm(tx, tw, tb, eps, residual=tr)
    # the sum as it is stored: float addition, one rounding
    sv, st = put((vx.astype(np.float32) + np.float32(vr)).astype(np.float32) if residual else vx, dtype)
    import torch
    assert torch.equal(s, st)
    n = O.layer_norm(sv, vw, vb, eps)
    close(y, n["y"], n["e_y"], dtype, "y")
    close(mean, n["mean"], n["e_mean"], "f32", "mean")
    close(rstd, n["rstd"], n["e_rstd"], "f32", "rstd")
    d = m3.layer_norm_backward(tdy, s, tw, mean, rstd, dsum=tds, want_bias=bias)
    w = O.layer_norm_backward(vdy, sv, vw, eps, vds)
    close(d["x"], w["dx"], w["e_dx"], dtype, "dx")
    close(d["weight"], w["dw"], w["e_dw"], "f32", "dw")
    assert ("bias" in d) == bias
    if bias:
        close(d["bias"], w["db"], w["e_db"], "f32", "db")
    return dict(x=tx, r=tr, w=tw, b=tb, dy=tdy, ds=tds, y=y, s=s, mean=mean, rstd=rstd, d=d)


SHAPES = [(1, 1), (1, 2), (3, 5), (2, 64), (7, 65), (5, 127), (1, 512), (70, 520), (300, 72), (9, 1001),
          (4, 2048), (1030, 264), (33, 4097), (6, 8192), (3, 16384), (2, 16383), (4101, 520), (5003, 1000), (1030, 4100), (7, 6001),
          # rows whose last vector is cut after 1 to 7 elements
          (5, 9), (41, 130), (40, 131), (300, 1100), (50, 2045), (260, 1030), (600, 2047)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d" % s)
def test_forward_and_gradients(shape, residual, dtype):
    M, D = shape
    log("layer norm %s residual=%s %s" % (shape, residual, dtype))
    run_case(M, D, dtype, residual, bias=(M % 2 == 1) or residual, seed=M * 7 + D)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offset_constant_and_huge_rows(dtype):
    """Rows far from zero (a difference of sums would lose the variance),
    constant rows, and rows near the square root of the largest float."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((12, 384))
    x[0:3] = x[0:3] * 0.25 + 300
    x[3] = 7.0
    x[4] = 0.0
    x[5:7] *= 1e15
    x[7:9] *= 1e-15
    run_case(12, 384, dtype, False, True, 6, x=x)


def test_nan_rows_stay_apart():
    """A row with a NaN or an infinity is NaN itself and no other row is."""
    import torch
    import state_space_sequence_exp_amd as m3
    x = torch.randn(9, 1000, device="cuda")
    w = torch.ones(1000, device="cuda")
    ref = m3.layer_norm(x, w)[0]
    bad = x.clone()
    bad[2, 999] = float("nan")
    bad[5, 0] = float("inf")
    y = m3.layer_norm(bad, w)[0]
    keep = [i for i in range(9) if i not in (2, 5)]
    assert y[2].isnan().all() and y[5].isnan().any() and torch.equal(y[keep], ref[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [256, 250])
def test_strided_and_in_place(D, dtype):
    """Strided rows give the dense call's results bit for bit; y, the sum and
    dx in the place of their inputs as well; nothing between the rows changes."""
    import torch
    import state_space_sequence_exp_amd as m3
    M = 40
    c = run_case(M, D, dtype, True, True, 8)
    wide = torch.full((M, 5 * D + 6), 3.0, device="cuda").to(torch_type(dtype))
    sl = [wide[:, i * (D + 1):i * (D + 1) + D] for i in range(5)]
    for s, k in zip(sl, ("x", "r", "dy", "ds")):
        s.copy_(c[k])
    keep = wide.clone()
    y, s, mean, rstd = m3.layer_norm(sl[0], c["w"], c["b"], 1e-5, residual=sl[1], y=sl[0], sum_out=sl[1])
    assert torch.equal(y, c["y"]) and torch.equal(s, c["s"]) and y.data_ptr() == sl[0].data_ptr()
    assert torch.equal(mean, c["mean"]) and torch.equal(rstd, c["rstd"])
    d = m3.layer_norm_backward(sl[2], sl[1], c["w"], mean, rstd, dsum=sl[3], dx=sl[2])
    assert torch.equal(d["x"], c["d"]["x"]) and torch.equal(d["weight"], c["d"]["weight"])
    d = m3.layer_norm_backward(c["dy"], sl[1], c["w"], mean, rstd, dsum=sl[3], dx=sl[3])
    assert torch.equal(sl[3], c["d"]["x"]) and torch.equal(d["bias"], c["d"]["bias"])
    for i in range(4):
        keep[:, i * (D + 1):i * (D + 1) + D] = sl[i]
    assert torch.equal(wide, keep)
    # the sum in the place of x, three dimensions, no statistics
    x3, r3 = c["x"].view(5, 8, D).clone(), c["r"].view(5, 8, D)
    y, s, mean, rstd = m3.layer_norm(x3, c["w"], c["b"], 1e-5, residual=r3, sum_out=x3, want_stats=False)
    assert mean is None and rstd is None and s is x3
    assert torch.equal(y.view(M, D), c["y"]) and torch.equal(s.view(M, D), c["s"])


def test_empty_rows():
    import torch
    import state_space_sequence_exp_amd as m3
    w = torch.ones(8, device="cuda")
    x = torch.empty(0, 8, device="cuda")
    y, s, mean, rstd = m3.layer_norm(x, w)
    assert y.shape == (0, 8) and mean.shape == (0,)
    d = m3.layer_norm_backward(x, s, w, mean, rstd)
    assert not d["weight"].any() and not d["bias"].any() and d["x"].shape == (0, 8)


def test_repeats_other_stream_and_graph():
    """Bit-for-bit repeats, on another stream, and in a graph replayed with new
    inputs between eager calls."""
    import torch
    import state_space_sequence_exp_amd as m3
    M, D = 700, 520
    w, b = torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    x, r, dy = (torch.randn(M, D, device="cuda").to(torch.bfloat16) for _ in range(3))

    def work(stream=None):
        y, s, mean, rstd = m3.layer_norm(x, w, b, residual=r, stream=stream)
        d = m3.layer_norm_backward(dy, s, w, mean, rstd, dsum=r, stream=stream)
        return [y, s, mean, rstd, d["x"], d["weight"], d["bias"]]

    first = work()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = work(side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, other))
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for k in range(4):
        for v in (x, r, dy):
            v.copy_(torch.randn(M, D, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        assert all(torch.equal(p, q) for p, q in zip(got, work()))
