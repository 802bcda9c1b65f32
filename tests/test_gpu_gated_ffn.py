"""GPU tests of the gated feed-forward projections and their gradients against
the fp64 oracle's bounds: one row to several tiles, odd widths, strided rows,
each gradient alone, streams and graphs."""
import numpy as np
import pytest
import torch

from gpu_util import from_gpu
from layer_util import HALF_STEP, close, stored
from oracle import selective as O
from test_gpu_selective import sliced

pytestmark = pytest.mark.gpu
TYPES = ["f32", "bf16"]


def inputs(seed, M, K, F, dtype):
    rng = np.random.default_rng(seed)
    v = dict(x=stored(rng, (M, K), dtype), wg=stored(rng, (F, K), dtype, 0.0, K ** -0.5),
             wu=stored(rng, (F, K), dtype, 0.0, K ** -0.5), dh=stored(rng, (M, F), dtype))
    return {k: a[0] for k, a in v.items()}, {k: a[1] for k, a in v.items()}


def check(r, t, dtype, back=True):
    import state_space_sequence_exp_amd as m3
    h, g, u = m3.gated_ffn(t["x"], t["wg"], t["wu"], want_pre=True)
    o = O.gated_ffn(r["x"], r["wg"], r["wu"])
    close(h, o["h"], o["e_h"], dtype, "h")
    close(g, o["g"], o["e_g"], "f32", "gate")
    close(u, o["u"], o["e_u"], "f32", "up")
    alone, none, _ = m3.gated_ffn(t["x"], t["wg"], t["wu"])
    assert none is None and torch.equal(alone, h)
    if not back:
        return
    d = m3.gated_ffn_backward(t["dh"], t["x"], t["wg"], t["wu"], g, u)
    w = O.gated_ffn_backward(r["dh"], r["x"], r["wg"], r["wu"], HALF_STEP[dtype] if dtype == "bf16" else 0.0)
    for k, q in (("x", "dx"), ("w_gate", "dw_gate"), ("w_up", "dw_up")):
        close(d[k], w[q], w["e_" + q], dtype, q)
    return h, g, u, d


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,F", [(1, 1, 1), (1, 64, 16), (2, 7, 33), (16, 100, 50), (17, 512, 40), (32, 31, 300),
                                   (33, 64, 64), (65, 130, 257), (128, 96, 128), (300, 520, 200), (7, 2050, 70)])
def test_ffn(dtype, M, K, F):
    r, t = inputs([M, K, F], M, K, F, dtype)
    check(r, t, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,F", [(1000, 264, 1100), (2050, 192, 1800), (2305, 129, 2817)])
def test_ffn_larger_tiles(dtype, M, K, F):
    """Sizes that take the larger tiles, with rests in every direction."""
    r, t = inputs([M, K, F], M, K, F, dtype)
    check(r, t, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,F", [(4090, 72, 4090), (4090, 71, 4090), (4090, 4090, 70), (70, 4090, 2040)])
def test_ffn_largest_tiles(dtype, M, K, F):
    """Sizes at which each of the three products fills the chip with its largest tiles,
    by rows and units picked from all over the outputs: a row of dx needs every unit,
    a unit's weights every row."""
    import state_space_sequence_exp_amd as m3
    r, t = inputs([9, M, K, F], M, K, F, dtype)
    h, g, u = m3.gated_ffn(t["x"], t["wg"], t["wu"], want_pre=True)
    d = m3.gated_ffn_backward(t["dh"], t["x"], t["wg"], t["wu"], g, u)
    rng = np.random.default_rng(2)
    pick = lambda n: np.unique(np.concatenate([rng.integers(0, n, 20), [0, n - 1]]))
    rows, units = pick(M), pick(F)
    half = HALF_STEP[dtype] if dtype == "bf16" else 0.0
    o = O.gated_ffn(r["x"][rows], r["wg"][units], r["wu"][units])
    at = np.ix_(rows, units)
    for got, k, kind in ((h, "h", dtype), (g, "g", "f32"), (u, "u", "f32")):
        close(torch.from_numpy(from_gpu(got)[at]), o[k], o["e_" + k], kind, k)
    w = O.gated_ffn_backward(r["dh"][rows], r["x"][rows], r["wg"], r["wu"], half)
    close(d["x"][rows], w["dx"], w["e_dx"], dtype, "dx")
    w = O.gated_ffn_backward(r["dh"][:, units], r["x"], r["wg"][units], r["wu"][units], half)
    for k in ("w_gate", "w_up"):
        close(d[k][units], w["d" + k], w["e_d" + k], dtype, "d" + k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [5, 90])
def test_ffn_strided(dtype, M):
    """Slices of wider rows, at odd elements, give the same bits; what lies beside
    the outputs' rows is left as it was."""
    import state_space_sequence_exp_amd as m3
    r, t = inputs([3, M], M, 72, 136, dtype)
    h, g, u, d = check(r, t, dtype)
    s = {k: sliced(v) for k, v in t.items()}
    outs = [sliced(torch.zeros_like(v)) for v in (h, g, u, d["x"], d["w_gate"], d["w_up"])]
    m3.gated_ffn(s["x"], s["wg"], s["wu"], h=outs[0], gate=outs[1], up=outs[2])
    m3.gated_ffn_backward(s["dh"], s["x"], s["wg"], s["wu"], outs[1], outs[2], dx=outs[3], dw_gate=outs[4],
                          dw_up=outs[5])
    for o, want in zip(outs, (h, g, u, d["x"], d["w_gate"], d["w_up"])):
        assert torch.equal(o, want)
        assert torch.isnan(o._base[..., :3]).all() and torch.isnan(o._base[..., -2:]).all()


def test_ffn_leading_axes_and_parts():
    import state_space_sequence_exp_amd as m3
    _, t = inputs(4, 30, 40, 48, "bf16")
    h, g, u = m3.gated_ffn(t["x"].view(2, 3, 5, 40), t["wg"], t["wu"], want_pre=True)
    assert h.shape == g.shape == (2, 3, 5, 48) and g.dtype == torch.float32
    args = (t["dh"].view(2, 3, 5, 48), t["x"].view(2, 3, 5, 40), t["wg"], t["wu"], g, u)
    d = m3.gated_ffn_backward(*args)
    only_x, only_w = m3.gated_ffn_backward(*args, want_weights=False), m3.gated_ffn_backward(*args, want_x=False)
    assert set(only_x) == {"x"} and torch.equal(only_x["x"], d["x"]) and d["x"].shape == (2, 3, 5, 40)
    assert set(only_w) == {"w_gate", "w_up"} and all(torch.equal(only_w[k], d[k]) for k in only_w)
    assert m3.gated_ffn_backward(*args, want_x=False, want_weights=False) == {}
    need = m3.gated_ffn_backward_workspace_size(30, 40, 48, torch.bfloat16)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")      # NaN
    again = m3.gated_ffn_backward(*args, workspace=ws)
    assert all(torch.equal(again[k], d[k]) for k in d) and (ws[need:] == 255).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,F", [(20, 48, 3000), (3, 131, 5000)])
def test_ffn_long_sums(dtype, M, K, F):
    """Few rows and inputs over many units: dx is summed in parts, kept in a workspace of
    any content, in a fixed order."""
    import state_space_sequence_exp_amd as m3
    r, t = inputs([10, M, K, F], M, K, F, dtype)
    h, g, u, d = check(r, t, dtype)
    kind = torch.bfloat16 if dtype == "bf16" else torch.float32
    need = m3.gated_ffn_backward_workspace_size(M, K, F, kind)
    assert need > M * 2 * -(-F // 64) * 64 * t["x"].element_size() + 512      # more than dg and du
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")      # NaN
    again = m3.gated_ffn_backward(t["dh"], t["x"], t["wg"], t["wu"], g, u, workspace=ws)
    assert all(torch.equal(again[k], d[k]) for k in d) and (ws[need:] == 255).all()
    wide = sliced(torch.zeros_like(d["x"]))
    m3.gated_ffn_backward(t["dh"], t["x"], t["wg"], t["wu"], g, u, dx=wide)
    assert torch.equal(wide, d["x"]) and torch.isnan(wide._base[..., :3]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,F", [(5001, 48, 40), (3000, 131, 70)])
def test_ffn_many_rows(dtype, M, K, F):
    """Many rows over few inputs and units: the weights' gradients are summed in parts, in a
    workspace of any content, in a fixed order, and written alone where they are asked alone."""
    import state_space_sequence_exp_amd as m3
    r, t = inputs([11, M, K, F], M, K, F, dtype)
    h, g, u, d = check(r, t, dtype)
    args = (t["dh"], t["x"], t["wg"], t["wu"], g, u)
    need = m3.gated_ffn_backward_workspace_size(M, K, F, torch.bfloat16 if dtype == "bf16" else torch.float32)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")      # NaN
    again = m3.gated_ffn_backward(*args, workspace=ws)
    assert all(torch.equal(again[k], d[k]) for k in d) and (ws[need:] == 255).all()
    only = m3.gated_ffn_backward(*args, want_x=False)
    assert all(torch.equal(only[k], d[k]) for k in ("w_gate", "w_up"))
    wide = {k: sliced(torch.zeros_like(d[k])) for k in ("w_gate", "w_up")}
    m3.gated_ffn_backward(*args, dw_gate=wide["w_gate"], dw_up=wide["w_up"])
    assert all(torch.equal(wide[k], d[k]) and torch.isnan(wide[k]._base[..., :3]).all() for k in wide)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,F", [(2050, 4096), (500, 200), (30, 200)])
def test_ffn_far_rows(dtype, M, F):
    """Rows as far apart as is taken, offsets past 32 bits: the results of dense ones."""
    import state_space_sequence_exp_amd as m3
    K, ld = 72, 2 ** 22 - 2
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    _, t = inputs([12, M, F], M, K, F, dtype)
    wide = torch.empty(M, ld, dtype=t["x"].dtype, device="cuda")
    x, dx, h, dh = wide[:, :K], wide[:, 100:100 + K], wide[:, 1000:1000 + F], wide[:, -F:]
    x.copy_(t["x"]), dh.copy_(t["dh"])
    want, g, u = m3.gated_ffn(t["x"], t["wg"], t["wu"], want_pre=True)
    got, gf, uf = m3.gated_ffn(x, t["wg"], t["wu"], want_pre=True, h=h)
    assert got is h and torch.equal(h, want) and torch.equal(gf, g) and torch.equal(uf, u)
    d = m3.gated_ffn_backward(t["dh"], t["x"], t["wg"], t["wu"], g, u)
    far = m3.gated_ffn_backward(dh, x, t["wg"], t["wu"], g, u, dx=dx)
    assert far["x"] is dx and all(torch.equal(far[k], d[k]) for k in d)
    with pytest.raises(Exception):
        m3.gated_ffn(torch.empty(2, 2 ** 22, dtype=x.dtype, device="cuda")[:, :K], t["wg"], t["wu"])


def test_ffn_no_rows():
    import state_space_sequence_exp_amd as m3
    _, t = inputs(5, 4, 24, 32, "f32")
    x, dh = t["x"][:0], t["dh"][:0]
    h, g, u = m3.gated_ffn(x, t["wg"], t["wu"], want_pre=True)
    assert h.shape == (0, 32)
    d = m3.gated_ffn_backward(dh, x, t["wg"], t["wu"], g, u)
    assert d["x"].shape == (0, 24) and not d["w_gate"].any() and not d["w_up"].any()


def test_ffn_no_rows_wide_weights():
    """More zeros to write than one launch has threads."""
    import state_space_sequence_exp_amd as m3
    F, K = 70000, 61400                                             # > 2^32 elements
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    new = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    kept = torch.empty(0, F, device="cuda")
    wg, wu = new(F, K), new(F, K)
    dg, du = torch.full_like(wg, float("nan")), torch.full_like(wu, float("nan"))
    d = m3.gated_ffn_backward(new(0, F), new(0, K), wg, wu, kept, kept, dw_gate=dg, dw_up=du)
    assert d["w_gate"] is dg
    for w in (dg, du):
        assert all(not piece.any() for piece in w.view(torch.int16).split(10000))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [3, 100])
def test_ffn_extremes(dtype, M):
    """A NaN or an infinity stays in the rows and units that it belongs to; gates far
    below zero give zeros, far above the product."""
    import state_space_sequence_exp_amd as m3
    _, t = inputs([6, M], M, 70, 90, dtype)
    h, _, _ = m3.gated_ffn(t["x"], t["wg"], t["wu"])
    t["x"][1, 69], t["wu"][80, 3] = float("nan"), float("inf")
    h2, _, _ = m3.gated_ffn(t["x"], t["wg"], t["wu"])
    assert h2[1].isnan().all() and not h2[[0, 2], 80].isfinite().any()
    keep = [i for i in range(M) if i != 1]
    cols = [i for i in range(90) if i != 80]
    assert torch.equal(h2[keep][:, cols], h[keep][:, cols])
    one = torch.ones(M, 8, dtype=t["x"].dtype, device="cuda")
    w = torch.full((4, 8), 1.0, dtype=one.dtype, device="cuda")
    w[1], w[2], w[3] = -200.0, 200.0, 0.0
    h3, g, u = m3.gated_ffn(one, w, torch.ones_like(w), want_pre=True)
    assert (h3[:, 1] == 0).all() and (h3[:, 2] == 12800).all() and (h3[:, 3] == 0).all()
    d = m3.gated_ffn_backward(torch.ones_like(h3), one, w, torch.ones_like(w), g, u)
    assert all(v.isfinite().all() for v in d.values())
    assert (d["w_gate"][1] == 0).all() and (d["w_gate"][2] == 8 * M).all() and (d["w_gate"][3] == 4 * M).all()


def test_ffn_gradients_by_differences():
    """The gradients against central differences of the forward pass itself, float32:
    steps of 1/64 make the difference's own error of third order, below 1e-3."""
    import state_space_sequence_exp_amd as m3
    _, t = inputs(7, 12, 24, 20, "f32")
    h, g, u = m3.gated_ffn(t["x"], t["wg"], t["wu"], want_pre=True)
    d = m3.gated_ffn_backward(t["dh"], t["x"], t["wg"], t["wu"], g, u)
    loss = lambda **k: float((m3.gated_ffn(*({**t, **k}[q] for q in ("x", "wg", "wu")))[0].double()
                              * t["dh"].double()).sum())
    rng = np.random.default_rng(1)
    for k, key in (("x", "x"), ("wg", "w_gate"), ("wu", "w_up")):
        for _ in range(5):
            at = tuple(int(rng.integers(0, n)) for n in t[k].shape)
            hi, lo = t[k].clone(), t[k].clone()
            hi[at] += 1 / 64
            lo[at] -= 1 / 64
            assert abs((loss(**{k: hi}) - loss(**{k: lo})) * 32 - float(d[key][at])) < 5e-3


def test_ffn_streams_and_graphs():
    import state_space_sequence_exp_amd as m3
    _, t = inputs(8, 70, 64, 96, "bf16")

    def both(t):
        h, g, u = m3.gated_ffn(t["x"], t["wg"], t["wu"], want_pre=True)
        return (h,) + tuple(m3.gated_ffn_backward(t["dh"], t["x"], t["wg"], t["wu"], g, u).values())

    want = both(t)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    h, g, u = m3.gated_ffn(t["x"], t["wg"], t["wu"], want_pre=True, stream=st)
    d = m3.gated_ffn_backward(t["dh"], t["x"], t["wg"], t["wu"], g, u, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((h,) + tuple(d.values()), want))
    graphs = []
    for _ in range(2):
        held = {k: v.clone() for k, v in t.items()}
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(held)
        graphs.append((g, held, out))
    for _ in range(3):
        ins = [{k: torch.randn_like(v) for k, v in t.items()} for _ in graphs]
        for (g, held, _), v in zip(graphs, ins):
            for k, a in v.items():
                held[k].copy_(a)
        for g, _, _ in graphs:
            g.replay()
        wants = [both(v) for v in ins]
        torch.cuda.synchronize()
        for (_, _, out), w in zip(graphs, wants):
            assert all(torch.equal(a, b) for a, b in zip(out, w))
