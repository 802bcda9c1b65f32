"""CPU pins of the fp64 oracle of the gated recurrence, layer norm and the
8-bit state rows: closed forms, central differences, and the format's own
properties."""
import numpy as np
import pytest
import torch

from oracle import layer as O


def test_gated_scan_closed_forms():
    # a constant gate and input: h_t = x + a^(t+1) (h0 - x)
    f, x, h0 = 1.3, -0.7, 2.0
    a = 1 / (1 + np.exp(-f))
    o = O.gated_scan(np.full((1, 9, 1), x), np.full((1, 9, 1), f), None, np.full((1, 1), h0))
    want = x + a ** np.arange(1, 10) * (h0 - x)
    assert np.allclose(o["y"][0, :, 0], want, rtol=1e-14)
    # f = 0 and g: halves, times silu
    o = O.gated_scan(np.array([[[1.0], [1.0]]]), np.zeros((1, 2, 1)), np.full((1, 2, 1), 2.0))
    silu = 2 / (1 + np.exp(-2.0))
    assert np.allclose(o["y"][0, :, 0], np.array([0.5, 0.75]) * silu, rtol=1e-14)


def test_gated_scan_masks():
    """f = +inf passes the state and does not look at x, f = -inf starts
    afresh and does not look at the state."""
    x = np.array([[[1.0], [np.nan], [3.0]]])
    f = np.array([[[-np.inf], [np.inf], [0.0]]])
    o = O.gated_scan(x, f, None, np.array([[np.nan]]))
    assert np.array_equal(o["h"][0, :, 0], [1.0, 1.0, 2.0])


@pytest.mark.parametrize("gate", [False, True])
def test_gated_scan_gradients_by_differences(gate):
    rng = np.random.default_rng(3)
    v = {k: rng.standard_normal((2, 7, 3)) for k in ("x", "f") + (("g",) if gate else ())}
    v["h0"] = rng.standard_normal((2, 3))
    dy, dl = rng.standard_normal((2, 7, 3)), rng.standard_normal((2, 3))

    def loss(p):
        o = O.gated_scan(p["x"], p["f"], p.get("g"), p["h0"])
        return (o["y"] * dy).sum() + (o["h_last"] * dl).sum()

    d = O.gated_scan_backward(dy, v["x"], v["f"], v.get("g"), v["h0"], dl)
    for k in v:
        for _ in range(6):
            at = tuple(rng.integers(0, n) for n in v[k].shape)
            hi, lo = ({q: w.copy() for q, w in v.items()} for _ in range(2))
            hi[k][at] += 1e-5
            lo[k][at] -= 1e-5
            assert abs((loss(hi) - loss(lo)) / 2e-5 - d["d" + k][at]) < 1e-8


def test_layer_norm_and_gradients_by_differences():
    # a hand-worked row: [1, 3] has mean 2, variance 1
    n = O.layer_norm(np.array([[1.0, 3.0]]), np.array([2.0, 2.0]), np.array([0.5, 0.5]), 0.0)
    assert np.allclose(n["y"], [[-1.5, 2.5]], rtol=1e-15)
    rng = np.random.default_rng(4)
    s, w, b, dy = (rng.standard_normal(z) for z in ((5, 6), (6,), (6,), (5, 6)))
    d = O.layer_norm_backward(dy, s, w, 1e-3)
    loss = lambda s, w, b: (O.layer_norm(s, w, b, 1e-3)["y"] * dy).sum()
    for i in range(5):
        for j in range(6):
            e = np.zeros((5, 6)); e[i, j] = 1e-5
            assert abs((loss(s + e, w, b) - loss(s - e, w, b)) / 2e-5 - d["dx"][i, j]) < 1e-8
    for j in range(6):
        e = np.zeros(6); e[j] = 1e-5
        assert abs((loss(s, w + e, b) - loss(s, w - e, b)) / 2e-5 - d["dw"][j]) < 1e-8
        assert abs((loss(s, w, b + e) - loss(s, w, b - e)) / 2e-5 - d["db"][j]) < 1e-8


def test_e4m3_codes_against_torch():
    """Every code's value, and rounding with ties, against torch's type."""
    codes = np.array([c for c in range(256) if c % 128 != 127], np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.code_values(codes, "e4m3"), t)
    vals = O.e4m3_values()
    mid = (vals[1:] + vals[:-1]) / 2
    v = np.concatenate([vals, mid, mid * 1.0000002, mid * 0.9999998,
                        np.random.default_rng(5).uniform(-448, 448, 4000)]).astype(np.float32)
    v = np.concatenate([v, -v])
    t = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.to_e4m3(v), t)


@pytest.mark.parametrize("fmt,half", [("int8", None), ("e4m3", 2.0 ** -4)])
def test_quantised_rows(fmt, half):
    rng = np.random.default_rng(6)
    h = (rng.standard_normal((50, 32)) * np.exp(rng.uniform(-40, 40, (50, 1)))).astype(np.float32)
    h[3] = 0
    h[4] = 1e-31
    h[5, 7] = np.inf
    h[6, 1] = np.nan
    codes, scales = O.quantise(h, fmt)
    back = O.dequantise(codes, scales, fmt)
    assert not scales[3:5].any() and not back[3:5].any()
    assert np.isnan(scales[5:7]).all() and np.isnan(back[5:7]).all()
    ok = np.r_[0:3, 7:50]
    top = np.abs(h[ok]).max(-1, keepdims=True).astype(np.float64)
    err = np.abs(back[ok].astype(np.float64) - h[ok])
    step = top / 254 if fmt == "int8" else np.maximum(half * np.abs(h[ok]), top / 448 * 2.0 ** -10)
    assert (err <= step * (1 + 1e-5) + top * 4 * O.U).all()
    # rows already on the grid come back as they are
    c2, s2 = O.quantise(back[ok], fmt)
    assert np.array_equal(O.code_values(c2, fmt), O.code_values(codes[ok], fmt))
