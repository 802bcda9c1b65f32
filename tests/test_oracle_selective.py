"""CPU pins of the fp64 oracle of the short convolution, the selective scan and
the gated feed-forward projections: closed forms, pieces against the whole,
PyTorch's own convolution, autograd and central differences."""
import numpy as np
import pytest
import torch

from oracle import selective as O


def test_conv_against_torch_and_pieces():
    rng = np.random.default_rng(1)
    for W in (2, 3, 4):
        x, w, b = rng.standard_normal((2, 11, 5)), rng.standard_normal((5, W)), rng.standard_normal(5)
        y, _, kept = O.causal_conv(x, w, b)
        t = torch.nn.functional.conv1d(torch.from_numpy(x).transpose(1, 2), torch.from_numpy(w)[:, None],
                                       torch.from_numpy(b), padding=W - 1, groups=5)[..., :11]
        assert np.allclose(y, t.transpose(1, 2).numpy(), atol=1e-14)
        for cut in (1, 2, 7):
            y1, _, k1 = O.causal_conv(x[:, :cut], w, b)
            y2, _, k2 = O.causal_conv(x[:, cut:], w, b, state=k1)
            assert np.array_equal(np.concatenate([y1, y2], 1), y) and np.array_equal(k2, kept)


def test_conv_lengths():
    """Behind a sequence's end nothing is looked at; a state of fewer tokens keeps old ones."""
    x = np.arange(12, dtype=np.float64).reshape(2, 6, 1)
    x[0, 1:], x[1, 0:] = np.nan, np.nan
    y, _, kept = O.causal_conv(x, np.ones((1, 3)), state=np.full((2, 2, 1), 5.0), lengths=np.array([1, -3]))
    assert np.array_equal(y[:, :, 0], [[10, 0, 0, 0, 0, 0], [0] * 6])
    assert np.array_equal(kept[:, :, 0], [[5, 0], [5, 5]])


def test_scan_closed_form():
    """A constant step and input: h_t = a^(t+1) h0 + s x B (1 - a^(t+1)) / (1 - a)."""
    s, A, x, Bn, h0 = 0.25, np.array([[-1.0, -3.0]]), 1.5, np.array([0.5, -2.0]), np.array([[[2.0, 1.0]]])
    dt = np.log(np.expm1(s))                     # softplus(dt) = s
    T = 7
    f = lambda v, n=1: np.full((1, T, n), v)
    o = O.selective_scan(f(x), f(dt - 0.5), A, np.tile(Bn, (1, T, 1)), f(1.0, 2), np.array([2.0]), None,
                         np.array([0.5]), h0=h0)
    a = np.exp(s * A)
    at = a ** np.arange(1, T + 1)[:, None]
    h = at * h0[0] + s * x * Bn * (1 - at) / (1 - a)
    assert np.allclose(o["y"][0, :, 0], h.sum(1) + 2 * x, rtol=1e-13)
    assert np.allclose(o["h_last"][0, 0], h[-1], rtol=1e-13)


def test_scan_pieces_lengths_and_gate():
    rng = np.random.default_rng(2)
    B, T, D, N = 3, 9, 4, 5
    v = [rng.standard_normal(s) for s in ((B, T, D), (B, T, D), (D, N), (B, T, N), (B, T, N), (D,), (B, T, D))]
    v[2] = -np.exp(v[2])
    whole = O.selective_scan(*v, plus=True)
    cut = lambda a, s: a[:, s] if a.ndim == 3 else a
    p1 = O.selective_scan(*(cut(a, slice(0, 4)) for a in v))
    p2 = O.selective_scan(*(cut(a, slice(4, T)) for a in v), h0=p1["h_last"])
    assert np.allclose(np.concatenate([p1["y"], p2["y"]], 1), whole["y"], rtol=1e-12)
    n = np.array([0, 4, 99])
    for a in (v[0], v[1], v[3], v[4], v[6]):
        a[0], a[1, 4:] = np.nan, np.nan
    o = O.selective_scan(*v, lengths=n)
    assert np.array_equal(o["y"][0], np.zeros((T, D))) and np.array_equal(o["h_last"][0], np.zeros((D, N)))
    assert np.allclose(o["y"][1, :4], whole["y"][1, :4]) and not o["y"][1, 4:].any()
    assert np.allclose(o["h_last"][1], p1["h_last"][1]) and np.allclose(o["y"][2], whole["y"][2])


def test_ffn_gradients():
    rng = np.random.default_rng(3)
    v = dict(x=rng.standard_normal((7, 5)), wg=rng.standard_normal((6, 5)), wu=rng.standard_normal((6, 5)))
    dh = rng.standard_normal((7, 6))
    d = O.gated_ffn_backward(dh, **v, half_step=0.0)
    t = {k: torch.from_numpy(a).requires_grad_() for k, a in v.items()}
    h = torch.nn.functional.silu(t["x"] @ t["wg"].T) * (t["x"] @ t["wu"].T)
    assert np.allclose(O.gated_ffn(**v)["h"], h.detach().numpy(), rtol=1e-13)
    for key, g in zip(("dx", "dw_gate", "dw_up"), torch.autograd.grad(h, list(t.values()), torch.from_numpy(dh))):
        assert np.allclose(d[key], g.numpy(), rtol=1e-11, atol=1e-13)
    loss = lambda p: (O.gated_ffn(**p)["h"] * dh).sum()
    for k, key in (("x", "dx"), ("wg", "dw_gate"), ("wu", "dw_up")):
        at = tuple(rng.integers(0, n) for n in v[k].shape)
        hi, lo = ({q: w.copy() for q, w in v.items()} for _ in range(2))
        hi[k][at] += 1e-5
        lo[k][at] -= 1e-5
        assert abs((loss(hi) - loss(lo)) / 2e-5 - d[key][at]) < 1e-8


@pytest.mark.parametrize("plus", [True, False])
def test_bounds_hold_for_float32(plus):
    """A float32 walk of the same formulas stays within the oracle's bounds."""
    rng = np.random.default_rng(4)
    B, T, D, N = 1, 200, 3, 4
    f32 = lambda *s: rng.standard_normal(s).astype(np.float32)
    x, dt, Bt, Ct, z = f32(B, T, D), f32(B, T, D) - 1, f32(B, T, N), f32(B, T, N), f32(B, T, D)
    dt = dt if plus else np.abs(dt)
    A, bias = -np.exp(f32(D, N)), f32(D) if plus else np.abs(f32(D))
    up = lambda a: a.astype(np.float64)
    o = O.selective_scan(up(x), up(dt), up(A), up(Bt), up(Ct), None, up(z), up(bias), plus)
    h = np.zeros((B, D, N), np.float32)
    for t in range(T):
        v = dt[:, t] + bias
        s = np.log1p(np.exp(v)) if plus else v
        h = np.exp(s[..., None] * A) * h + (s * x[:, t])[..., None] * Bt[:, t, None]
        y = (h * Ct[:, t, None]).sum(-1) * (z[:, t] / (1 + np.exp(-z[:, t])))
        assert y.dtype == np.float32
        assert (np.abs(y - o["y"][:, t]) <= o["e_y"][:, t]).all()
    assert (np.abs(h - o["h_last"]) <= o["e_h"]).all()
    assert (o["e_h"] < 1e-3 * np.abs(o["h_last"]).max()).all()     # and they are not idle
