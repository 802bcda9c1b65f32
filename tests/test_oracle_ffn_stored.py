"""CPU pins of the oracle of the feed-forward gradients with dg and du rounded to the
storage type: against the plain gradients, and that its bounds hold for a float
evaluation and are tight enough to show a product that loses a few terms of its
sum."""
import numpy as np
import pytest

from oracle import selective as O
from state_space_sequence_exp_amd import inputs as I

HALF = 2.0 ** -8                                   # of a bfloat16 step, relative


def bf16(v):
    return I._store(np.ascontiguousarray(v, dtype=np.float32), "bf16")[0].astype(np.float64)


def draw(seed, M, K, F):
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.standard_normal(s)
    f32 = lambda a: a.astype(np.float32).astype(np.float64)
    return dict(dh=bf16(n(M, F)), x=bf16(n(M, K)), wg=bf16(n(F, K) * K ** -0.5), wu=bf16(n(F, K) * K ** -0.5),
                g=f32(n(M, F)), u=f32(n(M, F)))


def test_without_rounding_it_is_the_gradient():
    v = draw(1, 9, 7, 12)
    f = O.gated_ffn(v["x"], v["wg"], v["wu"])
    d = O.gated_ffn_backward_stored(v["dh"], v["x"], v["wg"], v["wu"], f["g"], f["u"], lambda a: a)
    w = O.gated_ffn_backward(v["dh"], v["x"], v["wg"], v["wu"], 0.0)
    for k in ("dx", "dw_gate", "dw_up"):
        assert np.allclose(d[k], w[k], rtol=1e-12, atol=1e-14)
    # rounded, the gradients are within the looser bound of the same roundings
    d = O.gated_ffn_backward_stored(v["dh"], v["x"], v["wg"], v["wu"], f["g"], f["u"], bf16)
    w = O.gated_ffn_backward(v["dh"], v["x"], v["wg"], v["wu"], HALF)
    for k in ("dx", "dw_gate", "dw_up"):
        assert (np.abs(d[k] - w[k]) <= w["e_" + k]).all()


def products(v, lost=0):
    """A float32 evaluation with dg and du in bfloat16; `lost`: the last terms that each sum
    leaves out."""
    dh, x, wg, wu, g, u = (v[k].astype(np.float32) for k in ("dh", "x", "wg", "wu", "g", "u"))
    sg = 1 / (1 + np.exp(-g))
    du, dg = bf16(dh * (g * sg)), bf16(dh * u * (sg * (1 + g * (1 - sg))))
    f = lambda a: a.astype(np.float32)
    M, F = g.shape
    both, w = f(np.concatenate([dg, du], 1)), np.concatenate([wg, wu])
    return dict(dx=bf16(both[:, :2 * F - lost] @ w[:2 * F - lost]), dw_gate=bf16(f(dg[:M - lost]).T @ x[:M - lost]),
                dw_up=bf16(f(du[:M - lost]).T @ x[:M - lost]))


def outside(v, got):
    d = O.gated_ffn_backward_stored(v["dh"], v["x"], v["wg"], v["wu"], v["g"], v["u"], bf16)
    return {k: float((np.abs(got[k] - d[k]) > d["e_" + k] + HALF * (np.abs(d[k]) + d["e_" + k])).mean()) for k in got}


@pytest.mark.parametrize("M,K,F", [(70, 30, 2040), (4090, 72, 30), (300, 40, 300)])
def test_bounds_hold_and_show_lost_terms(M, K, F):
    v = draw([2, M, K, F], M, K, F)
    assert set(outside(v, products(v)).values()) == {0.0}
    long = [k for k, n in (("dx", 2 * F), ("dw_gate", M), ("dw_up", M)) if n >= 500]
    # A sum of n terms of rms 1 is within n^0.5 of 0; half a bfloat16 step of it, n^0.5 2^-8, and
    # the float sum's (n + 65) n 0.5 2^-24 leave, at n = 4090, 0.25 + 0.5.  One term, a product
    # of three normal factors, is larger than 0.75 in about one element of six, eight together
    # in most: a tenth and a third are asked for.
    for lost, share in ((1, 0.1), (8, 0.33)):
        seen = outside(v, products(v, lost))
        assert all(seen[k] > share for k in long), seen
