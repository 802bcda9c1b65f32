"""The cached decode step against its definition: the float operations that the
header lists, evaluated one by one in NumPy, give the codes and scales of every
form of the kernel to the last bit (a zero's sign aside).  What a float function
returns is not defined to the last bit, so the exponential, the sine and the
cosine are first read out of the kernel itself, as the y of states of ones."""
import numpy as np
import pytest

from layer_util import put, stored
from test_gpu_state_cache import cache_with, raw, rows

pytestmark = pytest.mark.gpu
F = np.float32


def factors(t):
    """alpha [S,H], cos and sin [S,H,N/2] as the kernel computes them from dt, A
    and theta (device tensors, float32): a step without inputs on states that
    are 1 in one column of every row pair's first row, read by a C that picks
    the first rows or the second ones."""
    import torch
    import state_space_sequence_exp_amd as m3
    S, H, K = t["theta"].shape
    N, P = 2 * K, 128
    codes = torch.zeros(S, H, N, P, dtype=torch.int8, device="cuda")
    at = torch.arange(K, device="cuda")
    codes[:, :, 2 * at, at] = 64
    scales = torch.full((S, H, N), 2.0 ** -6, device="cuda")
    none = torch.zeros(S, H, 1, P, device="cuda")
    zero = torch.zeros(S, H, 1, N, device="cuda")
    pick = torch.zeros(2, S, H, 1, N, device="cuda")
    pick[0, ..., 0::2] = 1
    pick[1, ..., 1::2] = 1

    def y(C, A, theta):
        out = m3.decode_step_cached(codes.clone(), scales.clone(), None, none, None, zero, None, C, t["dt"], A,
                                    None, theta)
        return out[:, :, 0, :K].cpu().numpy()

    still = torch.zeros_like(t["A"])
    assert (y(pick[0], still, None) == 1).all()            # exp(0) is 1: the rest reads true
    return y(pick[0], t["A"], None)[..., 0], y(pick[0], still, t["theta"]), y(pick[1], still, t["theta"])


def in_order(b, x):
    """sum_r b[r] x[r] over the third axis, each product and sum rounded."""
    t = b[:, :, 0, :, None] * x[:, :, 0, None, :]
    for r in range(1, b.shape[2]):
        t = t + b[:, :, r, :, None] * x[:, :, r, None, :]
    return t


def step(h, v, alpha, cos, sin, lam, theta):
    """The new states [S,H,N,P], float32 operation by float32 operation."""
    at = lambda a: a[..., None, None]
    la = v["lam"] if lam else np.ones_like(v["dt"])
    if lam:
        h = h + at((F(1) - la) * v["dt"]) * in_order(v["B_prev"], v["x_prev"])
    if theta:
        c, s, e, o = cos[..., None], sin[..., None], h[:, :, 0::2], h[:, :, 1::2]
        h = np.stack([c * e - s * o, s * e + c * o], 3).reshape(h.shape)
    return at(alpha) * h + at(la * v["dt"]) * in_order(v["B"], v["x"])


# S, H, N, P: by the kernel's rule a workgroup of four waves a unit, a wave a
# unit because it holds the whole unit, and a wave a unit because there are
# enough of them; for bfloat16 the matrix form too
FORMS = [(3, 2, 64, 64), (2, 3, 98, 16), (2, 2, 34, 32), (2, 2, 18, 128),
         (3, 5, 64, 16), (2, 2, 16, 64),
         (37, 28, 34, 32), (37, 28, 22, 64), (37, 28, 10, 128), (41, 25, 66, 16),
         (41, 25, 32, 64), (9, 128, 96, 64)]


@pytest.mark.parametrize("lam,theta", [(True, True), (False, False)], ids=["full", "reduced"])
@pytest.mark.parametrize("R", [1, 2, 4])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "s%d-h%d-n%d-p%d" % f)
def test_codes_are_the_definition_s(form, dtype, fmt, R, lam, theta):
    import torch
    import state_space_sequence_exp_amd as m3
    from oracle import layer as O
    S, H, N, P = form
    rng = np.random.default_rng(S + N + P + R)
    v, t = {}, {}
    for k, n in (("x", P), ("x_prev", P), ("B", N), ("B_prev", N), ("C", N)):
        v[k], t[k] = stored(rng, (S, H, R, n), dtype)
    for k, a in (("dt", np.log1p(np.exp(rng.standard_normal((S, H)) - 1))),
                 ("lam", 1 / (1 + np.exp(-rng.standard_normal((S, H))))),
                 ("theta", rng.uniform(-np.pi, np.pi, (S, H, N // 2))), ("A", -np.exp(rng.uniform(-2, 0, H)))):
        v[k], t[k] = put(a, "f32")
    v = {k: a.astype(F) for k, a in v.items()}
    alpha, cos, sin = factors(t)
    h = rows(rng, S, H, N, P)
    codes, scales = cache_with(h, fmt)
    old = O.dequantise(*O.quantise(h, fmt), fmt)
    m3.decode_step_cached(codes, scales, None, t["x"], t["x_prev"] if lam else None, t["B"],
                          t["B_prev"] if lam else None, t["C"], t["dt"], t["A"], t["lam"] if lam else None,
                          t["theta"] if theta else None)
    new = step(old, v, alpha, cos, sin, lam, theta)
    assert new.dtype == F
    c, s = O.quantise(new, fmt)
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(O.code_values(raw(codes), fmt), O.code_values(c, fmt))
