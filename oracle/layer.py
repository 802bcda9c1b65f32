"""fp64 oracle of the operators beside the recurrence: the gated linear
recurrence and its gradients, layer norm and its gradients, the 8-bit state
rows.  Plain NumPy from the formulas; shares no code with the HIP path.

The recurrence and the norm also return how far a float32 evaluation may be
from the exact values, by carrying each step's rounding through the same
formulas (running error analysis): with u = 2^-24, a gate's two values within
delta(f) = (8 + 2 |f|) u relative (the hardware exponential's argument f
log2(e) is rounded, |f| u, and its constant is, 0.3 |f| u; the exponential and
the reciprocal are within an ulp, 2 u, each; the sum and the product add 2 u),
every state update within C = 8 roundings of its terms (a state composed from
partial products takes up to that many)."""
import numpy as np

U = 2.0 ** -24
C = 8


def delta(f):
    """Relative error of a float sigmoid of f, and of one minus it."""
    return (8 + 2 * np.minimum(np.abs(f), 128)) * U


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def gated_scan(x, f, g=None, h0=None):
    """x, f, g [B,T,D] float64.  Returns dict: y, h (every token), before (the
    state each token meets), h_last, and the bounds e_h, e_y, e_last."""
    B, T, D = x.shape
    a, w, df = sigmoid(f), sigmoid(-f), delta(f)
    h = np.zeros((B, D)) if h0 is None else h0.astype(np.float64)
    e = np.zeros((B, D))
    hs, es, before, e_before = (np.empty((B, T, D)) for _ in range(4))
    for t in range(T):
        before[:, t], e_before[:, t] = h, e
        # masks: w = 0 does not look at x, a = 0 not at the state
        xt = np.where(w[:, t] == 0, 0.0, x[:, t])
        ht, et = np.where(a[:, t] == 0, 0.0, h), np.where(a[:, t] == 0, 0.0, e)
        e = a[:, t] * et + df[:, t] * w[:, t] * np.abs(xt) + \
            df[:, t] * np.minimum(a[:, t], w[:, t]) * np.abs(ht) + \
            C * U * (w[:, t] * np.abs(xt) + a[:, t] * np.abs(ht))
        h = a[:, t] * ht + w[:, t] * xt
        hs[:, t], es[:, t] = h, e
    out = dict(h=hs, before=before, e_h=es, e_before=e_before, h_last=h, e_last=e, a=a, w=w)
    if g is None:
        out.update(y=hs, e_y=es)
    else:
        s = g * sigmoid(g)
        out.update(y=hs * s, e_y=es * np.abs(s) + (delta(g) + 4 * U) * np.abs(hs * s))
    return out


def gated_scan_backward(dy, x, f, g=None, h0=None, dh_last=None):
    """Gradients of sum(y dy) + sum(h_last dh_last) and their bounds (keys
    e_dx, ...): the adjoint, token by token from the last."""
    B, T, D = x.shape
    s = gated_scan(x, f, g, h0)
    a, w, before = s["a"], s["w"], s["before"]
    out = {}
    dh, e_dh = dy, np.zeros_like(dy)
    if g is not None:
        sg = sigmoid(g)
        slope = sg * (1 + g * (1 - sg))
        out["dg"] = dy * s["h"] * slope
        # d slope = d sg (1 + g (1 - sg)) + sg g d(1 - sg), both within delta sg
        mag = sg * (1 + np.abs(g))
        out["e_dg"] = np.abs(dy) * (s["e_h"] * mag + np.abs(s["h"]) * mag * (2 * delta(g) + 8 * U))
        dh = dy * g * sg
        e_dh = (delta(g) + 4 * U) * np.abs(dh)
    u = np.zeros((B, D)) if dh_last is None else dh_last.astype(np.float64)
    e = np.zeros((B, D))
    out["dx"], out["df"], out["e_dx"], out["e_df"] = (np.empty((B, T, D)) for _ in range(4))
    for t in range(T - 1, -1, -1):
        G = dh[:, t] + u
        eG = e_dh[:, t] + e + C * U * (np.abs(dh[:, t]) + np.abs(u))
        at, wt, dt = a[:, t], w[:, t], delta(f[:, t])
        slope = at * wt
        diff = np.where(slope == 0, 0.0, before[:, t] - x[:, t])
        e_diff = s["e_before"][:, t] + 2 * U * (np.abs(before[:, t]) + np.abs(x[:, t]))
        e_diff = np.where(slope == 0, 0.0, e_diff)
        out["dx"][:, t] = G * wt
        out["e_dx"][:, t] = eG * wt + (dt + 4 * U) * np.abs(G * wt)
        out["df"][:, t] = G * diff * slope
        out["e_df"][:, t] = slope * (eG * np.abs(diff) + np.abs(G) * e_diff) + \
            (2 * dt + 8 * U) * np.abs(G * diff * slope)
        G, eG = np.where(at == 0, 0.0, G), np.where(at == 0, 0.0, eG)
        u = at * G
        e = at * eG + dt * np.minimum(at, wt) * np.abs(G) + C * U * np.abs(u)
    out["dh0"], out["e_dh0"] = u, e
    return out


def layer_norm(s, weight, bias, eps):
    """s [M,D] float64 (the stored sum).  Returns y, q, mean, rstd and bounds.
    A float32 mean of D values summed in pieces is within K u of the mean
    magnitude, K = 48 roundings (up to 16 in a lane, 6 in a wave, 16 between
    waves, and the division)."""
    K = 48
    mean = s.mean(-1, keepdims=True)
    c = s - mean
    var = (c * c).mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    q = c * rstd
    e_mean = K * U * np.abs(s).mean(-1, keepdims=True)
    e_c = e_mean + 2 * U * np.abs(c)
    # the variance: each square by 2 |c| e_c, the sum and division by K u
    e_var = (2 * np.abs(c) * e_c + e_c * e_c).mean(-1, keepdims=True) + K * U * var
    e_rstd = rstd * np.minimum(1.0, 0.5 * e_var / (var + eps) + 4 * U)
    e_q = e_c * rstd + np.abs(c) * e_rstd + 2 * U * np.abs(q)
    y = q * weight + bias
    e_y = e_q * np.abs(weight) + 2 * U * (np.abs(q * weight) + np.abs(bias))
    return dict(y=y, q=q, mean=mean[:, 0], rstd=rstd[:, 0], e_y=e_y, e_q=e_q,
                e_mean=e_mean[:, 0], e_rstd=e_rstd[:, 0])


def layer_norm_backward(dy, s, weight, eps, dsum=None):
    """Gradients dx, dw, db of layer norm and their bounds."""
    K = 48
    n = layer_norm(s, weight, np.zeros_like(weight), eps)
    q, rstd = n["q"], n["rstd"][:, None]
    p = dy * weight
    mp, mpq = p.mean(-1, keepdims=True), (p * q).mean(-1, keepdims=True)
    dx = rstd * (p - mp - q * mpq)
    e_mp = K * U * np.abs(p).mean(-1, keepdims=True)
    e_mpq = (np.abs(p) * n["e_q"]).mean(-1, keepdims=True) + K * U * np.abs(p * q).mean(-1, keepdims=True)
    size = np.abs(p) + np.abs(mp) + np.abs(q * mpq)
    e_dx = rstd * (e_mp + n["e_q"] * np.abs(mpq) + np.abs(q) * e_mpq + 6 * U * size) + \
        n["e_rstd"][:, None] * np.abs(p - mp - q * mpq)
    if dsum is not None:
        dx = dx + dsum
        e_dx = e_dx + U * np.abs(dx)
    # sums over the rows in any order: at most one rounding a row and term
    m = s.shape[0] + 8
    dw, db = (dy * q).sum(0), dy.sum(0)
    e_dw = (np.abs(dy) * n["e_q"]).sum(0) + m * U * np.abs(dy * q).sum(0)
    e_db = m * U * np.abs(dy).sum(0)
    return dict(dx=dx, dw=dw, db=db, e_dx=e_dx, e_dw=e_dw, e_db=e_db)


# ---- 8-bit rows ---------------------------------------------------------------

CODE_MAX = {"int8": np.float32(127), "e4m3": np.float32(448)}
TINY_ROW = np.float32(2.0 ** -100)


def e4m3_values():
    """The non-negative finite values of the OCP e4m3 format, by code."""
    out = [m * 2.0 ** -9 for m in range(8)]
    for e in range(1, 16):
        out += [(8 + m) * 2.0 ** (e - 10) for m in range(8) if (e, m) != (15, 7)]
    return np.array(out)


def to_e4m3(v):
    """float32 values within +-448 rounded to the nearest e4m3 value, ties to
    the even code; returns codes."""
    vals = e4m3_values()
    m = np.abs(v).astype(np.float64)
    hi = np.clip(np.searchsorted(vals, m), 0, len(vals) - 1)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = m - vals[lo], vals[hi] - m
    code = np.where(dlo < dhi, lo, np.where(dhi < dlo, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code + np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def quantise(h, fmt):
    """Rows (last axis) of float32 values -> (codes uint8, scales float32), as
    the format is defined: quotients and products rounded to float32."""
    h = h.astype(np.float32)
    q = CODE_MAX[fmt]
    with np.errstate(all="ignore"):
        amax = np.abs(h).max(-1)
        bad = ~np.isfinite(h).all(-1)
        held = ~bad & (amax >= TINY_ROW)
        safe = np.where(held, amax, np.float32(1))
        scale = np.where(held, safe * (np.float32(1) / q), np.float32(0)).astype(np.float32)
        inv = np.where(held, q / safe, np.float32(0)).astype(np.float32)
        v = np.where(bad[..., None], np.float32(0), h) * inv[..., None]
    v = np.clip(v.astype(np.float32), -q, q)
    scale = np.where(bad, np.float32(np.nan), scale)
    if fmt == "int8":
        return np.rint(v).astype(np.int8).view(np.uint8), scale
    return to_e4m3(v), scale


def code_values(codes, fmt):
    if fmt == "int8":
        return codes.view(np.int8).astype(np.float64)
    table = e4m3_values()
    table = np.concatenate([table, [np.nan], -table, [np.nan]])
    return table[codes]


def dequantise(codes, scales, fmt):
    """float32(code * scale)."""
    return (code_values(codes, fmt).astype(np.float32) * scales[..., None]).astype(np.float32)
