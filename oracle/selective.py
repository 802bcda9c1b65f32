"""fp64 oracle of the short causal convolution, the selective scan and the gated
feed-forward projections with their gradients.  Plain NumPy from the formulas;
shares no code with the HIP path.

Each also returns how far a float32 evaluation may be from the exact values, by
carrying the roundings through the same formulas (u = 2^-24):

* a sum of n products in any order is within (n + 1) u of the sum of the
  products' magnitudes;
* sigmoid and silu are within delta(v) relative (see layer.delta);
* softplus(v), v = dt + dt_bias: the sum is rounded (u |v|, times the slope
  sigmoid(v)); exp(-|v|) is within (2 + 2 |v|) u, what is made of it within
  another 8 u, relative to the result;
* a decay exp(s A): the exponent is s A with the error of s, two roundings of
  products and one of log2(e); where a sequence is cut, a segment's decay comes
  from the sum of its steps, up to 40 roundings in a chain of sums, all relative
  to the exponent; the exponential adds 2 u;
* a state update rounds s x (one rounding), times B (one) and the fused sum (one),
  a joined segment as often again: 8 u of its terms."""
import numpy as np

from .layer import U, delta, sigmoid


def silu(v):
    return v * sigmoid(v)


def _e_silu(v, e):
    """Error of a float silu of a value within e of v (its slope is within 1.1)."""
    return 1.1 * e + (delta(v) + 4 * U) * (np.abs(silu(v)) + 1.1 * e)


def _ends(lengths, B, T):
    return np.full(B, T) if lengths is None else np.clip(lengths, 0, T)


def causal_conv(x, w, bias=None, act=False, state=None, lengths=None):
    """x [B,T,D], w [D,W], state [B,W-1,D] float64.  Returns y, its bound, and the
    last W-1 inputs of each sequence."""
    B, T, D = x.shape
    W = w.shape[1]
    y, e, kept = np.zeros((B, T, D)), np.zeros((B, T, D)), np.zeros((B, W - 1, D))
    for b, n in enumerate(_ends(lengths, B, T)):
        old = np.zeros((W - 1, D)) if state is None else state[b]
        seq = np.concatenate([old, x[b, :n]])
        terms = np.stack([seq[k:k + n] * w[:, k] for k in range(W)])
        v, mag = terms.sum(0), np.abs(terms).sum(0)
        if bias is not None:
            v, mag = v + bias, mag + np.abs(bias)
        ev = (W + 2) * U * mag
        y[b, :n], e[b, :n] = (silu(v), _e_silu(v, ev)) if act else (v, ev)
        kept[b] = seq[n:]
    return y, e, kept


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def selective_scan(x, dt, A, Bt, Ct, skip=None, z=None, dt_bias=None, plus=True, h0=None, lengths=None):
    """x, dt, z [B,T,D], A [D,N], Bt, Ct [B,T,N], h0 [B,D,N] float64.  Returns a
    dict: y, h_last and their bounds e_y, e_h."""
    B, T, D = x.shape
    N = A.shape[1]
    h = np.zeros((B, D, N)) if h0 is None else h0.astype(np.float64)
    eh = np.zeros((B, D, N))
    y, ey = np.zeros((B, T, D)), np.zeros((B, T, D))
    ends = _ends(lengths, B, T)
    for t in range(T):
        on = ends > t
        if not on.any():
            break
        xt, v = x[on, t], dt[on, t] + (0 if dt_bias is None else dt_bias)
        if plus:
            s = softplus(v)
            es = U * np.abs(v) * sigmoid(v) + (10 + 2 * np.abs(v)) * U * s
        else:
            s, es = v, U * np.abs(v)
        sx, esx = (s * xt)[..., None], (es * np.abs(xt))[..., None]
        Bn, Cn = Bt[on, t][:, None], Ct[on, t][:, None]
        arg = s[..., None] * A
        a = np.exp(arg)
        rel = np.abs(A) * es[..., None] + np.abs(arg) * 44 * U + 2 * U
        hp, ep = h[on], eh[on]
        hn = a * hp + sx * Bn
        en = a * (1 + rel) * ep + a * rel * np.abs(hp) + esx * np.abs(Bn) + \
            8 * U * (np.abs(a * hp) + np.abs(sx * Bn))
        h[on], eh[on] = hn, en
        o, eo = (Cn * hn).sum(-1), (np.abs(Cn) * en).sum(-1) + (N + 2) * U * np.abs(Cn * hn).sum(-1)
        if skip is not None:
            eo = eo + 2 * U * (np.abs(o) + np.abs(skip * xt))
            o = o + skip * xt
        if z is not None:
            g = silu(z[on, t])
            eo = eo * np.abs(g) * (1 + 1e-4) + (delta(z[on, t]) + 4 * U) * np.abs(o * g)
            o = o * g
        y[on, t], ey[on, t] = o, eo
    return dict(y=y, e_y=ey, h_last=h, e_h=eh)


def gated_ffn(x, wg, wu):
    """x [M,K], wg, wu [F,K] float64.  Returns a dict: h, g, u and bounds e_h, e_g, e_u."""
    K = x.shape[1]
    g, u = x @ wg.T, x @ wu.T
    eg, eu = ((K + 1) * U * (np.abs(x) @ np.abs(w).T) for w in (wg, wu))
    s = silu(g)
    es = _e_silu(g, eg)
    return dict(h=s * u, e_h=es * np.abs(u) + (np.abs(s) + es) * eu + 2 * U * np.abs(s * u), g=g, u=u, e_g=eg,
                e_u=eu)


def gated_ffn_backward(dh, x, wg, wu, half_step):
    """Gradients of sum(h dh) and their bounds (keys e_dx, ...): dg and du are
    rounded to the storage type on the way, half a step of which is half_step
    relative."""
    M, K = x.shape
    F = wg.shape[0]
    f = gated_ffn(x, wg, wu)
    g, u, sg = f["g"], f["u"], sigmoid(f["g"])
    s, slope = g * sg, sg * (1 + g * (1 - sg))
    es = _e_silu(g, f["e_g"])
    # silu's second derivative is within 0.5; the slope's evaluation within 4 delta of its parts
    eslope = 0.5 * f["e_g"] + (4 * delta(g) + 8 * U) * sg * (1 + np.abs(g) * (1 - sg))
    du, dg = dh * s, dh * u * slope
    edu = np.abs(dh) * es + 2 * U * np.abs(du)
    edg = np.abs(dh) * (f["e_u"] * (np.abs(slope) + eslope) + np.abs(u) * eslope) + 4 * U * np.abs(dg)
    edu, edg = (e + half_step * (np.abs(v) + e) + 1e-38 for e, v in ((edu, du), (edg, dg)))
    ab = np.abs
    out = dict(dx=dg @ wg + du @ wu, dw_gate=dg.T @ x, dw_up=du.T @ x)
    out["e_dx"] = (edg @ ab(wg) + edu @ ab(wu)) + (2 * F + 130) * U * ((ab(dg) + edg) @ ab(wg) + (ab(du) + edu) @ ab(wu))
    for k, d, e in (("dw_gate", dg, edg), ("dw_up", du, edu)):
        out["e_" + k] = e.T @ ab(x) + (M + 65) * U * ((ab(d) + e).T @ ab(x))
    return out


def gated_ffn_backward_stored(dh, x, wg, wu, g, u, store):
    """Gradients from g and u as they were kept (float32 values, taken as exact), with dg and
    du rounded by `store` (float64 values to the storage type's) before the products, as
    the operator defines them; and bounds.  Half a step of dg and du is then no error: what
    is left of it is the elements that a float evaluation may round to the other side."""
    M, F = g.shape
    ab = np.abs
    sg = sigmoid(g)
    slope, mag = sg * (1 + g * (1 - sg)), sg * (1 + ab(g) * (1 - sg))
    du, dg = dh * g * sg, dh * u * slope
    edu = (delta(g) + 6 * U) * ab(du)
    edg = ab(dh * u) * (4 * delta(g) + 8 * U) * mag + 4 * U * ab(dg)
    (dg, edg), (du, edu) = ((store(v), np.maximum(store(v + e) - store(v), store(v) - store(v - e)) + 1e-38)
                            for v, e in ((dg, edg), (du, edu)))
    out = dict(dx=dg @ wg + du @ wu, dw_gate=dg.T @ x, dw_up=du.T @ x)
    out["e_dx"] = (edg @ ab(wg) + edu @ ab(wu)) + (2 * F + 130) * U * ((ab(dg) + edg) @ ab(wg) + (ab(du) + edu) @ ab(wu))
    for k, d, e in (("dw_gate", dg, edg), ("dw_up", du, edu)):
        out["e_" + k] = e.T @ ab(x) + (M + 65) * U * ((ab(d) + e).T @ ab(x))
    return out
