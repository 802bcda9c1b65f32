"""GPU tests of the short causal convolution and the selective scan, over prompts
and for single tokens, against the fp64 oracle's bounds: tokens from none to
several segments, odd widths, strided slices, padding that holds NaN, pools with
idle and twice-named slots, streams and graphs."""
import numpy as np
import pytest
import torch

from gpu_util import from_gpu
from layer_util import close, put, stored, torch_type
from oracle import selective as O

pytestmark = pytest.mark.gpu
TYPES = ["f32", "bf16"]


def f32(rng, shape, mean=0.0, std=1.0):
    return put((rng.standard_normal(shape) * std + mean).astype(np.float32), "f32")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def sliced(t, before=3, after=2):
    """The same values as a slice of wider rows, at an odd element."""
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + before + after,), float("nan"), dtype=t.dtype, device=t.device)
    s = wide[..., before:before + t.shape[-1]]
    s.copy_(t)
    return s


# ---- convolution ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,T,D,W", [(1, 1, 1, 2), (2, 2, 7, 4), (1, 9, 8, 4), (3, 33, 65, 3), (2, 300, 24, 2),
                                     (1, 70, 1030, 4)])
@pytest.mark.parametrize("extra", [False, True])
def test_conv(dtype, B, T, D, W, extra):
    import state_space_sequence_exp_amd as m3
    rng = np.random.default_rng([B, T, D, W, extra])
    x64, x = stored(rng, (B, T, D), dtype)
    w64, w = f32(rng, (D, W), std=W ** -0.5)
    b64, b = f32(rng, (D,))
    s64, s = stored(rng, (B, W - 1, D), dtype)
    if not extra:
        b64 = b = s64 = s = None
    y, kept = m3.causal_conv(x, w, b, silu=extra, state=s)
    want, e, k64 = O.causal_conv(x64, w64, b64, extra, s64)
    close(y, want, e, dtype, "y")
    assert np.array_equal(from_gpu(kept), k64)
    # a slice of a wider projection, into a slice of wider rows
    out = sliced(torch.zeros_like(x))
    y2, _ = m3.causal_conv(sliced(x), w, b, silu=extra, state=s, y=out, want_state=False)
    assert y2 is out and torch.equal(out, y)
    assert torch.isnan(out._base[..., :3]).all() and torch.isnan(out._base[..., -2:]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("silu", [False, True])
def test_conv_lengths(dtype, silu):
    """Padding that holds NaN is not looked at, its outputs are 0; lengths outside 0..T are taken as the nearest."""
    import state_space_sequence_exp_amd as m3
    rng = np.random.default_rng(5)
    n = np.array([0, 1, 2, 3, 40, 77, 1000, -7])
    B, T, D, W = len(n), 77, 20, 4
    x64, x = stored(rng, (B, T, D), dtype)
    w64, w = f32(rng, (D, W))
    s64, s = stored(rng, (B, W - 1, D), dtype)
    for b in range(B):
        x[b, max(0, n[b]):] = float("nan")
    y, kept = m3.causal_conv(x, w, silu=silu, state=s, lengths=ints(n))
    want, e, k64 = O.causal_conv(x64, w64, None, silu, s64, n)
    close(y, want, e, dtype, "y")
    assert np.array_equal(from_gpu(kept), k64)


def test_conv_pieces_and_empty():
    """A prompt in pieces, one of no tokens among them, is the prompt at once, bit for bit."""
    import state_space_sequence_exp_amd as m3
    rng = np.random.default_rng(6)
    _, x = stored(rng, (2, 50, 12), "bf16")
    _, w = f32(rng, (12, 4))
    whole, last = m3.causal_conv(x, w, silu=True)
    s, parts = None, []
    for a, b in ((0, 1), (1, 1), (1, 3), (3, 30), (30, 50)):
        y, s = m3.causal_conv(x[:, a:b].contiguous(), w, silu=True, state=s)
        parts.append(y)
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(s, last)
    y, s = m3.causal_conv(x[:0], w)
    assert y.shape == (0, 50, 12) and s.shape == (0, 3, 12)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("S,D,W", [(1, 1, 2), (5, 37, 3), (3, 2100, 4), (300, 16, 4)])
def test_conv_step(dtype, S, D, W):
    import state_space_sequence_exp_amd as m3
    rng = np.random.default_rng([S, D, W])
    x64, x = stored(rng, (S, D), dtype)
    w64, w = f32(rng, (D, W))
    b64, b = f32(rng, (D,))
    s64, s = stored(rng, (S + 2, W - 1, D), dtype)
    slots = rng.permutation(S + 2)[:S]
    y = m3.causal_conv_step(s, sliced(x), w, b, silu=True, slots=ints(slots))
    want, e, k64 = O.causal_conv(x64[:, None], w64, b64, True, s64[slots])
    close(y, want[:, 0], e[:, 0], dtype, "y")
    s64[slots] = k64
    assert np.array_equal(from_gpu(s), s64)


@pytest.mark.parametrize("op", ["conv", "scan"])
def test_step_slots(op):
    """Idle rows and rows that name a slot again leave y and the pool as they were."""
    import state_space_sequence_exp_amd as m3
    rng = np.random.default_rng(8)
    S, D, N, W, pool = 700, 12, 16, 4, 40
    _, x = stored(rng, (S, D), "bf16")
    _, w = f32(rng, (D, W))
    _, A = f32(rng, (D, N), std=0.1)
    _, Bt = stored(rng, (S, N), "bf16")
    A = -A.exp()
    slots = np.full(S, -1)
    slots[[3, 600, 650]], slots[[4, 699]], slots[5], slots[[10, 11]] = 17, 0, pool, (39, 2 ** 31 - 1)
    s0 = stored(rng, (pool, W - 1, D), "bf16")[1] if op == "conv" else f32(rng, (pool, D, N))[1]
    s, y = s0.clone(), torch.full_like(x, 7.0)
    step = (lambda st, xs, ks, **kw: m3.causal_conv_step(st, xs, w, **kw)) if op == "conv" else \
        (lambda st, xs, ks, **kw: m3.selective_scan_step(st, xs, xs, A, ks, ks, **kw))
    out = step(s, x, Bt, slots=ints(slots), y=y)
    assert out is y
    live, at = [3, 4, 10], [17, 0, 39]
    alone = s0[at].clone()
    want = step(alone, x[live].contiguous(), Bt[live].contiguous())
    assert torch.equal(y[live], want) and torch.equal(s[at], alone)
    rest = [i for i in range(S) if i not in live]
    assert (y[rest] == 7).all()
    others = [i for i in range(pool) if i not in at]
    assert torch.equal(s[others], s0[others])
    fresh = step(s0.clone(), x, Bt, slots=ints(slots))
    assert torch.equal(fresh[live], want) and not fresh[rest].any()
    # no pool at all, and a pool without slots
    assert not step(s0[:0].clone(), x, Bt, slots=ints(slots)).any()
    with pytest.raises(ValueError, match="pool"):
        step(s0.clone(), x, Bt)


# ---- scan ------------------------------------------------------------------------

def scan_inputs(seed, B, T, D, N, dtype, plus=True):
    rng = np.random.default_rng(seed)
    v = dict(x=stored(rng, (B, T, D), dtype), dt=stored(rng, (B, T, D), dtype, -1.0), A=f32(rng, (D, N)),
             B=stored(rng, (B, T, N), dtype), C=stored(rng, (B, T, N), dtype), skip=f32(rng, (D,)),
             z=stored(rng, (B, T, D), dtype), dt_bias=f32(rng, (D,)), h0=f32(rng, (B, D, N)))
    v["A"] = put(-np.exp(v["A"][0]).astype(np.float32), "f32")
    if not plus:
        for k in ("dt", "dt_bias"):
            v[k] = put(np.abs(v[k][0]).astype(np.float32), dtype if k == "dt" else "f32")
    return {k: a[0] for k, a in v.items()}, {k: a[1] for k, a in v.items()}


def oracle_scan(r, plus=True, lengths=None, **drop):
    r = {**r, **drop}
    return O.selective_scan(r["x"], r["dt"], r["A"], r["B"], r["C"], r["skip"], r["z"], r["dt_bias"], plus, r["h0"],
                            lengths)


def check_scan(y, h, o, dtype):
    close(y, o["y"], o["e_y"], dtype, "y")
    close(h, o["h_last"], o["e_h"], "f32", "h_last")


def run_scan(t, **kw):
    import state_space_sequence_exp_amd as m3
    return m3.selective_scan(t["x"], t["dt"], t["A"], t["B"], t["C"], t["skip"], t["z"],
                             **{"dt_bias": t["dt_bias"], "h0": t["h0"], **kw})


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,T,D,N", [(1, 1, 1, 1), (2, 3, 5, 16), (1, 16, 16, 8), (3, 65, 33, 16), (2, 130, 18, 17),
                                     (1, 100, 40, 64), (2, 64, 67, 33), (1, 200, 19, 3), (1, 1030, 20, 16),
                                     (2, 900, 35, 24)])
def test_scan(dtype, B, T, D, N):
    r, t = scan_inputs([B, T, D, N], B, T, D, N, dtype)
    y, h = run_scan(t)
    check_scan(y, h, oracle_scan(r), dtype)
    # slices of wider projections, into a slice of wider rows
    wide = {k: sliced(v) if k in ("x", "dt", "B", "C", "z") else v for k, v in t.items()}
    out = sliced(torch.zeros_like(t["x"]))
    y2, h2 = run_scan(wide, y=out)
    assert torch.equal(out, y) and torch.equal(h2, h)
    assert torch.isnan(out._base[..., :3]).all() and torch.isnan(out._base[..., -2:]).all()


@pytest.mark.parametrize("plus", [True, False])
@pytest.mark.parametrize("none", [("skip",), ("z",), ("dt_bias",), ("h0",), ("skip", "z", "dt_bias", "h0")])
def test_scan_options(plus, none):
    r, t = scan_inputs(11, 2, 90, 20, 16, "f32", plus)
    drop = {k: None for k in none}
    y, h = run_scan({**t, **drop}, softplus=plus)
    check_scan(y, h, oracle_scan(r, plus, **drop), "f32")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,D", [(150, 20), (1100, 17)])
def test_scan_lengths(dtype, T, D):
    """Padding that holds NaN is not looked at, in whole and in cut sequences: y is 0
    there, the state is the one after each sequence's last token."""
    n = np.array([0, 1, 63, 64, 65, T - 1, T, 5000, -2, T // 2])
    r, t = scan_inputs([T, D], len(n), T, D, 16, dtype)
    for k in ("x", "dt", "B", "C", "z"):
        for b in range(len(n)):
            t[k][b, max(0, n[b]):] = float("nan")
    y, h = run_scan(t, lengths=ints(n))
    check_scan(y, h, oracle_scan(r, lengths=n), dtype)


def test_scan_steep():
    """Decays that underflow, steps that vanish or are large, and states that do not decay."""
    B, T, D, N = 1, 260, 6, 16
    r, t = scan_inputs(12, B, T, D, N, "f32")
    put_in = lambda k, v: (r.__setitem__(k, v.astype(np.float64)), t[k].copy_(torch.from_numpy(v)))
    A = r["A"].astype(np.float32)
    A[0], A[1] = 0.0, -1e4
    put_in("A", A)
    dt = r["dt"].astype(np.float32)
    dt[..., 2], dt[..., 3], dt[..., 4] = -60.0, 30.0, -200.0
    dt[:, ::2, 5] = 12.0
    put_in("dt", dt)
    y, h = run_scan(t)
    check_scan(y, h, oracle_scan(r), "f32")


@pytest.mark.parametrize("B,T,D,N", [(1, 3000, 16, 16), (1, 2000, 130, 64), (3, 1500, 40, 5)])
def test_scan_cut(B, T, D, N):
    """Few channels over many tokens: cut into segments, whose states come from a
    workspace of any content; pieces give the whole."""
    import state_space_sequence_exp_amd as m3
    r, t = scan_inputs([B, T, D], B, T, D, N, "f32")
    need = m3.selective_scan_workspace_size(B, T, D, N, torch.float32)
    assert need > 0
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")       # NaN
    y, h = run_scan(t, workspace=ws)
    o = oracle_scan(r)
    check_scan(y, h, o, "f32")
    assert (ws[need:] == 255).all()
    y2, h2 = run_scan(t)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    cut = {k: v[:, :T // 3].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in t.items()}
    rest = {k: v[:, T // 3:].contiguous() if k in ("x", "dt", "B", "C", "z") else v for k, v in t.items()}
    y1, h1 = run_scan(cut)
    y2, h2 = run_scan({**rest, "h0": h1})
    check_scan(torch.cat([y1, y2], 1), h2, o, "f32")


def test_scan_empty():
    r, t = scan_inputs(13, 2, 5, 8, 16, "bf16")
    none = {k: v[:, :0] if k in ("x", "dt", "B", "C", "z") else v for k, v in t.items()}
    y, h = run_scan(none)
    assert y.shape == (2, 0, 8) and torch.equal(h, t["h0"])
    y, h = run_scan({**none, "h0": None})
    assert not h.any()
    y, h = run_scan({k: v[:0] if k in ("x", "dt", "B", "C", "z", "h0") else v for k, v in t.items()})
    assert y.shape == (0, 5, 8) and h.shape == (0, 8, 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("S,D,N", [(1, 1, 1), (2, 5, 4), (3, 70, 7), (5, 300, 16), (2, 33, 24), (4, 257, 64)])
@pytest.mark.parametrize("plain", [False, True])
def test_scan_step(dtype, S, D, N, plain):
    import state_space_sequence_exp_amd as m3
    r, t = scan_inputs([S, D, N], S, 1, D, N, dtype, not plain)
    drop = {"skip": None, "z": None, "dt_bias": None} if plain else {}
    slots = np.random.default_rng(S).permutation(S + 3)[:S]
    pool = torch.full((S + 3, D, N), 3.0, device="cuda")
    pool[slots] = t["h0"]
    v = {k: sliced(a[:, 0]) if k in ("x", "dt", "B", "C", "z") else a for k, a in t.items()}
    v.update(drop)
    y = m3.selective_scan_step(pool, v["x"], v["dt"], v["A"], v["B"], v["C"], v["skip"], v["z"],
                               dt_bias=v["dt_bias"], softplus=not plain, slots=ints(slots))
    o = oracle_scan(r, not plain, **drop)
    check_scan(y[:, None], pool[slots], o, dtype)
    rest = [i for i in range(S + 3) if i not in slots]
    assert (pool[rest] == 3).all()


# ---- streams and graphs -------------------------------------------------------------

def test_on_another_stream():
    import state_space_sequence_exp_amd as m3
    _, t = scan_inputs(14, 1, 2000, 24, 16, "bf16")
    _, w = f32(np.random.default_rng(1), (24, 4))
    want = run_scan(t)
    kept = m3.causal_conv(t["x"], w)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got, conv = run_scan(t, stream=st), m3.causal_conv(t["x"], w, stream=st.cuda_stream)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + conv, want + kept))


def test_captured():
    """A prompt (cut into segments) and a token, captured together and replayed with
    new inputs and eager calls between; two graphs with a workspace each."""
    import state_space_sequence_exp_amd as m3
    rng = np.random.default_rng(15)
    _, t = scan_inputs(16, 1, 1600, 20, 16, "bf16")
    _, w = f32(rng, (20, 4))
    slots = ints([1])
    new = lambda: {k: torch.randn_like(t[k]) for k in ("x", "dt", "B", "C", "z")}

    def both(t, conv, pool):
        x, s = m3.causal_conv(t["x"], w, silu=True)
        y, h = run_scan({**t, "x": x})
        pool[1].copy_(h[0])
        conv[1].copy_(s[0])
        x1 = m3.causal_conv_step(conv, t["x"][:, 0], w, silu=True, slots=slots)
        y1 = m3.selective_scan_step(pool, x1, t["dt"][:, 0], t["A"], t["B"][:, 0], t["C"][:, 0], t["skip"],
                                    t["z"][:, 0], dt_bias=t["dt_bias"], slots=slots)
        return y, y1, pool, conv

    fresh = lambda: (torch.zeros(3, 3, 20, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 20, 16, device="cuda"))
    both(t, *fresh())
    graphs = []
    for _ in range(2):
        held, state = {k: v.clone() for k, v in t.items()}, fresh()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(held, *state)
        graphs.append((g, held, out))
    for _ in range(3):
        ins = [new() for _ in graphs]
        for (g, held, _), v in zip(graphs, ins):
            for k, a in v.items():
                held[k].copy_(a)
        for g, _, _ in graphs:
            g.replay()
        wants = [both({**t, **v}, *fresh()) for v in ins]
        torch.cuda.synchronize()
        for (_, _, out), want in zip(graphs, wants):
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_far_rows():
    """Rows whose offsets pass 32 bits: tokens 2^20 elements apart, 2500 of them."""
    import state_space_sequence_exp_amd as m3
    r, t = scan_inputs(17, 1, 2500, 8, 4, "bf16")
    wide = torch.zeros((1, 2500, 1 << 20), dtype=torch.bfloat16, device="cuda")
    far = {}
    for i, k in enumerate(("x", "dt", "z")):
        far[k] = wide[..., 100 * i:100 * i + 8]
        far[k].copy_(t[k])
    for i, k in enumerate(("B", "C")):
        far[k] = wide[..., 500 + 100 * i:504 + 100 * i]
        far[k].copy_(t[k])
    out = wide[..., 1000:1008]
    y, h = run_scan({**t, **far}, y=out)
    want, hw = run_scan(t)
    assert torch.equal(out, want) and torch.equal(h, hw)
    _, w = f32(np.random.default_rng(2), (8, 3))
    m3.causal_conv(far["x"], w, y=out)
    assert torch.equal(out, m3.causal_conv(t["x"], w)[0])
