"""GPU parity of the 8-bit state cache: store and load against the format's
definition (equal to the last bit), the decode step on cached states against
the fp64 oracle, and a prefill handed over to it."""
import numpy as np
import pytest

from layer_util import put, stored, torch_type
from gpu_util import from_gpu, log, to_gpu_f32, to_gpu_storage

pytestmark = pytest.mark.gpu

FORMATS = ["int8", "e4m3"]


def code_type(fmt):
    import torch
    return torch.int8 if fmt == "int8" else torch.float8_e4m3fn


def rows(rng, *shape):
    """States whose rows differ in size, float32."""
    return (rng.standard_normal(shape) * np.exp2(rng.uniform(-12, 6, shape[:-1] + (1,)))).astype(np.float32)


def cache_with(h, fmt):
    """(codes, scales) device tensors holding the oracle's codes of h."""
    import torch
    from oracle import layer as O
    c, s = O.quantise(h, fmt)
    return torch.from_numpy(c).cuda().view(code_type(fmt)), torch.from_numpy(s).cuda()


def raw(codes):
    import torch
    return codes.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", [(1, 1, 2, 16), (3, 2, 64, 64), (2, 3, 34, 32), (5, 1, 128, 128), (2, 5, 256, 16),
                                   (70, 2, 18, 64)], ids=str)
def test_store_and_load(shape, fmt):
    import torch
    import state_space_sequence_exp_amd as m3
    from oracle import layer as O
    S, H, N, P = shape
    log("store and load %s %s" % (shape, fmt))
    rng = np.random.default_rng(sum(shape))
    h = rows(rng, *shape)
    h.reshape(-1, P)[0] = 0
    h.reshape(-1, P)[1, 3:] = 0.25                              # ties and equal values
    if S * H * N > 12:
        h.reshape(-1, P)[2] = 1e-31                             # below the smallest row
        h.reshape(-1, P)[3, -1] = np.inf
        h.reshape(-1, P)[4, 0] = np.nan
        h.reshape(-1, P)[5] = 3.4e38
        h.reshape(-1, P)[6] = np.arange(P) - P / 2              # halves fall between codes
    n_slots = S + 3
    slots = rng.permutation(n_slots)[:S].astype(np.int32)
    codes, scales = m3.state_cache(n_slots, H, N, P, code_type(fmt))
    codes.view(torch.uint8).fill_(77)
    scales.fill_(-5.0)
    m3.state_store(to_gpu_f32(h), codes, scales, torch.from_numpy(slots).cuda())
    wc, ws = np.full((n_slots, H, N, P), 77, np.uint8), np.full((n_slots, H, N), -5.0, np.float32)
    c, s = O.quantise(h, fmt)
    wc[slots], ws[slots] = c, s
    assert np.array_equal(raw(codes), wc)                       # the other slots stay
    assert np.array_equal(scales.cpu().numpy(), ws, equal_nan=True)
    back = m3.state_load(codes, scales, torch.from_numpy(slots).cuda())
    want = O.dequantise(c, s, fmt)
    assert np.array_equal(back.cpu().numpy(), want, equal_nan=True)
    b16 = m3.state_load(codes, scales, torch.from_numpy(slots).cuda(), dtype=torch.bfloat16)
    assert torch.equal(b16.cpu().nan_to_num(9.0), torch.from_numpy(want).to(torch.bfloat16).nan_to_num(9.0))
    # the whole pool, slot by slot, and states into slots by their number
    assert np.array_equal(m3.state_load(codes, scales)[slots].cpu().numpy(), want, equal_nan=True)
    c2, s2 = m3.state_cache(n_slots, H, N, P, code_type(fmt))
    m3.state_store(to_gpu_f32(h), c2, s2)
    assert np.array_equal(raw(c2)[:S], c) and not raw(c2)[S:].any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_idle_and_repeated_slots(fmt):
    """Negative and too large entries are skipped (load: zeros); of entries
    that name one slot the first is taken."""
    import torch
    import state_space_sequence_exp_amd as m3
    from oracle import layer as O
    rng = np.random.default_rng(9)
    S, H, N, P = 300, 1, 16, 16
    h = rows(rng, S, H, N, P)
    slots = np.full(S, -1, np.int32)
    slots[[0, 7, 13, 290, 299]] = [4, 2, 4, 2, 0]
    slots[20], slots[21], slots[22] = 5, 2147483647, -2147483648      # a pool of 5
    codes, scales = m3.state_cache(5, H, N, P, code_type(fmt))
    t = torch.from_numpy(slots).cuda()
    m3.state_store(to_gpu_f32(h), codes, scales, t)
    c, s = O.quantise(h[[299, 7, 0]], fmt)
    want = np.zeros((5, H, N, P), np.uint8)
    want[[0, 2, 4]] = c
    assert np.array_equal(raw(codes), want)
    back = m3.state_load(codes, scales, t).cpu().numpy()
    v = O.dequantise(c, s, fmt)
    for i in range(S):
        ref = {0: v[0], 2: v[1], 4: v[2]}.get(slots[i], np.zeros((H, N, P)))
        assert np.array_equal(back[i], ref), i


def decode_inputs(rng, S, H, N, P, R, dtype):
    v, t = {}, {}
    for k, shape in (("x", (S, H, R, P)), ("x_prev", (S, H, R, P)), ("B", (S, H, R, N)),
                     ("B_prev", (S, H, R, N)), ("C", (S, H, R, N))):
        v[k], t[k] = stored(rng, shape, dtype, 0.0, 1.0 if k[0] == "x" else N ** -0.5)
    for k, a in (("dt", np.log1p(np.exp(rng.standard_normal((S, H)) - 1))),
                 ("lam", 1 / (1 + np.exp(-rng.standard_normal((S, H))))),
                 ("theta", rng.uniform(-np.pi, np.pi, (S, H, N // 2))), ("A", -np.exp(rng.uniform(-2, 0, H)))):
        v[k], t[k] = put(a, "f32")
    return v, t


def step64(h, v, i, lam=True, theta=True):
    """One step of sequence i in float64 from h [H,N,P]; the new state, y, and
    the sum of the magnitudes that enter each."""
    dt = v["dt"][i][:, None, None]
    la = v["lam"][i][:, None, None] if lam else 1.0
    al = np.exp(dt * v["A"][:, None, None])
    z, mag = h.copy(), np.abs(h)
    if lam:
        add = (1 - la) * dt * np.einsum("hrn,hrp->hnp", v["B_prev"][i], v["x_prev"][i])
        z, mag = z + add, mag + np.abs((1 - la) * dt) * np.einsum(
            "hrn,hrp->hnp", np.abs(v["B_prev"][i]), np.abs(v["x_prev"][i]))
    if theta:
        p = v["dt"][i][:, None] * v["theta"][i]
        c, s = np.cos(p)[..., None], np.sin(p)[..., None]
        e, o = z[:, 0::2].copy(), z[:, 1::2].copy()
        z[:, 0::2], z[:, 1::2] = c * e - s * o, s * e + c * o
        e, o = mag[:, 0::2].copy(), mag[:, 1::2].copy()
        mag[:, 0::2] = mag[:, 1::2] = e + o
    new = al * z + la * dt * np.einsum("hrn,hrp->hnp", v["B"][i], v["x"][i])
    mag = al * mag + np.abs(la * dt) * np.einsum("hrn,hrp->hnp", np.abs(v["B"][i]), np.abs(v["x"][i]))
    y = np.einsum("hrn,hnp->hrp", v["C"][i], new)
    ymag = np.einsum("hrn,hnp->hrp", np.abs(v["C"][i]), mag)
    return new, mag, y, ymag


# A new state value is a sum of up to 2 R + 2 products of float coefficients
# (an exponential, a sine or cosine of an argument below 16, each within 8
# roundings and the argument's own rounding, 16 u): within 64 u of the
# magnitudes.  y adds N terms: N + 64 roundings.
E_STATE = 64 * 2.0 ** -24


def check_decode(codes, scales, y, old, live, slots, v, fmt, dtype, **form):
    """The cache and y after one step from the float32 states `old`."""
    from oracle import layer as O
    got = O.code_values(raw(codes), fmt) * scales.cpu().numpy().astype(np.float64)[..., None]
    y = from_gpu(y)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for i in live:
        new, mag, yr, ymag = step64(old[slots[i]].astype(np.float64), v, i, **form)
        err = E_STATE * mag
        top = (np.abs(new) + err).max(-1, keepdims=True)
        step = top / 254 if fmt == "int8" else np.maximum(2.0 ** -4 * (np.abs(new) + err), top / 448 * 2.0 ** -10)
        assert (np.abs(got[slots[i]] - new) <= step * (1 + 1e-5) + err + top * 2.0 ** -22 + 1e-30).all(), i
        # the largest value of a row takes the largest code
        sc = scales[slots[i]].cpu().numpy().astype(np.float64)
        q = 127 if fmt == "int8" else 448
        assert (np.abs(sc * q - np.abs(new).max(-1)) <= err.max(-1) + top[..., 0] * 2.0 ** -22).all(), i
        n = v["B"].shape[-1]
        bound = (E_STATE + n * 2.0 ** -24) * ymag
        assert (np.abs(y[i] - yr) <= bound + half * (np.abs(yr) + bound) + 1e-30).all(), i


CASES = [
    # S, H, N, P, R
    (1, 1, 2, 16, 1), (3, 2, 64, 64, 1), (2, 3, 34, 32, 2), (5, 2, 128, 64, 4), (2, 1, 128, 128, 1),
    (2, 1, 256, 16, 4), (1, 2, 22, 128, 2), (4, 3, 256, 64, 2),
    # a wave a unit: a wave for every SIMD and more, whole units, ragged pairs
    (37, 28, 66, 64, 1), (33, 32, 128, 64, 4), (130, 16, 98, 128, 2), (3, 5, 64, 16, 2), (1100, 1, 34, 32, 1),
    # bfloat16: sums over r on the matrix units
    (33, 32, 32, 64, 1), (9, 128, 96, 64, 2), (257, 4, 256, 64, 4), (1024, 1, 64, 64, 1),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "s%d-h%d-n%d-p%d-r%d" % c)
def test_decode_step(case, fmt, dtype):
    import torch
    import state_space_sequence_exp_amd as m3
    from oracle import layer as O
    S, H, N, P, R = case
    log("cached decode %s %s %s" % (case, fmt, dtype))
    rng = np.random.default_rng(sum(case))
    v, t = decode_inputs(rng, S, H, N, P, R, dtype)
    n_slots = S + 2
    h = rows(rng, n_slots, H, N, P)
    codes, scales = cache_with(h, fmt)
    old = O.dequantise(*O.quantise(h, fmt), fmt)
    slots = rng.permutation(n_slots)[:S].astype(np.int32)
    before = raw(codes).copy()
    y = m3.decode_step_cached(codes, scales, torch.from_numpy(slots).cuda(), t["x"], t["x_prev"], t["B"],
                              t["B_prev"], t["C"], t["dt"], t["A"], t["lam"], t["theta"])
    check_decode(codes, scales, y, old, range(S), slots, v, fmt, dtype)
    others = [s for s in range(n_slots) if s not in slots]
    assert np.array_equal(raw(codes)[others], before[others])


@pytest.mark.parametrize("lam,theta", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_reduced_forms_and_identity_slots(fmt, lam, theta):
    import state_space_sequence_exp_amd as m3
    from oracle import layer as O
    S, H, N, P, R = 3, 2, 64, 64, 2
    rng = np.random.default_rng(41)
    v, t = decode_inputs(rng, S, H, N, P, R, "bf16")
    h = rows(rng, S, H, N, P)
    codes, scales = cache_with(h, fmt)
    old = O.dequantise(*O.quantise(h, fmt), fmt)
    y = m3.decode_step_cached(codes, scales, None, t["x"], t["x_prev"] if lam else None, t["B"],
                              t["B_prev"] if lam else None, t["C"], t["dt"], t["A"],
                              t["lam"] if lam else None, t["theta"] if theta else None)
    check_decode(codes, scales, y, old, range(S), list(range(S)), v, fmt, "bf16", lam=lam, theta=theta)


@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_idle_repeated_and_poisoned(fmt):
    """Idle rows of a padded batch (their y and every other slot stay), a slot
    named twice (its first entry), zero states, and a NaN that stays in its
    head and row pair."""
    import torch
    import state_space_sequence_exp_amd as m3
    from oracle import layer as O
    S, H, N, P, R = 6, 2, 32, 32, 1
    rng = np.random.default_rng(43)
    v, t = decode_inputs(rng, S, H, N, P, R, "f32")
    h = rows(rng, 5, H, N, P)
    h[3] = 0
    codes, scales = cache_with(h, fmt)
    old = O.dequantise(*O.quantise(h, fmt), fmt)
    slots = np.array([3, -1, 0, 9, 3, 1], np.int32)
    y = torch.full((S, H, R, P), 7.0, device="cuda")
    before, sb = raw(codes).copy(), scales.clone()
    m3.decode_step_cached(codes, scales, torch.from_numpy(slots).cuda(), t["x"], t["x_prev"], t["B"],
                          t["B_prev"], t["C"], t["dt"], t["A"], t["lam"], t["theta"], y=y)
    check_decode(codes, scales, y, old, [0, 2, 5], slots, v, fmt, "f32")
    assert (y[[1, 3, 4]] == 7.0).all()
    assert np.array_equal(raw(codes)[[2, 4]], before[[2, 4]]) and torch.equal(scales[[2, 4]], sb[[2, 4]])
    # y of idle rows without a given y: zeros
    y2 = m3.decode_step_cached(codes, scales, torch.from_numpy(slots).cuda(), t["x"], t["x_prev"], t["B"],
                               t["B_prev"], t["C"], t["dt"], t["A"], t["lam"], t["theta"])
    assert not y2[[1, 3, 4]].any() and y2[[0, 2, 5]].isfinite().all()
    scales[1, 1, 6] = float("nan")
    y3 = m3.decode_step_cached(codes, scales, torch.from_numpy(slots).cuda(), t["x"], t["x_prev"], t["B"],
                               t["B_prev"], t["C"], t["dt"], t["A"], t["lam"], t["theta"])
    nan = scales.isnan()
    assert nan[1, 1, 6:8].all() and nan.sum() == 2
    assert y3[5, 1].isnan().all() and not y3[5, 0].isnan().any() and not y3[[0, 2]].isnan().any()


@pytest.mark.parametrize("fmt,tol", [("int8", 2e-2), ("e4m3", 1e-1)])
def test_prefill_store_decode_load(fmt, tol):
    """A prefill handed over to the cache and decoded for 24 tokens, beside the
    same tokens on float states.  Each step's rounding is at most half a step
    of the row's largest value (1/254, 1/16 of each value) and decays with the
    state, alpha about 0.8 a step here, so the state is off by at most about 5
    steps' roundings, adding up as independent errors: 0.6% x sqrt(2.8) of a
    row's rms for int8, 2.6% x sqrt(2.8) for e4m3; held to 2% and 10%."""
    import torch
    import state_space_sequence_exp_amd as m3
    from state_space_sequence_exp_amd import inputs as I
    from gpu_util import rel_l2
    B, T, H, N, P, R = 3, 124, 2, 64, 64, 2
    inp = I.prefill_inputs(B, T, H, N, P, R, "bf16", seed=77)
    g = {k: to_gpu_storage(inp[k + "_raw"], "bf16") for k in ("x", "B", "C")}
    g.update({k: to_gpu_f32(inp[k]) for k in ("dt", "lam", "theta", "A")})
    pre = {k: g[k][:, :100].contiguous() for k in g if k != "A"}
    _, h = m3.prefill(pre["x"], pre["dt"], g["A"], pre["lam"], pre["theta"], pre["B"], pre["C"], 64)
    codes, scales = m3.state_cache(8, H, N, P, code_type(fmt))
    slots = torch.tensor([6, 0, 3], dtype=torch.int32, device="cuda")
    m3.state_store(h, codes, scales, slots)
    for s in range(100, T):
        c, p = (lambda a: a[:, s].contiguous()), (lambda a: a[:, s - 1].contiguous())
        args = (c(g["x"]), p(g["x"]), c(g["B"]), p(g["B"]), c(g["C"]), c(g["dt"]), g["A"], c(g["lam"]),
                c(g["theta"]))
        y8 = m3.decode_step_cached(codes, scales, slots, *args)
        y, h = m3.decode_step(h, *args)
    back = m3.state_load(codes, scales, slots)
    eh, ey = rel_l2(from_gpu(back), from_gpu(h)), rel_l2(from_gpu(y8), from_gpu(y))
    log("   %s after 24 tokens: state %.2e, y %.2e" % (fmt, eh, ey))
    assert eh <= tol and ey <= tol


def test_offsets_past_32_bits():
    """A pool past 2^31 codes: its last slot works like any other."""
    import torch
    import state_space_sequence_exp_amd as m3
    H, N, P = 32, 128, 64
    n = (1 << 31) // (H * N * P) + 3
    codes, scales = m3.state_cache(n, H, N, P)
    assert codes.numel() > 1 << 31
    small, ss = m3.state_cache(1, H, N, P)
    h = torch.randn(1, H, N, P, device="cuda")
    last = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(3)
    _, t = decode_inputs(rng, 1, H, N, P, 1, "bf16")
    got = []
    for c, s, at in ((codes, scales, last), (small, ss, None)):
        m3.state_store(h, c, s, at)
        y = m3.decode_step_cached(c, s, at, t["x"], t["x_prev"], t["B"], t["B_prev"], t["C"], t["dt"], t["A"],
                                  t["lam"], t["theta"])
        got.append((y, m3.state_load(c, s, at)))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert not scales[:-1].any()


def test_captured_and_replayed():
    import torch
    import state_space_sequence_exp_amd as m3
    S, H, N, P, R = 4, 2, 64, 64, 4
    rng = np.random.default_rng(51)
    _, t = decode_inputs(rng, S, H, N, P, R, "bf16")
    h = torch.from_numpy(rows(rng, S, H, N, P)).cuda()
    slots = torch.tensor([5, 1, -1, 2], dtype=torch.int32, device="cuda")
    codes, scales = m3.state_cache(6, H, N, P)
    y = torch.zeros(S, H, R, P, dtype=torch.bfloat16, device="cuda")

    def work(codes, scales, y):
        m3.state_store(h, codes, scales, slots)
        m3.decode_step_cached(codes, scales, slots, t["x"], t["x_prev"], t["B"], t["B_prev"], t["C"], t["dt"],
                              t["A"], t["lam"], t["theta"], y=y)
        return m3.state_load(codes, scales, slots)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(codes, scales, y)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        back = work(codes, scales, y)
    for k in range(4):
        h.copy_(torch.from_numpy(rows(rng, S, H, N, P)))
        slots.copy_(torch.from_numpy(rng.permutation(6)[:S].astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        c2, s2 = m3.state_cache(6, H, N, P)
        y2 = torch.zeros_like(y)
        b2 = work(c2, s2, y2)
        at = slots.long()
        assert torch.equal(back, b2) and torch.equal(y, y2)
        assert torch.equal(codes[at], c2[at]) and torch.equal(scales[at], s2[at])


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_entries_repeated_slots(fmt):
    """The first of a slot's entries is found however far ahead it lies, and
    with the y of a call on another stream zero-filled there."""
    import torch
    import state_space_sequence_exp_amd as m3
    from oracle import layer as O
    S, H, N, P = 4500, 1, 4, 16
    rng = np.random.default_rng(10)
    slots = np.arange(S, dtype=np.int32)
    for first, later in ((0, 4499), (1, 2049), (300, 301), (511, 512), (2047, 4095), (7, 520), (2500, 2600)):
        slots[later] = first
    kept = np.flatnonzero(slots == np.arange(S))
    h = rows(rng, S, H, N, P)
    codes, scales = m3.state_cache(S, H, N, P, code_type(fmt))
    t = torch.from_numpy(slots).cuda()
    m3.state_store(to_gpu_f32(h), codes, scales, t)
    c, s = O.quantise(h[kept], fmt)
    want = np.zeros((S, H, N, P), np.uint8)
    want[kept] = c
    assert np.array_equal(raw(codes), want)
    _, g = decode_inputs(rng, S, H, N, P, 1, "bf16")
    args = (g["x"], g["x_prev"], g["B"], g["B_prev"], g["C"], g["dt"], g["A"], g["lam"], g["theta"])
    both = []
    for stream in (None, torch.cuda.Stream()):
        k = (codes.clone(), scales.clone())
        torch.cuda.synchronize()
        both.append((m3.decode_step_cached(*k, t, *args, stream=stream),) + k)
        torch.cuda.synchronize()
    for a, b in zip(*both):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    idle = np.setdiff1d(np.arange(S), kept)
    assert not both[0][0][idle].any() and both[0][0][kept].flatten(1).any(1).all()
    plain = (codes.clone(), scales.clone())
    y = m3.decode_step_cached(*plain, None, *args)        # every state its own slot
    assert torch.equal(y[kept], both[0][0][kept])


@pytest.mark.parametrize("lam,theta", [(True, True), (False, False), (False, True), (True, False)])
@pytest.mark.parametrize("R", [1, 2, 4])
@pytest.mark.parametrize("fmt", FORMATS)
def test_batch_size_does_not_change_the_cache(fmt, R, lam, theta):
    """A batch large enough for the matrix units writes the codes and scales
    that small batches write, to the last bit (a zero's sign aside), with idle
    and repeated entries, zero rows and a NaN among them.  Each y is a sum of N
    fused terms in two orders, either off by at most N 2^-24 of the terms' sum
    (a term is at most |C| times its row's largest value, Q scale), and rounded
    to bfloat16 twice."""
    import torch
    import state_space_sequence_exp_amd as m3
    S, H, N, P, step = 300, 4, 64, 64, 60
    Q = 127 if fmt == "int8" else 448
    rng = np.random.default_rng(61 + R)
    _, t = decode_inputs(rng, S, H, N, P, R, "bf16")
    h = rows(rng, S, H, N, P)
    h[5] = 0
    codes, scales = cache_with(h, fmt)
    scales[7, 1, 9] = float("nan")
    slots = torch.randperm(S, dtype=torch.int32, generator=torch.Generator().manual_seed(3))
    slots[[3, 50, 299]] = torch.tensor([-1, S, -7], dtype=torch.int32)
    slots[40] = slots[20]
    slots = slots.cuda()
    got = []
    for n in (S, step):
        c, s = codes.clone(), scales.clone()
        y = torch.full((S, H, R, P), 3.0, dtype=torch.bfloat16, device="cuda")
        for i in range(0, S, n):
            k = slice(i, i + n)
            m3.decode_step_cached(c, s, slots[k], t["x"][k], t["x_prev"][k] if lam else None, t["B"][k],
                                  t["B_prev"][k] if lam else None, t["C"][k], t["dt"][k], t["A"],
                                  t["lam"][k] if lam else None, t["theta"][k] if theta else None, y=y[k])
        got.append((c, s, y.double()))
    (c0, s0, y0), (c1, s1, y1) = got
    assert torch.equal(c0.float(), c1.float()) and torch.equal(s0.nan_to_num(-1.0), s1.nan_to_num(-1.0))
    assert (s0.isnan().sum() == 2) if theta else (s0.isnan().sum() == 1)
    live = [i for i in range(S) if i not in (3, 40, 50, 299)]
    assert (y0[[3, 40, 50, 299]] == 3).all()
    size = s0[slots[live].long()].double().nan_to_num(0.0) * Q            # [live, H, N]
    terms = (t["C"][live].double().abs() * size[:, :, None]).sum(-1)      # [live, H, R]
    off = 2 * N * 2.0 ** -24 * terms[..., None]
    nan = y0[live].isnan()
    assert torch.equal(nan, y1[live].isnan()) and nan.sum() == R * P
    tol = off + 2 * 2.0 ** -8 * (y1[live].abs() + off)
    assert ((y0[live] - y1[live]).abs() <= tol)[~nan].all()
