"""GPU parity of the gated linear recurrence (m3_gated_scan, its backward and
its one-token step) against the fp64 oracle, element by element within the
oracle's running error bounds plus one rounding to the storage type."""
import numpy as np
import pytest

from layer_util import close, put, stored, torch_type
from gpu_util import from_gpu, log, to_gpu_f32

pytestmark = pytest.mark.gpu


def draw(seed, B, T, D, dtype, gate, h0=True):
    rng = np.random.default_rng(seed)
    v, t = {}, {}
    v["x"], t["x"] = stored(rng, (B, T, D), dtype)
    v["f"], t["f"] = stored(rng, (B, T, D), dtype, 2.0, 2.0)
    v["g"], t["g"] = stored(rng, (B, T, D), dtype) if gate else (None, None)
    v["dy"], t["dy"] = stored(rng, (B, T, D), dtype)
    v["h0"], t["h0"] = put(rng.standard_normal((B, D)), "f32") if h0 else (None, None)
    v["dh_last"], t["dh_last"] = put(rng.standard_normal((B, D)), "f32") if h0 else (None, None)
    return v, t


def check_all(v, t, dtype, workspace=None):
    """Forward and backward through the binding against the oracle."""
    import state_space_sequence_exp_amd as m3
    from oracle import layer as O
    y, last, states = m3.gated_scan(t["x"], t["f"], t["g"], h0=t["h0"], want_states=True,
                                    workspace=workspace)
    d = m3.gated_scan_backward(t["dy"], t["x"], t["f"], t["g"], states, dh_last=t["dh_last"],
                               workspace=workspace)
    o = O.gated_scan(v["x"], v["f"], v["g"], v["h0"])
    w = O.gated_scan_backward(v["dy"], v["x"], v["f"], v["g"], v["h0"], v["dh_last"])
    close(y, o["y"], o["e_y"], dtype, "y")
    close(last, o["h_last"], o["e_last"], "f32", "h_last")
    at = np.arange(0, v["x"].shape[1], m3._binding.SCAN_CHUNK)
    close(states, o["before"][:, at], o["e_before"][:, at], "f32", "states")
    for k in ("x", "f", "g"):
        if v[k] is not None:
            close(d[k], w["d" + k], w["e_d" + k], dtype, "d" + k)
    close(d["h0"], w["dh0"], w["e_dh0"], "f32", "dh0")
    return y, last, states, d


CASES = [
    # B, T, D: one token, one chunk and its ends, ragged chunks, odd widths, several groups of chunks
    (1, 1, 8), (2, 1, 1), (3, 2, 65), (1, 7, 130), (2, 255, 64), (2, 256, 72), (1, 257, 200),
    (2, 63, 20), (1, 64, 64), (2, 65, 128), (2, 127, 64), (2, 128, 132), (1, 129, 200), (2, 513, 33), (3, 777, 129), (1, 2100, 16), (5, 300, 256), (1, 4500, 12),
    # cut vectors at the ends of rows and of tiles, rows narrower than a vector
    (2, 70, 2), (1, 200, 3), (2, 131, 131), (1, 140, 387), (3, 65, 67), (2, 1, 5),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [False, True], ids=["plain", "gate"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "b%d-t%d-d%d" % c)
def test_forward_and_gradients(case, gate, dtype):
    B, T, D = case
    log("gated scan %s gate=%s %s" % (case, gate, dtype))
    v, t = draw(B * 1000 + T + D, B, T, D, dtype, gate)
    check_all(v, t, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_optional_arguments(dtype):
    v, t = draw(11, 2, 300, 40, dtype, False, h0=False)
    check_all(v, t, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [9, 700, 9000])
def test_slow_and_fast_gates(T, dtype):
    """Memories of one token, of thousands, and of all (w near the type's
    smallest step), channel by channel."""
    rng = np.random.default_rng(12)
    v, t = draw(13, 1, T, 24, dtype, True)
    f = rng.standard_normal((1, T, 24)) * 0.3 + np.linspace(-30, 30, 24)
    v["f"], t["f"] = put(f, dtype)
    check_all(v, t, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(40, 16), (1100, 50)])
def test_masks(T, D, dtype):
    """Padding (f = +inf, x NaN or infinite behind it) and document starts (f
    = -inf, the state before poisoned) at chunk borders, at the first and last
    token, and a sequence that is padding throughout."""
    import torch
    import state_space_sequence_exp_amd as m3
    from oracle import layer as O
    B = 4
    v, t = draw(17, B, T, D, dtype, True)
    f, x = v["f"].copy(), v["x"].copy()
    f[0, T // 2:] = np.inf                    # padded behind the first half
    x[0, T // 2:] = np.nan
    f[1] = np.inf                             # nothing but padding
    x[1, ::2] = np.inf
    for s in (0, 5, 63, 64, T // 3, 127, 128, 255, 256, T - 1):
        if s < T:
            f[2, s] = -np.inf                 # documents
    big = -np.finfo(np.float32).max if dtype == "f32" else -3.3895e38
    f[3, T // 2] = big                        # the type's lowest value acts as -inf
    f[3, T // 4] = -big
    x[3, T // 4] = np.nan
    v["f"], t["f"] = put(f, dtype)
    v["x"], t["x"] = put(x, dtype)
    y, last, states, d = check_all(v, t, dtype)
    assert torch.equal(last[1], t["h0"][1])   # padding passes the state bit for bit
    assert not d["x"][0, T // 2:].any() and not d["f"][0, T // 2:].any()
    assert not d["x"][1].any() and not d["f"][1].any()
    # a poisoned state is dropped where a document starts
    h0 = t["h0"].clone()
    h0[2] = float("nan")
    y2, last2, _ = m3.gated_scan(t["x"], t["f"], t["g"], h0=h0)
    assert torch.equal(y2[2], y[2]) and torch.equal(last2, last)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 31])
def test_slices_of_a_projection(D, dtype):
    """x, f, g as slices of one projection, gradients into slices of one
    buffer, results equal to the dense call's bit for bit; what lies between
    the slices stays."""
    import torch
    import state_space_sequence_exp_amd as m3
    B, T = 2, 400
    v, t = draw(19, B, T, D, dtype, True)
    y, last, states = m3.gated_scan(t["x"], t["f"], t["g"], h0=t["h0"], want_states=True)
    d = m3.gated_scan_backward(t["dy"], t["x"], t["f"], t["g"], states, dh_last=t["dh_last"])
    W = 4 * D + 8
    wide = torch.randn(B, T, W, device="cuda").to(torch_type(dtype))
    at = {"x": 0, "f": D, "g": 2 * D + 3, "y": 3 * D + 5}
    sl = {k: wide[..., o:o + D] for k, o in at.items()}
    for k in "xfg":
        sl[k].copy_(t[k])
    keep = wide.clone()
    y2, last2, st2 = m3.gated_scan(sl["x"], sl["f"], sl["g"], h0=t["h0"], y=sl["y"], want_states=True)
    keep[..., at["y"]:at["y"] + D] = y
    assert torch.equal(wide, keep) and torch.equal(last, last2) and torch.equal(states, st2)
    dwide = torch.full((B, T, W), 7.0, device="cuda").to(torch_type(dtype))
    ds = {k: dwide[..., at[k]:at[k] + D] for k in "xfg"}
    dyw = torch.zeros(B, T, D + 3, device="cuda").to(torch_type(dtype))
    dyw[..., 1:D + 1] = t["dy"]
    keep = dwide.clone()
    d2 = m3.gated_scan_backward(dyw[..., 1:D + 1], sl["x"], sl["f"], sl["g"], states,
                                dh_last=t["dh_last"], dx=ds["x"], df=ds["f"], dg=ds["g"])
    for k in "xfg":
        keep[..., at[k]:at[k] + D] = d[k]
    assert torch.equal(dwide, keep) and torch.equal(d["h0"], d2["h0"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pieces_equal_the_whole(dtype):
    """A prompt in two pieces, then token by token: each piece continues from
    the state before; within the bounds of the whole."""
    import state_space_sequence_exp_amd as m3
    from oracle import layer as O
    B, T, D = 2, 620, 40
    v, t = draw(23, B, T, D, dtype, True)
    o = O.gated_scan(v["x"], v["f"], v["g"], v["h0"])
    ys, h = [], t["h0"]
    for a, b in ((0, 300), (300, 612)):
        y, h, _ = m3.gated_scan(*(t[k][:, a:b].contiguous() for k in "xfg"), h0=h)
        ys.append(from_gpu(y))
    for s in range(612, T):
        y, h = m3.gated_scan_step(h, *(t[k][:, s] for k in "xfg"))
        ys.append(from_gpu(y)[:, None])
    import torch
    close(torch.from_numpy(np.concatenate(ys, 1)), o["y"], o["e_y"], dtype, "y")
    close(h, o["h_last"], o["e_last"], "f32", "h")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,D", [(1, 1), (3, 7), (4, 2048), (37, 1001)])
@pytest.mark.parametrize("gate", [False, True], ids=["plain", "gate"])
def test_step(gate, B, D, dtype):
    import torch
    import state_space_sequence_exp_amd as m3
    from oracle import layer as O
    v, t = draw(29 + B, B, 1, D, dtype, gate)
    o = O.gated_scan(v["x"], v["f"], v["g"], v["h0"])
    args = [None if t[k] is None else t[k][:, 0] for k in "xfg"]
    out = torch.full_like(t["h0"], float("nan"))
    h_in = t["h0"].clone()
    y, h = m3.gated_scan_step(h_in, *args, h_out=out)
    assert h is out and torch.equal(h_in, t["h0"])
    close(y, o["y"][:, 0], o["e_y"][:, 0], dtype, "y")
    close(h, o["h_last"], o["e_last"], "f32", "h")
    y2, h2 = m3.gated_scan_step(h_in, *args)          # in place
    assert h2 is h_in and torch.equal(h2, h) and torch.equal(y2, y)
    # strided rows
    wide = torch.zeros(B, 3 * D + 5, device="cuda").to(torch_type(dtype))
    sl = [None if a is None else wide[:, i * D + i:(i + 1) * D + i] for i, a in enumerate(args)]
    for s, a in zip(sl, args):
        if a is not None:
            s.copy_(a)
    y3, h3 = m3.gated_scan_step(t["h0"].clone(), *sl)
    assert torch.equal(h3, h) and torch.equal(y3, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty_and_zero_length(dtype):
    import torch
    import state_space_sequence_exp_amd as m3
    ty = torch_type(dtype)
    e = lambda *s: torch.empty(s, dtype=ty, device="cuda")
    y, last, st = m3.gated_scan(e(0, 5, 8), e(0, 5, 8), want_states=True)
    assert y.shape == (0, 5, 8) and last.shape == (0, 8) and st.shape == (0, 1, 8)
    h0 = torch.randn(3, 8, device="cuda")
    y, last, st = m3.gated_scan(e(3, 0, 8), e(3, 0, 8), h0=h0, want_states=True)
    assert torch.equal(last, h0) and st.shape == (3, 0, 8)
    assert not m3.gated_scan(e(3, 0, 8), e(3, 0, 8))[1].any()
    d = m3.gated_scan_backward(e(3, 0, 8), e(3, 0, 8), e(3, 0, 8), None, st, dh_last=h0)
    assert torch.equal(d["h0"], h0) and d["x"].shape == (3, 0, 8)
    y, h = m3.gated_scan_step(torch.empty(0, 8, device="cuda"), e(0, 8), e(0, 8))
    assert y.shape == (0, 8)


def test_long_state_crosses_32_bit_offsets():
    """Arrays past 2^31 elements: the last sequence's results equal those of
    the same sequence by itself."""
    import torch
    import state_space_sequence_exp_amd as m3
    B, T, D = 3, 600, 16
    ld = (1 << 31) // (2 * T) + 1000            # token rows this far apart
    gen = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.empty((B, T, ld), dtype=torch.bfloat16, device="cuda")
    assert wide.numel() > 1 << 31
    x, f = wide[..., :D], wide[..., 4096:4096 + D]
    for s in (x, f):
        s.copy_(torch.randn((B, T, D), device="cuda", generator=gen).to(torch.bfloat16) + 1)
    y, last, st = m3.gated_scan(x, f, want_states=True)
    one = slice(B - 1, B)
    y1, last1, st1 = m3.gated_scan(x[one].contiguous(), f[one].contiguous(), want_states=True)
    assert torch.equal(y[one], y1) and torch.equal(last[one], last1) and torch.equal(st[one], st1)
    dy = torch.randn((B, T, D), device="cuda", generator=gen).to(torch.bfloat16)
    dx, df = wide[..., 8192:8192 + D], wide[..., 12288:12288 + D]
    d = m3.gated_scan_backward(dy, x, f, None, st, dx=dx, df=df)
    d1 = m3.gated_scan_backward(dy[one].contiguous(), x[one].contiguous(), f[one].contiguous(), None, st1)
    assert torch.equal(dx[one], d1["x"]) and torch.equal(df[one], d1["f"])
    assert torch.equal(d["h0"][one], d1["h0"])


def test_streams_workspace_and_repeats():
    """One workspace over calls of several shapes on another stream than the
    current one; repeated calls agree bit for bit."""
    import torch
    import state_space_sequence_exp_amd as m3
    shapes = [(2, 1500, 264), (1, 5000, 64), (4, 100, 40), (2, 1500, 264)]
    need = max(m3.gated_scan_workspace_size(*s, torch.bfloat16) for s in shapes)
    ws = torch.zeros(max(need, 1), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    first = {}
    for s in shapes * 2:
        v, t = draw(sum(s), *s, "bf16", True)
        torch.cuda.synchronize()
        y, last, st = m3.gated_scan(t["x"], t["f"], t["g"], h0=t["h0"], want_states=True,
                                    workspace=ws, stream=side)
        d = m3.gated_scan_backward(t["dy"], t["x"], t["f"], t["g"], st, dh_last=t["dh_last"],
                                   workspace=ws, stream=side)
        torch.cuda.synchronize()
        got = (y, last, st, d["x"], d["f"], d["g"], d["h0"])
        if s in first:
            assert all(torch.equal(a, b) for a, b in zip(got, first[s]))
        first[s] = got


def test_captured_and_replayed():
    """Forward, backward and step in one graph, replayed with new inputs and
    eager calls between the replays."""
    import torch
    import state_space_sequence_exp_amd as m3
    B, T, D = 2, 700, 72
    v, t = draw(31, B, T, D, "bf16", True)
    need = m3.gated_scan_workspace_size(B, T, D, torch.bfloat16)
    ws = torch.zeros(max(need, 1), dtype=torch.uint8, device="cuda")
    h = torch.empty(B, D, device="cuda")

    def work(ws):
        y, last, st = m3.gated_scan(t["x"], t["f"], t["g"], h0=t["h0"], want_states=True, workspace=ws)
        d = m3.gated_scan_backward(t["dy"], t["x"], t["f"], t["g"], st, dh_last=t["dh_last"], workspace=ws)
        y1, h1 = m3.gated_scan_step(last, t["x"][:, 0], t["f"][:, 0], t["g"][:, 0], h_out=h)
        return [y, last, st, d["x"], d["f"], d["g"], d["h0"], y1, h1]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work(ws)
    for k in range(4):
        _, n = draw(40 + k, B, T, D, "bf16", True)
        for q in ("x", "f", "g", "dy", "h0", "dh_last"):
            t[q].copy_(n[q])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for a, b in zip(got, work(None)):
            assert torch.equal(a, b)


def busy():
    """Work that keeps the current stream from what is enqueued behind it for
    some milliseconds."""
    import torch
    a = torch.zeros(4096, 4096, device="cuda")
    for _ in range(16):
        a = a @ a
    return a


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_own_allocations_are_on_the_call_s_stream(handle):
    """With `stream` the workspace that a call makes and zero-fills by itself
    is ordered with its kernels, not with the current stream's work."""
    import torch
    import state_space_sequence_exp_amd as m3
    _, t = draw(77, 3, 1100, 136, "bf16", True)
    args = (t["x"], t["f"], t["g"])
    want = m3.gated_scan(*args, h0=t["h0"], want_states=True)
    wd = m3.gated_scan_backward(t["dy"], *args, want[2], dh_last=t["dh_last"])
    side = torch.cuda.Stream()
    at = side.cuda_stream if handle else side
    dirty = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del dirty
    keep = busy()
    got = m3.gated_scan(*args, h0=t["h0"], want_states=True, stream=at)
    gd = m3.gated_scan_backward(t["dy"], *args, got[2], dh_last=t["dh_last"], stream=at)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(gd[k], wd[k]) for k in wd)
    torch.cuda.synchronize()
    del keep
    base = m3.gated_scan(*args, h0=t["h0"], stream=0)     # the default stream's handle
    torch.cuda.synchronize()
    assert torch.equal(base[0], want[0])


@pytest.mark.parametrize("ticket", [1 << 20, 1])
def test_dirty_workspace_is_reported(ticket):
    """A chain counter that is not zero on entry: the workgroups past the
    chain's end compute nothing and set error word 2, those inside it wait for
    a place that nobody takes until they see that word, and everything ends.  A
    zero-filled workspace serves again."""
    import torch
    import state_space_sequence_exp_amd as m3
    B, T, D = 1, 200, 64
    v, t = draw(78, B, T, D, "f32", False)
    ws = torch.zeros(m3.gated_scan_workspace_size(B, T, D, torch.float32), dtype=torch.uint8, device="cuda")
    ws[256:260].view(torch.int32)[0] = ticket
    y, _, st = m3.gated_scan(t["x"], t["f"], want_states=True, workspace=ws)
    assert m3.prefill_workspace_error(ws, clear=True) == 2
    if ticket == 1:
        assert y[:, 128:].isnan().all()
    ws.zero_()
    y, _, st = m3.gated_scan(t["x"], t["f"], want_states=True, workspace=ws)
    assert m3.prefill_workspace_error(ws) == 0 and not ws.any()
    assert torch.equal(y, m3.gated_scan(t["x"], t["f"])[0])


def test_two_calls_at_once():
    """Calls that overlap on two streams, each with its own workspace."""
    import torch
    import state_space_sequence_exp_amd as m3
    shapes = [(2, 3000, 520), (1, 6000, 200)]
    ins = [draw(90 + i, *s, "bf16", True)[1] for i, s in enumerate(shapes)]
    want = [m3.gated_scan(t["x"], t["f"], t["g"], want_states=True) for t in ins]
    wd = [m3.gated_scan_backward(t["dy"], t["x"], t["f"], t["g"], w[2]) for t, w in zip(ins, want)]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, (t, s) in enumerate(zip(ins, streams)):
            o = m3.gated_scan(t["x"], t["f"], t["g"], want_states=True, stream=s)
            d = m3.gated_scan_backward(t["dy"], t["x"], t["f"], t["g"], o[2], stream=s)
            got[i].append((o, d))
    torch.cuda.synchronize()
    for i in range(2):
        for o, d in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(o, want[i]))
            assert all(torch.equal(d[k], wd[i][k]) for k in d)


def test_graphs_share_a_workspace():
    """Two captured graphs and eager calls of other shapes on one workspace,
    one after the other."""
    import torch
    import state_space_sequence_exp_amd as m3
    shapes = [(2, 900, 136), (1, 2500, 72)]
    ins = [draw(95 + i, *s, "bf16", True)[1] for i, s in enumerate(shapes)]
    need = max(m3.gated_scan_workspace_size(*s, torch.bfloat16) for s in shapes)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def work(t):
        y, last, st = m3.gated_scan(t["x"], t["f"], t["g"], want_states=True, workspace=ws)
        d = m3.gated_scan_backward(t["dy"], t["x"], t["f"], t["g"], st, workspace=ws)
        return [y, last, st, d["x"], d["f"], d["g"], d["h0"]]

    want = [[o.clone() for o in work(t)] for t in ins]
    torch.cuda.synchronize()
    graphs = []
    for t in ins:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = work(t)
        graphs.append((graph, out))
    for k in range(4):
        for i, (graph, out) in enumerate(graphs):
            for o in out:
                o.zero_()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
            assert all(torch.equal(a, b) for a, b in zip(work(ins[1 - i]), want[1 - i]))
        torch.cuda.synchronize()
    assert not ws.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_single_tokens_of_long_sequences(dtype):
    """One token of every sequence, read out of arrays whose sequences lie
    further apart than a chunk's rows may."""
    import torch
    import state_space_sequence_exp_amd as m3
    B, T, D = 3, 4200, 1001
    assert T * D > 1 << 22
    _, t = draw(97, B, 1, D, dtype, True)
    wide = [torch.zeros(B, T, D, dtype=torch_type(dtype), device="cuda") for _ in range(3)]
    for w, k in zip(wide, "xfg"):
        w[:, 4100] = t[k][:, 0]
    want = m3.gated_scan(t["x"], t["f"], t["g"], h0=t["h0"], want_states=True)
    got = m3.gated_scan(*(w[:, 4100:4101] for w in wide), h0=t["h0"], want_states=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    d = m3.gated_scan_backward(t["dy"], *(w[:, 4100:4101] for w in wide), got[2])
    e = m3.gated_scan_backward(t["dy"], t["x"], t["f"], t["g"], want[2])
    assert all(torch.equal(d[k], e[k]) for k in d)
    y, h = m3.gated_scan_step(t["h0"].clone(), *(w[:, 4100] for w in wide))
    z, k = m3.gated_scan_step(t["h0"].clone(), t["x"][:, 0], t["f"][:, 0], t["g"][:, 0])
    assert torch.equal(y, z) and torch.equal(h, k)
