"""The gated recurrence where a state is not a number, or forgotten to the last
bit: only a gate of -inf drops a state, and what a channel holds does not
depend on the channels beside it."""
import numpy as np
import pytest

from layer_util import close, put
from gpu_util import from_gpu

pytestmark = pytest.mark.gpu


def same(a, b):
    """Equal to the last bit, any NaN equal to any other."""
    import torch
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


def both(t):
    import state_space_sequence_exp_amd as m3
    y, last, st = m3.gated_scan(t["x"], t["f"], t["g"], h0=t["h0"], want_states=True)
    d = m3.gated_scan_backward(t["dy"], t["x"], t["f"], t["g"], st)
    return dict(y=y, last=last, st=st, dx=d["x"], df=d["f"], dh0=d["h0"], **({} if t["g"] is None else {"dg": d["g"]}))


def draw(seed, T, D, dtype, gate):
    rng = np.random.default_rng(seed)
    v = dict(x=rng.uniform(1, 2, (1, T, D)), f=rng.standard_normal((1, T, D)) * 2,
             g=rng.standard_normal((1, T, D)) if gate else None, dy=rng.standard_normal((1, T, D)),
             h0=rng.standard_normal((1, D)))
    return v


def up(v, dtype):
    out, t = {}, {}
    for k, a in v.items():
        out[k], t[k] = (None, None) if a is None else put(a, "f32" if k == "h0" else dtype)
    return out, t


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [False, True], ids=["plain", "gate"])
@pytest.mark.parametrize("T", [30, 300])
def test_a_lost_state_stays_lost(T, gate, dtype):
    """A NaN state is NaN at every later token, however small the gates' product
    (the states are forgotten in float after a few tokens of f = -60) and
    whatever the output gate (0 at some tokens), until a gate of -inf drops it;
    a channel of masks beside it changes nothing."""
    D = 64
    v = draw(3, T, D, dtype, gate)
    v["f"][:, :, :8] = -60.0
    v["h0"][:, :8] = np.nan
    if gate:
        v["g"][:, ::3, :8] = 0.0
    v["f"][0, T // 2, 4:8] = -np.inf                  # four of them start afresh
    _, t = up(v, dtype)
    got = both(t)
    y = from_gpu(got["y"])
    assert np.isnan(y[0, :, :4]).all() and np.isnan(y[0, :T // 2, 4:8]).all()
    assert np.isfinite(y[0, T // 2:, 4:]).all() and np.isfinite(y[0, :, 8:]).all()
    last = from_gpu(got["last"])
    assert np.isnan(last[0, :4]).all() and np.isfinite(last[0, 4:]).all()
    # masks in other channels of the same waves
    w = {k: None if a is None else a.copy() for k, a in v.items()}
    w["f"][0, 1::5, 8:] = np.inf
    w["f"][0, 3::7, 8:] = -np.inf
    _, s = up(w, dtype)
    other = both(s)
    for k in got:
        assert same(got[k][..., :8], other[k][..., :8]), k
    # and without any mask in the first four
    w = {k: None if a is None else a[..., :4].copy() for k, a in v.items()}
    _, s = up(w, dtype)
    alone = both(s)
    for k in got:
        assert same(got[k][..., :4], alone[k]), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [1, 6, 63, 64, 128, 255])
def test_a_nan_gate_before_a_document(at, dtype):
    """A gate that is NaN spoils its document from there on, forward, and all
    before it in the gradients, but neither the next document nor the next one's
    gradients."""
    from oracle import layer as O
    T, D = 300, 40
    v = draw(5, T, D, dtype, True)
    v["f"][0, at, ::2] = np.nan
    v["f"][0, at + 1] = -np.inf
    v, t = up(v, dtype)
    got = both(t)
    after = slice(at + 1, T)
    o = O.gated_scan(v["x"][:, after], v["f"][:, after], v["g"][:, after])
    w = O.gated_scan_backward(v["dy"][:, after], v["x"][:, after], v["f"][:, after], v["g"][:, after])
    close(got["y"][:, after], o["y"], o["e_y"], dtype, "y")
    close(got["last"], o["h_last"], o["e_last"], "f32", "h_last")
    for k in ("dx", "df", "dg"):
        close(got[k][:, after], w[k], w["e_" + k], dtype, k)
    y, dh0 = from_gpu(got["y"]), from_gpu(got["dh0"])
    assert np.isnan(y[0, at, ::2]).all() and np.isfinite(y[0, :at]).all() and np.isfinite(y[0, at, 1::2]).all()
    assert np.isnan(dh0[0, ::2]).all() and np.isfinite(dh0[0, 1::2]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [40, 700])
def test_a_large_state_is_forgotten(T, dtype):
    """What underflow leaves of a state of 1e34 after gates of -20 is within the
    float evaluation's bound: a product of gates is held down to 2^-149."""
    from oracle import layer as O
    v = draw(7, T, 24, dtype, False)
    v["f"][:] = -20.0
    v["h0"][:] = 1e34
    v, t = up(v, dtype)
    got = both(t)
    o = O.gated_scan(v["x"], v["f"], None, v["h0"])
    close(got["y"], o["y"], o["e_y"], dtype, "y")
    close(got["last"], o["h_last"], o["e_last"], "f32", "h_last")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_arrays_between_each_other_s_rows(dtype):
    """A step whose y, x and f are slices of one wide array, and whose state lies
    dense between two of its rows: nothing overlaps, nothing is refused, and the
    results are those of arrays apart."""
    import torch
    import state_space_sequence_exp_amd as m3
    B, D = 2, 24
    ty = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(8)
    wide = torch.randn(B, 12 * D, device="cuda", generator=gen).to(ty)
    y, x, f = (wide[:, i * D:(i + 1) * D] for i in range(3))
    h = wide.view(-1)[4 * D:4 * D + B * D * 4 // wide.element_size()].view(torch.float32).view(B, D)
    h.copy_(torch.randn(B, D, device="cuda", generator=gen))
    keep = wide.clone()
    want_y, want_h = m3.gated_scan_step(h.clone(), x.clone(), f.clone())
    got_y, got_h = m3.gated_scan_step(h, x, f, y=y)
    assert got_y is y and got_h is h and torch.equal(y, want_y) and torch.equal(h, want_h)
    at = slice(4 * D, 4 * D + B * D * 4 // wide.element_size())
    keep[:, :D] = y
    keep.view(-1)[at] = wide.view(-1)[at]
    bits = lambda a: a.view(torch.uint8)              # (halves of a state may read as NaN in the storage type)
    assert torch.equal(bits(wide), bits(keep))
    for bad in (x, f, h if dtype == "f32" else x):
        with pytest.raises(m3.M3Error):
            m3.gated_scan_step(h, x, f, y=bad)
