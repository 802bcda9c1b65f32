"""CPU-only checks of the short convolution, the selective scan and the gated
feed-forward projections: every refusal comes from the host before any HIP call,
and the binding's own checks."""
import ctypes
import os

import pytest
import torch

import state_space_sequence_exp_amd as m3
from state_space_sequence_exp_amd import _binding as bnd

INV, UNS, WS, GOOD = m3.M3_ERR_INVALID_VALUE, m3.M3_ERR_NOT_SUPPORTED, m3.M3_ERR_WORKSPACE, m3.M3_SUCCESS
MIS = ctypes.c_void_p(0x100001)


def at(i, off=0):
    """The i-th array of a call, 2^40 bytes from the next."""
    return ctypes.c_void_p(((i + 1) << 40) + off)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(m3.LIB_PATH):
        from state_space_sequence_exp_amd import build
        build.build()
    return m3.load_library()


def dims(cls, base, **kw):
    s = cls(*base)
    for k, v in kw.items():
        setattr(s, k, v)
    return ctypes.byref(s)


conv_dims = lambda **kw: dims(bnd.M3ConvDims, (2, 300, 64, 4), **kw)
sel_dims = lambda **kw: dims(bnd.M3SelectDims, (2, 300, 64, 16), **kw)
ffn_dims = lambda **kw: dims(bnd.M3FfnDims, (8, 64, 96), **kw)

# x weight bias silu state_in lengths y state_out
CONV = [at(0), at(1), at(2), 1, at(3), at(4), at(5), at(6)]
# state slots n x weight bias silu y
CONV_STEP = [at(0), at(1), 5, at(2), at(3), at(4), 0, at(5)]
# x dt A B C skip z dt_bias softplus h0 lengths y h_last
SCAN = [at(0), at(1), at(2), at(3), at(4), at(5), at(6), at(7), 1, at(8), at(9), at(10), at(11)]
# h slots n x dt A B C skip z dt_bias softplus y
SCAN_STEP = [at(0), at(1), 5, at(2), at(3), at(4), at(5), at(6), at(7), at(8), at(9), 1, at(10)]
FFN = [at(i) for i in range(6)]          # x wg wu h gate up
FFN_BW = [at(i) for i in range(9)]       # dh x wg wu gate up dx dwg dwu
BIG = [at(20), 1 << 50]


def swap(args, **kw):
    a = list(args)
    for k, v in kw.items():
        a[int(k[1:])] = v
    return a


def conv(lib, args=CONV, dt=1, **kw):
    return lib.m3_causal_conv(conv_dims(**kw), dt, *args, None)


def conv_step(lib, args=CONV_STEP, dt=1, **kw):
    return lib.m3_causal_conv_step(conv_dims(**kw), dt, *args, None)


def scan(lib, args=SCAN, dt=1, ws=BIG, **kw):
    return lib.m3_selective_scan(sel_dims(**kw), dt, *args, *ws, None)


def scan_step(lib, args=SCAN_STEP, dt=1, **kw):
    return lib.m3_selective_scan_step(sel_dims(**kw), dt, *args, None)


def ffn(lib, args=FFN, dt=1, **kw):
    return lib.m3_gated_ffn(ffn_dims(**kw), dt, *args, None)


def ffn_bw(lib, args=FFN_BW, dt=1, ws=BIG, **kw):
    return lib.m3_gated_ffn_backward(ffn_dims(**kw), dt, *args, *ws, None)


@pytest.mark.parametrize("bad,code", [
    (dict(batch=-1), INV), (dict(seqlen=-1), INV), (dict(channels=0), INV), (dict(width=0), INV), (dict(width=1), UNS),
    (dict(width=5), UNS), (dict(ld_x=63), INV), (dict(ld_y=-1), INV), (dict(batch=1 << 32), UNS),
    (dict(channels=1 << 32), UNS), (dict(seqlen=1 << 32), UNS), (dict(ld_x=1 << 62), UNS), (dict(batch=1 << 30), UNS),
    (dict(batch=1 << 20, channels=1 << 20), UNS)])
def test_conv_shapes(lib, bad, code):
    assert conv(lib, **bad) == code
    if "seqlen" not in bad:
        assert conv_step(lib, swap(CONV_STEP, _2=1 << 31), **bad) in (code, UNS)


def test_conv_pointers(lib):
    assert conv(lib, dt=2) == INV and lib.m3_causal_conv(None, 1, *CONV, None) == INV
    for i in (0, 1, 2, 4, 5, 6, 7):
        assert conv(lib, swap(CONV, **{"_%d" % i: MIS})) == INV
    for i in (0, 1, 6):
        assert conv(lib, swap(CONV, **{"_%d" % i: None})) == INV
    assert conv(lib, [None] * 3 + [0] + [None] * 4, batch=0) == GOOD
    assert conv(lib, swap(CONV, _7=None), seqlen=0) == GOOD          # nothing to keep
    for i in (0, 1, 2, 4, 5):                                        # y, state_out over an input; over each other
        assert conv(lib, swap(CONV, _6=CONV[i])) == INV and conv(lib, swap(CONV, _7=CONV[i])) == INV
    assert conv(lib, swap(CONV, _7=CONV[6])) == INV
    assert conv(lib, swap(CONV, _6=at(0, 64))) == INV                # a shifted y lies over x


def test_conv_step_pointers(lib):
    for i in (0, 1, 3, 4, 5, 7):
        assert conv_step(lib, swap(CONV_STEP, **{"_%d" % i: MIS})) == INV
    for i in (0, 3, 4, 7):
        assert conv_step(lib, swap(CONV_STEP, **{"_%d" % i: None})) == INV
    assert conv_step(lib, swap(CONV_STEP, _2=-1)) == INV
    assert conv_step(lib, swap(CONV_STEP, _1=None, _2=1)) == INV     # two rows, a pool of one
    assert conv_step(lib, swap(CONV_STEP, _2=1 << 31)) == UNS
    assert conv_step(lib, swap(CONV_STEP, _2=0)) == GOOD and conv_step(lib, batch=0) == GOOD
    for i in (1, 3, 4, 5):
        assert conv_step(lib, swap(CONV_STEP, _0=CONV_STEP[i])) == INV
        assert conv_step(lib, swap(CONV_STEP, _7=CONV_STEP[i])) == INV
    # the whole pool counts: 5 x 3 x 64 bfloat16
    assert conv_step(lib, swap(CONV_STEP, _7=at(0, 5 * 3 * 64 * 2 - 2))) == INV


@pytest.mark.parametrize("bad,code", [
    (dict(batch=-1), INV), (dict(seqlen=-1), INV), (dict(channels=0), INV), (dict(dstate_n=0), INV),
    (dict(dstate_n=65), UNS), (dict(ld_x=63), INV), (dict(ld_dt=1), INV), (dict(ld_z=63), INV), (dict(ld_y=-1), INV),
    (dict(ld_b=15), INV), (dict(ld_c=15), INV), (dict(batch=1 << 32), UNS), (dict(channels=1 << 32), UNS),
    (dict(seqlen=1 << 32), UNS), (dict(ld_b=1 << 62), UNS), (dict(ld_z=1 << 62), UNS), (dict(batch=1 << 30), UNS)])
def test_scan_shapes(lib, bad, code):
    assert scan(lib, **bad) == code
    assert lib.m3_selective_scan_workspace_size(sel_dims(**bad), 1) == 0
    if "seqlen" not in bad:
        assert scan_step(lib, swap(SCAN_STEP, _2=1 << 31), **bad) in (code, UNS)


def test_scan_pointers(lib):
    assert scan(lib, dt=-1) == INV and lib.m3_selective_scan(None, 1, *SCAN, *BIG, None) == INV
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 9, 10, 11, 12):
        assert scan(lib, swap(SCAN, **{"_%d" % i: MIS})) == INV
    for i in (0, 1, 2, 3, 4, 11):
        assert scan(lib, swap(SCAN, **{"_%d" % i: None})) == INV
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 9, 10):
        assert scan(lib, swap(SCAN, _11=SCAN[i])) == INV and scan(lib, swap(SCAN, _12=SCAN[i])) == INV
    assert scan(lib, swap(SCAN, _12=SCAN[11])) == INV
    assert scan(lib, [None] * 8 + [0] + [None] * 4, batch=0) == GOOD
    assert scan(lib, swap(SCAN, _12=None), seqlen=0) == GOOD
    assert scan(lib, swap(SCAN, _12=at(8, 4)), seqlen=0) == INV       # h_last partly over h0


def test_scan_workspace(lib):
    """Few channels over many tokens are cut: their segments' states lie in the workspace."""
    need = lib.m3_selective_scan_workspace_size(sel_dims(batch=1, seqlen=8192), 1)
    assert need > 0 and need == m3.selective_scan_workspace_size(1, 8192, 64, 16, torch.bfloat16)
    assert need % (64 * 17 * 4) == 0
    kw = dict(batch=1, seqlen=8192)
    assert scan(lib, ws=[None, need], **kw) == WS and scan(lib, ws=[at(20), need - 1], **kw) == WS
    assert scan(lib, ws=[at(20, 8), need], **kw) == INV
    for i in (0, 2, 9, 11, 12):
        assert scan(lib, ws=[SCAN[i], need], **kw) == INV
    for b, t, d in ((1, 0, 64), (1, 64, 64), (1, 16384, 4096), (64, 2048, 2048)):
        assert lib.m3_selective_scan_workspace_size(sel_dims(batch=b, seqlen=t, channels=d), 1) == 0
    with pytest.raises(TypeError):
        m3.selective_scan_workspace_size(1, 8192, 64, 16, torch.float16)


def test_scan_step_pointers(lib):
    for i in (0, 1, 3, 4, 5, 6, 7, 8, 9, 10, 12):
        assert scan_step(lib, swap(SCAN_STEP, **{"_%d" % i: MIS})) == INV
    for i in (0, 3, 4, 5, 6, 7, 12):
        assert scan_step(lib, swap(SCAN_STEP, **{"_%d" % i: None})) == INV
    assert scan_step(lib, swap(SCAN_STEP, _2=-1)) == INV and scan_step(lib, swap(SCAN_STEP, _1=None, _2=1)) == INV
    assert scan_step(lib, swap(SCAN_STEP, _2=0)) == GOOD and scan_step(lib, batch=0) == GOOD
    for i in (1, 3, 4, 5, 6, 7, 8, 9, 10):
        assert scan_step(lib, swap(SCAN_STEP, _0=SCAN_STEP[i])) == INV
        assert scan_step(lib, swap(SCAN_STEP, _12=SCAN_STEP[i])) == INV
    assert scan_step(lib, swap(SCAN_STEP, _12=at(0, 5 * 64 * 16 * 4 - 2))) == INV


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), INV), (dict(channels=0), INV), (dict(hidden=0), INV), (dict(ld_x=63), INV),
    (dict(ld_wgate=63), INV), (dict(ld_wup=1), INV), (dict(ld_gate=95), INV), (dict(ld_up=-1), INV),
    (dict(ld_x=1 << 24), UNS), (dict(channels=1 << 24), UNS), (dict(hidden=1 << 33), UNS), (dict(rows=1 << 33), UNS),
    (dict(rows=1 << 30, hidden=1 << 20), UNS)])
def test_ffn_shapes(lib, bad, code):
    assert ffn(lib, **bad) == code and ffn_bw(lib, **bad) == code
    assert lib.m3_gated_ffn_backward_workspace_size(ffn_dims(**bad), 1) == 0


def test_ffn_largest_operands(lib):
    """Copies of rows that are not whole 16-byte chunks: as many as one launch takes."""
    size = lambda t, **kw: lib.m3_gated_ffn_backward_workspace_size(ffn_dims(hidden=1, **kw), t)
    big = dict(rows=4190000, ld_x=0, ld_wgate=0, ld_wup=0)
    assert size(0, channels=7701, **big) == 0 and size(0, channels=7700, **big) > 0
    assert size(1, channels=7701, **big) > 0 and size(0, channels=3901, **big) > 0
    assert ffn_bw(lib, dt=0, hidden=1, channels=7701, **big) == UNS


def test_ffn_pointers(lib):
    assert ffn(lib, dt=2) == INV and lib.m3_gated_ffn(None, 1, *FFN, None) == INV
    assert ffn(lib, ld_h=95) == INV
    for i in range(6):
        assert ffn(lib, swap(FFN, **{"_%d" % i: MIS})) == INV
        assert ffn(lib, swap(FFN, **{"_%d" % i: None})) == INV      # gate without up, too
    for o in (3, 4, 5):
        for i in range(6):
            if i != o:
                assert ffn(lib, swap(FFN, **{"_%d" % o: FFN[i]})) == INV
    assert ffn(lib, [None] * 6, rows=0) == GOOD


def test_ffn_backward_pointers(lib):
    for kw in (dict(ld_dh=95), dict(ld_dx=63), dict(ld_dwgate=1), dict(ld_dwup=63)):
        assert ffn_bw(lib, **kw) == INV
    for i in range(9):
        assert ffn_bw(lib, swap(FFN_BW, **{"_%d" % i: MIS})) == INV
        if i != 6:                                                  # dx may be absent, dwg only with dwu
            assert ffn_bw(lib, swap(FFN_BW, **{"_%d" % i: None})) == INV
    assert ffn_bw(lib, swap(FFN_BW, _6=None, _7=None, _8=None)) == GOOD
    for o in (6, 7, 8):
        for i in range(9):
            if i != o:
                assert ffn_bw(lib, swap(FFN_BW, **{"_%d" % o: FFN_BW[i]})) == INV
    need = lib.m3_gated_ffn_backward_workspace_size(ffn_dims(), 1)
    assert need == m3.gated_ffn_backward_workspace_size(8, 64, 96, torch.bfloat16) > 0
    assert ffn_bw(lib, ws=[None, need]) == WS and ffn_bw(lib, ws=[at(20), need - 1]) == WS
    assert ffn_bw(lib, ws=[at(20, 64), need]) == INV
    for i in range(9):
        assert ffn_bw(lib, ws=[FFN_BW[i], need]) == INV
    assert lib.m3_gated_ffn_backward_workspace_size(ffn_dims(rows=0), 1) == 0
    assert ffn_bw(lib, [None] * 9, rows=0) == GOOD
    assert ffn_bw(lib, swap(FFN_BW, _8=FFN_BW[7]), rows=0) == INV    # both gradients in one place


def test_binding_refuses():
    """What the wrappers refuse by themselves (CPU tensors: at the latest for that)."""
    f, h = torch.zeros, torch.bfloat16
    x, w = f(2, 6, 8), f(8, 4)
    with pytest.raises(ValueError, match="GPU"):
        m3.causal_conv(x, w)
    with pytest.raises(ValueError, match=r"\[B, T, D\]"):
        m3.causal_conv(f(6, 8), w)
    with pytest.raises(ValueError, match="weight"):
        m3.causal_conv(x, f(7, 4))
    with pytest.raises(TypeError):
        m3.causal_conv(x.half(), w)
    with pytest.raises(TypeError, match="state"):
        m3.causal_conv(x, w, state=f(2, 3, 8, dtype=h))
    with pytest.raises(ValueError, match="state"):
        m3.causal_conv(x, w, state=f(2, 4, 8))
    with pytest.raises(TypeError, match="lengths"):
        m3.causal_conv(x, w, lengths=f(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="pool"):
        m3.causal_conv_step(f(1, 3, 8), x[:, 0], w)
    with pytest.raises(ValueError, match="slots"):
        m3.causal_conv_step(f(4, 3, 8), x[:, 0], w, slots=f(3, dtype=torch.int32))
    A, B = f(8, 16), f(2, 6, 16)
    with pytest.raises(ValueError, match="GPU"):
        m3.selective_scan(x, x, A, B, B)
    with pytest.raises(ValueError, match="C:"):
        m3.selective_scan(x, x, A, B, f(2, 6, 15))
    with pytest.raises(TypeError, match="dt:"):
        m3.selective_scan(x, x.to(h), A, B, B)
    with pytest.raises(TypeError, match="A:"):
        m3.selective_scan(x, x, A.to(h), B, B)
    with pytest.raises(ValueError, match="h0"):
        m3.selective_scan(x, x, A, B, B, h0=f(2, 16, 8))
    with pytest.raises(ValueError, match="pool"):
        m3.selective_scan_step(f(1, 8, 16), x[:, 0], x[:, 0], A, B[:, 0], B[:, 0])
    g, r = f(12, 8), f(5, 8)
    with pytest.raises(ValueError, match="GPU"):
        m3.gated_ffn(r, g, g)
    with pytest.raises(ValueError, match="w_up"):
        m3.gated_ffn(r, g, f(11, 8))
    with pytest.raises(ValueError, match="together"):
        m3.gated_ffn(r, g, g, gate=f(5, 12))
    with pytest.raises(ValueError, match="wanted"):
        m3.gated_ffn_backward(f(5, 12), r, g, g, f(5, 12), f(5, 12), dx=f(5, 8), want_x=False)
    with pytest.raises(TypeError, match="gate"):
        m3.gated_ffn_backward(f(5, 12), r, g, g, f(5, 12, dtype=h), f(5, 12))
    with pytest.raises(ValueError, match="GPU"):
        m3.gated_ffn_backward(f(5, 12), r, g, g, f(5, 12), f(5, 12))
    with pytest.raises(ValueError, match="GPU"):
        m3.gated_ffn(w_up=g, w_gate=g, x=r, stream=0)
