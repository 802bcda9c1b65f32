"""CPU-only checks of the layer operators' entry points: every refusal comes
from the host before any HIP call, and the binding's own checks."""
import ctypes
import os

import pytest
import torch

import state_space_sequence_exp_amd as m3
from state_space_sequence_exp_amd import _binding as bnd

OK = ctypes.c_void_p(0x100000)
MIS = ctypes.c_void_p(0x100001)
HALF = ctypes.c_void_p(0x100008)   # 8-byte aligned
INV, UNS, WS = m3.M3_ERR_INVALID_VALUE, m3.M3_ERR_NOT_SUPPORTED, m3.M3_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(m3.LIB_PATH):
        from state_space_sequence_exp_amd import build
        build.build()
    return m3.load_library()


def scan_dims(b=2, t=300, d=64, **ld):
    s = bnd.M3ScanDims(b, t, d)
    for k, v in ld.items():
        setattr(s, k, v)
    return s


BAD_SCAN = [(dict(b=-1), INV), (dict(t=-1), INV), (dict(d=0), INV), (dict(ld_x=63), INV), (dict(ld_f=-1), INV),
            (dict(ld_g=1), INV), (dict(ld_y=63), INV), (dict(t=1 << 40), UNS), (dict(d=1 << 40), UNS),
            (dict(b=1 << 33), UNS), (dict(b=1 << 30), UNS), (dict(ld_x=1 << 62), UNS), (dict(ld_y=1 << 22), UNS)]


@pytest.mark.parametrize("bad,code", BAD_SCAN)
def test_scan_shapes(lib, bad, code):
    d = scan_dims(**bad)
    ws, n = OK, 1 << 40
    assert lib.m3_gated_scan(ctypes.byref(d), 0, *[OK] * 7, ws, n, None) == code
    assert lib.m3_gated_scan_backward(ctypes.byref(d), 0, *[OK] * 10, ws, n, None) == code
    assert lib.m3_gated_scan_workspace_size(ctypes.byref(d), 0) == 0
    if "t" not in bad and bad.get("ld_y") != 1 << 22:      # single tokens may lie that far apart
        assert lib.m3_gated_scan_step(ctypes.byref(d), 0, *[OK] * 6, None) == code


@pytest.mark.parametrize("b,t,d", [(1 << 23, 0, 64), (1 << 22, 64, 64), (1 << 17, 1, 1 << 12), (1, 1 << 29, 64)])
def test_scan_launch_size(lib, b, t, d):
    """No launch has 2^32 threads or more, whatever the memory would hold."""
    dims = ctypes.byref(scan_dims(b, t, d))
    assert lib.m3_gated_scan(dims, 1, *[OK] * 7, OK, 1 << 62, None) == UNS
    assert lib.m3_gated_scan_backward(dims, 1, *[OK] * 10, OK, 1 << 62, None) == UNS
    assert lib.m3_gated_scan_workspace_size(dims, 1) == 0
    if b > 1:
        assert lib.m3_gated_scan_step(ctypes.byref(scan_dims(1 << 23, 1, d)), 1, *[OK] * 6, None) == UNS


@pytest.mark.parametrize("t", [-1, 0, 1 << 40])
def test_step_ignores_the_length(lib, t):
    """The single-token form does not look at seqlen: what it refuses here is
    the pointer, and an empty batch passes."""
    args = [OK] * 5 + [MIS, None]
    assert lib.m3_gated_scan_step(ctypes.byref(scan_dims(t=t)), 0, *args) == INV
    assert lib.m3_gated_scan_step(ctypes.byref(scan_dims(t=t, b=0)), 0, *args) == m3.M3_SUCCESS


def test_scan_pointers(lib):
    d = scan_dims()
    ws = [OK, 1 << 40, None]
    call = lambda p, dt=0, dd=d, w=ws: lib.m3_gated_scan(ctypes.byref(dd), dt, *p, *w)
    assert call([OK] * 7, dt=2) == INV
    assert lib.m3_gated_scan(None, 0, *[OK] * 7, *ws) == INV
    for i in range(7):                    # x f g h0 y h_last states
        p = [OK] * 7
        p[i] = MIS
        assert call(p) == INV
        if i in (0, 1, 4):
            p[i] = None
            assert call(p) == INV
    need = lib.m3_gated_scan_workspace_size(ctypes.byref(d), 0)
    # 2 sequences x 1 tile of 64 floats: 256 bytes, their counters (256), 5
    # tiles of 64 tokens with a map and a state each, 64 words of 8 bytes
    assert need == 256 + 256 + 2 * 5 * 2 * 64 * 8
    # bfloat16 tiles are 128 channels wide
    assert lib.m3_gated_scan_workspace_size(ctypes.byref(scan_dims(t=4200, d=129)), 1) == \
        256 + 256 + 4 * 66 * 2 * 128 * 8
    assert call([OK] * 7, w=[None, need, None]) == WS and call([OK] * 7, w=[OK, need - 1, None]) == WS
    assert call([OK] * 7, w=[HALF, need, None]) == INV
    for t in (0, 1, 64):                  # one tile hands nothing on
        assert lib.m3_gated_scan_workspace_size(ctypes.byref(scan_dims(t=t)), 0) == 0
    bw = lambda p, dd=d: lib.m3_gated_scan_backward(ctypes.byref(dd), 1, *p, *ws)
    for i in range(10):                   # dy x f g states dh_last dx df dg dh0
        p = [OK] * 10
        p[i] = MIS
        assert bw(p) == INV
        if i not in (5, 9):               # dh_last, dh0 are optional; g and dg go together
            p[i] = None
            assert bw(p) == INV
    assert bw([OK] * 10, scan_dims(ld_dx=63)) == INV
    assert lib.m3_gated_scan_backward(ctypes.byref(d), 1, *[OK] * 10, OK, need - 1, None) == WS
    assert call([None] * 7, dd=scan_dims(b=0)) == m3.M3_SUCCESS
    assert bw([None] * 10, scan_dims(b=0)) == m3.M3_SUCCESS
    st = lambda p, dd=d: lib.m3_gated_scan_step(ctypes.byref(dd), 0, *p, None)
    for i in range(6):                    # h_in h_out x f g y
        p = [OK] * 6
        p[i] = MIS
        assert st(p) == INV
        if i != 4:
            p[i] = None
            assert st(p) == INV
    p = [OK] * 6
    p[1] = ctypes.c_void_p(0x100000 + 64)   # partly over h_in
    assert st(p) == INV
    assert st([None] * 6, scan_dims(b=0)) == m3.M3_SUCCESS


def norm_dims(m=4, d=64, **ld):
    s = bnd.M3NormDims(m, d)
    for k, v in ld.items():
        setattr(s, k, v)
    return s


def test_layer_norm(lib):
    def fwd(d=norm_dims(), p=None, eps=1e-5, dt=0):
        p = p or [OK, ctypes.c_void_p(0x200000), OK, OK, ctypes.c_void_p(0x300000), ctypes.c_void_p(0x400000), OK, OK]
        return lib.m3_layer_norm(ctypes.byref(d), dt, *p[:4], eps, *p[4:], None)
    for bad, code in ((dict(m=-1), INV), (dict(d=0), INV), (dict(d=16385), UNS), (dict(ld_x=63), INV),
                      (dict(ld_residual=5), INV), (dict(ld_sum=5), INV), (dict(ld_y=-64), INV),
                      (dict(m=1 << 33), UNS)):
        assert fwd(norm_dims(**bad)) == code, bad
    assert fwd(dt=5) == INV and fwd(eps=-1.0) == INV and fwd(eps=float("nan")) == INV
    base = [OK, ctypes.c_void_p(0x200000), OK, OK, ctypes.c_void_p(0x300000), ctypes.c_void_p(0x400000), OK, OK]
    for i in range(8):                    # x residual weight bias y sum mean rstd
        p = list(base)
        p[i] = MIS
        assert fwd(p=p) == INV
        if i in (0, 2, 4):
            p[i] = None
            assert fwd(p=p) == INV
    p = list(base)
    p[5] = p[4]                           # y and the sum in one place
    assert fwd(p=p) == INV
    p = list(base)
    p[4] = p[0]                           # in place, but another distance of rows
    assert fwd(norm_dims(ld_y=65), p) == INV
    p[4], p[5] = base[4], base[1]
    assert fwd(norm_dims(ld_sum=65), p) == INV
    assert fwd(norm_dims(m=0), [None] * 8) == m3.M3_SUCCESS

    need = lib.m3_layer_norm_backward_workspace_size(ctypes.byref(norm_dims()), 0)
    assert need > 0 and lib.m3_layer_norm_backward_workspace_size(ctypes.byref(norm_dims(d=1 << 20)), 0) == 0
    base = [OK, OK, OK, OK, OK, ctypes.c_void_p(0x200000), ctypes.c_void_p(0x300000), OK, OK]

    def bwd(d=norm_dims(), p=base, ws=OK, n=need):
        return lib.m3_layer_norm_backward(ctypes.byref(d), 0, *p, ws, n, None)
    for i in range(9):                    # dy s weight mean rstd dsum dx dweight dbias
        p = list(base)
        p[i] = MIS
        assert bwd(p=p) == INV
        if i not in (5, 8):
            p[i] = None
            assert bwd(p=p) == INV
    assert bwd(ws=None) == WS and bwd(n=need - 1) == WS and bwd(ws=HALF) == INV
    p = list(base)
    p[6] = p[5]
    assert bwd(norm_dims(ld_dx=70), p) == INV
    for k in ("ld_sum", "ld_dy", "ld_dsum", "ld_dx"):
        assert bwd(norm_dims(**{k: 3})) == INV


def cdims(b=2, h=2, p=64, n=64, r=2):
    return bnd.M3Dims(b, 1, h, p, n, r)


BAD_CACHE = [(dict(n=15), INV), (dict(n=0), INV), (dict(h=0), INV), (dict(b=-1), INV), (dict(p=24), UNS),
             (dict(n=258), UNS), (dict(p=128, n=256), UNS), (dict(b=1 << 33), UNS), (dict(b=1 << 20, h=1 << 20), UNS)]


@pytest.mark.parametrize("bad,code", BAD_CACHE)
def test_cache_shapes(lib, bad, code):
    d = ctypes.byref(cdims(**bad))
    assert lib.m3_state_store(d, 0, OK, OK, OK, OK, 9, None) == code
    assert lib.m3_state_load(d, 0, 0, OK, OK, OK, 9, OK, None) == code
    assert lib.m3_decode_step_cached(d, 0, 0, OK, OK, OK, 9, *[OK] * 10, None) == code


def test_cache_launch_size(lib):
    d = ctypes.byref(cdims(b=1 << 12, h=1 << 12))
    assert lib.m3_state_store(d, 0, OK, OK, OK, OK, 9, None) == UNS
    assert lib.m3_state_load(d, 0, 0, OK, OK, OK, 9, OK, None) == UNS
    assert lib.m3_decode_step_cached(d, 0, 0, OK, OK, OK, 9, *[OK] * 10, None) == UNS


def test_cache_pointers(lib):
    d = ctypes.byref(cdims())
    store = lambda h=OK, c=OK, s=OK, at=OK, n=9, code=0: lib.m3_state_store(d, code, h, c, s, at, n, None)
    assert store(code=2) == INV and store(n=-1) == INV and store(n=1 << 33) == UNS
    assert store(at=None, n=1) == INV          # two states, one slot
    assert store(h=HALF) == INV and store(c=HALF) == INV and store(s=MIS) == INV and store(at=MIS) == INV
    assert store(h=None) == INV and store(c=None) == INV and store(s=None) == INV
    assert store(n=0) == m3.M3_SUCCESS
    load = lambda dt=0, c=OK, s=OK, at=OK, n=9, h=OK, code=0: lib.m3_state_load(d, code, dt, c, s, at, n, h, None)
    assert load(dt=2) == INV and load(code=-1) == INV and load(h=None) == INV and load(h=HALF) == INV
    assert load(c=None) == INV and load(s=MIS) == INV and load(at=None, n=1) == INV
    dec = lambda p, dt=0, code=0, dd=d, n=9: lib.m3_decode_step_cached(dd, dt, code, *p[:3], n, *p[3:], None)
    base = [OK] * 13     # codes scales slots | x_t x_prev B_t B_prev C_t dt A lam theta y_t
    assert dec(base, dt=9) == INV and dec(base, code=9) == INV
    for i in range(13):
        p = list(base)
        p[i] = MIS
        assert dec(p) == INV, i
        if i not in (2, 10, 11):
            p[i] = None
            assert dec(p) == INV, i
    p = list(base)
    p[2] = None
    assert dec(p, n=1) == INV
    assert dec(base, dd=ctypes.byref(cdims(r=3))) == UNS
    assert dec(base, dd=ctypes.byref(cdims(r=0))) == INV
    assert dec([None] * 13, dd=ctypes.byref(cdims(b=0))) == m3.M3_SUCCESS
    assert dec(base, n=0) == m3.M3_SUCCESS


def test_binding_refuses():
    """The binding's own checks, on CPU tensors (a call that passes them all is
    refused for not being on a GPU)."""
    x = torch.zeros(2, 5, 8)
    with pytest.raises(ValueError, match="GPU"):
        m3.gated_scan(x, x)
    with pytest.raises(TypeError):
        m3.gated_scan(x.half(), x.half())
    with pytest.raises(TypeError):
        m3.gated_scan(x, x.bfloat16())
    with pytest.raises(ValueError):
        m3.gated_scan(x, x[:, :4])
    with pytest.raises(ValueError):
        m3.gated_scan(x[0], x[0])
    with pytest.raises(ValueError, match="last dimension"):
        m3.gated_scan(torch.zeros(2, 5, 16)[..., ::2], x)
    with pytest.raises(ValueError, match="one distance"):
        m3.gated_scan(torch.zeros(2, 9, 8)[:, :5], x)           # a gap between the sequences
    with pytest.raises(ValueError, match="one distance"):
        m3.gated_scan(torch.zeros(1, 5, 8).expand(2, 5, 8), x)  # a broadcast input
    with pytest.raises(ValueError):
        m3.gated_scan(x, x, h0=torch.zeros(2, 7))
    with pytest.raises(ValueError):
        m3.gated_scan_backward(x, x, x, None, torch.zeros(2, 2, 8))
    with pytest.raises(ValueError):
        m3.gated_scan_backward(x, x, x, None, torch.zeros(2, 1, 8), dg=x)
    with pytest.raises(ValueError):
        m3.gated_scan_step(torch.zeros(2, 8), x, x)
    with pytest.raises(ValueError, match="GPU"):
        m3.gated_scan(x, x, stream=0)
    with pytest.raises(ValueError, match="GPU"):
        m3.gated_scan(x=x, f=x, stream=0)
    w = torch.ones(8)
    with pytest.raises(ValueError, match="GPU"):
        m3.layer_norm(x, w)
    with pytest.raises(TypeError):
        m3.layer_norm(x, w.bfloat16())
    with pytest.raises(ValueError):
        m3.layer_norm(x, torch.ones(7))
    with pytest.raises(ValueError):
        m3.layer_norm(x, w, residual=x[:1])
    with pytest.raises(ValueError):
        m3.layer_norm_backward(x, x, w, torch.zeros(10), torch.zeros(2, 5))
    c, s = m3.state_cache(4, 2, 16, 16, device="cpu")
    h = torch.zeros(4, 2, 16, 16)
    with pytest.raises(ValueError, match="GPU"):
        m3.state_store(h, c, s)
    with pytest.raises(TypeError):
        m3.state_store(h, c.view(torch.uint8), s)
    with pytest.raises(TypeError):
        m3.state_cache(4, 2, 16, 16, torch.float32, device="cpu")
    with pytest.raises(TypeError):
        m3.state_store(h, c, s, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        m3.state_store(h[:3], c, s, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        m3.state_load(c, s[:, :1])
    with pytest.raises(TypeError):
        m3.state_load(c, s, dtype=torch.float16)
    t = torch.zeros(4, 2, 1, 16)
    z = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="required with lam"):
        m3.decode_step_cached(c, s, None, t, None, t, None, t, z, torch.zeros(2), z, None)
    with pytest.raises(ValueError):
        m3.decode_step_cached(c, s, torch.zeros(3, dtype=torch.int32), t, t, t, t, t, z, torch.zeros(2), z, None)


def at(address):
    return ctypes.c_void_p(address)


def apart(n, first=0x10000000):
    """n addresses 16 MiB apart."""
    return [first + (i << 24) for i in range(n)]


def refused(call, args, i, j, shift, **dims):
    p = list(args)
    p[i] = args[j] + shift
    return call([at(a) for a in p], **dims) == INV


def test_scan_overlaps(lib):
    """An output over an input or another output is refused before anything is
    enqueued; slices of one wider array are told apart by the length of a row."""
    B, T, D = 2, 300, 64
    fwd = lambda p, **ld: lib.m3_gated_scan(ctypes.byref(scan_dims(B, T, D, **ld)), 0, *p, OK, 1 << 40, None)
    p = apart(7)                          # x f g h0 y h_last states
    for i, j in ((4, 0), (4, 1), (4, 2)):
        for shift in (0, 4, -4, 4 * (B * T * D - 1), -4 * (B * T * D - 1)):
            assert refused(fwd, p, i, j, shift)
    for shift in (0, 4, 4 * (B * D - 1)):
        assert refused(fwd, p, 5, 3, shift)
    wide = dict(ld_x=3 * D, ld_y=3 * D)   # x, then y: D, 2 D elements on
    for shift in (0, 4 * (D - 1), 4 * (2 * D + 1), 4 * (7 * 3 * D - 1), -4 * (D - 1), -4 * (2 * D + 1)):
        assert refused(fwd, p, 4, 0, shift, **wide)
    assert refused(fwd, p, 4, 0, 4 * D, ld_x=3 * D, ld_y=2 * D)
    bwd = lambda p: lib.m3_gated_scan_backward(ctypes.byref(scan_dims(B, T, D)), 0, *p, OK, 1 << 40, None)
    p = apart(10)                         # dy x f g states dh_last dx df dg dh0
    for i in (6, 7, 8):
        for j in (0, 1, 2, 3, 6, 7, 8):
            if i != j:
                assert refused(bwd, p, i, j, 0) and refused(bwd, p, i, j, 4 * (B * T * D - 1))
    assert refused(bwd, p, 9, 5, 0) and refused(bwd, p, 9, 5, -4)
    step = lambda p: lib.m3_gated_scan_step(ctypes.byref(scan_dims(B, 1, D)), 0, *p, None)
    p = apart(6)                          # h_in h_out x f g y
    for j in (2, 3, 4):
        assert refused(step, p, 5, j, 0) and refused(step, p, 5, j, 4 * (2 * D - 1))


def test_norm_and_cache_overlaps(lib):
    M, D = 4, 64
    fwd = lambda p, **ld: lib.m3_layer_norm(ctypes.byref(norm_dims(M, D, **ld)), 0, *p[:4], 1e-5, *p[4:], None)
    p = apart(8)                          # x residual weight bias y sum mean rstd
    for i, j in ((4, 0), (4, 1), (5, 0), (5, 1), (4, 5)):
        for shift in (4, -4, 4 * (M * D - 1)):
            assert refused(fwd, p, i, j, shift)
    assert refused(fwd, p, 4, 5, 0)
    assert refused(fwd, p, 4, 0, 4 * (D - 1), ld_x=2 * D, ld_y=2 * D)
    need = lib.m3_layer_norm_backward_workspace_size(ctypes.byref(norm_dims(M, D)), 0)
    bwd = lambda p: lib.m3_layer_norm_backward(ctypes.byref(norm_dims(M, D)), 0, *p, OK, need, None)
    p = apart(9)                          # dy s weight mean rstd dsum dx dweight dbias
    for j, shift in ((0, 4), (5, -4), (1, 0), (1, 4 * D)):
        assert refused(bwd, p, 6, j, shift)
    dec = lambda p: lib.m3_decode_step_cached(ctypes.byref(cdims()), 0, 0, *p[:3], 9, *p[3:], None)
    p = apart(13)                         # codes scales slots | x_t x_prev B_t B_prev C_t dt A lam theta y_t
    for j in (3, 4, 5, 6, 7):
        assert refused(dec, p, 12, j, 0) and refused(dec, p, 12, j, 4 * (2 * 2 * 2 * 64 - 1))
