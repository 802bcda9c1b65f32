"""CPU-only checks that the layer operators refuse an output that lies over an
input, another output or the workspace, the float arrays among them, before
any HIP call."""
import ctypes
import os

import pytest

import state_space_sequence_exp_amd as m3
from state_space_sequence_exp_amd import _binding as bnd

INV = m3.M3_ERR_INVALID_VALUE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(m3.LIB_PATH):
        from state_space_sequence_exp_amd import build
        build.build()
    return m3.load_library()


def apart(n, first=0x10000000):
    """n addresses 16 MiB apart."""
    return [first + (i << 24) for i in range(n)]


def hits(sizes, i, j):
    """Offsets at which array i still meets array j: first bytes together, the
    last of j, the last of i."""
    return (0, sizes[j] - 4, 4 - sizes[i])


def all_refused(call, sizes, pairs):
    p = apart(len(sizes))
    for i, j in pairs:
        for shift in hits(sizes, i, j):
            q = list(p)
            q[i] = p[j] + shift
            assert call([ctypes.c_void_p(a) for a in q]) == INV, (i, j, shift)


def test_scan_step(lib):
    """y over the state would store the state and then write y over it."""
    B, D = 2, 64
    d = bnd.M3ScanDims(B, 1, D)
    call = lambda p: lib.m3_gated_scan_step(ctypes.byref(d), 0, *p, None)
    n = 4 * B * D                          # h_in h_out x f g y
    all_refused(call, [n] * 6, [(5, 0), (5, 1), (1, 2), (1, 3), (1, 4)])
    p = apart(6)
    p[1] = p[5] = p[0]                     # h_out in h_in's place, and y there too
    assert call([ctypes.c_void_p(a) for a in p]) == INV
    wide = bnd.M3ScanDims(B, 1, D, 0, 0, 0, 3 * D)
    p = apart(6)
    p[0] = p[5] + 4 * (2 * D + 1)          # the state between y's rows reaches into the second
    assert lib.m3_gated_scan_step(ctypes.byref(wide), 0, *[ctypes.c_void_p(a) for a in p], None) == INV


def test_scan(lib):
    B, T, D = 2, 300, 64
    d = bnd.M3ScanDims(B, T, D)
    ws = lib.m3_gated_scan_workspace_size(ctypes.byref(d), 0)
    call = lambda p: lib.m3_gated_scan(ctypes.byref(d), 0, *p, 1 << 40, None)
    row, state, states = 4 * B * T * D, 4 * B * D, 4 * B * 5 * D
    sizes = [row, row, row, state, row, state, states, ws]     # x f g h0 | y h_last states workspace
    pairs = [(i, j) for i in (4, 5, 6) for j in range(7) if i != j]
    all_refused(call, sizes, pairs)
    p = apart(8)
    for j in range(7):
        q = p[:7] + [p[j]]
        assert call([ctypes.c_void_p(a) for a in q]) == INV, j


def test_scan_backward(lib):
    B, T, D = 2, 300, 64
    d = bnd.M3ScanDims(B, T, D)
    call = lambda p: lib.m3_gated_scan_backward(ctypes.byref(d), 0, *p, 1 << 40, None)
    row, state, states = 4 * B * T * D, 4 * B * D, 4 * B * 5 * D
    # dy x f g states dh_last | dx df dg dh0 workspace
    sizes = [row] * 4 + [states, state] + [row] * 3 + [state]
    pairs = [(i, j) for i in (6, 7, 8, 9) for j in range(10) if i != j]
    all_refused(lambda p: call(p + [ctypes.c_void_p(0x7000000000)]), sizes, pairs)
    p = apart(11)
    for j in range(10):
        q = p[:10] + [p[j]]
        assert call([ctypes.c_void_p(a) for a in q]) == INV, j


def test_layer_norm(lib):
    M, D = 40, 64
    d = bnd.M3NormDims(M, D)
    call = lambda p: lib.m3_layer_norm(ctypes.byref(d), 0, *p[:4], 1e-5, *p[4:], None)
    row, col, stat = 4 * M * D, 4 * D, 4 * M
    sizes = [row, row, col, col, row, row, stat, stat]      # x residual weight bias | y sum mean rstd
    pairs = [(i, j) for i in (4, 5) for j in (2, 3, 6, 7)]
    pairs += [(i, j) for i in (6, 7) for j in range(8) if i != j]
    all_refused(call, sizes, pairs)


def test_layer_norm_backward(lib):
    M, D = 40, 64
    d = bnd.M3NormDims(M, D)
    ws = lib.m3_layer_norm_backward_workspace_size(ctypes.byref(d), 0)
    call = lambda p: lib.m3_layer_norm_backward(ctypes.byref(d), 0, *p, 1 << 40, None)
    row, col, stat = 4 * M * D, 4 * D, 4 * M
    # dy s weight mean rstd dsum | dx dweight dbias workspace
    sizes = [row, row, col, stat, stat, row, row, col, col, ws]
    all_refused(call, sizes, [(6, j) for j in (1, 2, 3, 4, 7, 8)] + [(7, 6), (7, 8), (8, 6), (8, 7)])
    p = apart(10)
    for j in range(9):
        for shift in (0, -(ws - 16)):
            q = p[:9] + [p[j] + shift]
            assert call([ctypes.c_void_p(a) for a in q]) == INV, j
    d.rows = 0                                               # zeros to both, one over the other
    p[8] = p[7] + 4
    assert call([ctypes.c_void_p(a) for a in p]) == INV


def test_state_cache(lib):
    """The whole pool counts, its last slot as its first."""
    S, H, N, P, slots = 2, 3, 34, 32, 5
    d = bnd.M3Dims(S, 1, H, P, N, 1)
    codes, scales, at, h = slots * H * N * P, 4 * slots * H * N, 4 * S, 4 * S * H * N * P
    all_sizes = [h, codes, scales, at]

    def aligned(sizes, pairs, call):
        p = apart(len(sizes))
        for i, j in pairs:
            for shift in (0, (sizes[j] - 4) // 16 * 16, -((sizes[i] - 4) // 16 * 16)):
                q = list(p)
                q[i] = p[j] + shift
                assert call([ctypes.c_void_p(a) for a in q]) == INV, (i, j, shift)

    store = lambda p: lib.m3_state_store(ctypes.byref(d), 0, *p, slots, None)
    aligned(all_sizes, [(1, 0), (1, 2), (1, 3), (2, 0), (2, 3)], store)
    load = lambda p: lib.m3_state_load(ctypes.byref(d), 0, 0, p[1], p[2], p[3], slots, p[0], None)
    aligned(all_sizes, [(0, 1), (0, 2), (0, 3)], load)


def test_decode_cached(lib):
    S, H, N, P, R, slots = 2, 3, 34, 32, 2, 5
    d = bnd.M3Dims(S, 1, H, P, N, R)
    x, b, each = 4 * S * H * R * P, 4 * S * H * R * N, 4 * S * H
    # codes scales slots | x_t x_prev B_t B_prev C_t dt A lam theta y_t
    sizes = [slots * H * N * P, 4 * slots * H * N, 4 * S, x, x, b, b, b, each, 4 * H, each, each * N // 2, x]
    call = lambda p: lib.m3_decode_step_cached(ctypes.byref(d), 0, 0, *p[:3], slots, *p[3:], None)
    p = apart(13)
    for i in (0, 1, 12):
        for j in range(13):
            if i == j:
                continue
            for shift in (0, (sizes[j] - 4) // 16 * 16, -((sizes[i] - 4) // 16 * 16)):
                q = list(p)
                q[i] = p[j] + shift
                assert call([ctypes.c_void_p(a) for a in q]) == INV, (i, j, shift)


def test_pool_that_no_memory_holds(lib):
    """Its size does not wrap round to one that misses the states."""
    d = bnd.M3Dims(1, 1, 1 << 22, 128, 128, 1)
    p = [ctypes.c_void_p(a) for a in apart(4)]
    slots = (1 << 31) - 1
    assert lib.m3_state_store(ctypes.byref(d), 0, *p, slots, None) == INV
    assert lib.m3_state_load(ctypes.byref(d), 0, 0, p[1], p[2], p[3], slots, p[0], None) == INV
