"""More CPU checks of the host's refusals: the short convolution, the selective
scan and the gated feed-forward projections."""
import pytest

from test_selective_abi_cpu import (CONV, CONV_STEP, FFN_BW, GOOD, INV, UNS, conv, conv_step,  # noqa: F401
                                    ffn_bw, ffn_dims, lib, swap)


def test_ffn_backward_without_rows(lib):  # noqa: F811
    """The weights' gradients of no rows are zeros, and are not written over the weights."""
    assert ffn_bw(lib, swap(FFN_BW, _7=None, _8=None), rows=0) == GOOD
    for o in (7, 8):
        for w in (2, 3):
            assert ffn_bw(lib, swap(FFN_BW, **{"_%d" % o: FFN_BW[w]}), rows=0) == INV


@pytest.mark.parametrize("rows,K,F,good", [
    (1 << 22, 64, 96, True), (100000000, 64, 96, True), (230000000, 1, 1, True), (1 << 23, 1024, 1800, True),
    (110000000, 64, 96, False), (1 << 28, 1, 1, False), (1 << 23, 1024, 2048, False), (1 << 23, 4000, 64, False)])
def test_ffn_rows_bounded_by_tiles_alone(lib, rows, K, F, good):  # noqa: F811
    """Forward and backward take the same rows: as many as the tiles of one launch, rows x units
    and rows x channels (an unaligned gate tells a call that would be taken)."""
    kw = dict(rows=rows, channels=K, hidden=F)
    for dt in (0, 1):
        size = lib.m3_gated_ffn_backward_workspace_size(ffn_dims(**kw), dt)
        assert (size > rows * 2 * F * (4 - 2 * dt)) if good else size == 0
        off = swap(FFN_BW, _5=FFN_BW[5].value + 1)
        assert ffn_bw(lib, off, dt=dt, **kw) == (INV if good else UNS)


def test_ffn_backward_counts_the_copies_it_makes(lib):  # noqa: F811
    """The first launch holds dg and the copies of arrays whose rows are not whole chunks at
    multiples of 4 bytes: a call of aligned arrays is not refused for copies it does not make."""
    kw = dict(rows=4190000, channels=7744, hidden=512)
    assert lib.m3_gated_ffn_backward_workspace_size(ffn_dims(**kw), 1) > 4190000 * (2 * 512 + 7744) * 2
    off = swap(FFN_BW, _5=FFN_BW[5].value + 1)                     # (tells a call that would be taken)
    assert ffn_bw(lib, off, **kw) == INV
    assert ffn_bw(lib, swap(off, _2=FFN_BW[2].value + 2), **kw) == INV    # copies of the weights: few
    assert ffn_bw(lib, swap(off, _1=FFN_BW[1].value + 2), **kw) == UNS    # of x: 65 GB more to write
    assert ffn_bw(lib, off, ld_x=7745, **kw) == UNS
    assert lib.m3_gated_ffn_backward_workspace_size(ffn_dims(ld_x=7745, **kw), 1) == 0
    assert ffn_bw(lib, off, ld_x=7746, **kw) == INV
    for less in (dict(kw, channels=7743), dict(kw, channels=7740)):      # rows that are no whole chunks
        assert ffn_bw(lib, off, **less) == UNS
        assert lib.m3_gated_ffn_backward_workspace_size(ffn_dims(**less), 1) == 0


@pytest.mark.parametrize("batch,seqlen,channels,dt,good", [
    (1 << 20, 4094 * 16, 8, 1, True), (1 << 20, 4095 * 16, 8, 1, False), (1 << 20, 4094 * 16, 9, 1, False),
    (1 << 20, 2046 * 16, 9, 1, True), (1 << 20, 4094 * 16, 4, 0, True), (1 << 20, 4094 * 16, 5, 0, False),
    (1, (1 << 31) - 1, 200, 1, True), ((1 << 31) - 256, 1, 8, 1, True), ((1 << 31) - 256, 17, 8, 1, False)])
def test_conv_largest(lib, batch, seqlen, channels, dt, good):  # noqa: F811
    """At most 2^24 - 1 workgroups of 256 items: 16 tokens of 16 bytes of channels, or a sequence's
    kept inputs of these (a misaligned weight tells a call that would be taken)."""
    off = swap(CONV, _1=CONV[1].value + 1)
    kw = dict(batch=batch, seqlen=seqlen, channels=channels, ld_x=0, ld_y=0)
    assert conv(lib, off, dt=dt, **kw) == (INV if good else UNS)


@pytest.mark.parametrize("batch,channels,good", [
    ((1 << 24) - 1, 2048, True), (1 << 24, 2048, False), (1 << 23, 2049, False), ((1 << 23) - 1, 4096, True)])
def test_conv_step_largest(lib, batch, channels, good):  # noqa: F811
    off = swap(CONV_STEP, _4=CONV_STEP[4].value + 1)
    assert conv_step(lib, off, batch=batch, channels=channels, ld_x=0, ld_y=0) == (INV if good else UNS)
