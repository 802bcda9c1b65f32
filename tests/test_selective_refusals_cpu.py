"""More CPU checks of the host's refusals: the short convolution, the selective
scan and the gated feed-forward projections."""
from test_selective_abi_cpu import FFN_BW, GOOD, INV, ffn_bw, lib, swap  # noqa: F401


def test_ffn_backward_without_rows(lib):  # noqa: F811
    """The weights' gradients of no rows are zeros, and are not written over the weights."""
    assert ffn_bw(lib, swap(FFN_BW, _7=None, _8=None), rows=0) == GOOD
    for o in (7, 8):
        for w in (2, 3):
            assert ffn_bw(lib, swap(FFN_BW, **{"_%d" % o: FFN_BW[w]}), rows=0) == INV
