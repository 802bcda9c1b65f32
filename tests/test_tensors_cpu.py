"""CPU checks of the compiled look at a call's tensors: any number of dimensions,
rows of slices, and what is not an array of rows."""
import gc
import sys

import pytest
import torch

import state_space_sequence_exp_amd as m3
from state_space_sequence_exp_amd import _binding as bnd


@pytest.fixture(scope="module")
def look():
    return bnd._look()


@pytest.mark.parametrize("dims", [1, 2, 8, 9, 20])
def test_any_number_of_dimensions(look, dims):
    shape = (2,) * (min(dims, 10) - 1) + (1,) * max(0, dims - 10) + (6,)
    t = torch.empty(shape)
    assert len(shape) == dims
    assert look.dense(torch.float32, shape, -1, t) == (t.data_ptr(),)
    assert look.rows(torch.float32, shape, -1, t) == (t.data_ptr(), 0)
    wide = torch.empty(shape[:-1] + (11,))[..., 3:9]
    assert look.rows(torch.float32, shape, -1, wide) == (wide.data_ptr(), 0 if dims == 1 else 11)
    other = shape[:-1] + (5,)
    for bad in (other, shape + (1,), shape[:-1]):
        assert look.rows(torch.float32, bad, -1, t) is None and look.dense(torch.float32, bad, -1, t) is None
    new = look.empty(torch.bfloat16, shape, t)
    assert new.shape == shape and new.dtype == torch.bfloat16 and new.device == t.device


@pytest.mark.parametrize("dims", [8, 9, 12])
def test_feed_forward_takes_any_leading_axes(dims):
    """CPU tensors: everything but their device is in order."""
    lead = (2,) * (dims - 1)
    x, w, pre = torch.zeros(lead + (6,)), torch.zeros(5, 6), torch.zeros(lead + (5,))
    with pytest.raises(ValueError, match="GPU"):
        m3.gated_ffn(x, w, w)
    with pytest.raises(ValueError, match="GPU"):
        m3.gated_ffn_backward(pre, x, w, w, pre, pre)
    with pytest.raises(ValueError, match="dh: expected shape"):
        m3.gated_ffn_backward(pre[..., :4], x, w, w, pre, pre)
    with pytest.raises(ValueError, match="x: its last dimension"):
        m3.gated_ffn(torch.zeros(lead[:-1] + (6, 2)).transpose(-1, -2), w, w)
    with pytest.raises(ValueError, match="x: its rows must follow"):
        m3.gated_ffn(torch.zeros(lead[:-2] + (3, 2, 6)).transpose(-2, -3)[..., :2, :], w, w)


def test_refused_address_keeps_nothing(look):
    """Where torch refuses a tensor's address, the call raises and what it had made is
    given up: a handful of objects for the test itself, not some for every call."""
    t, grown = torch.empty(3), []

    def f(v):  # a batched tensor, which has none
        def go():
            try:
                look.dense(torch.float32, (3,), -1, t, t, t, t, v)
            except RuntimeError:
                return True
        assert all(go() for _ in range(20))
        gc.collect()
        before = sys.getallocatedblocks()
        for _ in range(500):
            go()
        grown.append(sys.getallocatedblocks() - before)
        return v
    torch.vmap(f)(torch.empty(2, 3))
    assert grown[0] < 500
