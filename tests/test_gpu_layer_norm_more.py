"""GPU checks of layer norm beside those of its formulas: the sum that a call
returns, and rows of large values."""
import numpy as np
import pytest

from layer_util import put
from test_gpu_layer_norm import run_case

pytestmark = pytest.mark.gpu


def test_no_sum_where_y_takes_the_place_of_x():
    """Without a residual the norm's input is x itself: a y in its place leaves
    none to return (the backward pass would take y for it)."""
    import torch
    import state_space_sequence_exp_amd as m3
    x, w = torch.randn(6, 40, device="cuda"), torch.ones(40, device="cuda")
    want, s, _, _ = m3.layer_norm(x, w)
    assert s is x
    a = x.clone()
    y, s, mean, rstd = m3.layer_norm(a, w, y=a)
    assert torch.equal(y, want) and y is a and s is None
    a, kept = x.clone(), torch.empty_like(x)
    y, s, _, _ = m3.layer_norm(a, w, y=a, sum_out=kept)
    assert torch.equal(y, want) and s is kept and torch.equal(s, x)
    y, s, _, _ = m3.layer_norm(x, w, y=torch.empty_like(x))
    assert torch.equal(y, want) and s is x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_near_the_root_of_the_largest_float(dtype):
    """Values up to 2^57: the sums of 384 of their squares stay below 2^123, so
    in float."""
    rng = np.random.default_rng(15)
    x = rng.standard_normal((4, 384))
    x = np.clip(x, -4, 4) * np.array([[2.0 ** 55], [2.0 ** 55], [2.0 ** 55], [2.0 ** -55]])
    run_case(4, 384, dtype, False, True, 16, x=x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(5, 8193), (3, 12281), (300, 513), (70, 1025), (40, 2049), (2, 16377)],
                         ids=lambda s: "%dx%d" % s)
def test_one_element_behind_the_last_vector(shape, dtype):
    """Rows whose last vector holds one element, in every size of team."""
    run_case(*shape, dtype, shape[0] % 2 == 0, True, seed=sum(shape))
