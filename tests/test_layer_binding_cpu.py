"""CPU-only checks of the layer operators' Python entry points."""
import pytest
import torch

import state_space_sequence_exp_amd as m3


def test_scan_workspace_size_of_other_types():
    """Only the two storage types have a size; another one's would be a wrong
    one."""
    for dtype in (torch.float16, torch.float64, torch.int32, 2, -1):
        with pytest.raises(TypeError):
            m3.gated_scan_workspace_size(2, 300, 64, dtype)
    for code, dtype in ((m3.M3_F32, torch.float32), (m3.M3_BF16, torch.bfloat16)):
        assert m3.gated_scan_workspace_size(2, 300, 64, code) == m3.gated_scan_workspace_size(2, 300, 64, dtype) > 0


def test_stream_with_arguments_by_name():
    """The call's device is its first tensor's, in whatever order the arguments
    are named (CPU tensors: refused for that, not for the order)."""
    x, w = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises(ValueError, match="GPU"):
        m3.layer_norm(eps=1e-5, residual=None, weight=w, x=x, stream=0)
    c, s = m3.state_cache(4, 2, 16, 16, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        m3.state_load(slots=None, scales=s, codes=c, stream=0)
    with pytest.raises(ValueError, match="GPU"):
        m3.gated_scan(g=None, f=torch.zeros(1, 2, 8), x=torch.zeros(1, 2, 8), stream=0)
    with pytest.raises(TypeError, match="'x'"):
        m3.layer_norm(weight=w, stream=0)


def test_each_name_is_defined_once():
    """A helper of the layer operators does not replace one that the other
    entry points use."""
    import ast
    import collections
    from state_space_sequence_exp_amd import _binding
    names = collections.Counter(n.name for n in ast.parse(open(_binding.__file__).read()).body
                                if isinstance(n, (ast.FunctionDef, ast.ClassDef)))
    assert [n for n, k in names.items() if k > 1] == []
