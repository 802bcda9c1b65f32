"""Helpers of the layer operators' GPU tests: seeded storage-typed inputs and
the element-wise comparison against the fp64 oracle's running error bounds."""
import numpy as np

from gpu_util import from_gpu, to_gpu_storage
from state_space_sequence_exp_amd import inputs as I

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # rounding to the storage type
TINY = 1e-30                                        # what underflow may leave out


def torch_type(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def stored(rng, shape, dtype, mean=0.0, std=1.0):
    """(values as float64, device tensor) of normal draws in the storage type."""
    v32 = (rng.standard_normal(shape) * std + mean).astype(np.float32)
    return put(v32, dtype)


def put(v32, dtype):
    v, raw = I._store(np.ascontiguousarray(v32, dtype=np.float32), dtype)
    return v.astype(np.float64), to_gpu_storage(raw, dtype)


def close(got, want, bound, dtype, what):
    """|got - want| within the float evaluation's bound and one rounding to
    the storage type, element by element."""
    got = from_gpu(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    tol = bound + HALF_STEP[dtype] * (np.abs(want) + bound) + TINY
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(np.isnan(got), np.inf, np.abs(got - want) / tol)), got.shape)
        raise AssertionError("%s: %d of %d out of bounds, worst at %s: got %r, want %r, bound %.3g"
                             % (what, bad.sum(), bad.size, at, got[at], want[at], tol[at]))
