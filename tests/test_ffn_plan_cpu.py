"""Every kernel that the feed-forward products may take is run by a GPU test
against the oracle: the plan (csrc/ffn_plan.h, compiled here for the host) of those
tests' sizes reaches each tile, with k whole and cut and with rows straight into the
LDS and through registers, that sizes drawn from the whole range reach.  A change of
the plan's rule that moves a kernel out of the tests' reach fails here."""
import ctypes
import math
import random
import shutil
import subprocess

import pytest

import test_gpu_gated_ffn as first
import test_gpu_gated_ffn_more as more
from state_space_sequence_exp_amd import build as B

SHIM = """#include "ffn_plan.h"
extern "C" void plan(int64_t M, int64_t cols, int64_t K, int es, int cut, int64_t* out) {
  const m3::Plan p = m3::plan_gemm(M, cols, K, es, cut != 0);
  out[0] = p.tile, out[1] = p.parts, out[2] = p.each;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    gxx = shutil.which("g++") or pytest.skip("no g++")
    d = tmp_path_factory.mktemp("plan")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I", B.CSRC,
                    str(d / "shim.cpp"), "-o", str(d / "shim.so")], check=True)
    lib = ctypes.CDLL(str(d / "shim.so"))
    lib.plan.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 2 + [ctypes.c_void_p]

    def of(M, cols, K, es, cut):
        out = (ctypes.c_int64 * 3)()
        lib.plan(M, cols, K, es, cut, out)
        return tuple(out)
    return of


def kernels(plan, M, K, F, es):
    """What the forward and backward products of dense arrays of this size run on."""
    wide = 2 * (-(-F // 64) * 64)
    if M > 32:                                              # (fewer rows: another kernel)
        yield es, "both", plan(M, 2 * F, K, es, 0)[0], "registers" if es * K % 4 else "straight"
    for kind, sizes in (("inputs", (M, K, wide)), ("weights", (wide, K, M))):
        tile, parts, each = plan(*sizes, es, 1)
        assert (parts - 1) * each < sizes[2] <= parts * each and each % (128 // es) == 0
        yield es, kind, tile, "cut" if parts > 1 else "whole"


def sizes_of(test):
    """The (M, K, F) that a test is run with, in both types."""
    marks = {m.args[0]: m.args[1] for m in test.pytestmark if m.name == "parametrize"}
    assert marks["dtype"] == ["f32", "bf16"]
    return marks["M,K,F"]


TESTED = [s for t in (first.test_ffn, first.test_ffn_larger_tiles, first.test_ffn_largest_tiles,
                      first.test_ffn_long_sums, first.test_ffn_many_rows, more.test_ffn_other_kernels)
          for s in sizes_of(t)]


def test_every_kernel_is_run(plan):
    rng = random.Random(1)
    size = lambda most: int(round(math.exp(rng.uniform(0, math.log(most)))))
    drawn = {k for _ in range(60000) for k in kernels(plan, size(60000), size(20000), size(20000), rng.choice([2, 4]))}
    run = {k for s in TESTED for es in (2, 4) for k in kernels(plan, *s, es)}
    assert not drawn - run
    # four tiles in bfloat16, three in float, each whole at the least, each product of them
    assert {(es, kind, t) for es, kind, t, _ in drawn} == \
        {(es, kind, t) for es in (2, 4) for kind in ("both", "inputs", "weights") for t in range(es // 4, 4)}
