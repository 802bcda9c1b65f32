"""The 8-bit cache's codes are defined by float operations that are each
rounded, none fused: the compiler must not be left free to contract any in the
source that computes them."""
import os
import re
import shutil
import subprocess

import pytest

from state_space_sequence_exp_amd import build as b

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_no_operation_may_be_fused(tmp_path):
    """In the device code as the front end hands it to the optimiser, no sum or
    product of the library's own functions carries leave to be contracted."""
    out = str(tmp_path / "state_cache.ll")
    r = subprocess.run([HIPCC] + b.compile_flags() + ["--cuda-device-only", "-S", "-emit-llvm", "-Xclang",
                        "-disable-llvm-passes", os.path.join(b.CSRC, "state_cache.hip"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    seen, free, name = set(), [], ""
    for line in open(out):
        if line.startswith("define"):
            name = re.search(r"@([^(]+)\(", line).group(1)
        elif name.startswith("_ZN2m3") and re.search(r"= f(mul|add|sub) ", line):
            seen.add(name)
            if " contract " in line:
                free.append(name)
    for part in ("pack4", "quantise8", "quantise16", "unpack16", "rank_sum", "decode_kernel", "decode_outer_kernel"):
        assert any(part in n for n in seen), part
    # m3_device.h's lane sums are not used for what is kept
    assert not [n for n in free if "_GLOBAL__N_1" in n], sorted(set(free))
