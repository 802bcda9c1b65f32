"""Host sanitizer run (CPU only) of the layer operators' argument checks: the
sizes' products, the workspace queries and the overlap arithmetic, over sweeps of
ordinary and extreme dimensions."""
import os

import pytest

from state_space_sequence_exp_amd import build as B
from test_sanitize_cpu import CLANG, DRIVERS, ENV, _run, sanitized_library  # noqa: F401


@pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm clang not found")
def test_layer_validation_under_asan_ubsan(sanitized_library, tmp_path):  # noqa: F811
    exe = str(tmp_path / "driver_layer_abi")
    _run([CLANG, "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
          "-fno-omit-frame-pointer", "-I", B.INCLUDE, os.path.join(DRIVERS, "driver_layer_abi.c"),
          sanitized_library, "-Wl,-rpath," + os.path.dirname(sanitized_library), "-o", exe])
    r = _run([exe], env=ENV)
    assert " 0 failures" in r.stdout
    assert "runtime error" not in r.stderr
