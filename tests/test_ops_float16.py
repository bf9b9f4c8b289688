"""Which kept values are exact in float16 (ops_internal.h), on the CPU."""
import os
import shutil
import subprocess

import pytest

from test_sanitizers import C, ENV, ROCM, ROOT, SAN, _run


def test_float16_holds_what_a_rounding_leaves(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    if not os.path.exists(os.path.join(ROCM, "include", "hip",
                                       "hip_runtime.h")):
        pytest.skip("HIP headers not found")
    exe = str(tmp_path / "float16_holds")
    _run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__",
          f"-I{ROCM}/include", f"-I{ROOT}/include", "-o", exe,
          os.path.join(C, "float16_holds.cpp")], tmp_path)
    r = subprocess.run([exe], capture_output=True, text=True, env=ENV,
                       timeout=60)
    assert r.returncode == 0, r.stderr
    assert "same" in r.stdout
