"""The host side of include/mta_matrix.h (matrix_host.cpp) under AddressSanitizer
and UndefinedBehaviorSanitizer, on the CPU: tests/c/san_matrix.c makes random and
extreme calls that have to be refused and sweeps the workspace sizes, with the
kernel launchers replaced by stubs that must never be reached.  Host code only,
built with gcc / g++."""
import os
import shutil
import subprocess

import pytest

from test_sanitizers import C, ENV, ROCM, ROOT, SAN, _run


def test_matrix_host_side_under_sanitizers(tmp_path):
    for tool in ("gcc", "g++"):
        if shutil.which(tool) is None:
            pytest.skip(f"{tool} not found")
    if not os.path.exists(os.path.join(ROCM, "include", "hip",
                                       "hip_runtime.h")):
        pytest.skip("HIP headers not found")
    csrc = os.path.join(ROOT, "mixed_precision_optimizer_mta_amd", "csrc")
    objs = []
    for src in (os.path.join(csrc, "mta_host.cpp"),
                os.path.join(csrc, "matrix_host.cpp"),
                os.path.join(C, "san_stubs.cpp"),
                os.path.join(C, "san_matrix_stubs.cpp"),
                os.path.join(C, "san_matrix.c")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        cc = ["gcc", "-std=c11"] if src.endswith(".c") else \
            ["g++", "-std=c++17"]
        _run([*cc, *SAN, "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
              f"-I{ROOT}/include", "-c", "-o", obj, src], tmp_path)
        objs.append(obj)
    exe = str(tmp_path / "san_matrix")
    _run(["g++", *SAN, "-o", exe, *objs, f"-L{ROCM}/lib", "-lamdhip64",
          f"-Wl,-rpath,{ROCM}/lib"], tmp_path)
    r = subprocess.run([exe], capture_output=True, text=True, env=ENV,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    assert "clean" in r.stdout
