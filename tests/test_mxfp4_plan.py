"""Host logic of the MXFP4 linear's split form from C++ (tests/mxfp4_plan_check.cpp; no GPU is touched)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a C++ compiler")
def test_split_plans(lib, tmp_path):
    """Shared memory that there is, and one order of summation for codes and for a bf16 x, whatever the number of SMs."""
    exe, so = tmp_path / "mxfp4_plan_check", lib.LIB_PATH
    cmd = ["g++", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "moe_router_gemm_gb300", "csrc"), os.path.join(ROOT, "tests", "mxfp4_plan_check.cpp"),
           "-o", str(exe), so, "-Wl,-rpath," + os.path.dirname(so)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[:2000]
