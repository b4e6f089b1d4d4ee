"""Launch sizes of the training operators: a dimension of a grid holds less than 2^32 work-items."""
import ctypes
import os
import shutil
import subprocess

import pytest

from helpers import ROOT, ensure_built

CSRC = os.path.join(ROOT, "linear_bound_propagation_amd", "csrc")


def test_grids_of_many_workgroups(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    exe = str(tmp_path / "grid_checks")
    cmd = [gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
           "-I", CSRC, os.path.join(ROOT, "tests", "sanitize", "grid_checks.cpp"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0 and " 0 failure(s)" in run.stdout, run.stdout


def test_clipping_of_more_than_a_launch_holds_is_refused():
    """2^38 numbers take 2^24 chunks, one workgroup each."""
    ensure_built()
    import linear_bound_propagation_amd as lbp
    out = ctypes.c_size_t(0)
    call = lbp.lib().vb_clip_grad_norm_workspace
    for sizes, status in (([2 ** 38 - 16384], 0), ([2 ** 38], -1), ([2 ** 37, 2 ** 37], -1), ([2 ** 37 - 16384, 2 ** 37], 0)):
        assert call(len(sizes), (ctypes.c_int64 * len(sizes))(*sizes), ctypes.byref(out)) == status, sizes
