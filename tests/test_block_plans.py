"""Which way the layers' products and layer norm's sums take, seen from the workspaces that the
library asks for (no GPU: fake addresses, nothing is dereferenced)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from helpers import ROOT, ensure_built

ensure_built()
import linear_bound_propagation_amd as lbp  # noqa: E402
from linear_bound_propagation_amd import train  # noqa: E402

L = lbp.lib()
F32, BF16, F16 = 0, 1, 2


def size(fn, *args):
    out = ctypes.c_size_t(0)
    assert fn(*args, ctypes.byref(out)) == 0
    return out.value


def gated(rows, n_in, n_out, dtype, ld_w=None, weight=1 << 20):
    return size(L.vb_gated_linear_forward_workspace, ctypes.byref(train.vb_gated_linear_fwd(
        rows=rows, n_in=n_in, n_out=n_out, dtype=dtype, act=3, x=4096, ld_x=n_in, weight=weight, ld_w=ld_w or n_in)))


@pytest.mark.parametrize("rows, n_in, n_out, dtype", [
    (7, 8191, 2048, F32), (16, 8191, 2048, F32), (5, 5001, 1000, F32), (7, 4097, 300, F32), (31, 2049, 300, F32),
    (7, 8193, 2048, BF16), (16, 8193, 2048, F16), (5, 12001, 1500, BF16)])
def test_gated_few_rows_do_not_copy_many_weights(rows, n_in, n_out, dtype):
    """Weights off 16-byte boundaries, of a size whose copy costs more than a split reduction gains."""
    weights = 2 * n_out * n_in * (4 if dtype == F32 else 2)
    assert gated(rows, n_in, n_out, dtype) < weights // 8
    # rows that end on boundaries but start off them
    even = n_in // 8 * 8
    assert gated(rows, even, n_out, dtype, ld_w=even + 1) < weights // 8
    assert gated(rows, even, n_out, dtype, weight=(1 << 20) + 4) < weights // 8


def test_gated_few_rows_split_long_reductions():
    """Few weights: the reduction is split, and its parts are in the workspace."""
    for rows, n_in, n_out, dtype in ((16, 8192, 300, BF16), (7, 8192, 300, F32), (31, 2048, 300, F32), (16, 8193, 300, BF16)):
        assert gated(rows, n_in, n_out, dtype) >= 2 * rows * 2 * n_out * 4, (rows, n_in, n_out)


def test_tiles_of_both_backward_products(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    package = os.path.join(ROOT, "linear_bound_propagation_amd")
    exe = str(tmp_path / "plan_checks")
    res = subprocess.run([gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
                          "-I", os.path.join(ROOT, "include"), "-I", os.path.join(package, "csrc"),
                          os.path.join(ROOT, "tests", "sanitize", "plan_checks.cpp"), lbp.LIB_PATH,
                          "-Wl,-rpath," + package, "-L/opt/rocm/lib", "-Wl,-rpath,/opt/rocm/lib", "-lamdhip64", "-o", exe],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0 and " 0 failure(s)" in run.stdout, run.stdout


def norm_sums(rows, n, dtype):
    """Parts of dweight and dbias: two float32 rows each, rounded up to 16 bytes."""
    return size(L.vb_layer_norm_backward_workspace, rows, n, dtype) // (8 * ((n + 3) // 4 * 4))


def test_parts_of_layer_norm_sums_are_bounded():
    """Each part is a term of a float32 sum.  (The workspace is rounded up to 256 bytes, at most eight parts.)"""
    for rows in (2 ** 20, 2 ** 27, 2 ** 31 - 1):
        for n, dtype in ((1, F32), (3, F32), (7, F16), (7, BF16), (100, F32), (4096, BF16), (20000, F32), (2 ** 20, F16)):
            assert norm_sums(rows, n, dtype) <= 1024 + 8, (rows, n, dtype)


@pytest.mark.parametrize("rows, n, dtype, columns", [
    (64, 8192, BF16, True), (70, 8192, BF16, False), (256, 8192, F16, True), (512, 16384, BF16, True), (640, 8192, BF16, False),
    (100, 6001, BF16, False), (200, 6001, F32, False), (256, 4096, BF16, False), (128, 4096, F32, False), (256, 8192, F32, True),
    (200, 5000, F32, True), (400, 8192, F32, False), (2048, 8192, BF16, False), (300, 8193, F32, True)])
def test_way_of_layer_norm_sums(rows, n, dtype, columns):
    """By columns in parts of 64 rows, or a part per workgroup of rows."""
    assert (norm_sums(rows, n, dtype) <= (rows + 63) // 64) == columns
