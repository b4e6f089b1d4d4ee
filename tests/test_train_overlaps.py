"""Outputs that share memory with another argument are refused on the host (fake device
addresses: nothing is dereferenced), and the test for it is right."""
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
P = ctypes.c_void_p
CSRC = os.path.join(ROOT, "linear_bound_propagation_amd", "csrc")


def test_shared_bytes(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    exe = str(tmp_path / "overlap_checks")
    cmd = [gxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__",
           "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(ROOT, "tests", "sanitize", "overlap_checks.cpp"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and " 0 failure(s)" in run.stdout, run.stdout + run.stderr


def refused(status, what):
    message = L.vb_last_error().decode()
    assert status == -1 and "overlaps" in message and what in message, (status, message)


def test_linear():
    base = dict(rows=40, n_in=12, n_out=10, dtype=0, act=0, x=1 << 16, ld_x=12, weight=1 << 17, ld_w=12, bias=1 << 18,
                residual=1 << 19, ld_res=10, y=1 << 20, ld_y=10, pre=1 << 21, ld_pre=10)
    for kw, what in ((dict(y=1 << 16), "y overlaps x"), (dict(y=(1 << 16) + 40 * 48 - 4), "y overlaps x"),
                     (dict(y=1 << 17), "y overlaps weight"), (dict(y=(1 << 18) + 36), "y overlaps bias"),
                     (dict(y=(1 << 19) + 4), "y overlaps residual"), (dict(pre=1 << 20), "y overlaps pre"),
                     (dict(pre=1 << 19), "pre overlaps residual"), (dict(pre=(1 << 16) - 40), "pre overlaps x")):
        refused(L.vb_linear_forward(ctypes.byref(train.vb_linear_fwd(**{**base, **kw})), 1 << 24, 1 << 24, None), what)
    refused(L.vb_linear_forward(ctypes.byref(train.vb_linear_fwd(**{**base, "n_in": 11, "x": (1 << 24) + 1024})), 1 << 24, 1 << 24, None),
            "the workspace overlaps x")     # x lies in the workspace that its copy takes


def test_linear_backward():
    base = dict(rows=40, n_in=10, n_out=10, dtype=0, act=1, dy=1 << 16, ld_dy=10, x=1 << 17, ld_x=10, weight=1 << 18, ld_w=10,
                saved=1 << 19, ld_saved=10, dx=1 << 20, ld_dx=10, dweight=1 << 21, ld_dw=10, dbias=1 << 22, dresidual=1 << 23,
                ld_dres=10)
    for kw, what in ((dict(dx=1 << 16), "dx overlaps dy"), (dict(dx=1 << 17), "dx overlaps x"), (dict(dx=1 << 18), "dx overlaps weight"),
                     (dict(dweight=1 << 17), "dweight overlaps x"), (dict(dresidual=(1 << 16) + 8), "dresidual overlaps dy"),
                     (dict(dresidual=1 << 19), "dresidual overlaps saved"), (dict(dbias=(1 << 20) + 8), "dx overlaps dbias"),
                     (dict(dweight=1 << 23), "dresidual overlaps dweight"), (dict(saved=1 << 24), "the workspace overlaps saved")):
        refused(L.vb_linear_backward(ctypes.byref(train.vb_linear_bwd(**{**base, **kw})), 1 << 24, 1 << 24, None), what)


def test_cross_entropy():
    base = dict(rows=40, classes=10, dtype=0, logits=1 << 16, ld=10, labels=1 << 17, ignore_index=-1, loss=1 << 18, row_loss=1 << 19,
                dlogits=1 << 20, ld_d=10)
    for kw, what in ((dict(dlogits=(1 << 16) + 4), "dlogits overlaps logits"), (dict(dlogits=(1 << 16) - 16), "dlogits overlaps logits"),
                     (dict(row_loss=1 << 17), "row_loss overlaps labels"), (dict(loss=(1 << 16) + 36), "loss overlaps logits"),
                     (dict(loss=(1 << 19) + 8), "loss overlaps row_loss"), (dict(logits=1 << 24), "the workspace overlaps logits")):
        refused(L.vb_cross_entropy(ctypes.byref(train.vb_cross_entropy_args(**{**base, **kw})), 1 << 24, 1 << 24, None), what)


@pytest.mark.parametrize("n", [2, 3, 64, 65, 300])
def test_clip(n):
    def call(grads, out, norm=1 << 12):
        g, o = (P * n)(*grads), None if out is None else (P * n)(*out)
        s, d = (ctypes.c_int64 * n)(*[100] * n), (ctypes.c_int32 * n)(*[0] * n)
        return L.vb_clip_grad_norm(n, g, o, s, d, 1.0, norm, 1 << 24, 1 << 20, None)

    apart = [(1 << 16) + 400 * i for i in range(n)]
    other = [(1 << 22) + 400 * i for i in range(n)]
    refused(call([apart[0]] + apart[:-1], None), "written")              # a gradient twice, in place
    refused(call(apart[:-1] + [apart[0] + 396], None), "written")
    refused(call(apart, [apart[1], apart[0]] + apart[2:]), "written")    # outputs in another order
    refused(call(apart, [a + 4 for a in apart]), "written")
    refused(call(apart, [other[0]] + other[:-1]), "written")             # an output twice
    refused(call(apart, other, norm=other[-1] + 40), "written")
    refused(call([1 << 24] + apart[1:], other), "written")               # a gradient in the workspace
