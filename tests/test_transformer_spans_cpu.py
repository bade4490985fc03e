"""CPU checks of the transformer operators' limits on how far a tensor reaches:
2^52 elements from first to last, however extents and strides multiply."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
X, Y, G = P(0x100000), P(0x900000), P(0x3000000)
FAR = (1 << 40) - 1  # the longest stride taken


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


@pytest.fixture(scope="module")
def lib():
    import seam_blending_patch_amd as sb
    return sb._lib


def refused(lib, rc, name):
    message = lib.seamblend_last_error()
    assert rc == -2 and message == name + b" spans 2^52 elements or more", (rc, message)


def test_span_against_an_exact_count(tmp_path):
    exe = str(tmp_path / "span_check")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                    "-I", os.path.join(ROOT, "seam_blending_patch_amd", "csrc"),
                    os.path.join(ROOT, "tests", "csrc", "span_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    cases, wide = [int(w) for w in r.stdout.replace(",", "").split() if w.isdigit()]
    assert cases == 200000 and 0.01 * cases < wide < 0.99 * cases


# (outer extent, stride): 2^52 and a little, past 2^63, a multiple of 2^64 less a little
@pytest.mark.parametrize("rows", [(1 << 12) + 2, (1 << 23) + 1, (1 << 24) + 1, (1 << 30)])
def test_layer_norm_rows_that_reach_too_far(lib, rows):
    shape, near, far = i64(rows, 1, 64), i64(64, 0), i64(FAR, 0)
    refused(lib, lib.layer_norm_forward(X, far, shape, 1e-6, None, None, 0, 0, Y, near, None, 0, None), b"x")
    refused(lib, lib.layer_norm_forward(X, near, shape, 1e-6, None, None, 0, 0, P(1 << 45), far, None, 0, None), b"out")
    work = (P(0x4000000), 1 << 30)
    backward = lambda dy, x, dx: lib.layer_norm_backward(  # noqa: E731
        P(1 << 45), dy, X, x, shape, 1e-6, None, 0, 0, P(1 << 46), dx, None, None, *work, None)
    refused(lib, backward(far, near, near), b"dy")
    refused(lib, backward(near, far, near), b"x")
    refused(lib, backward(near, near, far), b"dx")


@pytest.mark.parametrize("tokens", [(1 << 12) + 2, (1 << 23) + 1, (1 << 24) + 1, (1 << 30)])
@pytest.mark.parametrize("axis", [0, 1])
def test_rotary_tensors_that_reach_too_far(lib, tokens, axis):
    shape = i64(tokens, 1, 64) if axis == 0 else i64(1, tokens, 64)
    near, far = i64(64, 64, 64), i64(FAR, FAR, 64)
    call = lambda q, qo, k, ko: lib.rotary_apply(  # noqa: E731
        X, q, P(1 << 45), qo, 1, P(1 << 46), k, P(1 << 47), ko, 1, shape, 0, G, 64, 0, P(0x3100000), 8, i64(0, 0, 0),
        i64(32), 1, 1.0, 0, None)
    refused(lib, call(far, near, near, near), b"q")
    refused(lib, call(near, far, near, near), b"q_out")
    refused(lib, call(near, near, far, near), b"k")
    refused(lib, call(near, near, near, far), b"k_out")
