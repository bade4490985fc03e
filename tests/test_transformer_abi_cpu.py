"""CPU checks of the transformer operators' C entry points: bad arguments are
refused on the host, before any device work, with a code and a message."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
X, Y, W, G, B = P(0x100000), P(0x900000), P(0x2000000), P(0x3000000), P(0x3100000)


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


@pytest.fixture(scope="module")
def lib():
    import seam_blending_patch_amd as sb
    return sb._lib


def refused(lib, code, rc, word):
    assert rc == code, (rc, lib.seamblend_last_error())
    assert word in lib.seamblend_last_error(), lib.seamblend_last_error()


def test_strided_overlap_check_against_a_count_of_elements(tmp_path):
    exe = str(tmp_path / "overlap_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-I",
                    os.path.join(ROOT, "seam_blending_patch_amd", "csrc"),
                    os.path.join(ROOT, "tests", "csrc", "overlap_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    cases, disjoint, told = [int(w) for w in r.stdout.replace(",", "").split() if w.isdigit()]
    assert cases == 60000 and told > 0.5 * disjoint


@pytest.mark.parametrize("change,code,word", [
    (dict(x=None), -1, b"null x"),
    (dict(out=None), -1, b"null out"),
    (dict(shape=None), -1, b"shape"),
    (dict(shape=i64(2, 3, 0)), -1, b"row length"),
    (dict(shape=i64(-1, 3, 64)), -1, b"row counts"),
    (dict(shape=i64(1 << 20, 1 << 20, 64)), -2, b"2^31 rows"),
    (dict(shape=i64(2, 3, (1 << 28) + 1)), -2, b"2^28"),
    (dict(x_stride=i64(-64, 64)), -2, b"strides of x"),
    (dict(x_stride=i64(1 << 40, 64)), -2, b"strides of x"),
    (dict(out_stride=i64(192, 0)), -1, b"overlaps itself"),
    (dict(out_stride=i64(192, 63)), -1, b"overlaps itself"),
    (dict(x=P(0x100002)), -1, b"aligned"),
    (dict(gamma=P(0x3000001)), -1, b"aligned"),
    (dict(dtype=3), -1, b"dtype"),
    (dict(wdtype=1), -1, b"weights"),
    (dict(eps=-1.0), -1, b"eps"),
    (dict(eps=float("nan")), -1, b"eps"),
    (dict(out=P(0x100000 + 4)), -1, b"overlaps x"),
    (dict(out=P(0x100000 + 64 * 4)), -1, b"overlaps x"),
])
def test_layer_norm_forward_refusals(lib, change, code, word):
    a = dict(x=X, x_stride=i64(192, 64), shape=i64(2, 3, 64), eps=1e-6, gamma=G, beta=B, dtype=0, wdtype=0, out=Y,
             out_stride=i64(192, 64)) | change
    refused(lib, code, lib.layer_norm_forward(a["x"], a["x_stride"], a["shape"], a["eps"], a["gamma"], a["beta"],
                                              a["dtype"], a["wdtype"], a["out"], a["out_stride"], None, 0, None), word)


def test_layer_norm_forward_workspace(lib):
    assert lib.layer_norm_forward_workspace_bytes(i64(1, 60000, 16384), 0) == 0
    assert lib.layer_norm_forward_workspace_bytes(i64(1, 60000, 32768), 2) == 0
    need = lib.layer_norm_forward_workspace_bytes(i64(1, 3, 40000), 2)
    assert need >= 3 * 6 * 32
    assert lib.layer_norm_forward_workspace_bytes(i64(1, 3, 0), 2) == ctypes.c_size_t(-1).value
    assert lib.layer_norm_forward_workspace_bytes(i64(1, 3, 64), 7) == ctypes.c_size_t(-1).value
    st = i64(0, 40000)
    call = lambda w, n: lib.layer_norm_forward(X, st, i64(1, 3, 40000), 1e-6, None, None, 2, 2, Y, st, w, n, None)  # noqa: E731
    refused(lib, -1, call(None, 0), b"workspace")
    refused(lib, -1, call(P(0x4000008), need), b"16-byte")
    refused(lib, -3, call(W, need - 1), b"too small")


@pytest.mark.parametrize("change,code,word", [
    (dict(dy=None), -1, b"null dy"),
    (dict(dx=None), -1, b"null dx"),
    (dict(workspace=None), -1, b"workspace"),
    (dict(workspace=P(0x4000008)), -1, b"16-byte"),
    (dict(room=64), -3, b"too small"),
    (dict(dx=P(0x100000 + 64)), -1, b"overlaps x"),
    (dict(dx=P(0x500000 + 64)), -1, b"overlaps dy"),
    (dict(dgamma=P(0x3200002)), -1, b"aligned"),
    (dict(wdtype=2), -1, b"weights"),
])
def test_layer_norm_backward_refusals(lib, change, code, word):
    a = dict(dy=P(0x500000), x=X, shape=i64(1, 6, 64), dtype=0, wdtype=0, dx=Y, dgamma=P(0x3200000),
             workspace=P(0x4000000), room=1 << 24) | change
    st = i64(0, 64)
    refused(lib, code, lib.layer_norm_backward(a["dy"], st, a["x"], st, a["shape"], 1e-6, G, a["dtype"], a["wdtype"],
                                               a["dx"], st, a["dgamma"], None, a["workspace"], a["room"], None), word)


def test_layer_norm_workspace(lib):
    small = lib.layer_norm_backward_workspace_bytes(i64(1, 6, 64), 0)
    large = lib.layer_norm_backward_workspace_bytes(i64(1, 60000, 4096), 0)
    assert 0 < small < large
    assert lib.layer_norm_backward_workspace_bytes(i64(1, 0, 64), 0) > 0
    assert lib.layer_norm_backward_workspace_bytes(i64(1, 6, 0), 0) == 0
    assert lib.layer_norm_backward_workspace_bytes(i64(1, 6, 64), 9) == 0


def test_layer_norm_without_rows_reads_nothing(lib):
    st = i64(0, 64)
    assert lib.layer_norm_forward(None, st, i64(4, 0, 64), 1e-6, None, None, 0, 0, None, st, None, 0, None) == 0
    assert lib.layer_norm_backward(None, st, None, st, i64(0, 4, 64), 1e-6, None, 0, 0, None, st, None, None, None, 0,
                                   None) == 0


ROT = dict(q=X, qs=i64(4096, 512, 64), qo=Y, qos=i64(4096, 512, 64), hq=8, k=None, ks=None, ko=None, kos=None, hk=0,
           shape=i64(2, 8, 64), dtype=2, freqs=P(0x3000000), rot=64, layout=0, pos=P(0x3100000), pb=8, ps=i64(0, 0, 1),
           sections=i64(32), n=1, scale=1.0)


@pytest.mark.parametrize("change,code,word", [
    (dict(q=None), -1, b"null q"),
    (dict(qo=None), -1, b"null q_out"),
    (dict(hk=2), -1, b"null k"),
    (dict(shape=None), -1, b"shape"),
    (dict(shape=i64(2, -8, 64)), -1, b"negative"),
    (dict(shape=i64(2, 8, 0)), -2, b"head length"),
    (dict(shape=i64(1 << 16, 1 << 16, 64)), -2, b"2^31 tokens"),
    (dict(hq=5000), -2, b"heads"),
    (dict(rot=0), -1, b"rot_dim"),
    (dict(rot=63), -1, b"rot_dim"),
    (dict(rot=66), -1, b"rot_dim"),
    (dict(layout=2), -1, b"layout"),
    (dict(dtype=5), -1, b"dtype"),
    (dict(pb=2), -1, b"positions"),
    (dict(pos=P(0x3100004)), -1, b"aligned"),
    (dict(freqs=P(0x3000004)), -1, b"aligned"),
    (dict(freqs=None), -1, b"null freqs"),
    (dict(ps=i64(0, 0, -1)), -2, b"strides of positions"),
    (dict(sections=i64(31)), -1, b"pairs"),
    (dict(sections=i64(40, -8), n=2), -1, b"section"),
    (dict(n=5), -1, b"sections"),
    (dict(scale=float("inf")), -1, b"scale"),
    (dict(qos=i64(4096, 512, 32)), -1, b"overlaps itself"),
    (dict(qo=P(0x100000 + 128)), -1, b"overlaps q"),
    (dict(k=P(0x100000), ks=i64(4096, 512, 64), ko=P(0xa00000), kos=i64(4096, 512, 64), hk=8, qo=X), -1, b"q_out overlaps k"),
    (dict(k=P(0x500000), ks=i64(4096, 512, 64), ko=Y, kos=i64(4096, 512, 64), hk=8), -1, b"q_out overlaps k_out"),
])
def test_rotary_refusals(lib, change, code, word):
    a = ROT | change
    refused(lib, code, lib.rotary_apply(a["q"], a["qs"], a["qo"], a["qos"], a["hq"], a["k"], a["ks"], a["ko"], a["kos"],
                                        a["hk"], a["shape"], a["dtype"], a["freqs"], a["rot"], a["layout"], a["pos"],
                                        a["pb"], a["ps"], a["sections"], a["n"], a["scale"], 0, None), word)


def ptrs(*v):
    return (ctypes.c_void_p * len(v))(*v)


def ints(*v):
    return (ctypes.c_int * len(v))(*v)


CLIP = dict(grads=ptrs(0x100000, 0x200000), outs=None, numels=i64(100, 50), types=ints(0, 2), out_types=None, n=2,
            max_norm=1.0, eps=1e-6, norm=P(0x3000000), work=P(0x4000000), room=4096)


@pytest.mark.parametrize("change,code,word", [
    (dict(grads=None), -1, b"table"),
    (dict(grads=ptrs(0x100000, 0)), -1, b"gradient 1"),
    (dict(grads=ptrs(0x100002, 0x200000)), -1, b"gradient 0"),
    (dict(numels=i64(100, -1)), -1, b"tensor 1"),
    (dict(numels=i64(1 << 44, 50)), -2, b"2^44"),
    (dict(types=ints(0, 3)), -1, b"dtype"),
    (dict(outs=ptrs(0x500000, 0x600000), out_types=ints(0, 1)), -1, b"output"),
    (dict(outs=ptrs(0x500000, 0), out_types=ints(0, 2)), -1, b"output 1"),
    (dict(outs=ptrs(0x500000, 0x600000)), -1, b"table"),
    (dict(outs=ptrs(0x100004, 0x600000), out_types=ints(0, 2)), -1, b"overlaps"),
    (dict(outs=ptrs(0x100000, 0x200000), out_types=ints(0, 0)), -1, b"overlaps"),
    (dict(n=-1), -2, b"tensors"),
    (dict(n=(1 << 20) + 1), -2, b"tensors"),
    (dict(max_norm=-0.5), -1, b"max_norm"),
    (dict(max_norm=float("nan")), -1, b"max_norm"),
    (dict(eps=float("inf")), -1, b"eps"),
    (dict(norm=None), -1, b"norm"),
    (dict(work=None), -1, b"workspace"),
    (dict(room=8), -3, b"too small"),
])
def test_grad_norm_clip_refusals(lib, change, code, word):
    a = CLIP | change
    refused(lib, code, lib.grad_norm_clip(a["grads"], a["outs"], a["numels"], a["types"], a["out_types"], a["n"],
                                          a["max_norm"], a["eps"], a["norm"], a["work"], a["room"], None), word)


def test_grad_norm_workspace(lib):
    assert lib.grad_norm_workspace_bytes(i64(100, 50), 2) >= 16
    assert lib.grad_norm_workspace_bytes(i64(), 0) > 0
    assert lib.grad_norm_workspace_bytes(i64(1 << 36), 1) <= 1 << 20
    assert lib.grad_norm_workspace_bytes(i64(-1), 1) == 0
