"""CPU checks of attention's C entry points: bad arguments are refused on the
host, before any device work, with a code and a message; workspaces."""
from __future__ import annotations

import ctypes

import pytest

P = ctypes.c_void_p


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


@pytest.fixture(scope="module")
def lib():
    import seam_blending_patch_amd as sb
    return sb._lib


def refused(lib, code, rc, word):
    assert rc == code, (rc, lib.seamblend_last_error())
    assert word in lib.seamblend_last_error(), lib.seamblend_last_error()


# fp16: q, out [2, 8, 4, 32], k, v [2, 9, 2, 32]
BASE = dict(q=P(0x100000), qs=i64(1024, 128, 32), k=P(0x200000), ks=i64(576, 64, 32), v=P(0x300000),
            vs=i64(576, 64, 32), shape=i64(2, 8, 9, 4, 2, 32), dtype=1, scale=0.1, causal=0, ql=None, kl=None,
            out=P(0x400000), os=i64(1024, 128, 32), lse=P(0x500000), work=P(0x600000), room=1 << 24)


def forward(lib, **change):
    a = BASE | change
    return lib.attention_forward(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["shape"], a["dtype"], a["scale"],
                                 a["causal"], a["ql"], a["kl"], a["out"], a["os"], a["lse"], a["work"], a["room"], None)


COMMON = [
    (dict(q=None), -1, b"null q"), (dict(k=None), -1, b"null k"), (dict(v=None), -1, b"null v"),
    (dict(out=None), -1, b"null out"), (dict(vs=None), -1, b"strides of v"), (dict(shape=None), -1, b"null shape"),
    (dict(dtype=5), -1, b"dtype"), (dict(scale=0.0), -1, b"scale"), (dict(scale=-1.0), -1, b"scale"),
    (dict(scale=float("nan")), -1, b"scale"), (dict(scale=float("inf")), -1, b"scale"), (dict(scale=3e38), -1, b"scale"),
    (dict(shape=i64(2, 8, 9, 4, 3, 32)), -1, b"multiple"), (dict(shape=i64(2, 8, 9, 4, 0, 32)), -1, b"multiple"),
    (dict(shape=i64(2, 8, 9, 0, 2, 32)), -1, b"multiple"), (dict(shape=i64(2, -1, 9, 4, 2, 32)), -1, b"negative"),
    (dict(shape=i64(2, 8, 9, 4, 2, 0)), -2, b"head length"), (dict(shape=i64(2, 8, 9, 4, 2, 257)), -2, b"head length"),
    (dict(shape=i64(2, 8, 9, 8192, 2, 32)), -2, b"heads"), (dict(shape=i64(2, 1 << 29, 9, 4, 2, 32)), -2, b"2^30"),
    (dict(shape=i64(2, 8, 1 << 29, 4, 2, 32)), -2, b"2^30"), (dict(shape=i64(1 << 29, 8, 9, 4, 2, 32)), -2, b"2^30"),
    (dict(shape=i64(2, 1 << 62, 9, 4, 2, 32)), -2, b"2^30"),
    (dict(qs=i64(-1, 128, 32)), -2, b"strides of q"), (dict(ks=i64(576, 1 << 40, 32)), -2, b"strides of k"),
    (dict(q=P(0x100001)), -1, b"aligned"), (dict(kl=P(0x700002)), -1, b"aligned"), (dict(ql=P(0x700001)), -1, b"aligned"),
    (dict(lse=P(0x500002)), -1, b"aligned"),
]


@pytest.mark.parametrize("change,code,word", COMMON + [
    (dict(os=i64(1024, 128, 31)), -1, b"overlaps itself"), (dict(os=i64(0, 128, 32)), -1, b"overlaps itself"),
    (dict(out=P(0x100000)), -1, b"out overlaps q"), (dict(out=P(0x200000 - 64)), -1, b"out overlaps k"),
    (dict(out=P(0x300000 + 512)), -1, b"out overlaps v"),
])
def test_forward_refusals(lib, change, code, word):
    refused(lib, code, forward(lib, **change), word)


def backward(lib, **change):
    a = BASE | dict(dout=P(0x800000), gs=i64(1024, 128, 32), dq=P(0x900000), dqs=i64(1024, 128, 32), dk=P(0xa00000),
                    dks=i64(576, 64, 32), dv=P(0xb00000), dvs=i64(576, 64, 32)) | change
    return lib.attention_backward(a["dout"], a["gs"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["out"], a["os"],
                                  a["lse"], a["shape"], a["dtype"], a["scale"], a["causal"], a["ql"], a["kl"], a["dq"],
                                  a["dqs"], a["dk"], a["dks"], a["dv"], a["dvs"], a["work"], a["room"], None)


@pytest.mark.parametrize("change,code,word", COMMON + [
    (dict(dout=None), -1, b"null dout"), (dict(lse=None), -1, b"lse"), (dict(dq=None), -1, b"null dq"),
    (dict(dv=None), -1, b"null dv"), (dict(dk=P(0xb00000)), -1, b"dv overlaps dk"), (dict(dq=P(0x100000)), -1, b"overlaps q"),
    (dict(dk=P(0x200000)), -1, b"overlaps k"), (dict(dv=P(0x400000)), -1, b"overlaps out"),
    (dict(dq=P(0x800040)), -1, b"overlaps dout"), (dict(dks=i64(0, 64, 32)), -1, b"overlaps itself"),
    (dict(work=None), -1, b"workspace"), (dict(work=P(0x600008)), -1, b"16-byte"), (dict(room=16), -3, b"too small"),
])
def test_backward_refusals(lib, change, code, word):
    refused(lib, code, backward(lib, **change), word)


def test_workspaces(lib):
    f, b = lib.attention_forward_workspace_bytes, lib.attention_backward_workspace_bytes
    bad = ctypes.c_size_t(-1).value
    assert f(i64(1, 20280, 20280, 12, 12, 128), 2) == 0  # blocks enough: no splits
    split = f(i64(8, 1, 16384, 32, 8, 128), 2)
    assert split >= 2 * 8 * 32 * 129 * 4
    assert f(i64(2, 8, 9, 4, 3, 32), 1) == bad and f(i64(2, 8, 9, 4, 2, 32), 7) == bad and b(None, 1) == bad
    assert b(i64(2, 8, 9, 4, 2, 32), 1) >= 2 * 8 * 4 * 4
    assert f(i64(0, 8, 9, 4, 2, 32), 1) == 0 and f(i64(2, 0, 9, 4, 2, 32), 1) == 0
    refused(lib, -3, forward(lib, shape=i64(2, 1, 4096, 4, 2, 32), ks=i64(1 << 20, 64, 32), vs=i64(1 << 20, 64, 32),
                             v=P(0x9000000), out=P(0x5000000), room=64), b"too small")
    refused(lib, -1, forward(lib, shape=i64(2, 1, 4096, 4, 2, 32), ks=i64(1 << 20, 64, 32), vs=i64(1 << 20, 64, 32),
                             v=P(0x9000000), out=P(0x5000000), work=P(0x600004)), b"16-byte")


def test_an_empty_call_reads_nothing(lib):
    none = dict(q=None, qs=None, k=None, ks=None, v=None, vs=None, out=None, os=None, lse=None, work=None, room=0)
    assert forward(lib, shape=i64(0, 8, 9, 4, 2, 32), **none) == 0
    assert forward(lib, shape=i64(2, 0, 9, 4, 2, 32), **none) == 0
    assert backward(lib, shape=i64(0, 8, 9, 4, 2, 32), dout=None, dq=None, dk=None, dv=None, **none) == 0
