"""CPU checks of the C entry points of the channels-last group norm and of
dropout: bad arguments are refused on the host; and of the tests' generator."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import channels_ref

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


def test_generator_against_the_published_answers():
    """the known answers that its authors give: zeros, ones and the digits of pi"""
    cases = [((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
             ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
             ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
              (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))]
    for counter, key, want in cases:
        assert tuple(int(w) for w in channels_ref.philox(np.array([counter], np.uint64), key)[0]) == want


GN = dict(x=P(0x100000), xs=i64(384, 64), shape=i64(2, 6, 64), groups=4, eps=1e-6, gamma=P(0x500000), beta=P(0x600000),
          act=1, dtype=1, wdtype=1, out=P(0x200000), os=i64(384, 64), stats=P(0x700000), work=P(0x800000), room=1 << 20)
GN_BAD = [
    (dict(x=None), -1, b"null x"), (dict(xs=None), -1, b"strides of x"), (dict(shape=None), -1, b"null shape"),
    (dict(shape=i64(2, 6, 0)), -1, b"channels"), (dict(shape=i64(-1, 6, 64)), -1, b"samples"),
    (dict(shape=i64(2, 6, 66)), -1, b"multiple"), (dict(groups=0), -1, b"multiple"), (dict(dtype=4), -1, b"dtype"),
    (dict(shape=i64(2, 6, 1 << 17)), -2, b"channels"), (dict(shape=i64(2, 1 << 30, 64)), -2, b"2^30"),
    (dict(shape=i64(1 << 20, 6, 64)), -2, b"2^22"), (dict(shape=i64(1 << 62, 6, 64)), -2, b"2^22"),
    (dict(act=2), -1, b"activation"), (dict(wdtype=2), -1, b"weights"), (dict(gamma=P(0x500001)), -1, b"aligned"),
    (dict(xs=i64(384, -64)), -2, b"strides of x"), (dict(xs=i64(1 << 40, 64)), -2, b"strides of x"),
    (dict(x=P(0x100001)), -1, b"aligned"), (dict(work=None), -1, b"workspace"), (dict(work=P(0x800004)), -1, b"16-byte"),
    (dict(room=32), -3, b"too small"), (dict(stats=P(0x700002)), -1, b"aligned"),
]


@pytest.mark.parametrize("change,code,word", GN_BAD + [
    (dict(eps=-1.0), -1, b"eps"), (dict(eps=float("inf")), -1, b"eps"), (dict(out=None), -1, b"null out"),
    (dict(os=i64(384, 63)), -1, b"overlaps itself"), (dict(out=P(0x100000 + 128)), -1, b"overlaps x"),
    (dict(out=P(0x100000), os=i64(768, 64)), -1, b"overlaps x"),
])
def test_group_norm_forward_refusals(lib, change, code, word):
    a = GN | change
    refused(lib, code, lib.group_norm_forward(a["x"], a["xs"], a["shape"], a["groups"], a["eps"], a["gamma"], a["beta"],
                                              a["act"], a["dtype"], a["wdtype"], a["out"], a["os"], a["stats"], a["work"],
                                              a["room"], None), word)


def backward(lib, **change):
    a = GN | dict(dy=P(0x900000), ys=i64(384, 64), dgamma=P(0xa00000), dbeta=P(0xb00000)) | change
    return lib.group_norm_backward(a["dy"], a["ys"], a["x"], a["xs"], a["shape"], a["groups"], a["stats"], a["gamma"],
                                   a["beta"], a["act"], a["dtype"], a["wdtype"], a["out"], a["os"], a["dgamma"],
                                   a["dbeta"], a["work"], a["room"], None)


@pytest.mark.parametrize("change,code,word", GN_BAD + [
    (dict(dy=None), -1, b"null dy"), (dict(stats=None), -1, b"stats"), (dict(out=None), -1, b"null dx"),
    (dict(out=P(0x900000 + 2)), -1, b"dx overlaps dy"), (dict(dgamma=P(0xa00001)), -1, b"aligned"),
])
def test_group_norm_backward_refusals(lib, change, code, word):
    refused(lib, code, backward(lib, **change), word)


def test_group_norm_workspace(lib):
    f, bad = lib.group_norm_workspace_bytes, ctypes.c_size_t(-1).value
    assert f(i64(2, 6, 64), 4, 1) >= (2 * 2 * 64 + 2 * 4 * 3) * 4
    assert f(i64(2, 6, 64), 5, 1) == bad and f(i64(2, 6, 64), 4, 9) == bad and f(None, 4, 1) == bad
    # partial sums by channel stay a small part of the activation
    assert f(i64(2, 512 * 512, 256), 32, 1) < 2 * 512 * 512 * 256 * 2 // 50
    none = dict(x=None, xs=None, out=None, os=None, work=None, room=0, stats=None, gamma=None, beta=None)
    assert backward(lib, shape=i64(2, 0, 64), dy=None, dgamma=None, dbeta=None, **none) == 0
    a = GN | none | dict(shape=i64(0, 6, 64))
    assert lib.group_norm_forward(a["x"], a["xs"], a["shape"], 4, 1e-6, None, None, 0, 1, 1, None, None, None, None, 0,
                                  None) == 0


@pytest.mark.parametrize("change,code,word", [
    (dict(x=None), -1, b"null x"), (dict(out=None), -1, b"null out"), (dict(shape=None), -1, b"null shape"),
    (dict(state=None), -1, b"state"), (dict(state=P(0x700004)), -1, b"state"), (dict(p=1.0), -1, b"p must"),
    (dict(p=-0.5), -1, b"p must"), (dict(p=float("nan")), -1, b"p must"), (dict(dtype=3), -1, b"dtype"),
    (dict(shape=i64(-1, 3, 64)), -1, b"negative"), (dict(shape=i64(1 << 20, 1 << 20, 4)), -2, b"2^31"),
    (dict(shape=i64(1 << 20, 1, 1 << 20)), -2, b"2^34"), (dict(shape=i64(1, 1, 1 << 60)), -2, b"2^34"),
    (dict(xs=i64(-1, 64)), -2, b"strides of x"), (dict(rs=i64(192, 1 << 41)), -2, b"strides of residual"),
    (dict(os=i64(192, 63)), -1, b"overlaps itself"), (dict(out=P(0x100004)), -1, b"out overlaps x"),
    (dict(out=P(0x300100)), -1, b"out overlaps residual"), (dict(x=P(0x100002)), -1, b"aligned"),
])
def test_dropout_refusals(lib, change, code, word):
    a = dict(x=P(0x100000), xs=i64(192, 64), shape=i64(2, 3, 64), dtype=0, p=0.1, state=P(0x700000), res=P(0x300000),
             rs=i64(192, 64), out=P(0x200000), os=i64(192, 64)) | change
    refused(lib, code, lib.dropout_apply(a["x"], a["xs"], a["shape"], a["dtype"], a["p"], a["state"], 0, a["res"], a["rs"],
                                         a["out"], a["os"], None), word)


def test_dropout_of_nothing_reads_nothing(lib):
    for shape in (i64(0, 3, 64), i64(2, 0, 64), i64(2, 3, 0)):
        assert lib.dropout_apply(None, None, shape, 0, 0.1, None, 0, None, None, None, None, None) == 0
