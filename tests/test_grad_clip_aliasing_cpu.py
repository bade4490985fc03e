"""CPU checks of what grad_norm_clip refuses to write: memory that another
tensor of the call has too.  A refusal comes before any device work."""
from __future__ import annotations

import ctypes
import random

import pytest

P = ctypes.c_void_p
BYTES = {0: 4, 1: 2, 2: 2}


@pytest.fixture(scope="module")
def lib():
    import seam_blending_patch_amd as sb
    return sb._lib


def call(lib, grads, outs=None, function="grad_norm_clip"):
    """(code, message) of a call over (address, elements, dtype) tensors."""
    n = len(grads)
    ptrs = lambda ts: (ctypes.c_void_p * n)(*[t[0] for t in ts])  # noqa: E731
    ints = lambda ts: (ctypes.c_int * n)(*[t[2] for t in ts])  # noqa: E731
    numels = (ctypes.c_int64 * n)(*[t[1] for t in grads])
    tail = (P(0x10), P(0x20), 1 << 30, None)
    if function == "grad_norm":
        rc = lib.grad_norm(ptrs(grads), numels, ints(grads), n, *tail)
    else:
        rc = lib.grad_norm_clip(ptrs(grads), None if outs is None else ptrs(outs), numels, ints(grads),
                                None if outs is None else ints(outs), n, 1.0, 1e-6, *tail)
    return rc, lib.seamblend_last_error()


A, B, C = 0x100000, 0x200000, 0x300000


@pytest.mark.parametrize("grads,outs,word", [
    # in place: gradients that share elements
    ([(A, 100, 0), (A + 16, 96, 0)], None, b"gradient 1 shares memory with gradient 0"),
    ([(A + 16, 96, 0), (A, 100, 0)], None, b"gradient 0 shares memory with gradient 1"),
    ([(A, 100, 0), (B, 7, 2), (A + 396, 1, 0)], None, b"gradient 2 shares memory with gradient 0"),
    ([(A, 100, 0), (A, 100, 0)], None, b"shares memory with gradient"),
    ([(A, 100, 0), (A + 200, 4, 2), (A + 396, 1, 0)], None, b"shares memory with gradient 0"),
    ([(A, 100, 1), (A + 199, 1, 0)], None, b"gradient 1"),  # (not aligned: refused all the same)
    # outputs that share elements
    ([(A, 100, 0), (B, 100, 0)], [(C, 100, 0), (C + 396, 100, 0)], b"output 1 shares memory with output 0"),
    ([(A, 100, 2), (B, 100, 2)], [(C + 396, 100, 0), (C, 100, 0)], b"output 0 shares memory with output 1"),
    ([(A, 1, 2), (B, 100, 2)], [(C + 4, 1, 2), (C, 100, 2)], b"shares memory with output"),
    # an output over another tensor's gradient
    ([(A, 100, 0), (B, 100, 0)], [(B, 100, 0), (C, 100, 0)], b"output 0 shares memory with gradient 1"),
    ([(A, 100, 0), (B, 100, 0)], [(B, 100, 0), (A, 100, 0)], b"shares memory with gradient"),
    ([(A, 100, 2), (A + 200, 100, 2)], [(A, 100, 2), (A + 398, 100, 2)], b"output 1 overlaps its gradient"),
    ([(A, 100, 2), (A + 200, 100, 2), (B, 1, 2)], [(A, 100, 2), (A + 200, 100, 2), (A + 398, 1, 2)],
     b"shares memory with"),
    ([(A, 100, 0), (A + 40, 10, 0)], [(A, 100, 0), (C, 10, 0)], b"output 0 shares memory with gradient 1"),
])
def test_refused(lib, grads, outs, word):
    rc, message = call(lib, grads, outs)
    assert rc == -1 and word in message, (rc, message)


@pytest.mark.parametrize("grads,outs", [
    ([(A, 100, 0), (A + 400, 100, 0)], None),  # neighbours in a bucket, in any order
    ([(A + 400, 100, 0), (A, 100, 0)], None),
    ([(A + 200, 50, 2), (A, 50, 0)], None),
    ([(A, 100, 0), (0, 0, 0), (A, 0, 0), (A + 40, 0, 2)], None),  # nothing in the others
    ([(A, 100, 0), (A, 100, 0)], [(B, 100, 0), (C, 100, 0)]),  # read twice, written apart
    ([(A, 100, 0), (A + 40, 10, 0)], [(B, 100, 0), (B + 400, 10, 0)]),
    ([(A, 100, 0), (B, 50, 2)], [(A, 100, 0), (C, 50, 0)]),  # one in place, one out
])
def test_taken(lib, grads, outs):
    """(What a call without a refusal runs into here is the missing GPU.)"""
    if _gpu():
        pytest.skip("the addresses are made up")
    rc, message = call(lib, grads, outs)
    assert rc == -4, (rc, message)


def _gpu():
    import torch
    return torch.cuda.is_available()


def test_a_norm_alone_takes_shared_memory(lib):
    if _gpu():
        pytest.skip("the addresses are made up")
    rc, message = call(lib, [(A, 100, 0), (A + 16, 96, 0), (A, 100, 0)], function="grad_norm")
    assert rc == -4, (rc, message)


def _shared(a, b):
    return a[1] and b[1] and a[0] < b[0] + b[1] * BYTES[b[2]] and b[0] < a[0] + a[1] * BYTES[a[2]]


def test_against_every_pair(lib):
    """Random small lists in a few hundred bytes: refused exactly where a written
    tensor shares a byte with another one (or with its own gradient, unless it
    is that gradient)."""
    if _gpu():
        pytest.skip("the addresses are made up")
    rng = random.Random(7)
    answers = {True: 0, False: 0}
    for _ in range(6000):
        n = rng.randint(1, 6)
        room = rng.choice((160, 640, 2560))
        tensor = lambda k, types: (A + 4 * rng.randrange(room), k, rng.choice(types))  # noqa: E731
        grads = [tensor(rng.choice((0, 1, 3, 17, 40)), (0, 1, 2)) for _ in range(n)]
        outs = None
        if rng.random() < 0.6:
            outs = [g if rng.random() < 0.3 else tensor(g[1], (0, g[2])) for g in grads]
        written = grads if outs is None else outs
        bad = any(_shared(written[i], written[j]) for i in range(n) for j in range(i))
        for i in range(n):
            for j in range(n):
                if outs is not None and not (i == j and outs[i][0] == grads[i][0] and outs[i][2] == grads[i][2]):
                    bad = bad or bool(_shared(outs[i], grads[j]))
        rc, message = call(lib, grads, outs)
        assert rc == (-1 if bad else -4 if any(g[1] for g in grads) else rc), (grads, outs, rc, message)
        answers[bad] += 1
    assert min(answers.values()) > 500, answers


def test_many_tensors(lib):
    """As many as a call takes, in an order far from their addresses'."""
    n = 1 << 16
    order = list(range(n))
    random.Random(1).shuffle(order)
    grads = [(A + 16 * k, 4, 0) for k in order]
    grads[77] = (grads[76][0] + 12, 4, 0)  # one element of the one before, and three of the next
    rc, message = call(lib, grads)
    assert rc == -1 and b"shares memory with gradient" in message
    rc, message = call(lib, grads + [(A, 1, 0)])
    assert rc == -2 and b"2^16 tensors" in message
