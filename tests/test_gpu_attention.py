"""attention and attention_backward against their definition in 64 bits, at the
sizes, masks and layouts where a kernel can go wrong."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_ref as ref
from transformer_ref import assert_near, f64

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


def draw(seed, b, nq, nk, hq, hk, d, dtype, sharp=1.0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    q, k, v, g = n(b, nq, hq, d) * sharp, n(b, nk, hk, d), n(b, nk, hk, d) + 0.5 * n(b, 1, hk, d), n(b, nq, hq, d)
    return [t.to(DT[dtype]).cuda() for t in (q, k, v, g)]


def lens(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def check_forward(sb, q, k, v, what, scale=None, **how):
    s = q.shape[-1] ** -0.5 if scale is None else scale
    (out, lse), (tol, tol_lse) = ref.forward(q, k, v, s, how.get("causal", False), how.get("query_lengths"),
                                             how.get("key_lengths"))
    got, got_lse = sb.attention(q, k, v, return_lse=True, scale=scale, **how)
    assert_near(got_lse, lse, tol_lse, what + " lse")
    assert_near(got, out, tol, what + " out")
    return out, lse


def check_backward(sb, q, k, v, g, what, scale=None, **how):
    s = q.shape[-1] ** -0.5 if scale is None else scale
    lengths = how.get("query_lengths"), how.get("key_lengths")
    (out, lse), _ = ref.forward(q, k, v, s, how.get("causal", False), *lengths)
    out, lse = torch.from_numpy(out).to(q.dtype).cuda(), torch.from_numpy(lse).float().cuda()
    want, tol = ref.backward(g, q, k, v, out, lse, s, how.get("causal", False), *lengths)
    got = sb.attention_backward(g, q, k, v, out, lse, scale=scale, **how)
    for name, a, b, t in zip(("dq", "dk", "dv"), got, want, tol):
        assert_near(a, b, t, f"{what} {name}")


SIZES = [
    # b, queries, keys, heads, key heads, D
    (1, 1, 1, 1, 1, 1), (1, 1, 1, 2, 1, 64), (2, 1, 5, 4, 2, 40), (1, 3, 2, 1, 1, 7), (1, 31, 33, 2, 2, 32),
    (1, 32, 32, 1, 1, 128), (2, 33, 31, 3, 1, 64), (1, 64, 65, 2, 2, 96), (1, 65, 64, 1, 1, 80),
    (1, 127, 129, 2, 1, 128), (1, 129, 127, 1, 1, 72), (1, 200, 300, 2, 2, 160), (1, 130, 70, 2, 1, 192),
    (1, 97, 140, 1, 1, 256), (1, 40, 50, 1, 1, 255), (1, 150, 61, 1, 1, 127), (1, 70, 90, 5, 1, 16),
    (1, 45, 77, 8, 8, 31),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("causal", [False, True])
def test_forward(sb, dtype, size, causal):
    q, k, v, _ = draw(1, *size, dtype)
    check_forward(sb, q, k, v, f"{size} {dtype}", causal=causal)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("causal", [False, True])
def test_backward(sb, dtype, size, causal):
    q, k, v, g = draw(2, *size, dtype)
    check_backward(sb, q, k, v, g, f"{size} {dtype}", causal=causal)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("size", [(2, 1, 3000, 8, 2, 128), (1, 4, 1100, 4, 1, 64), (1, 2, 2500, 2, 2, 40),
                                  (1, 40, 1500, 2, 1, 96), (1, 1, 700, 3, 3, 256)], ids=str)
@pytest.mark.parametrize("causal", [False, True])
def test_few_rows_over_many_keys(sb, dtype, size, causal):
    """split over the keys and joined"""
    q, k, v, g = draw(3, *size, dtype)
    assert sb.attention_workspace_bytes(q, k) > 0
    check_forward(sb, q, k, v, f"{size} {dtype}", causal=causal)
    check_backward(sb, q, k, v, g, f"{size} {dtype}", causal=causal)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("size", [(1, 1500, 40, 2, 1, 64), (2, 1030, 77, 2, 2, 40), (1, 700, 9, 1, 1, 256)], ids=str)
@pytest.mark.parametrize("causal", [False, True])
def test_many_rows_over_few_keys(sb, dtype, size, causal):
    """the keys' gradients split over the rows"""
    q, k, v, g = draw(4, *size, dtype)
    check_forward(sb, q, k, v, f"{size} {dtype}", causal=causal)
    check_backward(sb, q, k, v, g, f"{size} {dtype}", causal=causal)


MANY = [
    # samples and heads that fill the chip: the kernels for many rows
    (16, 40, 50, 32, 32, 128), (16, 70, 33, 32, 32, 96), (8, 65, 130, 64, 64, 192), (16, 33, 64, 32, 32, 160),
    (8, 90, 70, 96, 32, 104), (9, 300, 140, 32, 32, 64), (32, 50, 40, 24, 8, 128), (16, 257, 20, 16, 16, 32),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("size", MANY, ids=str)
@pytest.mark.parametrize("causal", [False, True])
def test_many_rows(sb, dtype, size, causal):
    q, k, v, g = draw(17, *size, dtype)
    check_forward(sb, q, k, v, f"{size} {dtype}", causal=causal)
    check_backward(sb, q, k, v, g, f"{size} {dtype}", causal=causal)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("size", [(2, 1060, 1060, 16, 4, 32), (1, 2100, 2050, 4, 4, 64)], ids=str)
def test_causal_tiles_that_share_compute_units(sb, dtype, size):
    """more tiles than units' shares of the chip: the order that sets long ones beside short ones"""
    q, k, v, g = draw(25, *size, dtype)
    check_forward(sb, q, k, v, f"{size} {dtype}", causal=True)
    check_backward(sb, q, k, v, g, f"{size} {dtype}", causal=True)


@pytest.mark.parametrize("size", [(16, 40, 50, 32, 32, 128), (9, 300, 140, 32, 32, 64), (8, 90, 70, 96, 32, 104)], ids=str)
@pytest.mark.parametrize("causal", [False, True])
def test_many_rows_of_unlike_lengths(sb, size, causal):
    q, k, v, g = draw(18, *size, "bf16")
    gen = torch.Generator().manual_seed(19)
    ql = torch.randint(0, size[1] + 1, (size[0],), generator=gen).tolist()
    kl = torch.randint(0, size[2] + 1, (size[0],), generator=gen).tolist()
    ql[0], kl[0], kl[1] = 0, size[2], 0
    kept = [t.clone() for t in (q, k, v, g)]
    for b in range(size[0]):
        q[b, ql[b]:] = g[b, ql[b]:] = float("nan")
        k[b, kl[b]:] = v[b, kl[b]:] = float("inf")
    how = dict(causal=causal, query_lengths=lens(ql), key_lengths=lens(kl))
    scale = size[-1] ** -0.5
    (out, lse), tol = ref.forward(*kept[:3], scale, causal, ql, kl)
    got, got_lse = sb.attention(q, k, v, return_lse=True, **how)
    assert_near(got, out, tol[0], "out")
    assert_near(got_lse, lse, tol[1], "lse")
    out, lse = torch.from_numpy(out).to(q.dtype).cuda(), torch.from_numpy(lse).float().cuda()
    want, tol = ref.backward(kept[3], *kept[:3], out, lse, scale, causal, ql, kl)
    for name, a, w, t in zip(("dq", "dk", "dv"), sb.attention_backward(g, q, k, v, out, lse, **how), want, tol):
        assert_near(a, w, t, name)


LENGTHS = [
    # batch of 4: query lengths, key lengths
    (None, [0, 1, 64, 150]), ([0, 1, 33, 90], None), ([90, 5, 64, 0], [150, 70, 0, 32]), ([90, 40, 1, 2], [20, 40, 9, 1]),
    ([-3, 1000, 90, 90], [1 << 30, 150, -1, 149]),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("of", LENGTHS, ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_lengths(sb, dtype, of, causal, bad):
    """what lies behind a length may hold anything and is not read"""
    q, k, v, g = draw(5, 4, 90, 150, 4, 2, 64, dtype)
    (ql, kl), (want_q, want_k) = of, ref.lengths(*of, q, k)
    for b in range(4):
        q[b, want_q[b]:] = g[b, want_q[b]:] = bad
        k[b, want_k[b]:] = v[b, want_k[b]:] = bad
    how = dict(causal=causal, query_lengths=lens(ql), key_lengths=lens(kl))
    zero = lambda t: torch.where(torch.isfinite(t), t, torch.zeros_like(t))  # noqa: E731
    (out, lse), tol = ref.forward(zero(q), zero(k), zero(v), 0.125, causal, ql, kl)
    got, got_lse = sb.attention(q, k, v, return_lse=True, **how)
    assert_near(got, out, tol[0], "out")
    assert_near(got_lse, lse, tol[1], "lse")
    out, lse = torch.from_numpy(out).to(q.dtype).cuda(), torch.from_numpy(lse).float().cuda()
    want, tol = ref.backward(zero(g), zero(q), zero(k), zero(v), out, lse, 0.125, causal, ql, kl)
    for b in range(4):
        out[b, want_q[b]:] = bad
    for name, a, w, t in zip(("dq", "dk", "dv"), sb.attention_backward(g, q, k, v, out, lse, **how), want, tol):
        assert_near(a, w, t, name)


def test_a_decoding_cache_with_lengths(sb):
    """single tokens over a long cache, lengths ending inside tiles and splits,
    the cache laid out head by head"""
    q, k, v, _ = draw(6, 5, 1, 2000, 8, 2, 128, "bf16")
    kl = [2000, 1999, 513, 1, 0]
    k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
    for b, n in enumerate(kl):
        k[b, n:] = v[b, n:] = float("nan")
    zero = lambda t: torch.nan_to_num(t)  # noqa: E731
    for causal in (False, True):
        (out, lse), tol = ref.forward(q, zero(k), zero(v), 128 ** -0.5, causal, None, kl)
        got, got_lse = sb.attention(q, k, v, causal=causal, key_lengths=lens(kl), return_lse=True)
        assert_near(got, out, tol[0], "out")
        assert_near(got_lse, lse, tol[1], "lse")


@pytest.mark.parametrize("dtype", DT)
def test_no_keys_or_no_queries(sb, dtype):
    q, k, v, g = draw(7, 2, 6, 0, 2, 1, 64, dtype)
    out, lse = sb.attention(q, k, v, return_lse=True)
    assert not out.any() and torch.isinf(lse).all() and (lse < 0).all()
    dq, dk, dv = sb.attention_backward(g, q, k, v, out, lse)
    assert not dq.any() and dk.numel() == dv.numel() == 0
    q, k, v, g = draw(7, 2, 0, 6, 2, 1, 64, dtype)
    out, lse = sb.attention(q, k, v, return_lse=True)
    dq, dk, dv = sb.attention_backward(g, q, k, v, out, lse)
    assert not dk.any() and not dv.any() and out.numel() == dq.numel() == 0
    q, k, v, g = draw(7, 0, 6, 6, 2, 1, 64, dtype)
    assert sb.attention(q, k, v).shape == q.shape


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d", [64, 80, 33])
def test_views(sb, dtype, d):
    """a packed projection read and its gradient written in place; rows at odd
    offsets; [T, heads, D]; a broadcast key"""
    gen = torch.Generator().manual_seed(8)
    whole = torch.randn(2, 75, 6, d + 3, generator=gen).to(DT[dtype]).cuda()
    packed = whole[..., 1:d + 1]
    q, k, v = packed[:, :, :2], packed[:, :, 2:4], packed[:, :, 4:]
    g = torch.randn(2, 75, 2, d, generator=gen).to(DT[dtype]).cuda()
    check_forward(sb, q, k, v, "packed")
    check_backward(sb, q, k, v, g, "packed")
    scale = d ** -0.5
    out, lse = sb.attention(q, k, v, return_lse=True)
    dwhole = torch.full_like(whole, 7.0)
    to = dwhole[..., 1:d + 1]
    plain = sb.attention_backward(g, q, k, v, out, lse)
    views = to[:, :, :2], to[:, :, 2:4], to[:, :, 4:]
    sb.attention_backward(g, q, k, v, out, lse, dq=views[0], dk=views[1], dv=views[2])
    for a, b in zip(views, plain):
        assert torch.equal(a, b)
    assert (dwhole[..., 0] == 7.0).all() and (dwhole[..., d + 1:] == 7.0).all()
    room = torch.full((2, 75, 2, d + 5), 7.0, dtype=DT[dtype], device="cuda")
    sb.attention(q, k, v, out=room[..., 3:d + 3])
    assert torch.equal(room[..., 3:d + 3], out) and (room[..., :3] == 7.0).all() and (room[..., d + 3:] == 7.0).all()
    flat = sb.attention(q[0], k[0], v[0])
    assert torch.equal(flat, out[0])
    one = k[:1].expand(2, -1, -1, -1)
    check_forward(sb, q, one, v, "broadcast", scale=scale)
    # without `out=`, a broadcast tensor's gradient is one for each of its uses
    check_backward(sb, q, one, v, g, "broadcast", scale=scale)


@pytest.mark.parametrize("dtype", DT)
def test_large_scores_and_scale(sb, dtype):
    """scores of hundreds: the running maximum moves often, most of P vanishes"""
    q, k, v, g = draw(9, 1, 70, 200, 2, 1, 64, dtype, sharp=30.0)
    check_forward(sb, q, k, v, "sharp")
    check_backward(sb, q, k, v, g, "sharp")
    k = k * torch.linspace(0.0, 1.0, 200, device="cuda").to(k.dtype)[:, None, None]  # growing along the keys
    check_forward(sb, q, k, v, "growing", causal=True)
    check_forward(sb, q, k, v, "scale", scale=0.7)
    check_backward(sb, q, k, v, g, "scale", scale=1e-3)


def test_nan_and_infinity_reach_their_rows(sb):
    q, k, v, _ = draw(10, 1, 40, 50, 1, 1, 64, "bf16")
    q[0, 3] = float("nan")
    out, lse = sb.attention(q, k, v, return_lse=True)
    assert torch.isnan(out[0, 3]).all() and torch.isnan(lse[0, 0, 3])
    rest = torch.arange(40, device="cuda") != 3
    assert torch.isfinite(out[0, rest]).all() and torch.isfinite(lse[0, 0, rest]).all()
    v[0, 7, 0, 5] = float("inf")
    out = sb.attention(q, k, v)
    assert torch.isinf(out[0, rest, 0, 5]).all() and torch.isfinite(out[0, rest, 0, :5]).all()


def test_gradient_against_differences(sb):
    """the gradients' products with a direction against the loss's differences, the
    loss from the 64-bit definition"""
    q, k, v, g = draw(11, 1, 40, 45, 2, 1, 48, "fp32")
    out, lse = sb.attention(q, k, v, causal=True, return_lse=True)
    grads = [f64(t) for t in sb.attention_backward(g, q, k, v, out, lse, causal=True)]
    gen = torch.Generator().manual_seed(12)
    step = 1e-4
    for i, (x, d) in enumerate(zip((q, k, v), grads)):
        way = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        losses = []
        for sign in (1, -1):
            moved = [t.cpu().double() for t in (q, k, v)]
            moved[i] = moved[i] + sign * step * way
            p = [m.numpy() for m in moved]
            loss = 0.0
            for h in range(2):
                pr, _, _, _ = ref.probabilities(p[0][0, :, h], p[1][0, :, 0], 48 ** -0.5, True, torch.float32)
                loss += (f64(g)[0, :, h] * (pr @ p[2][0, :, 0])).sum()
            losses.append(loss)
        # the differences' own error is their third derivative's, step^2; the gradient's
        # some 1e-6 of the sum of its terms' magnitudes
        want = (losses[0] - losses[1]) / (2 * step)
        assert abs(want - (d * way.numpy()).sum()) <= 1e-5 * np.abs(d * way.numpy()).sum()


@pytest.mark.parametrize("dtype", DT)
def test_same_bits_every_time(sb, dtype):
    for size in ((2, 1, 3000, 8, 2, 128), (1, 300, 260, 4, 2, 64), (16, 60, 70, 32, 32, 128)):
        q, k, v, g = draw(13, *size, dtype)
        out, lse = sb.attention(q, k, v, return_lse=True)
        grads = sb.attention_backward(g, q, k, v, out, lse)
        for _ in range(3):
            again = sb.attention(q, k, v, return_lse=True)
            assert torch.equal(again[0], out) and torch.equal(again[1], lse)
            assert all(torch.equal(a, b) for a, b in zip(sb.attention_backward(g, q, k, v, out, lse), grads))


@pytest.mark.parametrize("size", [(3, 1, 1500, 4, 2, 64), (1, 200, 150, 4, 2, 64), (1, 900, 30, 2, 2, 32)], ids=str)
def test_prepared_calls_in_a_graph(sb, size):
    """captured, replayed on changed inputs and lengths, with eager work between"""
    q, k, v, g = draw(14, *size, "bf16")
    kl = lens([size[2]] * size[0])
    forward = sb.Attention(q, k, v, key_lengths=kl, return_lse=True)
    forward()
    back = sb.AttentionBackward(g, q, k, v, forward.out, forward.lse, key_lengths=kl)
    back()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward()
        back()
    for turn in range(4):
        fresh = draw(20 + turn, *size, "bf16")
        for t, f in zip((q, k, v, g), fresh):
            t.copy_(f)
        kl.copy_(lens([max(0, size[2] - 7 * turn - b) for b in range(size[0])]))
        graph.replay()
        torch.cuda.synchronize()
        out, lse = sb.attention(*fresh[:3], key_lengths=kl, return_lse=True)
        assert torch.equal(forward.out, out) and torch.equal(forward.lse, lse)
        for a, b in zip(back.out, sb.attention_backward(fresh[3], *fresh[:3], out, lse, key_lengths=kl)):
            assert torch.equal(a, b)


def test_two_streams_at_once(sb):
    sets = [draw(30 + i, 2, 1, 2000, 8, 2, 128, "fp16") for i in range(2)]
    want = [sb.attention(*s[:3]) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for i, (s, t) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(s):
                got[i].append(sb.attention(*t[:3]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_writes_raise_the_version(sb):
    q, k, v, g = draw(15, 1, 8, 9, 2, 1, 32, "fp32")
    out, lse = torch.empty_like(q), torch.empty(1, 2, 8, device="cuda")
    grads = [torch.empty_like(t) for t in (q, k, v)]
    for what, call in ((out, lambda: sb.attention(q, k, v, out=out)), (lse, lambda: sb.attention(q, k, v, lse=lse)),
                       (out, sb.Attention(q, k, v, out=out, lse=lse)), (lse, sb.Attention(q, k, v, out=out, lse=lse)),
                       (grads[0], lambda: sb.attention_backward(g, q, k, v, out, lse, dq=grads[0])),
                       (grads[1], lambda: sb.attention_backward(g, q, k, v, out, lse, dk=grads[1])),
                       (grads[2], sb.AttentionBackward(g, q, k, v, out, lse, dv=grads[2]))):
        before, read = what._version, [t._version for t in (q, k, v, g)]
        call()
        assert what._version > before and [t._version for t in (q, k, v, g)] == read


def test_refusals(sb):
    q, k, v, g = draw(16, 2, 8, 9, 4, 2, 32, "fp16")
    out, lse = sb.attention(q, k, v, return_lse=True)
    bad = [
        (TypeError, lambda: sb.attention(q.cpu(), k, v)), (TypeError, lambda: sb.attention(q.double(), k, v)),
        (ValueError, lambda: sb.attention(q, k.float(), v)), (ValueError, lambda: sb.attention(q, k, v[:, :5])),
        (ValueError, lambda: sb.attention(q, k[:1], v[:1])), (ValueError, lambda: sb.attention(q, k[..., :16], v[..., :16])),
        (ValueError, lambda: sb.attention(q, k[0], v[0])), (ValueError, lambda: sb.attention(q[..., ::2], k, v)),
        (ValueError, lambda: sb.attention(q, k, v, key_lengths=torch.ones(2, device="cuda"))),
        (ValueError, lambda: sb.attention(q, k, v, key_lengths=lens([1]))),
        (ValueError, lambda: sb.attention(q, k, v, query_lengths=torch.ones(2, dtype=torch.int32))),
        (ValueError, lambda: sb.attention(q, k, v, out=out.float())), (ValueError, lambda: sb.attention(q, k, v, lse=lse[:1])),
        (sb.SeamBlendError, lambda: sb.attention(q, k, v, scale=0.0)),
        (sb.SeamBlendError, lambda: sb.attention(q, k, v, scale=float("nan"))),
        (sb.SeamBlendError, lambda: sb.attention(q[:, :, :3], k, v)),
        (sb.SeamBlendError, lambda: sb.attention(q, k, v, out=q)),
        (sb.SeamBlendError, lambda: sb.attention_backward(g, q, k, v, out, lse, dq=q)),
        (sb.SeamBlendError, lambda: sb.attention_backward(g, q, k, v, out, lse, dq=g)),
        (sb.SeamBlendError, lambda: sb.attention_backward(g, q, k, v, out, lse, dk=out[:1, :9 - 1].new_empty(1, 9, 2, 32).expand(2, -1, -1, -1))),
        (ValueError, lambda: sb.attention_backward(g[:, :3], q, k, v, out, lse)),
        (ValueError, lambda: sb.attention_backward(g, q, k, v, out, lse.half())),
        (ValueError, lambda: sb.attention(q, k, v, workspace=torch.empty(8, dtype=torch.uint8))),
    ]
    for k_, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {k_} was not refused")
    far = torch.empty(2, 3000, 2, 32, dtype=torch.float16, device="cuda")
    with pytest.raises(sb.SeamBlendError, match="workspace too small"):
        sb.attention(q[:, :1], far, far, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
