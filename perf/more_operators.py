"""What the library's operators of a block over latents are measured on.

Latents are made by transformers over latent tokens and by U-Nets, and decoded
by a VAE.  Measured here are what their blocks need beside layer norm, rotary
embedding and clipping:

  attention     of query heads over key and value heads, forward and backward
                (the probabilities are formed again), from single tokens over a
                long cache to a clip's tokens among each other;
  group norm    channels last, with its activation, forward and backward;
  dropout       from a counter-based generator, the residual added.

Every pass runs either in a plain form (elementary torch operations in 32
bits) or, where ``own`` is set, as the call a user makes of the library.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
#: what the largest listed cases cost: products of attention, elements of the others
MOST_FORWARD = 4 * 20280 ** 2 * 12 * 128
MOST_BACKWARD = 10 * 10140 ** 2 * 12 * 128
MOST_SCORES = 20280 ** 2 * 12
MOST_NORM = 2 * 512 * 512 * 256
MOST_NORM_GRAD = 256 * 256 * 512
MOST_DROPOUT = 65536 * 2048


def listed():
    return [
        # one new token for each of 8 requests over a cache filled to different
        # lengths, 4 query heads to a key head
        attention("attention_token", "forward", 8, 1, 16384, 32, 8, 128, "bf16", True, "keys"),
        # image tokens attend to a short text, padded to different lengths: one
        # level of a U-Net, heads of 40
        attention("attention_text", "forward", 2, 4096, 77, 8, 8, 40, "fp16", False, "keys"),
        # the latent tokens of a 49-frame 480x832 clip (13 x 30 x 52), read in place
        # from the packed query-key-value projection
        attention("attention_video", "forward", 1, 20280, 20280, 12, 12, 128, "bf16", False, "none", packed=True),
        # a text encoder's causal layer in full precision, odd length, shared key heads
        attention("attention_causal", "forward", 2, 2049, 2049, 16, 4, 80, "fp32", True, "none"),
        # training on a padded batch (its last sample empty), causal, shared key heads
        attention("attention_grad_causal", "backward", 3, 1537, 1537, 16, 4, 64, "fp16", True, "both"),
        # a training step over the tokens of a 49-frame 480x416 clip (13 x 30 x 26)
        attention("attention_grad_video", "backward", 1, 10140, 10140, 12, 12, 128, "bf16", False, "none",
                  packed=True),
        # the middle of a U-Net at a batch of 2: 32 x 32 positions, 10 channels a group
        group_norm("group_norm_latent", "forward", 2, 32 * 32, 320, 32, "fp16", "silu", "same"),
        # a VAE decoder's last level for two 512 x 512 tiles: the largest activation
        group_norm("group_norm_decoder", "forward", 2, 512 * 512, 256, 32, "fp16", "silu", "same"),
        # fine-tuning a decoder's level in 16 bits, master weights in 32
        group_norm("group_norm_grad_decoder", "backward", 1, 256 * 256, 512, 32, "bf16", "silu", "fp32"),
        # odd sizes in full precision, 3 channels a group, no activation
        group_norm("group_norm_grad_ragged", "backward", 3, 33 * 47, 96, 32, "fp32", "none", "fp32"),
        # adapter training on one short text
        dropout("dropout_text", 77, 768, "fp32", 0.1, False, "forward"),
        # behind the projection of a 4096 x 4096 image's tokens, onto the residual stream
        dropout("dropout_image", 65536, 2048, "bf16", 0.1, True, "forward"),
    ]


def attention(name, way, batch, queries, keys, q_heads, k_heads, width, dtype, causal, ragged, packed=False):
    """``ragged``: which lengths differ over the batch: none, those of the keys, or
    both (then the queries are as long as the keys)."""
    return {"name": name, "kind": "attention", "way": way, "batch": batch, "queries": queries, "keys": keys,
            "q_heads": q_heads, "k_heads": k_heads, "width": width, "dtype": dtype, "causal": causal,
            "ragged": ragged, "packed": packed}


def group_norm(name, way, batch, positions, channels, groups, dtype, activation, weights):
    return {"name": name, "kind": "group_norm", "way": way, "batch": batch, "positions": positions,
            "channels": channels, "groups": groups, "dtype": dtype, "activation": activation, "weights": weights}


def dropout(name, tokens, width, dtype, p, residual, way):
    return {"name": name, "kind": "dropout", "way": way, "tokens": tokens, "width": width, "dtype": dtype, "p": p,
            "residual": residual}


def log_uniform(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    kind = rng.choice(("attention_forward", "attention_backward", "group_norm_forward", "group_norm_backward",
                       "dropout"))
    dtype = rng.choice(("fp32", "fp16", "bf16"))
    if kind.startswith("attention"):
        way = kind[10:]
        k_heads = log_uniform(rng, 1, 16)
        q_heads = k_heads * rng.choice((1, 1, 2, 4))
        width = rng.choice((32, 40, 64, 72, 80, 96, 128, 128, 160, 256))
        batch = log_uniform(rng, 1, 8)
        form = rng.choice(("token", "text", "self")) if way == "forward" else rng.choice(("text", "self", "self"))
        each, most = (4, MOST_FORWARD) if way == "forward" else (10, MOST_BACKWARD)
        if dtype == "fp32":
            most //= 16  # the matrix cores take fp32 at a sixteenth of the 16-bit rate
        pairs = min(most // (each * width), MOST_SCORES) // (batch * q_heads)
        if form == "token":
            queries, keys = rng.randint(1, 4), log_uniform(rng, 1, min(32768, pairs // 4))
        elif form == "text":
            # one key alone takes any weight whatever its score: nothing but rounding is its gradient
            keys = log_uniform(rng, 1 if way == "forward" else 8, 512)
            queries = log_uniform(rng, 16, min(16384, pairs // keys))
        else:
            queries = keys = log_uniform(rng, 16, min(16384, math.isqrt(pairs)))
        ragged = rng.choice(("none", "keys", "both") if form == "self" else ("none", "keys"))
        case = attention("", way, batch, queries, keys, q_heads, k_heads, width, dtype,
                         form != "text" and rng.random() < 0.5, ragged, packed=form == "self" and rng.random() < 0.4)
    elif kind.startswith("group_norm"):
        way = kind[11:]
        groups = rng.choice((1, 8, 16, 32, 32))
        channels = groups * rng.choice((1, 2, 3, 4, 8, 10, 16, 20, 30))
        most = MOST_NORM if way == "forward" else MOST_NORM_GRAD
        room = most // (2 if dtype == "fp32" else 1)
        batch = log_uniform(rng, 1, 8)
        # a group of a few numbers has next to no gradient: its values cannot but be what they are
        positions = log_uniform(rng, 1 if way == "forward" else 24, min(262144, room // (channels * batch)))
        case = group_norm("", way, batch, positions, channels, groups, dtype, rng.choice(("silu", "silu", "none")),
                          rng.choice(("fp32", "same", "none")))
    else:
        way = rng.choice(("forward", "forward", "backward"))
        width = log_uniform(rng, 16, 8192)
        room = MOST_DROPOUT // (2 if dtype == "fp32" else 1) // width
        case = dropout("", log_uniform(rng, 1, min(65536, room)), width, dtype, rng.choice((0.0, 0.1, 0.25, 0.5)),
                       way == "forward" and rng.random() < 0.6, way)
    del case["name"]
    return case


def lengths(case):
    """(query lengths, key lengths) of a batch, as lists: falling evenly from whole
    to empty (none is empty in a batch of 1 or 2).  Without lengths of their own
    all are whole."""
    b = case["batch"]
    steps = [(b - k) / b for k in range(b)] if b < 3 else [(b - 1 - k) / (b - 1) for k in range(b)]
    of = lambda n: [math.ceil(n * s) for s in steps]  # noqa: E731
    q = of(case["queries"]) if case["ragged"] == "both" else [case["queries"]] * b
    return q, of(case["keys"]) if case["ragged"] != "none" else [case["keys"]] * b


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"attention": prepare_attention, "group_norm": prepare_group_norm,
            "dropout": prepare_dropout}[case["kind"]](case, gen)


def normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def prepare_attention(case, gen):
    dt, b, d = DTYPES[case["dtype"]], case["batch"], case["width"]
    nq, nk, hq, hk = case["queries"], case["keys"], case["q_heads"], case["k_heads"]
    if case["packed"]:  # query, key and value heads of one projection
        whole = normal(gen, b, nq, hq + 2 * hk, d)
        q, k, v = whole.split((hq, hk, hk), 2)
    else:
        q, k, v = normal(gen, b, nq, hq, d), normal(gen, b, nk, hk, d), normal(gen, b, nk, hk, d)
    # normed heads whose learned gains differ: diffuse heads beside sharp ones
    q *= (0.5 + 2.0 * torch.rand(hq, 1, generator=gen, device="cuda"))
    v += 0.5 * normal(gen, b, 1, hk, d)
    q_len = k_len = None
    if case["ragged"] != "none":
        lq, lk = lengths(case)
        k_len = torch.tensor(lk, dtype=torch.int32, device="cuda")
        past = torch.arange(nk, device="cuda") >= k_len[:, None]
        for t in (k, v):  # a cache's rows behind its length were never written
            t.masked_fill_(past[:, :, None, None], math.nan)
        if case["ragged"] == "both":
            q_len = torch.tensor(lq, dtype=torch.int32, device="cuda")
            q.masked_fill_((torch.arange(nq, device="cuda") >= q_len[:, None])[:, :, None, None], math.nan)
    if case["packed"]:
        q, k, v = whole.to(dt).split((hq, hk, hk), 2)
    else:
        q, k, v = q.to(dt), k.to(dt), v.to(dt)
    s = {"case": case, "q": q, "k": k, "v": v, "q_len": q_len, "k_len": k_len, "scale": d ** -0.5}
    if case["way"] == "backward":  # what the forward pass left
        left = plain_attention(s)
        s["dout"] = normal(gen, b, nq, hq, d).to(dt)
        s["out"], s["lse"] = left["out"], left["lse"]
    return s


def prepare_group_norm(case, gen):
    dt, b, n, c, g = DTYPES[case["dtype"]], case["batch"], case["positions"], case["channels"], case["groups"]
    # what a convolution leaves: a mean of its own in every channel, some loud ones
    x = normal(gen, b, n, c)
    x *= 0.3 + normal(gen, c).abs()
    x = x.add_(normal(gen, c)).to(dt)
    gamma = beta = None
    if case["weights"] != "none":
        wt = torch.float32 if case["weights"] == "fp32" else dt
        gamma, beta = (1 + 0.2 * normal(gen, c)).to(wt), (0.2 * normal(gen, c)).to(wt)
    s = {"case": case, "x": x, "gamma": gamma, "beta": beta,
         "activation": None if case["activation"] == "none" else case["activation"]}
    if case["way"] == "backward":
        s["dy"] = normal(gen, b, n, c).to(dt)
        # what the forward pass left: each group's mean as the sum of two numbers,
        # and one over its deviation
        h = x.view(b, n, g, c // g)
        mean = h.mean((1, 3), dtype=torch.float64)
        var = (h.float() - mean.float()[:, None, :, None]).square().mean((1, 3), dtype=torch.float64) \
            - (mean.float() - mean).square()
        s["stats"] = torch.stack((mean.float(), (mean - mean.float()).float(), torch.rsqrt(var + EPS).float()), -1)
    return s


def prepare_dropout(case, gen):
    dt = DTYPES[case["dtype"]]
    x = normal(gen, case["tokens"], case["width"]).to(dt)
    residual = normal(gen, case["tokens"], case["width"]).to(dt) if case["residual"] else None
    # the generator's seed and the step's offset
    state = torch.randint(1 << 62, (2,), generator=gen, device="cuda")
    return {"case": case, "x": x, "residual": residual, "state": state, "site": 3}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        return run_own(s, case)
    if case["kind"] == "attention":
        return plain_attention(s) if case["way"] == "forward" else plain_attention_backward(s)
    if case["kind"] == "group_norm":
        return plain_group_norm(s) if case["way"] == "forward" else plain_group_norm_backward(s)
    return plain_dropout(s)


def run_own(s, case):
    import seam_blending_patch_amd as sb
    if case["kind"] == "attention":
        how = dict(causal=case["causal"], scale=s["scale"], query_lengths=s["q_len"], key_lengths=s["k_len"])
        if case["way"] == "forward":
            out, lse = sb.attention(s["q"], s["k"], s["v"], return_lse=True, **how)
            return {"out": out, "lse": lse}
        dq, dk, dv = sb.attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], **how)
        return {"dq": dq, "dk": dk, "dv": dv}
    if case["kind"] == "group_norm":
        if case["way"] == "forward":
            return {"y": sb.group_norm(s["x"], case["groups"], s["gamma"], s["beta"], eps=EPS,
                                       activation=s["activation"])}
        dx, dgamma, dbeta = sb.group_norm_backward(s["dy"], s["x"], case["groups"], s["stats"], s["gamma"], s["beta"],
                                                   activation=s["activation"])
        return {"dx": dx} if dgamma is None else {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if case["way"] == "forward":
        return {"y": sb.dropout(s["x"], case["p"], s["state"], site=s["site"], residual=s["residual"])}
    return {"dx": sb.dropout_backward(s["x"], case["p"], s["state"], site=s["site"])}


def hidden(s):
    """[B, 1, 1, queries, keys] of True where a query does not see a key, or None."""
    case = s["case"]
    b, nq, nk = case["batch"], case["queries"], case["keys"]
    if s["k_len"] is None and not case["causal"]:
        return None
    i, j = torch.arange(nq, device="cuda")[:, None], torch.arange(nk, device="cuda")
    lk = torch.full((b, 1, 1), nk, device="cuda") if s["k_len"] is None else s["k_len"][:, None, None]
    lq = torch.full((b, 1, 1), nq, device="cuda") if s["q_len"] is None else s["q_len"][:, None, None]
    no = (j >= lk) | (i >= lq)
    if case["causal"]:  # the last query sees the last key
        no = no | (j > i + (lk - lq))
    return no[:, None, None]


def heads_first(t, groups, live=None):
    """[B, T, H, D] as [B, groups, H / groups, T, D] in 32 bits; rows past a
    length, which may hold anything, as zeros."""
    t = t.unflatten(2, (groups, -1)).permute(0, 2, 3, 1, 4).float()
    if live is not None:
        past = torch.arange(t.shape[3], device="cuda") >= live[:, None]
        t = t.masked_fill(past[:, None, None, :, None], 0.0)
    return t.contiguous()


def tokens_first(t, dtype):
    return t.permute(0, 3, 1, 2, 4).flatten(2, 3).to(dtype).contiguous()


def plain_weights(s, q, k):
    """(probabilities, log of their sums): rows that see no key are zeros and -inf."""
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    no = hidden(s)
    if no is not None:
        p.masked_fill_(no, -math.inf)
    most = p.amax(-1, keepdim=True)
    p.sub_(most.masked_fill(most == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(total.masked_fill(total == 0.0, 1.0))
    return p, (most + torch.log(total)).squeeze(-1)


def plain_attention(s):
    hk = s["case"]["k_heads"]
    q, k, v = heads_first(s["q"], hk, s["q_len"]), heads_first(s["k"], hk, s["k_len"]), heads_first(s["v"], hk, s["k_len"])
    p, lse = plain_weights(s, q, k)
    return {"out": tokens_first(torch.matmul(p, v), s["q"].dtype), "lse": lse.flatten(1, 2)}


def plain_attention_backward(s):
    hk, dt = s["case"]["k_heads"], s["q"].dtype
    q, k, v = heads_first(s["q"], hk, s["q_len"]), heads_first(s["k"], hk, s["k_len"]), heads_first(s["v"], hk, s["k_len"])
    dout = heads_first(s["dout"], hk, s["q_len"])
    p, _ = plain_weights(s, q, k)
    dv = torch.matmul(p.transpose(-1, -2), dout).sum(2, keepdim=True)
    ds = torch.matmul(dout, v.transpose(-1, -2))
    ds.sub_((ds * p).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2, keepdim=True)
    return {"dq": tokens_first(torch.matmul(ds, k), dt), "dk": tokens_first(dk, dt), "dv": tokens_first(dv, dt)}


def plain_group_norm(s):
    case = s["case"]
    x = s["x"].float().unflatten(-1, (case["groups"], -1))
    d = x - x.mean((1, 3), keepdim=True)
    y = (d * torch.rsqrt((d * d).mean((1, 3), keepdim=True) + EPS)).flatten(-2)
    if s["gamma"] is not None:
        y = y * s["gamma"].float() + s["beta"].float()
    if s["activation"] is not None:
        y = y / (1 + torch.exp(-y))
    return {"y": y.to(s["x"].dtype)}


def plain_group_norm_backward(s):
    case = s["case"]
    mean, rest, rstd = (t[:, None, :, None] for t in s["stats"].unbind(-1))
    h = ((s["x"].float().unflatten(-1, (case["groups"], -1)) - mean) - rest) * rstd
    flat = h.flatten(-2)
    g = s["dy"].float()
    if s["activation"] is not None:
        z = flat if s["gamma"] is None else flat * s["gamma"].float() + s["beta"].float()
        t = 1 / (1 + torch.exp(-z))
        g = g * (t * (1 + z * (1 - t)))
    a = (g if s["gamma"] is None else g * s["gamma"].float()).unflatten(-1, (case["groups"], -1))
    dx = (rstd * (a - a.mean((1, 3), keepdim=True) - h * (a * h).mean((1, 3), keepdim=True))).flatten(-2)
    if s["gamma"] is None:
        return {"dx": dx.to(s["x"].dtype)}
    wt = s["gamma"].dtype
    return {"dx": dx.to(s["x"].dtype), "dgamma": (g * flat).sum((0, 1)).to(wt), "dbeta": g.sum((0, 1)).to(wt)}


def wide_product(m, x):
    """(high, low) 32 bits of the product of two 32-bit numbers held in 64-bit
    ones, x in two halves so that nothing passes 63 bits."""
    low, high = m * (x & 0xFFFF), m * (x >> 16)
    return (high + (low >> 16)) >> 16, (low + ((high & 0xFFFF) << 16)) & 0xFFFFFFFF


def plain_words(n, state, site):
    """The generator's 32-bit words for elements 0..n: Philox4x32 with ten rounds
    (Salmon, Moraes, Dror and Shaw, 2011), four words to a counter."""
    blocks = torch.arange((n + 3) // 4, device="cuda")
    k0, k1 = state[0] & 0xFFFFFFFF, (state[0] >> 32) & 0xFFFFFFFF
    a, b = blocks, torch.full_like(blocks, site)
    c, d = (state[1] & 0xFFFFFFFF).expand_as(blocks), ((state[1] >> 32) & 0xFFFFFFFF).expand_as(blocks)
    for _ in range(10):  # the generator's rounds
        (h0, l0), (h1, l1) = wide_product(0xD2511F53, a), wide_product(0xCD9E8D57, c)
        a, b, c, d = h1 ^ b ^ k0, l1, h0 ^ d ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return torch.stack((a, b, c, d), -1).flatten()[:n]


def plain_dropout(s):
    x, p = s["x"], s["case"]["p"]
    keep = plain_words(x.numel(), s["state"], s["site"]).view_as(x) >= int(p * 2 ** 32)
    y = torch.where(keep, x.float() * (1 / (1 - p)), 0.0)
    if s["case"]["way"] == "backward":
        return {"dx": y.to(x.dtype)}
    return {"y": (y if s["residual"] is None else y + s["residual"].float()).to(x.dtype)}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["kind"] == "attention":
        lq, lk = lengths(case)
        pairs = queries = keys = 0
        for a, b in zip(lq, lk):
            if case["causal"]:  # query i sees keys up to i + b - a
                first = max(0, a - b)
                seen = (a - first) * (first + b - a + 1 + b) // 2
            else:
                seen = a * b
            pairs, queries, keys = pairs + seen, queries + a, keys + b
        d, hq, hk = case["width"], case["q_heads"], case["k_heads"]
        rows = case["batch"] * case["queries"] * hq
        if case["way"] == "forward":  # q, k, v; out, lse
            return {"bytes": size * d * (queries * hq + 2 * keys * hk + rows) + 4 * rows, "flops": 4 * pairs * hq * d}
        # q, out, dout, k, v, lse; dq, dk, dv
        return {"bytes": size * d * (3 * queries * hq + 2 * keys * hk + rows + 2 * case["batch"] * case["keys"] * hk)
                + 4 * queries * hq, "flops": 10 * pairs * hq * d}
    if case["kind"] == "group_norm":
        n = case["batch"] * case["positions"] * case["channels"]
        each = 0 if case["weights"] == "none" else 4 if case["weights"] == "fp32" else size
        act = 0 if case["activation"] == "none" else 1
        if case["way"] == "forward":
            return {"bytes": 2 * n * size + 2 * case["channels"] * each, "flops": (8 + 4 * act) * n}
        return {"bytes": 3 * n * size + 4 * case["channels"] * each, "flops": (16 + 8 * act) * n}
    n = case["tokens"] * case["width"]
    return {"bytes": (3 if case["residual"] else 2) * n * size, "flops": 30 * n}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "group_norm":
        return exact_group_norm(s, case)
    if case["kind"] == "dropout":
        return exact_dropout(s, case)
    out = exact_outputs(s, case)
    lq, lk = lengths(case)
    group = case["q_heads"] // case["k_heads"]
    for b in range(case["batch"]):  # sample by sample and head by head: only what a length lets in is read
        for h in range(case["q_heads"]):
            if lq[b] and lk[b]:
                exact_head(s, case, out, b, h, h // group, lq[b], lk[b])
    return out


def exact_outputs(s, case):
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    if case["way"] == "forward":
        return {"out": z(s["q"]), "lse": torch.full((case["batch"], case["q_heads"], case["queries"]), -math.inf,
                                                    dtype=torch.float64, device="cuda")}
    return {"dq": z(s["q"]), "dk": z(s["k"]), "dv": z(s["v"])}


def exact_head(s, case, out, b, h, g, nq, nk):
    """One head's rows that see a key, by the softmax's Jacobian diag(p) - p p'."""
    first = max(0, nq - nk) if case["causal"] else 0
    q = s["q"][b, first:nq, h].double()
    k, v = s["k"][b, :nk, g].double(), s["v"][b, :nk, g].double()
    score = torch.mm(q * s["scale"], k.t())
    if case["causal"]:
        score += torch.full_like(score, -math.inf).triu_(first + nk - nq + 1)
    lse = torch.logsumexp(score, -1)
    p = torch.exp(score.sub_(lse[:, None]))
    del score
    if case["way"] == "forward":
        out["lse"][b, h, first:nq] = lse
        out["out"][b, first:nq, h] = torch.mm(p, v)
        return
    dout = s["dout"][b, first:nq, h].double()
    out["dv"][b, :nk, g] += torch.mm(p.t(), dout)
    mixed = torch.linalg.vecdot(dout, torch.mm(p, v))
    ds = torch.mm(dout, v.t()).sub_(mixed[:, None]).mul_(p)
    out["dq"][b, first:nq, h] = torch.mm(ds, k) * s["scale"]
    out["dk"][b, :nk, g] += torch.mm(ds.t(), q) * s["scale"]


def exact_group_norm(s, case):
    """The gradient is the formula's Jacobian applied to what reaches the norm."""
    x = s["x"].double()
    c = case["channels"]
    h = x.view(case["batch"], -1, case["groups"], c // case["groups"]).transpose(1, 2)  # [B, G, positions, C / G]
    var, mean = torch.var_mean(h, (2, 3), correction=0, keepdim=True)
    sigma = torch.sqrt(var + EPS)
    h = (h - mean) / sigma
    rows = lambda t: t.transpose(1, 2).reshape(x.shape)  # noqa: E731
    z = rows(h)
    if s["gamma"] is not None:
        z = torch.addcmul(s["beta"].double(), z, s["gamma"].double())
    if case["way"] == "forward":
        return {"y": z * torch.sigmoid(z) if s["activation"] else z}
    g = s["dy"].double()
    if s["activation"]:
        t = torch.sigmoid(z)
        g = g * t + g * z * t * (1 - t)
    out = {}
    if s["gamma"] is not None:
        out = {"dgamma": (g * rows(h)).sum((0, 1)), "dbeta": g.sum((0, 1))}
        g = g * s["gamma"].double()
    g = g.view(case["batch"], -1, case["groups"], c // case["groups"]).transpose(1, 2)
    g = g - g.mean((2, 3), keepdim=True)
    g = g - h * (h * g).mean((2, 3), keepdim=True)
    return {"dx": rows(g / sigma), **out}


def exact_dropout(s, case):
    """The generator with 64-bit products that wrap: their bits are those of the
    unsigned product.  Four columns of words, each round one rotation of them."""
    x, low = s["x"], 0xFFFFFFFF
    at = torch.arange(-(-x.numel() // 4), device="cuda")
    seed, offset = (int(v) for v in s["state"])
    word = [at, torch.zeros_like(at) + s["site"], torch.zeros_like(at) + (offset & low),
            torch.zeros_like(at) + (offset >> 32 & low)]
    for k in range(10):
        key = [(seed + k * 0x9E3779B9) & low, ((seed >> 32) + k * 0xBB67AE85) & low]
        one, two = word[0] * 0xD2511F53, word[2] * 0xCD9E8D57
        word = [((two >> 32) & low) ^ word[1] ^ key[0], two & low, ((one >> 32) & low) ^ word[3] ^ key[1], one & low]
    drop = torch.stack(word, 1).view(-1)[:x.numel()].view_as(x) < math.floor(case["p"] * 4294967296.0)
    y = x.double().div_(1 - case["p"]).masked_fill_(drop, 0.0)
    if case["way"] == "backward":
        return {"dx": y}
    return {"y": y if s["residual"] is None else y + s["residual"].double()}
