"""Cases and plain forms of the 8-bit cache's operators and of the verification of drafted tokens.

A paged key/value cache held in 8 bits: e4m3 numbers with one power-of-two
scale (an exponent byte e, the number 2^(e - 127)) for each block of tokens and
head, keys and values apart.

  store   a step's keys and values quantised into the blocks they belong to; a
          block that already holds tokens keeps the larger scale, and its
          tokens are quantised again where that scale grows
  load    rows of the cache read back in 16 bits
  attn    attention of a step's tokens over such a cache
  verify  drafted tokens accepted or rejected against the target's
          probabilities by given random numbers, and the token that follows

`run` computes a case in its plain form (elementary torch operations in 32
bits, in 64 beside the borders of a draw) or, where `own` is true, with the
library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode batch: one token for each of 64 requests, most into blocks that hold tokens already
        dict(name="store-decode", op="store", B=64, ctx_lo=1, ctx_hi=4096, n_lo=1, n_hi=1, Hkv=4, D=128, dtype="bf16",
             page=16, block=16, layout="token", pad=0, mix=1),
        # drafted trees of an odd batch: heads of 64, blocks shorter than pages, padded rows
        dict(name="store-f16-odd", op="store", B=23, ctx_lo=0, ctx_hi=1500, n_lo=0, n_hi=37, Hkv=8, D=64, dtype="f16",
             page=64, block=32, layout="head", pad=24, mix=2),
        # prompts' chunks of one step, 8192 tokens
        dict(name="store-chunk", op="store", B=4, ctx_lo=0, ctx_hi=3000, n_lo=2048, n_hi=2048, Hkv=8, D=128,
             dtype="bf16", page=64, block=64, layout="token", pad=0, mix=3),
        # the accepted tokens of a step, read back to be stored in their places
        dict(name="load-accepted", op="load", n=77, Hkv=4, D=128, dtype="bf16", page=16, block=16, pages=4096,
             layout="token", run=3, mix=4),
        # a prefix of 32768 tokens handed on in 16 bits
        dict(name="load-prefix", op="load", n=32768, Hkv=8, D=128, dtype="f16", page=64, block=32, pages=600,
             layout="head", run=64, mix=5),
        # single-token decode of one request: latency, split over the context
        dict(name="attn-one-token", op="attn", B=1, ctx_lo=4096, ctx_hi=4096, n_lo=1, n_hi=1, Hq=32, Hkv=4, D=128,
             dtype="bf16", page=16, block=16, layout="token", mix=6),
        # a served batch in decode: 64 single tokens, ragged contexts
        dict(name="attn-decode", op="attn", B=64, ctx_lo=100, ctx_hi=16384, n_lo=1, n_hi=1, Hq=32, Hkv=4, D=128,
             dtype="bf16", page=64, block=64, layout="token", mix=7),
        # odd sizes: five query heads to a key head, small trees, contexts that may be empty
        dict(name="attn-f16-odd", op="attn", B=5, ctx_lo=0, ctx_hi=3001, n_lo=1, n_hi=37, Hq=40, Hkv=8, D=64,
             dtype="f16", page=32, block=16, layout="head", mix=8),
        # trees of drafted tokens over long contexts
        dict(name="attn-long", op="attn", B=32, ctx_lo=8192, ctx_hi=32768, n_lo=24, n_hi=32, Hq=32, Hkv=4, D=128,
             dtype="bf16", page=64, block=64, layout="token", mix=9),
        # one request's four drafted tokens, one after another
        dict(name="verify-one", op="verify", B=1, n_lo=5, n_hi=5, V=131072, dtype="f32", tree=False, draft=True, pad=0,
             mix=10),
        # looked-up drafts (no probabilities of their own) of an odd batch, odd vocabulary, padded 16-bit rows
        dict(name="verify-bf16-odd", op="verify", B=37, n_lo=1, n_hi=9, V=50021, dtype="bf16", tree=True, draft=False,
             pad=27, mix=11),
        # a served batch's drafted trees, sampled from a smaller model
        dict(name="verify-trees", op="verify", B=64, n_lo=9, n_hi=17, V=131072, dtype="f32", tree=True, draft=True,
             pad=0, mix=12),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["store", "load", "attn", "attn", "verify", "verify"])
    mix = rng.randrange(1 << 30)
    if op == "verify":
        V = _spread(rng, 1000, 131072)
        tree = rng.random() < 0.6
        n_hi = _spread(rng, 1, 33 if tree else 9)
        most = max(1, 64 * 17 * 131072 // (n_hi * V))
        return dict(op=op, B=_spread(rng, 1, min(256, most)), n_lo=rng.choice([1, max(1, n_hi // 2), n_hi]), n_hi=n_hi,
                    V=V, dtype=rng.choice(["f32", "f32", "bf16", "f16"]), tree=tree, draft=rng.random() < 0.6,
                    pad=rng.choice([0, 0, 3, 64]), mix=mix)
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (16, 32, 64, 128) if b <= page])
    common = dict(Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "f16"]), page=page, block=block,
                  layout=rng.choice(["token", "head"]), mix=mix)
    if op == "store":
        n_hi = _spread(rng, 1, 2048)
        return dict(op=op, B=_spread(rng, 1, min(256, max(1, 8192 // n_hi))), ctx_lo=0, ctx_hi=_spread(rng, 1, 4096),
                    n_lo=rng.choice([0, 1, n_hi]), n_hi=n_hi, pad=rng.choice([0, 0, 8, 40]), **common)
    if op == "load":
        pages = max(2, _spread(rng, 256, 38400) // page)
        return dict(op=op, n=_spread(rng, 1, min(32768, pages * page)), pages=pages, run=rng.choice([1, 5, 16, 64]),
                    **common)
    G = rng.choice([1, 2, 3, 4, 5, 8])
    n_hi = rng.choice([1, _spread(rng, 1, 64)])
    ctx_hi = _spread(rng, 8, 32768)
    most = int(0.6 * 32 * 32768 * 4 * 128 * min(1.0, 8 * 32 / (G * n_hi)) / (ctx_hi * Hkv * D))
    return dict(op=op, B=_spread(rng, 1, max(1, min(64, most))), ctx_lo=rng.choice([0, ctx_hi // 4]), ctx_hi=ctx_hi,
                n_lo=rng.choice([1, max(1, n_hi // 2)]), n_hi=n_hi, Hq=Hkv * G, **common)


def _new(case):
    """New-token counts of a case's requests: its own, whatever the seed of the values."""
    rng = random.Random(case["mix"])
    new = [rng.randint(case["n_lo"], case["n_hi"]) for _ in range(case["B"])]
    new[-1] = case["n_hi"]
    return new


def _contexts(case):
    rng = random.Random(case["mix"] + 1)
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    ctx[-1] = case["ctx_hi"]
    return ctx


def _size(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    """The bytes and operations a pass cannot do without."""
    op = case["op"]
    if op == "verify":
        # one row of the target's probabilities to draw from, and the draft's beside it
        rows = case["B"] * (2 if case["draft"] else 1)
        return dict(bytes=rows * case["V"] * _size(case["dtype"]) + 20 * sum(_new(case)) + 8 * case["B"],
                    flops=3 * rows * case["V"])
    Hkv, D, block = case["Hkv"], case["D"], case["block"]
    if op == "load":
        n = case["n"]
        return dict(bytes=2 * n * Hkv * D * 3 + 8 * n + 2 * Hkv * -(-n // block), flops=2 * n * Hkv * D)
    ctx, new = _contexts(case), _new(case)
    if op == "store":
        T = sum(new)
        blocks = sum(-(-(c + n) // block) - c // block for c, n in zip(ctx, new) if n)
        return dict(bytes=2 * T * Hkv * D * 3 + 2 * Hkv * blocks + 12 * case["B"], flops=4 * T * Hkv * D)
    Hq, e = case["Hq"], _size(case["dtype"])
    keys, T = sum(ctx) + sum(new), sum(new)
    blocks = sum(-(-(c + n) // block) for c, n in zip(ctx, new))
    pairs = sum(n * c + n for c, n in zip(ctx, new))
    return dict(bytes=2 * keys * Hkv * D + 2 * blocks * Hkv + T * Hq * (2 * D * e + 4), flops=4 * pairs * Hq * D)


# ---------------------------------------------------------------- inputs

def _trees(new, rng):
    """Parents of every request's tokens (row 0 is the last one told): a few branches at each depth."""
    parents = []
    for n in new:
        parents += [-1 if i == 0 else rng.randint(max(0, i - 5), i - 1) for i in range(n)]
    return parents


def _masks(parents, new, words):
    """Every token's ancestors and itself as bits, `words` 32-bit words a token."""
    out, at = np.zeros((max(1, sum(new)), words), dtype=np.uint32), 0
    for n in new:
        bits = []
        for i in range(n):
            p = parents[at + i]
            bits.append((0 if p < 0 else bits[p]) | (1 << i))
        for i, b in enumerate(bits):
            for w in range(words):
                out[at + i, w] = (b >> (32 * w)) & 0xFFFFFFFF
        at += n
    return out[:sum(new)].view(np.int32)


def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype).to(DEV)


def _starts(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


def _rows(shape, g):
    """Keys or values as a model makes them: some heads larger than others, a few outlying channels and tokens."""
    *tokens, heads, D = shape
    x = torch.randn(shape, device=DEV, generator=g)
    x *= torch.exp(0.5 * torch.randn((heads, 1), device=DEV, generator=g))
    x *= 1 + 5 * (torch.rand((heads, D), device=DEV, generator=g) < 0.03)
    x *= 1 + 3 * (torch.rand((*tokens, 1, 1), device=DEV, generator=g) < 0.02)
    return x


def _scale_bytes(most):
    """The exponent byte of the least power of two that 448 of reach `most` (float32, at least 0)."""
    bits = most.view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000)).clamp(0, 254)


def _power(e):
    """2^e in 64 bits for whole numbers e."""
    return torch.ldexp(torch.ones_like(e, dtype=torch.float64), e)


def _empty(case, pages):
    """A cache of zeros and a view of it as [page, token, head, D]."""
    P, Hkv, D = case["page"], case["Hkv"], case["D"]
    shape = (pages, P, Hkv, D) if case["layout"] == "token" else (pages, Hkv, P, D)
    t = torch.zeros(shape, device=DEV, dtype=torch.uint8)
    return t if case["layout"] == "token" else t.transpose(1, 2)


def _held(case, pages, g):
    """A cache that holds tokens in every row: codes and scale bytes of keys and of values."""
    P, Hkv, D, block = case["page"], case["Hkv"], case["D"], case["block"]
    out = []
    for _ in range(2):
        codes = _empty(case, pages)
        scale = torch.zeros((pages, P // block, Hkv), device=DEV, dtype=torch.uint8)
        part = max(1, (1 << 26) // (P * Hkv * D))
        for p in range(0, pages, part):
            n = min(part, pages - p)
            x = _rows((n, P, Hkv, D), g).unflatten(1, (P // block, block))  # [page, block, token, head, D]
            e = _scale_bytes(x.abs().amax((2, 4)))
            scale[p:p + n] = e.to(torch.uint8)
            x *= _power(127 - e).float()[:, :, None, :, None]
            codes[p:p + n] = x.to(E4M3).view(torch.uint8).flatten(1, 2)
        out += [codes, scale]
    return out


def _pages(case, ctx, new, g):
    """Block tables of requests whose pages lie anywhere in the cache, and the number of its pages."""
    P = case["page"]
    held = [-(-(c + n) // P) for c, n in zip(ctx, new)]
    pages, width = sum(held) + 7, max(held) + 1
    ids = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
    col = torch.arange(width, device=DEV)[None, :]
    held_t, first = _int(held, torch.int64)[:, None], _int(_starts(held)[:-1], torch.int64)[:, None]
    return torch.where(col < held_t, ids[(first + col).clamp_(max=pages - 1)], -1).to(torch.int32), pages, max(held)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = random.Random(seed)
    s = dict(case=case)
    if case["op"] == "verify":
        _prepare_verify(s, case, g, rng)
        return s
    dt = DTYPES[case["dtype"]]
    if case["op"] == "load":
        s["k"], s["k_scale"], s["v"], s["v_scale"] = _held(case, case["pages"], g)
        slots, total, run = [], case["pages"] * case["page"], case["run"]
        while len(slots) < case["n"]:  # runs of tokens that follow one another
            at = rng.randrange(total)
            slots += range(at, min(at + run, total, at + case["n"] - len(slots)))
        s["slots"] = _int(slots, torch.int64)
        for name in ("k_out", "v_out"):
            s[name] = torch.zeros((case["n"], case["Hkv"], case["D"]), device=DEV, dtype=dt)
        return s
    ctx, new = _contexts(case), _new(case)
    T = sum(new)
    s["ctx"], s["q_start"] = _int(ctx), _int(_starts(new))
    s["table"], pages, s["width"] = _pages(case, ctx, new, g)
    s["k"], s["k_scale"], s["v"], s["v_scale"] = _held(case, pages, g)
    s["T"], s["n_max"] = T, max(new)
    if case["op"] == "store":
        kv = torch.zeros((T, 2 * case["Hkv"] * case["D"] + case["pad"]), device=DEV, dtype=dt)
        for i, name in enumerate(("k_rows", "v_rows")):
            s[name] = kv[:, i * case["Hkv"] * case["D"]:][:, :case["Hkv"] * case["D"]].unflatten(1, (case["Hkv"], case["D"]))
            s[name].copy_(_rows((T, case["Hkv"], case["D"]), g))
        return s
    Hq, D = case["Hq"], case["D"]
    s["q"] = torch.randn((T, Hq, D), device=DEV, generator=g).to(dt)
    s["mask"] = torch.from_numpy(_masks(_trees(new, rng), new, (case["n_hi"] + 31) // 32)).to(DEV)
    s["scale"] = 0.7 * D ** -0.5
    s["out"] = torch.zeros((T, Hq, D), device=DEV, dtype=dt)
    s["lse"] = torch.zeros((T, Hq), device=DEV)
    return s


def _prepare_verify(s, case, g, rng):
    new, V, pad = _new(case), case["V"], case["pad"]
    T, B, dt = sum(new), case["B"], DTYPES[case["dtype"]]
    start = _starts(new)
    parents = _trees(new, rng) if case["tree"] else [i - 1 for n in new for i in range(n)]
    first = [start[b] for b, n in enumerate(new) for _ in range(n)]
    above = _int([f + p if p >= 0 else -1 for f, p in zip(first, parents)], torch.int64)  # the parent's row
    s["probs"] = torch.zeros((T, V + pad), device=DEV, dtype=dt)[:, :V]
    s["draft"] = torch.zeros((T, V + pad), device=DEV, dtype=dt)[:, :V] if case["draft"] else None
    tokens = torch.zeros(T, device=DEV, dtype=torch.int64)
    for t0 in range(0, T, 128):
        n = min(128, T - t0)
        x = torch.randn((n, V), device=DEV, generator=g).mul_(1.5)
        likely = torch.randint(0, V, (n, 12), device=DEV, generator=g)
        x.scatter_add_(1, likely, 5 * torch.rand((n, 12), device=DEV, generator=g) + 7)
        s["probs"][t0:t0 + n] = torch.softmax(x, 1)
        mine = (above >= t0) & (above < t0 + n)  # tokens drafted after one of these rows
        rows = above[mine] - t0
        if s["draft"] is not None:
            q = torch.softmax(x + 0.6 * torch.randn((n, V), device=DEV, generator=g), 1).to(dt)
            s["draft"][t0:t0 + n] = q
            u = torch.rand((int(rows.numel()), V), device=DEV, generator=g).clamp_(min=1e-30)
            tokens[mine] = (q.float()[rows].log() - (-u.log()).log()).argmax(1)
        else:  # what followed the same words before: often the likeliest token, else another likely one
            pick = torch.randint(0, 12, (int(rows.numel()), 1), device=DEV, generator=g)
            other = likely[rows].gather(1, pick)[:, 0]
            take = torch.rand(int(rows.numel()), device=DEV, generator=g) < 0.5
            tokens[mine] = torch.where(take, x.argmax(1)[rows], other)
    s["tokens"] = tokens.to(torch.int32)
    s["parents"] = _int(parents) if case["tree"] else None
    s["q_start"] = _int(start)
    s["accept_u"] = torch.rand(T, device=DEV, generator=g)
    s["draw_u"] = torch.rand(B, device=DEV, generator=g)
    s["T"], s["n_max"] = T, max(new)
    s["accepted"] = torch.zeros(T, device=DEV, dtype=torch.int32)
    s["n_accepted"] = torch.zeros(B, device=DEV, dtype=torch.int32)
    s["next_token"] = torch.zeros(B, device=DEV, dtype=torch.int32)


# ---------------------------------------------------------------- plain forms

def _owners(start, T):
    """For each of T rows laid out request by request: its request and its place in it."""
    counts = start[1:] - start[:-1]
    b = torch.repeat_interleave(torch.arange(counts.numel(), device=counts.device), counts, output_size=T)
    return b, torch.arange(T, device=counts.device) - start[b]


def _fits(dtype, e):
    """The largest code whose value the 16-bit type holds: 448, or 240 where 2 * 128 * 2^e would pass it."""
    return torch.where(e >= (135 if dtype == torch.float16 else 247), 240.0, 448.0)


def _plain_store(s):
    c, T = s["case"], s["T"]
    P, block, Hkv = c["page"], c["block"], c["Hkv"]
    per = P // block
    ctx, start = s["ctx"].long(), s["q_start"].long()
    b, i = _owners(start, T)
    pos = ctx[b] + i
    page = s["table"][b, pos // P].long()
    unit = page * per + pos % P // block  # the row's block in the cache
    edge = ctx % block  # tokens that a request's first block holds
    part = (edge > 0) & (start[1:] > start[:-1])
    old_unit = s["table"][torch.arange(ctx.numel(), device=DEV), ctx // P].long().clamp(min=0) * per + ctx % P // block
    r = torch.arange(block, device=DEV)
    for name in ("k", "v"):
        x, codes, scale = s[name + "_rows"].float(), s[name], s[name + "_scale"].view(-1, Hkv)
        most = torch.zeros(scale.shape, device=DEV).index_reduce_(0, unit, x.abs().amax(-1), "amax")
        need = _scale_bytes(most)
        was = torch.zeros_like(need)
        was[old_unit] = torch.where(part[:, None], scale[old_unit].int(), 0)
        e = torch.maximum(was, need)
        # the tokens of blocks begun before, at the larger scale
        op, orow = old_unit // per, old_unit % per * block
        rows = codes[op[:, None], orow[:, None] + r].view(E4M3).float()  # [request, token, head, D]
        grow = torch.ldexp(torch.ones_like(e, dtype=torch.float32), (was - e).clamp(min=-126))[old_unit]
        rows = (rows * grow[:, None, :, None]).to(E4M3).view(torch.uint8)
        keep = part[:, None] & (r[None, :] < edge[:, None])
        codes[op[:, None].expand_as(keep)[keep], (orow[:, None] + r)[keep]] = rows[keep]
        y = (x.double() * _power(127 - e[unit])[:, :, None]).float()
        top = _fits(s[name + "_rows"].dtype, e[unit])[:, :, None]
        codes[page, pos % P] = torch.minimum(torch.maximum(y, -top), top).to(E4M3).view(torch.uint8)
        scale[unit] = e[unit].to(torch.uint8)
    return dict(k=s["k"].view(E4M3), k_scale=s["k_scale"], v=s["v"].view(E4M3), v_scale=s["v_scale"])


def _values(codes, scale, block, wide):
    """[..., token, head, D] codes with [..., token / block, head] scale bytes as numbers of the type `wide`."""
    x = codes.view(E4M3).to(wide).unflatten(-3, (-1, block))
    return (x * _power(scale.int() - 127).to(wide)[..., :, None, :, None]).flatten(-4, -3)


def _plain_load(s):
    c = s["case"]
    P, block = c["page"], c["block"]
    page, row = s["slots"] // P, s["slots"] % P
    out = {}
    for name in ("k", "v"):
        e = s[name + "_scale"][page, row // block].int()  # [token, head]
        x = s[name][page, row].view(E4M3).float() * _power(e - 127).float()[:, :, None]
        out[name] = x.to(s["k_out"].dtype)
    return out


def _plain_attn(s):
    c, T, n = s["case"], s["T"], s["n_max"]
    Hkv, D = c["Hkv"], c["D"]
    G = c["Hq"] // Hkv
    ctx, start = s["ctx"].long(), s["q_start"].long()
    new = start[1:] - start[:-1]
    pages = s["table"][:, :s["width"]].long().clamp(min=0)
    k, v = (_values(s[x][pages].flatten(1, 2), s[x + "_scale"][pages].flatten(1, 2), c["block"], torch.float32)
            .permute(0, 2, 1, 3) for x in ("k", "v"))  # [B, Hkv, K, D]
    K, B = k.shape[2], ctx.numel()
    row = (start[:-1, None] + torch.arange(n, device=DEV)).clamp(max=T - 1)
    q = s["q"][row].float().view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    x = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, n, G, K).mul_(s["scale"])
    j = torch.arange(K, device=DEV)[None, :] - ctx[:, None]  # place among the new tokens
    word = (j >> 5).clamp(0, s["mask"].shape[1] - 1)[:, None, :].expand(B, n, K)
    bit = (torch.gather(s["mask"][row].long(), 2, word) >> (j & 31)[:, None, :]) & 1
    seen = (j < 0)[:, None, :] | ((j[:, None, :] < new[:, None, None]) & (bit == 1) & (j >= 0)[:, None, :])
    x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, n * G, K), v).view(B, Hkv, n, G, D) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total))[..., 0]
    b, i = _owners(start, T)
    out = o.permute(0, 2, 1, 3, 4)[b, i].reshape(T, c["Hq"], D).to(s["q"].dtype)
    return dict(out=out, lse=lse.permute(0, 2, 1, 3)[b, i].reshape(T, c["Hq"]))


def _plain_verify(s):
    c, n = s["case"], s["n_max"]
    B, V = c["B"], c["V"]
    start = s["q_start"].long()
    new = start[1:] - start[:-1]
    each = torch.arange(B, device=DEV)
    at = torch.zeros(B, device=DEV, dtype=torch.int64)        # the last accepted token's place
    a = s["probs"][start[:-1]].double()                       # what the next token is drawn from, not normalised
    total = torch.ones(B, device=DEV, dtype=torch.float64)
    first = a.clone()                                         # the same before any rejection
    accepted = torch.full((B, n), -1, device=DEV, dtype=torch.int64)
    count = torch.zeros(B, device=DEV, dtype=torch.int64)
    for i in range(1, n):
        row = (start[:-1] + i).clamp(max=s["T"] - 1)
        parent = s["parents"][row].long() if s["parents"] is not None else torch.full_like(at, i - 1)
        live = (i < new) & (parent == at)
        x = s["tokens"][row].long()
        u = s["accept_u"][row].double()
        if s["draft"] is not None:
            q = s["draft"][start[:-1] + at].double()
        else:
            q = torch.zeros((B, V), device=DEV, dtype=torch.float64).scatter_(1, x[:, None], 1.0)
        yes = live & (u * q[each, x] * total < a[each, x])
        no = live & ~yes
        less = (a - q * total[:, None]).clamp_(min=0)
        a = torch.where(no[:, None], less, a)
        total = torch.where(no, a.sum(1), total)
        at = torch.where(yes, i, at)
        fresh = s["probs"][start[:-1] + at].double()
        a = torch.where(yes[:, None], fresh, a)
        first = torch.where(yes[:, None], fresh, first)
        total = torch.where(yes, 1.0, total)
        accepted[each, count.clamp(max=n - 1)] = torch.where(yes, i, accepted[each, count.clamp(max=n - 1)])
        count += yes
    a = torch.where(a.sum(1, keepdim=True) > 0, a, first)
    run = a.cumsum(1)
    token = (run <= s["draw_u"].double()[:, None] * run[:, -1:]).sum(1)
    b, i = _owners(start, s["T"])
    return dict(accepted=accepted[b, i].to(torch.int32), n_accepted=count.to(torch.int32), next_token=token.to(torch.int32))


_PLAIN = dict(store=_plain_store, load=_plain_load, attn=_plain_attn, verify=_plain_verify)


# ---------------------------------------------------------------- the library's calls

def _at(t):
    return 0 if t is None else t.data_ptr()


def _library_dtype(ft, t):
    return {torch.bfloat16: ft.FT_DTYPE_BF16, torch.float16: ft.FT_DTYPE_F16, torch.float32: ft.FT_DTYPE_F32}[t.dtype]


def _library_cache(ft, s):
    k, v = s["k"], s["v"]
    return ft.make_kv8_cache(k=_at(k), v=_at(v), k_scale=_at(s["k_scale"]), v_scale=_at(s["v_scale"]),
                             num_pages=k.shape[0], page_size=k.shape[1], block_size=s["case"]["block"],
                             kv_heads=k.shape[2], head_dim=k.shape[3], k_page_stride=k.stride(0),
                             k_token_stride=k.stride(1), k_head_stride=k.stride(2), v_page_stride=v.stride(0),
                             v_token_stride=v.stride(1), v_head_stride=v.stride(2))


def _library_call(s):
    """The call on a state's buffers and what it writes: a program that keeps its buffers fills the arguments once."""
    import expert_cache_host_gb300 as ft
    c = s["case"]
    if c["op"] == "store":
        args = ft.make_kv8_store_args(k=_at(s["k_rows"]), v=_at(s["v_rows"]), q_start=_at(s["q_start"]),
                                      ctx_len=_at(s["ctx"]), block_table=_at(s["table"]),
                                      k_stride=s["k_rows"].stride(0), v_stride=s["v_rows"].stride(0),
                                      dtype=_library_dtype(ft, s["k_rows"]), max_tokens=s["T"], num_reqs=c["B"],
                                      table_width=s["table"].shape[1], cache=_library_cache(ft, s))
        return ft.ft_kv8_store, args, dict(k=s["k"].view(E4M3), k_scale=s["k_scale"], v=s["v"].view(E4M3),
                                           v_scale=s["v_scale"])
    if c["op"] == "load":
        args = ft.make_kv8_load_args(k=_at(s["k_out"]), v=_at(s["v_out"]), slots=_at(s["slots"]),
                                     k_stride=s["k_out"].stride(0), v_stride=s["v_out"].stride(0),
                                     dtype=_library_dtype(ft, s["k_out"]), T=c["n"], cache=_library_cache(ft, s))
        return ft.ft_kv8_load, args, dict(k=s["k_out"], v=s["v_out"])
    if c["op"] == "attn":
        args = ft.make_kv8_attn_args(q=_at(s["q"]), out=_at(s["out"]), lse=_at(s["lse"]), q_start=_at(s["q_start"]),
                                     ctx_len=_at(s["ctx"]), block_table=_at(s["table"]), mask=_at(s["mask"]),
                                     q_stride=s["q"].stride(0), out_stride=s["out"].stride(0),
                                     dtype=_library_dtype(ft, s["q"]), max_tokens=s["T"], max_new=s["n_max"],
                                     num_reqs=c["B"], q_heads=c["Hq"], table_width=s["table"].shape[1],
                                     mask_words=s["mask"].shape[1], scale=s["scale"], cache=_library_cache(ft, s))
        s["workspace"] = torch.zeros(ft.ft_kv8_attention_workspace(args), dtype=torch.uint8, device=DEV)
        args.workspace, args.workspace_bytes = _at(s["workspace"]), s["workspace"].numel()
        return ft.ft_kv8_attention, args, dict(out=s["out"], lse=s["lse"])
    p, q = s["probs"], s["draft"]
    args = ft.make_verify_args(probs=_at(p), draft_probs=_at(q), tokens=_at(s["tokens"]), parents=_at(s["parents"]),
                               accept_u=_at(s["accept_u"]), draw_u=_at(s["draw_u"]), q_start=_at(s["q_start"]),
                               accepted=_at(s["accepted"]), n_accepted=_at(s["n_accepted"]),
                               next_token=_at(s["next_token"]), probs_stride=p.stride(0),
                               draft_stride=0 if q is None else q.stride(0), dtype=_library_dtype(ft, p),
                               max_tokens=s["T"], num_reqs=c["B"], V=c["V"])
    return ft.ft_verify_drafts, args, {name: s[name] for name in ("accepted", "n_accepted", "next_token")}


def run(state):
    if not own:
        return _PLAIN[state["case"]["op"]](state)
    if "call" not in state:
        state["call"] = _library_call(state)
    call, args, out = state["call"]
    call(args, torch.cuda.current_stream().cuda_stream)
    return out


# ---------------------------------------------------------------- 64 bits

def _exact_store(s):
    """Scale bytes, and every code as the number that is rounded to it."""
    c = s["case"]
    P, block, Hkv = c["page"], c["block"], c["Hkv"]
    ctx, start, table = s["ctx"].tolist(), s["q_start"].tolist(), s["table"].cpu().numpy()
    out = {}
    for name in ("k", "v"):
        codes = s[name].view(E4M3).double()
        scale = s[name + "_scale"].clone()
        rows = s[name + "_rows"].double()
        for b, n0 in enumerate(ctx):
            n = start[b + 1] - start[b]
            at = n0
            while at < n0 + n:
                end = min(n0 + n, (at // block + 1) * block)
                page, first = int(table[b, at // P]), at % P // block * block
                x = rows[start[b] + at - n0:start[b] + end - n0]
                most = x.abs().amax((0, 2))
                exponent = torch.ceil(torch.log2(most / 448)).clamp(min=-127)
                exponent += (most > 448 * _power(exponent.int())).double()
                exponent -= (most <= 448 * _power(exponent.int() - 1)).double()
                e = exponent.clamp(min=-127) + 127
                if at % block:
                    was = scale[page, first // block].double()
                    e = torch.maximum(e, was)
                    old = codes[page, first:first + at % block]
                    codes[page, first:first + at % block] = old * torch.exp2(was - e)[None, :, None]
                top = torch.where(e >= (135 if c["dtype"] == "f16" else 247), 240.0, 448.0)[None, :, None]
                y = x * torch.exp2(127 - e)[None, :, None]
                codes[page, at % P:at % P + end - at] = torch.minimum(torch.maximum(y, -top), top)
                scale[page, first // block] = e.to(torch.uint8)
                at = end
        out[name], out[name + "_scale"] = codes, scale
    return out


def _exact_load(s):
    c = s["case"]
    page, row = s["slots"] // c["page"], s["slots"] % c["page"]
    return {name: _values(s[name], s[name + "_scale"], c["block"], torch.float64)[page, row] for name in ("k", "v")}


def _exact_attn(s):
    c = s["case"]
    Hq, Hkv, D, P = c["Hq"], c["Hkv"], c["D"], c["page"]
    ctx, start = s["ctx"].tolist(), s["q_start"].tolist()
    out = torch.zeros((s["T"], Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["T"], Hq), dtype=torch.float64, device=DEV)
    masks = s["mask"].cpu().numpy().view(np.uint32)
    for b, n0 in enumerate(ctx):
        t0, t1 = start[b], start[b + 1]
        n = t1 - t0
        if not n:
            continue
        pages = s["table"][b, :-(-(n0 + n) // P)].long()
        k, v = (_values(s[x][pages], s[x + "_scale"][pages], c["block"], torch.float64).flatten(0, 1)[:n0 + n].transpose(0, 1)
                for x in ("k", "v"))
        bits = np.array([[(int(masks[t0 + i, j >> 5]) >> (j & 31)) & 1 for j in range(n)] for i in range(n)])
        hidden = torch.from_numpy(bits == 0).to(DEV)
        for h in range(Hq):
            x = s["q"][t0:t1, h].double() @ k[h * Hkv // Hq].T * s["scale"]
            x[:, n0:] = x[:, n0:].masked_fill(hidden, -math.inf)
            lse[t0:t1, h] = torch.logsumexp(x, -1)
            out[t0:t1, h] = torch.softmax(x, -1) @ v[h * Hkv // Hq]
    return dict(out=out, lse=lse)


def _exact_verify(s):
    c = s["case"]
    start, tokens, u = s["q_start"].tolist(), s["tokens"].tolist(), s["accept_u"].tolist()
    parents = s["parents"].tolist() if s["parents"] is not None else None
    accepted, counts, following = [-1] * s["T"], [], []
    for b, draw_u in enumerate(s["draw_u"].tolist()):
        t0, n = start[b], start[b + 1] - start[b]
        children = [[] for _ in range(n)]
        for i in range(1, n):
            children[parents[t0 + i] if parents else i - 1].append(i)
        at, path = 0, []
        while True:
            p = s["probs"][t0 + at].double()
            rest, mass, step = p, 1.0, None
            for i in children[at]:
                x = tokens[t0 + i]
                q = s["draft"][t0 + at].double() if s["draft"] is not None else \
                    torch.nn.functional.one_hot(torch.tensor(x, device=DEV), c["V"]).double()
                if u[t0 + i] * float(q[x]) * mass < float(rest[x]):
                    step = i
                    break
                rest = torch.relu(rest - mass * q)
                mass = float(rest.sum())
            if step is None:
                break
            accepted[t0 + len(path)] = at = step
            path.append(step)
        if not float(rest.sum()) > 0:
            rest = p
        ends = torch.cumsum(rest, 0)
        following.append(int(torch.searchsorted(ends, ends[-1:] * draw_u, right=True)))
        counts.append(len(path))
    return dict(accepted=_int(accepted), n_accepted=_int(counts), next_token=_int(following))


_EXACT = dict(store=_exact_store, load=_exact_load, attn=_exact_attn, verify=_exact_verify)


def exact(case, seed):
    """The outputs from the definitions in 64 bits."""
    return _EXACT[case["op"]](prepare(case, seed))
