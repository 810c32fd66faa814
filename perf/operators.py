"""Cases and plain forms of the attention-side operators of a serving step.

A step of a request takes one new token, a prompt's tokens or a tree of drafted
tokens.  Four operators carry it around the expert layers:

  plan      block tables, slot map, positions and ancestor masks from the
            requests' lengths (and the drafted tokens' parents)
  qk        per-head norms of queries and keys with the position rotation, keys
            and values written into the paged cache at their slots
  attn      attention of the step's tokens over the paged cache, each drafted
            token seeing the context and its ancestors
  logprob   log probability of the given token, entropy and top alternatives of
            every row of logits

`run` computes a case in its plain form (elementary torch operations in 32
bits) or, where `own` is true, with the library's calls.
"""
import bisect
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"
LOG2_WORD = 5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode batch's bookkeeping: one token for each of 64 requests
        dict(name="plan-decode", op="plan", B=64, ctx_lo=1, ctx_hi=8192, n_lo=1, n_hi=1, page=16, tree=False, mix=1),
        # 256 requests, each with a tree of up to 33 drafted tokens, some new and some idle
        dict(name="plan-trees", op="plan", B=256, ctx_lo=0, ctx_hi=32768, n_lo=0, n_hi=33, page=16, tree=True, mix=2),
        # one token of one request: latency only
        dict(name="qk-one-token", op="qk", T=1, Hq=32, Hkv=4, D=128, rot=128, pairs=False, dtype="bf16", page=16,
             layout="token", pad=0, mix=3),
        # an odd batch of drafted tokens: half of each head rotated, neighbours paired, padded rows
        dict(name="qk-f16-odd", op="qk", T=777, Hq=40, Hkv=8, D=64, rot=32, pairs=True, dtype="f16", page=32,
             layout="head", pad=24, mix=4),
        # a prompt chunk of 8192 tokens
        dict(name="qk-chunk", op="qk", T=8192, Hq=32, Hkv=4, D=128, rot=128, pairs=False, dtype="bf16", page=16,
             layout="token", pad=0, mix=5),
        # single-token decode of one request: latency, split over the context
        dict(name="attn-one-token", op="attn", B=1, ctx_lo=4096, ctx_hi=4096, n_lo=1, n_hi=1, Hq=32, Hkv=4, D=128,
             dtype="bf16", page=16, layout="token", mix=6),
        # a served batch: single tokens beside small trees, ragged contexts
        dict(name="attn-batch", op="attn", B=24, ctx_lo=100, ctx_hi=8192, n_lo=1, n_hi=17, Hq=32, Hkv=4, D=128,
             dtype="bf16", page=16, layout="token", mix=7),
        # odd sizes: five query heads to a key head, contexts that may be empty
        dict(name="attn-f16-odd", op="attn", B=5, ctx_lo=0, ctx_hi=3001, n_lo=1, n_hi=37, Hq=40, Hkv=8, D=64,
             dtype="f16", page=32, layout="head", mix=8),
        # trees of drafted tokens over long contexts
        dict(name="attn-long", op="attn", B=32, ctx_lo=8192, ctx_hi=32768, n_lo=24, n_hi=32, Hq=32, Hkv=4, D=128,
             dtype="bf16", page=64, layout="token", mix=9),
        # the one row a single request samples from
        dict(name="logprob-one-row", op="logprob", T=1, V=131072, top=5, dtype="bf16", pad=0, banned=0.0, mix=10),
        # constrained sampling: a third of an odd vocabulary banned, padded 32-bit rows
        dict(name="logprob-f32-banned", op="logprob", T=61, V=50021, top=20, dtype="f32", pad=27, banned=0.33, mix=11),
        # the drafted tokens of a large batch, or a prompt that is scored
        dict(name="logprob-rows", op="logprob", T=1024, V=131072, top=8, dtype="bf16", pad=0, banned=0.0, mix=12),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["plan", "qk", "attn", "attn", "logprob"])
    mix = rng.randrange(1 << 30)
    if op == "plan":
        tree = rng.random() < 0.6
        n_hi = _spread(rng, 1, 64 if tree else 512)
        return dict(op=op, B=_spread(rng, 1, 256), ctx_lo=0, ctx_hi=_spread(rng, 16, 32768), n_lo=rng.choice([0, 1]),
                    n_hi=n_hi, page=rng.choice([16, 32, 64, 128]), tree=tree, mix=mix)
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    common = dict(Hq=Hkv * G, Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "f16"]), page=rng.choice([16, 32, 64, 128]),
                  layout=rng.choice(["token", "head"]), mix=mix)
    if op == "qk":
        rot = rng.choice([D, D, D // 2])
        most = 8192 * 40 * 128 // ((Hkv * G + 2 * Hkv) * D)
        return dict(op=op, T=_spread(rng, 1, min(8192, most)), rot=rot, pairs=rng.random() < 0.3,
                    pad=rng.choice([0, 0, 8, 40]), **common)
    if op == "attn":
        n_hi = _spread(rng, 1, 64)
        ctx_hi = _spread(rng, 8, 32768)
        keys = ctx_hi * Hkv * D
        most = int(0.6 * 32 * 32768 * 4 * 128 * min(1.0, 8 * 32 / (G * n_hi)) / keys)
        return dict(op=op, B=_spread(rng, 1, max(1, min(64, most))), ctx_lo=rng.choice([0, ctx_hi // 4]), ctx_hi=ctx_hi,
                    n_lo=rng.choice([1, max(1, n_hi // 2)]), n_hi=n_hi, **common)
    V = _spread(rng, 1000, 131072)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    return dict(op=op, T=_spread(rng, 1, 1024 if dtype != "f32" else 512), V=V, top=rng.choice([0, 1, 5, 20, 32]),
                dtype=dtype, pad=rng.choice([0, 0, 3, 64]), banned=rng.choice([0.0, 0.0, 0.33]), mix=mix)


def _lengths(case):
    """Context and new-token counts of a case's requests: its own, whatever the seed of the values."""
    rng = random.Random(case["mix"])
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    new = [rng.randint(case["n_lo"], case["n_hi"]) for _ in range(case["B"])]
    ctx[-1] = case["ctx_hi"]
    new[-1] = case["n_hi"]
    return ctx, new


def _size(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    """The bytes and operations a pass cannot do without."""
    op = case["op"]
    if op == "plan":
        ctx, new = _lengths(case)
        T, page = sum(new), case["page"]
        fresh = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, new))
        words = _words(case)
        per_token = 8 + 4 + ((4 + 4 * words) if case["tree"] else 0)
        return dict(bytes=8 * case["B"] + 4 * (case["B"] + 1) + 8 * fresh + T * per_token, flops=4 * T)
    if op == "qk":
        T, Hq, Hkv, D, e = case["T"], case["Hq"], case["Hkv"], case["D"], _size(case["dtype"])
        rows = T * (Hq + 2 * Hkv) * D
        return dict(bytes=2 * rows * e + T * (12 + 4 * case["rot"]) + 2 * D * e, flops=T * (Hq + Hkv) * (4 * D + 3 * case["rot"]))
    if op == "attn":
        ctx, new = _lengths(case)
        Hq, Hkv, D, e = case["Hq"], case["Hkv"], case["D"], _size(case["dtype"])
        keys, T = sum(ctx) + sum(new), sum(new)
        pairs = sum(n * c + n for c, n in zip(ctx, new))
        return dict(bytes=2 * keys * Hkv * D * e + T * Hq * (2 * D * e + 4), flops=4 * pairs * Hq * D)
    T, V = case["T"], case["V"]
    return dict(bytes=T * V * _size(case["dtype"]) + T * (12 + 8 * case["top"]), flops=6 * T * V)


# ---------------------------------------------------------------- inputs

def _words(case):
    return (case["n_hi"] + 31) >> LOG2_WORD


def _tree(new, rng):
    """Parents of every request's drafted tokens (-1: the context): a few branches at each depth, as a drafter
    that keeps the likeliest continuations proposes them."""
    parents = []
    for n in new:
        own_parents = []
        for i in range(n):
            own_parents.append(-1 if i == 0 else rng.randint(max(-1, i - 6), i - 1))
        parents += own_parents
    return parents


def _depths(parents, new):
    """The length of every token's chain of ancestors."""
    out, at = [], 0
    for n in new:
        d = []
        for i in range(n):
            p = parents[at + i]
            d.append(0 if p < 0 else d[p] + 1)
        out += d
        at += n
    return out


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


def _cache(case, pages, g):
    """Keys and values of `pages` pages, [page, token, head, D] or [page, head, token, D] in memory, seen as the former."""
    P, Hkv, D = case["page"], case["Hkv"], case["D"]
    shape = (pages, P, Hkv, D) if case["layout"] == "token" else (pages, Hkv, P, D)
    kv = [torch.randn(shape, device=DEV, generator=g, dtype=DTYPES[case["dtype"]]) for _ in range(2)]
    return [t if case["layout"] == "token" else t.transpose(1, 2) for t in kv]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = random.Random(seed)
    s = dict(case=case)
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        P, B, T = case["page"], case["B"], sum(new)
        width = -(-(case["ctx_hi"] + case["n_hi"]) // P) + 1
        held = [-(-c // P) for c in ctx]
        fresh = sum(-(-(c + n) // P) - h for c, n, h in zip(ctx, new, held))
        ids = list(range(sum(held) + fresh + 32))
        rng.shuffle(ids)
        table, at = np.full((B, width), -1, dtype=np.int32), 0
        for b, h in enumerate(held):
            table[b, :h] = ids[at:at + h]
            at += h
        s.update(ctx=_int(ctx), new=_int(new), free=_int(ids[at:]), free_count=_int([len(ids) - at]),
                 table=torch.from_numpy(table).to(DEV), T=T)
        s["parents"], s["depth"] = None, 0
        if case["tree"]:
            parents = _tree(new, rng)
            s["parents"], s["depth"] = _int(parents), 1 + max(_depths(parents, new), default=0)
        words = _words(case)
        s.update(q_start=torch.zeros(B + 1, dtype=torch.int32, device=DEV),
                 slots=torch.zeros(T, dtype=torch.int64, device=DEV),
                 positions=torch.zeros(T, dtype=torch.int32, device=DEV),
                 mask=torch.zeros((T, words), dtype=torch.int32, device=DEV) if case["tree"] else None,
                 free_left=torch.zeros(1, dtype=torch.int32, device=DEV))
    elif case["op"] == "qk":
        T, Hq, Hkv, D, P = case["T"], case["Hq"], case["Hkv"], case["D"], case["page"]
        dt = DTYPES[case["dtype"]]
        ld = (Hq + 2 * Hkv) * D + case["pad"]
        qkv = torch.randn((T, ld), device=DEV, generator=g, dtype=torch.float32).mul_(1.7).to(dt)
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = qkv[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].unflatten(1, (Hkv, D))
        for name in ("q_weight", "k_weight"):
            s[name] = (1 + 0.2 * torch.randn(D, device=DEV, generator=g)).to(dt)
        pages = -(-T // P) + 3
        s["k_cache"], s["v_cache"] = (t.zero_() for t in _cache(case, pages, g))
        s["slots"] = torch.randperm(pages * P, device=DEV, generator=g)[:T].contiguous()
        s["max_pos"] = 16384
        half = case["rot"] // 2
        angle = torch.arange(s["max_pos"], device=DEV, dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half))
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["positions"] = torch.randint(0, s["max_pos"], (T,), device=DEV, generator=g, dtype=torch.int32)
        s["q_out"] = torch.zeros((T, Hq, D), device=DEV, dtype=dt)
        s["eps"] = 1e-6
    elif case["op"] == "attn":
        ctx, new = _lengths(case)
        B, P, T, Hq, D = case["B"], case["page"], sum(new), case["Hq"], case["D"]
        dt = DTYPES[case["dtype"]]
        held = [-(-(c + n) // P) for c, n in zip(ctx, new)]
        pages = sum(held) + 7
        s["k_cache"], s["v_cache"] = _cache(case, pages, g)
        ids = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
        width = max(held) + 1
        row = torch.arange(width, device=DEV)[None, :]
        held_t, first = _int(held, torch.int64)[:, None], _int(_starts(held)[:-1], torch.int64)[:, None]
        s["table"] = torch.where(row < held_t, ids[(first + row).clamp_(max=pages - 1)], -1).to(torch.int32)
        s["q"] = torch.randn((T, Hq, D), device=DEV, generator=g, dtype=torch.float32).to(dt)
        s["ctx"], s["q_start"] = _int(ctx), _int(_starts(new))
        s["mask"] = torch.from_numpy(_masks(_tree(new, rng), new, _words(case))).to(DEV)
        s.update(T=T, n_max=max(new), width=max(held), scale=D ** -0.5)
        s["out"] = torch.zeros((T, Hq, D), device=DEV, dtype=dt)
        s["lse"] = torch.zeros((T, Hq), device=DEV)
    else:
        T, V = case["T"], case["V"]
        x = torch.randn((T, V + case["pad"]), device=DEV, generator=g).mul_(2.5)
        likely = torch.randint(0, V, (T, 12), device=DEV, generator=g)
        x.scatter_add_(1, likely, 4 * torch.rand((T, 12), device=DEV, generator=g) + 5)
        if case["banned"]:
            x.masked_fill_(torch.rand(x.shape, device=DEV, generator=g) < case["banned"], -math.inf)
        s["logits"] = x.to(DTYPES[case["dtype"]])[:, :V]
        pick = torch.randint(0, 12, (T, 1), device=DEV, generator=g)
        s["tokens"] = torch.where(torch.rand(T, device=DEV, generator=g) < 0.8, likely.gather(1, pick)[:, 0],
                                  torch.randint(0, V, (T,), device=DEV, generator=g)).to(torch.int32)
        s["logprob"] = torch.zeros(T, device=DEV)
        s["entropy"] = torch.zeros(T, device=DEV)
        s["top_ids"] = torch.zeros((T, case["top"]), dtype=torch.int32, device=DEV)
        s["top_logprobs"] = torch.zeros((T, case["top"]), device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

def _owners(counts, T):
    """For each of T rows laid out request by request: its request and its place in it."""
    start = torch.cumsum(counts, 0) - counts
    b = torch.repeat_interleave(torch.arange(counts.numel(), device=counts.device), counts, output_size=T)
    return b, torch.arange(T, device=counts.device) - start[b], start


def _plain_plan(s):
    c, P = s["case"], s["case"]["page"]
    ctx, new, table = s["ctx"].long(), s["new"].long(), s["table"]
    held, need = (ctx + P - 1) // P, (ctx + new + P - 1) // P
    fresh = need - held
    first = torch.cumsum(fresh, 0) - fresh
    col = torch.arange(table.shape[1], device=DEV)[None, :]
    is_new = (col >= held[:, None]) & (col < need[:, None])
    at = s["free_count"].long() - 1 - (first[:, None] + col - held[:, None])
    table.copy_(torch.where(is_new, s["free"][at.clamp(0, s["free"].numel() - 1)], table))
    b, i, start = _owners(new, s["T"])
    slot = table[b, (ctx[b] + i) // P].long() * P + (ctx[b] + i) % P
    q_start = torch.cat([start, start[-1:] + new[-1:]]).to(torch.int32)
    out = dict(table=table, q_start=q_start, slots=slot, free_left=(s["free_count"] - fresh.sum()).to(torch.int32))
    if s["parents"] is None:
        out["positions"] = (ctx[b] + i).to(torch.int32)
        return out
    words = _words(c)
    word = torch.arange(words, device=DEV)[None, :]
    at, depth, mask = i, torch.full_like(i, -1), torch.zeros((s["T"], words), dtype=torch.int64, device=DEV)
    for _ in range(s["depth"]):
        alive = at >= 0
        bit = torch.where(alive, torch.ones_like(at) << (at & 31), torch.zeros_like(at))
        mask |= torch.where(word == (at >> LOG2_WORD)[:, None], bit[:, None], 0)
        depth += alive
        up = s["parents"][(start[b] + at).clamp(min=0)].long()
        at = torch.where(alive, up, at)
    out["positions"] = (ctx[b] + depth).to(torch.int32)
    out["mask"] = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32)
    return out


def _rotated(x, cos, sin, rot, pairs):
    """The first `rot` numbers of each head turned by the token's angles: number i with i + rot/2, or neighbours."""
    a, rest = x[..., :rot], x[..., rot:]
    u, v = (a[..., 0::2], a[..., 1::2]) if pairs else a.chunk(2, -1)
    u, v = u * cos - v * sin, v * cos + u * sin
    a = torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)
    return torch.cat([a, rest], -1)


def _qk(s, wide):
    """Norm and rotation of a case's queries and keys in the type `wide`."""
    c = s["case"]
    cos, sin = s["cos_sin"][s["positions"].long()].to(wide)[:, None, :].chunk(2, -1)
    out = []
    for name in ("q", "k"):
        x = s[name].to(wide)
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * s[name + "_weight"].to(wide)
        out.append(_rotated(x, cos, sin, c["rot"], c["pairs"]))
    return out


def _plain_qk(s):
    P, slots = s["case"]["page"], s["slots"]
    q, k = _qk(s, torch.float32)
    s["k_cache"][slots // P, slots % P] = k.to(s["k_cache"].dtype)
    s["v_cache"][slots // P, slots % P] = s["v"]
    return dict(q=q.to(s["q"].dtype), k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_attn(s):
    c, T, n = s["case"], s["T"], s["n_max"]
    Hkv, D = c["Hkv"], c["D"]
    G = c["Hq"] // Hkv
    ctx, start = s["ctx"].long(), s["q_start"].long()
    new = start[1:] - start[:-1]
    pages = s["table"][:, :s["width"]].long().clamp(min=0)
    k, v = (t[pages].flatten(1, 2).permute(0, 2, 1, 3).float() for t in (s["k_cache"], s["v_cache"]))  # [B, Hkv, K, D]
    K, B = k.shape[2], ctx.numel()
    row = (start[:-1, None] + torch.arange(n, device=DEV)).clamp(max=T - 1)
    q = s["q"][row].float().view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    x = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, n, G, K).mul_(s["scale"])
    j = torch.arange(K, device=DEV)[None, :] - ctx[:, None]  # place among the new tokens
    word = (j >> LOG2_WORD).clamp(0, s["mask"].shape[1] - 1)[:, None, :].expand(B, n, K)
    bit = (torch.gather(s["mask"][row].long(), 2, word) >> (j & 31)[:, None, :]) & 1
    seen = (j < 0)[:, None, :] | ((j[:, None, :] < new[:, None, None]) & (bit == 1) & (j >= 0)[:, None, :])
    x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, n * G, K), v).view(B, Hkv, n, G, D) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total))[..., 0]
    b, i, _ = _owners(new, T)
    out = o.permute(0, 2, 1, 3, 4)[b, i].reshape(T, c["Hq"], D).to(s["q"].dtype)
    return dict(out=out, lse=lse.permute(0, 2, 1, 3)[b, i].reshape(T, c["Hq"]))


def _plain_logprob(s):
    x = s["logits"].float()
    T, V = x.shape
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    logs = (x - m) - torch.log(total)
    entropy = -torch.where(e > 0, e * logs, torch.zeros_like(e)).sum(-1) / total[:, 0]
    out = dict(logprob=logs.gather(1, s["tokens"].long()[:, None])[:, 0], entropy=entropy)
    if s["case"]["top"]:
        bits = x.view(torch.int32).long()  # a whole number in the logits' order, the lower index first among equals
        order = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF))
        key = (order << 20) + (V - 1 - torch.arange(V, device=DEV))[None, :]
        best = torch.topk(key, s["case"]["top"], dim=1)[0]
        ids = V - 1 - (best & ((1 << 20) - 1))
        out.update(top_ids=ids.to(torch.int32), top_logprobs=logs.gather(1, ids))
    return out


_PLAIN = dict(plan=_plain_plan, qk=_plain_qk, attn=_plain_attn, logprob=_plain_logprob)


# ---------------------------------------------------------------- the library's calls

def _at(t):
    return 0 if t is None else t.data_ptr()


def _library_cache(ft, s):
    k, v = s["k_cache"], s["v_cache"]
    return ft.make_kv_cache(k=_at(k), v=_at(v), dtype=_library_dtype(ft, k), num_pages=k.shape[0], page_size=k.shape[1],
                            kv_heads=k.shape[2], head_dim=k.shape[3], k_page_stride=k.stride(0),
                            k_token_stride=k.stride(1), k_head_stride=k.stride(2), v_page_stride=v.stride(0),
                            v_token_stride=v.stride(1), v_head_stride=v.stride(2))


def _library_dtype(ft, t):
    return {torch.bfloat16: ft.FT_DTYPE_BF16, torch.float16: ft.FT_DTYPE_F16, torch.float32: ft.FT_DTYPE_F32}[t.dtype]


def _library_call(s):
    """The call on a state's buffers and what it writes: a program that keeps its buffers fills the arguments once."""
    import expert_cache_host_gb300 as ft
    c = s["case"]
    if c["op"] == "plan":
        args = ft.make_plan_args(ctx_len=_at(s["ctx"]), new_len=_at(s["new"]), parents=_at(s["parents"]),
                                 free_pages=_at(s["free"]), free_count=_at(s["free_count"]),
                                 block_table=_at(s["table"]), q_start=_at(s["q_start"]), slots=_at(s["slots"]),
                                 positions=_at(s["positions"]), mask=_at(s["mask"]), free_left=_at(s["free_left"]),
                                 num_reqs=c["B"], page_size=c["page"], table_width=s["table"].shape[1],
                                 max_tokens=s["T"], mask_words=_words(c) if c["tree"] else 0)
        names = ["table", "q_start", "slots", "free_left", "positions"] + (["mask"] if c["tree"] else [])
        return ft.ft_kv_plan, args, {n: s[n] for n in names}
    if c["op"] == "qk":
        args = ft.make_qk_args(q=_at(s["q"]), k=_at(s["k"]), v=_at(s["v"]), q_weight=_at(s["q_weight"]),
                               k_weight=_at(s["k_weight"]), cos_sin=_at(s["cos_sin"]), positions=_at(s["positions"]),
                               slots=_at(s["slots"]), q_out=_at(s["q_out"]), q_stride=s["q"].stride(0),
                               k_stride=s["k"].stride(0), v_stride=s["v"].stride(0), q_out_stride=s["q_out"].stride(0),
                               T=c["T"], q_heads=c["Hq"], rot_dim=c["rot"], max_pos=s["max_pos"],
                               interleaved=c["pairs"], eps=s["eps"], cache=_library_cache(ft, s))
        return ft.ft_qk_norm_rope, args, dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    if c["op"] == "attn":
        args = ft.make_attn_args(q=_at(s["q"]), out=_at(s["out"]), lse=_at(s["lse"]), q_start=_at(s["q_start"]),
                                 ctx_len=_at(s["ctx"]), block_table=_at(s["table"]), mask=_at(s["mask"]),
                                 q_stride=s["q"].stride(0), out_stride=s["out"].stride(0), max_tokens=s["T"],
                                 num_reqs=c["B"], q_heads=c["Hq"], table_width=s["table"].shape[1],
                                 mask_words=s["mask"].shape[1], scale=s["scale"], cache=_library_cache(ft, s))
        s["workspace"] = torch.zeros(ft.ft_tree_attention_workspace(args), dtype=torch.uint8, device=DEV)
        args.workspace, args.workspace_bytes = _at(s["workspace"]), s["workspace"].numel()
        return ft.ft_tree_attention, args, dict(out=s["out"], lse=s["lse"])
    x = s["logits"]
    args = ft.make_logprob_args(logits=_at(x), tokens=_at(s["tokens"]), logprob=_at(s["logprob"]),
                                entropy=_at(s["entropy"]), top_ids=_at(s["top_ids"]),
                                top_logprobs=_at(s["top_logprobs"]), row_stride=x.stride(0),
                                dtype=_library_dtype(ft, x), T=c["T"], V=c["V"], top_n=c["top"])
    names = ["logprob", "entropy"] + (["top_ids", "top_logprobs"] if c["top"] else [])
    return ft.ft_token_logprobs, args, {n: s[n] for n in names}


def run(state):
    if not own:
        return _PLAIN[state["case"]["op"]](state)
    if "call" not in state:
        state["call"] = _library_call(state)
    call, args, out = state["call"]
    call(args, torch.cuda.current_stream().cuda_stream)
    return out


# ---------------------------------------------------------------- 64 bits

def _exact_plan(s):
    c, P = s["case"], s["case"]["page"]
    ctx, new = s["ctx"].tolist(), s["new"].tolist()
    table, free = s["table"].cpu().numpy().copy(), s["free"].tolist()
    left = s["free_count"].item()
    slots, positions = [], []
    for b, (n0, n) in enumerate(zip(ctx, new)):
        for page in range(-(-n0 // P), -(-(n0 + n) // P)):
            left -= 1
            table[b, page] = free[left]
        for at in range(n0, n0 + n):
            slots.append(int(table[b, at // P]) * P + at % P)
            positions.append(at)
    starts = _starts(new)
    out = dict(table=torch.from_numpy(table).to(DEV), q_start=_int(starts), slots=_int(slots, torch.int64),
               free_left=_int([left]), positions=_int(positions))
    if c["tree"]:
        parents = s["parents"].tolist()
        owner = [bisect.bisect_right(starts, t) - 1 for t in range(len(slots))]
        out["positions"] = _int([ctx[b] + d for b, d in zip(owner, _depths(parents, new))])
        out["mask"] = torch.from_numpy(_masks(parents, new, _words(c))).to(DEV)
    return out


def _exact_qk(s):
    c, P = s["case"], s["case"]["page"]
    angle = s["cos_sin"].double()[s["positions"].long()]
    half = c["rot"] // 2
    turn = torch.complex(angle[:, :half], angle[:, half:])[:, None, :]
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s[name + "_weight"].double()
        place = torch.arange(c["rot"], device=DEV).view(half, 2) if c["pairs"] else \
            torch.arange(c["rot"], device=DEV).view(2, half).t()
        z = torch.complex(x[..., place[:, 0]], x[..., place[:, 1]]) * turn
        x[..., place[:, 0]], x[..., place[:, 1]] = z.real, z.imag
        out[name] = x
    page, row = s["slots"] // P, s["slots"] % P
    caches = {"k_cache": out.pop("k"), "v_cache": s["v"].double()}
    for name, rows in caches.items():
        out[name] = torch.zeros(s[name].shape, dtype=torch.float64, device=DEV)
        out[name][page, row] = rows
    return out


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
        k, v = (t[pages].flatten(0, 1)[:n0 + n].double().transpose(0, 1) for t in (s["k_cache"], s["v_cache"]))
        bits = np.array([[(int(masks[t0 + i, j >> 5]) >> (j & 31)) & 1 for j in range(n)] for i in range(n)])
        hidden = torch.from_numpy(bits == 0).to(DEV)
        for h in range(Hq):
            x = s["q"][t0:t1, h].double() @ k[h * Hkv // Hq].T * s["scale"]
            x[:, n0:] = x[:, n0:].masked_fill(hidden, -math.inf)
            lse[t0:t1, h] = torch.logsumexp(x, -1)
            out[t0:t1, h] = torch.softmax(x, -1) @ v[h * Hkv // Hq]
    return dict(out=out, lse=lse)


def _exact_logprob(s):
    x = s["logits"].double()
    logs = torch.log_softmax(x, -1)
    p = logs.exp()
    entropy = -(p * logs.masked_fill(p == 0, 0.0)).sum(-1)
    out = dict(logprob=logs[torch.arange(x.shape[0], device=DEV), s["tokens"].long()], entropy=entropy)
    if s["case"]["top"]:
        ids = torch.argsort(x, dim=-1, descending=True, stable=True)[:, :s["case"]["top"]]
        out.update(top_ids=ids.to(torch.int32), top_logprobs=torch.gather(logs, 1, ids))
    return out


_EXACT = dict(plan=_exact_plan, qk=_exact_qk, attn=_exact_attn, logprob=_exact_logprob)


def exact(case, seed):
    """The outputs from the definitions in 64 bits."""
    return _EXACT[case["op"]](prepare(case, seed))
