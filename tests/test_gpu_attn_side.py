"""The attention-side operators against plain 64-bit implementations.

Tolerances, from the arithmetic (u = 2^-8 for bf16, 2^-11 for f16, the half
spacing of the type; sums in fp32):
 - norm + rotation: one rounding at the end, |err| <= u |y| (2^-25 for f16's
   subnormal numbers) plus 2^-18 of the pair's size for the fp32 steps (a
   rotation can cancel).
 - attention: every probability is rounded to the type (u each) and the output
   once: |err| <= u sum p |v| + u |o|, plus 2^-16 sum p |v| for the scores' fp32
   sums and exponentials; f16 probabilities below 2^-14 have a fixed spacing of
   2^-24: sum over keys of 2^-25 |v| at a softmax sum >= 1.
   lse: 2^-16 max(1, largest |score|).
 - log probabilities: V-term fp32 sums in 512-way partial sums and a 2^-22
   exponential: 1e-5 + 1e-6 |value|.
Whole numbers are equal.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module")
def ft():
    from expert_cache_host_gb300 import build as ftbuild
    ftbuild.build()
    import expert_cache_host_gb300 as lib
    lib.load()
    return lib


def code(ft, t):
    return {torch.bfloat16: ft.FT_DTYPE_BF16, torch.float16: ft.FT_DTYPE_F16, torch.float32: ft.FT_DTYPE_F32}[t.dtype]


def at(t):
    return 0 if t is None else t.data_ptr()


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def stream():
    return torch.cuda.current_stream().cuda_stream


def kv(ft, k, v):
    """ft_kv_cache of two [page, row, head, D] views."""
    return ft.make_kv_cache(k=at(k), v=at(v), dtype=code(ft, k), num_pages=k.shape[0], page_size=k.shape[1],
                            kv_heads=k.shape[2], head_dim=k.shape[3], k_page_stride=k.stride(0),
                            k_token_stride=k.stride(1), k_head_stride=k.stride(2), v_page_stride=v.stride(0),
                            v_token_stride=v.stride(1), v_head_stride=v.stride(2))


# ---------------------------------------------------------------- plan

def plan_reference(ctx, new, parents, free, table, P, max_tokens, words):
    table, left = table.copy(), len(free)
    slots, pos, masks, starts = [], [], [], [0]
    for b, (c, n) in enumerate(zip(ctx, new)):
        for page in range(-(-c // P), -(-(c + n) // P)):
            left -= 1
            table[b, page] = free[left]
        depth, anc, base = [], [], starts[-1]
        for i in range(n):
            slots.append(int(table[b, (c + i) // P]) * P + (c + i) % P)
            p = parents[base + i] if parents is not None else i - 1
            depth.append(0 if p < 0 else depth[p] + 1)
            anc.append((0 if p < 0 else anc[p]) | (1 << i))
            pos.append(c + (depth[i] if parents is not None else i))
            masks.append([(anc[i] >> (32 * w)) & 0xFFFFFFFF for w in range(words)])
        starts.append(base + n)
    pad = max_tokens - len(slots)
    return (table, starts, slots + [-1] * pad, pos + [0] * pad,
            np.array(masks + [[0] * words] * pad, dtype=np.uint32).reshape(max_tokens, words), left)


def run_plan(ft, ctx, new, parents, free, table, P, max_tokens, words=0, free_count=None):
    B = len(ctx)
    t = dict(ctx=dev(ctx), new=dev(new), parents=None if parents is None else dev(parents + [-1] * (max_tokens - len(parents))),
             free=dev(free if len(free) else [0]), count=dev([len(free) if free_count is None else free_count]),
             table=dev(table), q_start=dev([-7] * (B + 1)), slots=dev([-7] * max(1, max_tokens), torch.int64),
             pos=dev([-7] * max(1, max_tokens)), mask=dev(np.full((max(1, max_tokens), max(1, words)), -7)),
             left=dev([-7]), status=dev([0]))
    args = ft.make_plan_args(ctx_len=at(t["ctx"]), new_len=at(t["new"]), parents=at(t["parents"]), free_pages=at(t["free"]),
                             free_count=at(t["count"]), block_table=at(t["table"]), q_start=at(t["q_start"]),
                             slots=at(t["slots"]), positions=at(t["pos"]), mask=at(t["mask"]) if parents is not None else 0,
                             free_left=at(t["left"]), status=at(t["status"]), num_reqs=B, page_size=P,
                             table_width=table.shape[1], max_tokens=max_tokens, mask_words=words)
    ft.ft_kv_plan(args, stream())
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in t.items() if v is not None}


def random_plan(rng, B, ctx_hi, n_lo, n_hi, P, tree):
    ctx = [int(rng.integers(0, ctx_hi + 1)) for _ in range(B)]
    new = [int(rng.integers(n_lo, n_hi + 1)) for _ in range(B)]
    width = (ctx_hi + n_hi) // P + 2
    held = [-(-c // P) for c in ctx]
    ids = rng.permutation(sum(held) + sum(-(-(c + n) // P) - h for c, n, h in zip(ctx, new, held)) + 5).tolist()
    table = np.full((B, width), -1, dtype=np.int32)
    for b, h in enumerate(held):
        table[b, :h] = ids[:h]
        ids = ids[h:]
    parents = [int(rng.integers(-1, i)) if i else -1 for n in new for i in range(n)] if tree else None
    return ctx, new, parents, ids, table


@pytest.mark.parametrize("B,ctx_hi,n_lo,n_hi,P,tree", [
    (1, 0, 1, 1, 16, False), (1, 5, 0, 0, 16, False), (1, 100, 700, 700, 8, False), (7, 300, 0, 40, 16, True),
    (300, 64, 0, 3, 1, False), (1030, 500, 0, 9, 32, True), (2100, 40, 1, 1, 16, False), (3, 10, 200, 300, 64, True),
    (40, 2000, 1, 65, 128, True)])
def test_plan(ft, B, ctx_hi, n_lo, n_hi, P, tree):
    rng = np.random.default_rng(B * 1000 + n_hi)
    ctx, new, parents, free, table = random_plan(rng, B, ctx_hi, n_lo, n_hi, P, tree)
    words = (n_hi + 31) // 32 if tree else 0
    T = sum(new) + 3
    want = plan_reference(ctx, new, parents, free, table, P, T, words)
    got = run_plan(ft, ctx, new, parents, free, table, P, T, words)
    assert got["status"][0] == 0
    for name, w in zip(("table", "q_start", "slots", "pos"), want):
        assert np.array_equal(got[name], np.asarray(w)), name
    if tree:
        assert np.array_equal(got["mask"].view(np.uint32), want[4])
    assert got["left"][0] == want[5]


def test_plan_chain_given_as_parents_is_the_sequence(ft):
    n, P = 70, 16
    table = np.full((1, 8), -1, dtype=np.int32)
    a = run_plan(ft, [3], [n], list(range(-1, n - 1)), list(range(20)), np.where(np.arange(8) < 1, 19, -1).astype(np.int32)[None], P, n, 3)
    b = run_plan(ft, [3], [n], None, list(range(20)), np.where(np.arange(8) < 1, 19, -1).astype(np.int32)[None], P, n)
    assert np.array_equal(a["pos"], b["pos"]) and np.array_equal(a["slots"], b["slots"])
    want = [(1 << (i + 1)) - 1 for i in range(n)]
    got = [sum(int(w) << (32 * k) for k, w in enumerate(r)) for r in a["mask"].view(np.uint32)]
    assert got == want


def test_plan_out_of_pages_columns_and_rows(ft):
    P = 16
    table = np.array([[5, -1, -1], [-1, -1, -1]], dtype=np.int32)
    # 3 fresh pages wanted (request 0: column 1; request 1: columns 0, 1), 2 there
    r = run_plan(ft, [10, 0], [10, 20], None, [7, 8], table, P, 30)
    assert r["status"][0] == ft.FT_ST_NO_ROOM and r["left"][0] == 0
    assert r["table"].tolist() == [[5, 8, -1], [7, -1, -1]]
    assert r["slots"].tolist() == [5 * 16 + 10 + i for i in range(6)] + [8 * 16 + i for i in range(4)] + \
        [7 * 16 + i for i in range(16)] + [-1] * 4
    # a request longer than its row of the table
    r = run_plan(ft, [40], [20], None, [3, 4], np.array([[0, 1, 2]], dtype=np.int32), P, 20)
    assert r["status"][0] == ft.FT_ST_NO_ROOM and r["slots"].tolist() == [2 * 16 + 8 + i for i in range(8)] + [-1] * 12
    # 30 new tokens, rows for 14: the last request is cut
    r = run_plan(ft, [0, 0], [10, 20], None, [0, 1, 2, 3], np.full((2, 3), -1, dtype=np.int32), P, 14)
    assert r["status"][0] == ft.FT_ST_NO_ROOM and r["q_start"].tolist() == [0, 10, 14]
    assert r["left"][0] == 2 and r["slots"].tolist() == [3 * 16 + i for i in range(10)] + [2 * 16 + i for i in range(4)]
    # a negative length is an empty request
    r = run_plan(ft, [-4, 0], [5, 2], None, [0, 1], np.full((2, 3), -1, dtype=np.int32), P, 4)
    assert r["status"][0] == ft.FT_ST_NO_ROOM and r["q_start"].tolist() == [0, 0, 2]


def test_plan_bad_parents_and_small_mask(ft):
    table = np.full((1, 4), -1, dtype=np.int32)
    r = run_plan(ft, [0], [4], [-1, 1, 0, -5], [0, 1], table, 16, 4, 1)  # 1's parent is itself, 3's is none at all
    assert r["status"][0] == ft.FT_ST_BAD_TREE
    assert r["mask"].tolist() == [[1], [2], [5], [8]] and r["pos"].tolist() == [0, 0, 1, 0]
    r = run_plan(ft, [0], [40], [i - 1 for i in range(40)], [0, 1, 2], table, 16, 40, 1)
    assert r["status"][0] == ft.FT_ST_BAD_TREE
    assert r["mask"].view(np.uint32)[:, 0].tolist() == [(1 << (i + 1)) - 1 if i < 32 else 0xFFFFFFFF for i in range(40)]


def test_plan_without_requests_marks_padding(ft):
    r = run_plan(ft, [], [], None, [1, 2], np.zeros((1, 1), dtype=np.int32)[:0].reshape(0, 1), 16, 5)
    assert r["q_start"].tolist() == [0] and r["left"][0] == 2
    assert r["slots"].tolist() == [-1] * 5 and r["pos"].tolist() == [0] * 5


# ---------------------------------------------------------------- norm + rotation

def rope_table(max_pos, rot):
    half = rot // 2
    ang = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(half) / max(1, half))
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float().cuda()


def rope_reference(x, w, cs, pos, rot, pairs, eps):
    x, w, cs = x.double().cpu().numpy(), w.double().cpu().numpy(), cs.double().cpu().numpy()
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    half = rot // 2
    size = np.abs(y)
    for t, p in enumerate(pos):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
            c, s = cs[p, i], cs[p, half + i]
            ya, yb = y[t, :, a].copy(), y[t, :, b].copy()
            y[t, :, a], y[t, :, b] = ya * c - yb * s, yb * c + ya * s
            size[t, :, a] = size[t, :, b] = np.hypot(ya, yb)
    return y, size


def check_rope(got, y, size, u, where):
    got = got.double().cpu().numpy()
    tol = np.maximum(u * np.abs(y), 2.0 ** -25 if u == U["f16"] else 0) + 2.0 ** -18 * size + 1e-30
    assert np.isfinite(got).all(), where
    assert (np.abs(got - y) <= tol * (1 + 1e-6)).all(), (where, np.max(np.abs(got - y) / tol))


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,pairs,dtype,P,layout,pad", [
    (1, 32, 4, 128, 128, False, "bf16", 16, "token", 0), (1, 1, 1, 64, 64, True, "f16", 8, "head", 0),
    (37, 5, 5, 64, 32, False, "f16", 32, "head", 8), (130, 7, 1, 128, 64, True, "bf16", 64, "token", 3),
    (3, 8, 2, 256, 64, False, "bf16", 16, "token", 0), (9, 8, 2, 256, 256, False, "f16", 16, "head", 1),
    (2000, 6, 2, 128, 128, False, "bf16", 16, "token", 40), (1500, 12, 4, 64, 64, False, "f16", 128, "head", 5),
    (5, 4, 2, 128, 0, False, "bf16", 16, "token", 0), (5, 4, 2, 128, 16, False, "bf16", 16, "token", 0)])
def test_qk_norm_rope(ft, T, Hq, Hkv, D, rot, pairs, dtype, P, layout, pad):
    g = torch.Generator(device="cuda").manual_seed(T * 7 + D)
    dt = DT[dtype]
    ld = (Hq + 2 * Hkv) * D + pad
    qkv = (torch.randn((T, ld), generator=g, device="cuda") * 2).to(dt)
    qkv[0] *= 1e-3  # eps matters
    if T > 1:
        qkv[1] = 0
    q, k, v = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D]
    qw, kw = ((torch.randn(D, generator=g, device="cuda") + 1).to(dt) for _ in range(2))
    pages, max_pos = -(-T // P) + 2, 300
    shape = (pages, P, Hkv, D) if layout == "token" else (pages, Hkv, P, D)
    kc, vc = (torch.full(shape, 7.0, device="cuda", dtype=dt) for _ in range(2))
    if layout == "head":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    slots = torch.randperm(pages * P, generator=g, device="cuda")[:T].contiguous()
    pos = torch.randint(0, max_pos, (T,), generator=g, device="cuda", dtype=torch.int32)
    cs = rope_table(max_pos, rot) if rot else torch.zeros(4, device="cuda")
    out = torch.full((T, Hq * D + pad), 3.0, device="cuda", dtype=dt)
    status = dev([0])
    args = ft.make_qk_args(q=at(q), k=at(k), v=at(v), q_weight=at(qw), k_weight=at(kw), cos_sin=at(cs), positions=at(pos),
                           slots=at(slots), q_out=at(out), status=at(status), q_stride=ld, k_stride=ld, v_stride=ld,
                           q_out_stride=out.stride(0), T=T, q_heads=Hq, rot_dim=rot, max_pos=max_pos, interleaved=pairs,
                           eps=1e-5, cache=kv(ft, kc, vc))
    ft.ft_qk_norm_rope(args, stream())
    torch.cuda.synchronize()
    assert status.item() == 0
    u, p = U[dtype], pos.tolist()
    check_rope(out[:, :Hq * D].unflatten(1, (Hq, D)), *rope_reference(q.unflatten(1, (Hq, D)), qw, cs, p, rot, pairs, 1e-5), u, "q")
    assert pad == 0 or bool((out[:, Hq * D:] == 3).all())
    at_slot = lambda c: c[slots // P, slots % P]
    check_rope(at_slot(kc), *rope_reference(k.unflatten(1, (Hkv, D)), kw, cs, p, rot, pairs, 1e-5), u, "k")
    assert torch.equal(at_slot(vc), v.unflatten(1, (Hkv, D)))
    free = torch.ones(pages * P, dtype=torch.bool, device="cuda")
    free[slots] = False
    idle = free.nonzero()[:, 0]
    for c in (kc, vc):
        assert bool((c[idle // P, idle % P] == 7).all())
    # in place
    want = out[:, :Hq * D].clone()
    args.q_out, args.q_out_stride = at(q), ld
    ft.ft_qk_norm_rope(args, stream())
    torch.cuda.synchronize()
    assert torch.equal(q, want)


def test_qk_padding_and_faults(ft):
    T, Hq, Hkv, D, P = 6, 2, 1, 64, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((T, h * D), generator=g, device="cuda").half() for h in (Hq, Hkv, Hkv))
    w = torch.ones(D, device="cuda").half()
    kc, vc = (torch.full((2, P, Hkv, D), 7.0, device="cuda").half() for _ in range(2))
    out = torch.full((T, Hq * D), 3.0, device="cuda").half()
    cs = rope_table(10, D)

    def call(slots, pos):
        status = dev([0])
        s, p = dev(slots, torch.int64), dev(pos)
        ft.ft_qk_norm_rope(ft.make_qk_args(q=at(q), k=at(k), v=at(v), q_weight=at(w), k_weight=at(w), cos_sin=at(cs),
                                           positions=at(p), slots=at(s), q_out=at(out), status=at(status), q_stride=Hq * D,
                                           k_stride=D, v_stride=D, q_out_stride=Hq * D, T=T, q_heads=Hq, rot_dim=D,
                                           max_pos=10, interleaved=0, eps=1e-6, cache=kv(ft, kc, vc)), stream())
        torch.cuda.synchronize()
        return status.item()

    assert call([-1, 3, -1, 4, -1, -1], [0, 1, 2, 3, 4, 5]) == 0  # padding
    written = [i for i in range(16) if not bool((kc.view(16, D)[i] == 7).all())]
    assert written == [3, 4] and bool((out != 3).any(1).all())
    assert call([0, 16, -1, -1, -1, -1], [0] * 6) == ft.FT_ST_BAD_SLOT
    assert call([5, 6, -1, -1, -1, -1], [10, -1, 0, 0, 0, 0]) == ft.FT_ST_BAD_TOKEN
    assert bool((out[:2] == 0).all()) and bool((out[2:] != 0).any(1).all())
    assert bool((kc.view(16, D)[5:7] == 7).all()) and bool((vc.view(16, D)[5:7] == 7).all())


# ---------------------------------------------------------------- attention

class Attn:
    """A batch of requests over a paged cache whose unused rows hold NaN."""

    def __init__(self, ft, ctx, new, Hq, Hkv, D, dtype, P, layout="token", mask="tree", seed=0, scale=None, spare=3, bias=0.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ft, self.ctx, self.new, self.D, self.P, self.dtype = ft, ctx, new, D, P, dtype
        self.Hq, self.Hkv = Hq, Hkv
        dt = DT[dtype]
        held = [-(-(c + n) // P) for c, n in zip(ctx, new)]
        pages = sum(held) + spare
        shape = (pages, P, Hkv, D) if layout == "token" else (pages, Hkv, P, D)
        self.k, self.v = (torch.full(shape, float("nan"), device="cuda", dtype=dt) for _ in range(2))
        if layout == "head":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        ids = rng.permutation(pages)
        self.width = max(held + [1]) + 2
        table = np.full((len(ctx), self.width), -1, dtype=np.int32)
        self.rows = []  # each request's (page, row) of every key
        for b, h in enumerate(held):
            table[b, :h], ids = ids[:h], ids[h:]
            idx = np.arange(ctx[b] + new[b])
            self.rows.append((torch.from_numpy(table[b, idx // P].astype(np.int64)).cuda(), torch.from_numpy(idx % P).cuda()))
            for c in (self.k, self.v):
                c[self.rows[b]] = (torch.randn((len(idx), Hkv, D), generator=g, device="cuda") + bias).to(dt)
        self.table = dev(table)
        self.T = sum(new)
        self.q = torch.randn((max(1, self.T), Hq, D), generator=g, device="cuda").to(dt)
        self.start = np.concatenate([[0], np.cumsum(new)]).tolist()
        self.seen = []  # [n, n] of each request
        words = (max(new + [1]) + 31) // 32
        m = np.zeros((max(1, self.T), words), dtype=np.uint32)
        for b, n in enumerate(new):
            s = np.zeros((n, n), dtype=bool)
            for i in range(n):
                if mask == "chain":
                    s[i, :i + 1] = True
                elif mask == "tree":
                    p = int(rng.integers(-1, i)) if i else -1
                    if p >= 0:
                        s[i] = s[p]
                    s[i, i] = True
                elif mask == "random":
                    s[i] = rng.random(n) < 0.4
                elif mask == "none":
                    pass
            self.seen.append(s)
            for i in range(n):
                for j in np.nonzero(s[i])[0]:
                    m[self.start[b] + i, j >> 5] |= np.uint32(1 << (j & 31))
        self.mask = None if mask == "chain" else torch.from_numpy(m.view(np.int32)).cuda()
        self.words = 0 if mask == "chain" else words
        self.scale = D ** -0.5 if scale is None else scale
        self.out = torch.full((max(1, self.T), Hq, D), 5.0, device="cuda", dtype=dt)
        self.lse = torch.full((max(1, self.T), Hq), 5.0, device="cuda")
        self.status = dev([0])
        self.d_start, self.d_ctx = dev(self.start), dev(ctx if len(ctx) else [0])
        self.args = ft.make_attn_args(q=at(self.q), out=at(self.out), lse=at(self.lse), q_start=at(self.d_start),
                                      ctx_len=at(self.d_ctx), block_table=at(self.table), mask=at(self.mask),
                                      status=at(self.status), q_stride=Hq * D, out_stride=Hq * D, max_tokens=self.T,
                                      num_reqs=len(ctx), q_heads=Hq, table_width=self.width, mask_words=self.words,
                                      scale=self.scale, cache=kv(ft, self.k, self.v))
        self.ws = torch.zeros(ft.ft_tree_attention_workspace(self.args), dtype=torch.uint8, device="cuda")
        self.args.workspace, self.args.workspace_bytes = at(self.ws), self.ws.numel()

    def run(self, st=None):
        self.ft.ft_tree_attention(self.args, stream() if st is None else st)
        torch.cuda.synchronize()
        return self

    def reference(self):
        """(out, lse, sum p|v|, largest |score|, keys) in 64 bits; rows that see nothing: 0, -inf."""
        T, Hq, D, G = self.T, self.Hq, self.D, self.Hq // self.Hkv
        out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
        lse, top = np.full((T, Hq), -np.inf), np.ones((T, Hq))
        q = self.q.double().cpu().numpy()
        for b, (c, n) in enumerate(zip(self.ctx, self.new)):
            k, v = (x[self.rows[b]].double().cpu().numpy() for x in (self.k, self.v))
            for i in range(n):
                keys = np.concatenate([np.arange(c), c + np.nonzero(self.seen[b][i])[0]]).astype(int)
                if not len(keys):
                    continue
                t = self.start[b] + i
                for h in range(Hq):
                    s = k[keys, h // G] @ q[t, h] * self.scale
                    m = s.max()
                    p = np.exp(s - m)
                    lse[t, h] = m + math.log(p.sum())
                    p /= p.sum()
                    out[t, h], mag[t, h] = p @ v[keys, h // G], p @ np.abs(v[keys, h // G])
                    top[t, h] = max(1.0, np.abs(s).max())
        return out, lse, mag, top

    def check(self, where=""):
        out, lse, mag, top = self.reference()
        got = self.out.double().cpu().numpy()[:self.T]
        u = U[self.dtype]
        tol = u * mag + u * np.abs(out) + 2.0 ** -16 * mag + 1e-30
        if self.dtype == "f16":
            tol = tol + 2.0 ** -25 * (max(c + n for c, n in zip(self.ctx, self.new)) * 6.0)
        assert np.isfinite(got).all(), where
        bad = np.abs(got - out) / tol
        assert bad.max(initial=0) <= 1, (where, bad.max(), np.unravel_index(bad.argmax(), bad.shape))
        got_lse = self.lse.double().cpu().numpy()[:self.T]
        empty = np.isinf(lse)
        assert np.array_equal(np.isinf(got_lse), empty), where
        err = np.abs(got_lse[~empty] - lse[~empty]) / (2.0 ** -16 * top[~empty])
        assert err.max(initial=0) <= 1, (where, err.max())


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,dtype,P,layout,mask", [
    ([0], [1], 1, 1, 64, "bf16", 8, "token", "chain"), ([1], [1], 8, 1, 128, "bf16", 16, "token", "chain"),
    ([127], [1], 32, 4, 128, "bf16", 16, "token", "chain"), ([128], [1], 32, 4, 128, "f16", 16, "head", "chain"),
    ([1000], [1], 16, 2, 64, "f16", 64, "token", "chain"), ([3000], [1], 32, 4, 128, "bf16", 16, "token", "tree"),
    ([5, 0, 260, 77], [1, 1, 1, 1], 8, 2, 128, "bf16", 16, "head", "chain"),
    ([100, 0, 300, 7], [17, 5, 0, 33], 8, 2, 128, "bf16", 16, "token", "tree"),
    ([100, 0, 300, 7], [17, 5, 0, 33], 10, 2, 64, "f16", 32, "head", "tree"),
    ([250, 511], [64, 64], 16, 2, 128, "bf16", 128, "token", "tree"),
    ([40], [100], 8, 1, 128, "bf16", 16, "token", "random"), ([0, 130], [40, 70], 3, 3, 64, "bf16", 256, "head", "random"),
    ([900, 10], [31, 2], 7, 1, 128, "f16", 16, "token", "chain"), ([0], [300], 4, 2, 128, "bf16", 16, "token", "chain"),
    ([2000], [40], 128, 1, 64, "bf16", 512, "token", "tree"), ([129, 1], [200, 1], 5, 5, 64, "f16", 8, "head", "chain"),
    ([4000, 3, 1200, 0, 640], [2, 3, 9, 1, 16], 48, 8, 128, "bf16", 16, "token", "tree")])
def test_attention(ft, ctx, new, Hq, Hkv, D, dtype, P, layout, mask):
    a = Attn(ft, ctx, new, Hq, Hkv, D, dtype, P, layout, mask, seed=len(ctx) + D + P).run()
    a.check()
    assert a.status.item() == 0


def test_attention_rows_that_see_nothing(ft):
    """An empty context and an empty mask: zeros and -inf, beside rows of other requests that see keys."""
    a = Attn(ft, [0, 50, 0], [3, 3, 20], 8, 2, 128, "bf16", 16, mask="none", seed=3).run()
    a.check()
    assert bool((a.out[:3] == 0).all()) and bool((a.out[6:] == 0).all()) and bool((a.out[3:6] != 0).any())


def test_attention_without_lse_and_twice(ft):
    """The workspace is ready again after every call; results repeat bit by bit."""
    a = Attn(ft, [3000, 20, 900], [9, 1, 40], 32, 4, 128, "bf16", 16, seed=4).run()
    first, lse = a.out.clone(), a.lse.clone()
    for _ in range(3):
        a.out.fill_(1)
        a.run()
        assert torch.equal(a.out, first) and torch.equal(a.lse, lse)
    a.args.lse = None
    a.out.fill_(1)
    a.lse.fill_(9)
    a.run()
    assert torch.equal(a.out, first) and bool((a.lse == 9).all())


@pytest.mark.parametrize("scale,bias", [(3.0, 0.0), (-0.5, 0.0), (0.0, 0.0), (1.0, 2.0)])
def test_attention_scales(ft, scale, bias):
    """Sharp, reversed and flat softmax, and scores that grow along the context."""
    a = Attn(ft, [700, 90], [5, 12], 16, 4, 64, "bf16", 16, seed=5, scale=scale, bias=bias)
    a.run().check()


def test_attention_growing_scores(ft):
    """Each key's score above the one before it: the running maximum moves at every step."""
    a = Attn(ft, [600], [3], 8, 1, 128, "bf16", 16, seed=6, scale=1.0)
    ramp = torch.linspace(-40, 60, 603, device="cuda")
    a.k[a.rows[0]] = 0
    a.q.zero_()
    a.q[:, :, 0] = 1
    kk = a.k[a.rows[0]]
    kk[:, :, 0] = ramp[:, None].to(kk.dtype)
    a.k[a.rows[0]] = kk
    a.run().check()


@pytest.mark.parametrize("dtype,size,scale", [("f16", 8000.0, 0.25), ("bf16", 1e6, None), ("bf16", 1e15, None),
                                              ("bf16", 1e6, -0.1), ("f16", 1000.0, None), ("bf16", 3000.0, -0.1)])
def test_attention_scores_far_from_zero(ft, dtype, size, scale):
    """Scores of 1e6 to 1e31: the row is its largest score's value wherever that stands clear of the scores' fp32 sums."""
    ctx, new = [700, 33, 0], [3, 20, 5]
    a = Attn(ft, ctx, new, 8, 2, 128, dtype, 16, mask="chain", seed=17, scale=scale)
    a.q.mul_(size)
    a.k.mul_(size)
    a.run()
    got, lse = a.out.double().cpu().numpy(), a.lse.double().cpu().numpy()
    assert np.isfinite(got).all() and np.isfinite(lse).all()
    q, clear = a.q.double().cpu().numpy(), 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        k, v = (x[a.rows[b]].double().cpu().numpy() for x in (a.k, a.v))
        for i in range(n):
            for h in range(8):
                kk, t = k[:c + i + 1, h // 4], a.start[b] + i
                s = kk @ q[t, h] * a.scale
                err = 2.0 ** -17 * np.max(np.abs(kk) @ np.abs(q[t, h])) * abs(a.scale)  # 128 fp32 sums
                first, second = s.argmax(), np.sort(s)[-2] if len(s) > 1 else -np.inf
                assert abs(lse[t, h] - s.max()) <= err + 10
                if s.max() - second > 2 * err + 40:
                    clear += 1
                    want = v[first, h // 4]
                    assert (np.abs(got[t, h] - want) <= 2 * U[dtype] * np.abs(want) + 2.0 ** -16).all()
    assert clear > 8 * 28 // 2


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min])
def test_attention_unseen_keys_take_no_part(ft, value):
    """Unusual numbers in new keys and values that a row does not see (other branches of its tree) and past the
    request's end; the rows that see one are left out of the comparison."""
    a = Attn(ft, [130, 20], [12, 40], 8, 2, 128, "bf16", 16, mask="tree", seed=7)
    bad = {0: 4, 1: 33}
    for b, j in bad.items():
        a.seen[b][:j, j] = False
    clean = a.run().out.clone()
    a.check()
    for b, j in bad.items():
        page, row = a.rows[b][0][a.ctx[b] + j], a.rows[b][1][a.ctx[b] + j]
        a.k[page, row] = value
        a.v[page, row] = value
    a.run()
    for b, j in bad.items():
        for i in range(a.new[b]):
            t = a.start[b] + i
            if not a.seen[b][i, j]:
                assert torch.equal(a.out[t], clean[t]), (b, i)


def test_attention_seen_nan_and_inf_reach_the_output(ft):
    a = Attn(ft, [130], [6], 8, 2, 128, "bf16", 16, mask="chain", seed=8)
    page, row = a.rows[0][0][132], a.rows[0][1][132]  # new token 2
    a.v[page, row, 0, 5] = float("inf")
    a.v[page, row, 1, 7] = float("nan")
    a.run()
    got = a.out.float().cpu().numpy()
    assert np.isfinite(got[:2]).all()
    assert np.isposinf(got[2:, :4, 5]).all() and np.isnan(got[2:, 4:, 7]).all()
    got[2:, :4, 5] = got[2:, 4:, 7] = 0
    assert np.isfinite(got).all()


def test_attention_seen_inf_where_a_cta_has_both_streams(ft):
    """Enough requests that one CTA has an item's context tile and its new tokens' tile: every column of a row that
    sees an infinity gets it, whichever warps write the column."""
    a = Attn(ft, [250] * 80, [4] * 80, 32, 8, 128, "bf16", 16, mask="chain", seed=15)
    for b in range(80):
        a.v[a.rows[b][0][251], a.rows[b][1][251]] = float("inf")  # new token 1, all heads and columns
    for _ in range(3):
        a.out.zero_()
        a.run()
        got = a.out.float().view(80, 4, 32, 128)
        assert bool(torch.isfinite(got[:, 0]).all()) and bool(torch.isposinf(got[:, 1:]).all())


def test_attention_strided_rows_and_shared_buffer(ft):
    """Keys and values interleaved in one buffer, q and out as slices of wider rows."""
    a = Attn(ft, [200, 5], [3, 9], 8, 2, 128, "bf16", 16, seed=9)
    both = torch.full((a.k.shape[0], 16, 2, 2, 128), float("nan"), device="cuda", dtype=a.k.dtype)
    both[:, :, 0], both[:, :, 1] = a.k, a.v
    a.k, a.v = both[:, :, 0], both[:, :, 1]
    wide_q = torch.zeros((a.T, 8 * 128 + 24), device="cuda", dtype=a.k.dtype)
    wide_q[:, 8:8 + 1024] = a.q.view(a.T, -1)
    wide_o = torch.full((a.T, 8 * 128 + 40), 2.0, device="cuda", dtype=a.k.dtype)
    a.args.cache = kv(ft, a.k, a.v)
    a.args.q, a.args.q_stride = at(wide_q) + 16, wide_q.stride(0)
    a.args.out, a.args.out_stride = at(wide_o) + 32, wide_o.stride(0)
    a.run()
    a.out = wide_o[:, 16:16 + 1024].unflatten(1, (8, 128))
    a.check()
    assert bool((wide_o[:, :16] == 2).all()) and bool((wide_o[:, 1040:] == 2).all())


def test_attention_bad_pages_are_reported_and_absent(ft):
    a = Attn(ft, [100, 40], [4, 4], 8, 2, 128, "bf16", 16, mask="chain", seed=10)
    a.table[0, 2] = a.k.shape[0]  # keys 32..47 of request 0
    a.table[1, 1] = -1            # keys 16..31 of request 1
    a.run()
    assert a.status.item() == ft.FT_ST_BAD_SLOT
    # the same as requests without those keys
    for b, lo in ((0, 32), (1, 16)):
        keep = [i for i in range(a.ctx[b] + a.new[b]) if not lo <= i < lo + 16]
        a.rows[b] = tuple(x[keep] for x in a.rows[b])
        a.ctx[b] -= 16
    a.check()


@pytest.mark.parametrize("ctx", [(1 << 31) - 1, (1 << 31) - 256])
def test_attention_request_of_too_many_keys_is_reported_and_left(ft, ctx):
    a = Attn(ft, [100, 20, 300], [4, 3, 5], 8, 2, 128, "bf16", 16, mask="chain", seed=16)
    a.d_ctx[1] = ctx
    a.run()
    assert a.status.item() == ft.FT_ST_BAD_SLOT
    assert bool((a.out[4:7] == 5).all()) and bool((a.lse[4:7] == 5).all())
    got, lse = a.out.clone(), a.lse.clone()
    a.d_ctx[1] = 20
    a.status.zero_()
    a.run()
    a.check()
    for rows in (slice(0, 4), slice(7, 12)):  # split elsewhere, so close and not the same
        assert bool(torch.allclose(got[rows].float(), a.out[rows].float(), atol=2.0 ** -6, rtol=2.0 ** -6))
        assert bool(torch.allclose(lse[rows], a.lse[rows], atol=1e-3))


def test_attention_rows_past_the_last_request_stay(ft):
    a = Attn(ft, [60, 10], [3, 2], 4, 1, 64, "f16", 16, seed=11)
    a.d_start[2] = 4  # the second request's last token is not part of the step
    a.args.max_tokens = 5
    a.run()
    assert bool((a.out[4] == 5).all()) and bool((a.lse[4] == 5).all())
    assert bool((a.out[:4] != 5).any(2).any(1).all())


def test_attention_offsets_past_32_bits(ft):
    """Pages more than 2^32 elements apart."""
    stride = (1 << 32) + 8 * 64
    D, P, Hkv = 64, 16, 1
    buf = torch.empty(stride + 4 * P * D, dtype=torch.bfloat16, device="cuda")
    a = Attn(ft, [20], [2], 4, Hkv, D, "bf16", P, seed=12, spare=0)
    assert a.k.shape[0] == 2
    far = torch.as_strided(buf, (2, P, Hkv, D), (stride, D, D, 1))
    far2 = torch.as_strided(buf, (2, P, Hkv, D), (stride, D, D, 1), P * D)
    far.copy_(a.k)
    far2.copy_(a.v)
    a.k, a.v = far, far2
    a.args.cache = kv(ft, a.k, a.v)
    a.run().check()


def test_attention_on_another_stream_and_in_a_graph(ft):
    a = Attn(ft, [700, 33], [6, 1], 32, 4, 128, "bf16", 16, seed=13)
    want = a.run().out.clone()
    side = torch.cuda.Stream()
    a.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    a.run(side.cuda_stream)
    assert torch.equal(a.out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ft.ft_tree_attention(a.args, stream())
    for _ in range(2):
        a.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, want)


def test_attention_many_requests(ft):
    rng = np.random.default_rng(14)
    ctx = rng.integers(0, 60, 700).tolist()
    new = rng.integers(0, 4, 700).tolist()
    a = Attn(ft, ctx, new, 4, 2, 64, "bf16", 16, seed=14)
    a.run().check()


def gpu_reference(a):
    """Attn.reference on the GPU in 64 bits, for long contexts."""
    T, Hq, D, G = a.T, a.Hq, a.D, a.Hq // a.Hkv
    out, mag = (torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda") for _ in range(2))
    lse, top = (torch.full((T, Hq), v, dtype=torch.float64, device="cuda") for v in (-math.inf, 1.0))
    for b, (c, n) in enumerate(zip(a.ctx, a.new)):
        if n == 0:
            continue
        k, v = (x[a.rows[b]].double() for x in (a.k, a.v))
        hidden = torch.zeros((n, c + n), dtype=torch.bool, device="cuda")
        hidden[:, c:] = torch.from_numpy(~a.seen[b]).cuda()
        t = slice(a.start[b], a.start[b] + n)
        for h in range(Hq):
            s = (a.q[t, h].double() @ k[:, h // G].T * a.scale).masked_fill(hidden, -math.inf)
            top[t, h] = s.masked_fill(hidden, 0).abs().amax(1).clamp(min=1)
            lse[t, h] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            out[t, h], mag[t, h] = p @ v[:, h // G], p @ v[:, h // G].abs()
    return tuple(x.cpu().numpy() for x in (out, lse, mag, top))


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,dtype,P,layout", [
    # many tiles to a CTA, one and two row tiles side by side
    ([21000, 300, 9000, 33000, 5], [32, 1, 17, 5, 40], 32, 4, 128, "bf16", 16, "token"),
    ([30000, 17000, 128, 4097], [3, 50, 1, 64], 40, 8, 64, "f16", 64, "head"),
    ([5000] * 40 + [100] * 40, [1, 20] * 40, 16, 2, 128, "f16", 128, "token")])
def test_attention_long_contexts(ft, ctx, new, Hq, Hkv, D, dtype, P, layout):
    a = Attn(ft, ctx, new, Hq, Hkv, D, dtype, P, layout, seed=sum(new)).run()
    a.reference = lambda: gpu_reference(a)
    a.check()
    assert a.status.item() == 0


def test_attention_back_to_back(ft):
    """Calls of several batches one after another without a pause, each with the result it has alone."""
    batch = [Attn(ft, [9000, 60, 3000], [20, 1, 5], 32, 4, 128, "bf16", 16, seed=20 + i) for i in range(3)]
    want = []
    for a in batch:
        a.run()
        want.append((a.out.clone(), a.lse.clone()))
        a.out.zero_()
    for _ in range(20):
        for a in batch:
            ft.ft_tree_attention(a.args, stream())
    torch.cuda.synchronize()
    for a, (out, lse) in zip(batch, want):
        assert torch.equal(a.out, out) and torch.equal(a.lse, lse) and a.status.item() == 0


# ---------------------------------------------------------------- log probabilities

def run_logprob(ft, x, tokens, top):
    T, V = x.shape
    o = dict(logprob=torch.full((T,), 5.0, device="cuda"), entropy=torch.full((T,), 5.0, device="cuda"),
             ids=torch.full((T, max(1, top)), -7, dtype=torch.int32, device="cuda"),
             lps=torch.full((T, max(1, top)), 5.0, device="cuda"), status=dev([0]))
    tok = dev(tokens)
    ft.ft_token_logprobs(ft.make_logprob_args(logits=at(x), tokens=at(tok), logprob=at(o["logprob"]), entropy=at(o["entropy"]),
                                              top_ids=at(o["ids"]), top_logprobs=at(o["lps"]), status=at(o["status"]),
                                              row_stride=x.stride(0), dtype=code(ft, x), T=T, V=V, top_n=top), stream())
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in o.items()}


def logprob_reference(x, tokens, top):
    x = x.double().cpu().numpy()
    x = np.where(np.isnan(x), -np.inf, x)
    T, V = x.shape
    m = x.max(1, keepdims=True)
    safe = np.where(np.isinf(m), 0, m)
    e = np.exp(x - safe)
    s = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        lp = np.where(s > 0, x - safe - np.log(s), -np.inf)
        p = np.where(s > 0, e / s, 0)
        ent = -np.where(p > 0, p * lp, 0).sum(1)
    ids = np.stack([np.lexsort((np.arange(V), -np.where(np.isinf(r), -1e300, r)))[:top] for r in x]) if top else np.zeros((T, 0), int)
    return lp[np.arange(T), tokens], ent, ids, np.take_along_axis(lp, ids, 1)


def close(got, want):
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], want[inf])
    err = np.abs(got[~inf] - want[~inf]) / (1e-5 + 1e-6 * np.abs(want[~inf]))
    assert err.max(initial=0) <= 1, err.max()


def check_logprob(ft, x, top, seed=0):
    T, V = x.shape
    tokens = np.random.default_rng(seed).integers(0, V, T)
    got = run_logprob(ft, x, tokens, top)
    lp, ent, ids, lps = logprob_reference(x, tokens, top)
    close(got["logprob"], lp)
    close(got["entropy"], ent)
    if top:
        assert np.array_equal(got["ids"], ids)
        close(got["lps"], lps)
    return got


@pytest.mark.parametrize("T,V,top,dtype,pad,lead", [
    (1, 1, 1, "bf16", 0, 0), (3, 7, 7, "f32", 0, 0), (2, 8, 0, "f16", 0, 0), (5, 33, 32, "bf16", 1, 0), (4, 1000, 5, "bf16", 0, 3),
    (1, 131072, 20, "bf16", 0, 0), (2, 100003, 32, "f16", 5, 1), (3, 50021, 9, "f32", 2, 1), (70, 9001, 4, "bf16", 7, 2),
    (700, 4097, 3, "f32", 0, 0), (1300, 2000, 8, "bf16", 3, 5), (9, 16385, 1, "bf16", 0, 0), (40, 65536, 32, "f32", 4, 0)])
def test_logprobs(ft, T, V, top, dtype, pad, lead):
    g = torch.Generator(device="cuda").manual_seed(T + V)
    x = (torch.randn((T, V + pad + lead), generator=g, device="cuda") * 3).to(DT[dtype])[:, lead:lead + V]
    assert check_logprob(ft, x, top)["status"][0] == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "one hot", "two values", "banned", "all banned", "lowest",
                                  "huge", "zeros of both signs", "runs"])
def test_logprobs_unusual_rows(ft, kind, dtype):
    T, V = 3, 20011
    dt = DT[dtype]
    lowest = torch.finfo(dt).min
    i = torch.arange(V, device="cuda", dtype=torch.float64)
    g = torch.Generator(device="cuda").manual_seed(2)
    r = torch.randn((T, V), generator=g, device="cuda")
    x = {"equal": torch.full((T, V), 1.5), "rising": (i / V * 40 - 20).repeat(T, 1), "falling": (20 - i / V * 40).repeat(T, 1),
         "one hot": torch.where(i.cpu() == 12345, 0.0, float(lowest)).repeat(T, 1), "two values": (i % 3 == 0).double().repeat(T, 1),
         "banned": torch.where(r < 1.2, -math.inf, r), "all banned": torch.full((T, V), -math.inf),
         "lowest": torch.full((T, V), float(lowest)), "huge": r * 1e4, "zeros of both signs": torch.where(i % 2 == 0, -0.0, 0.0).repeat(T, 1),
         "runs": (i // 700 % 5).repeat(T, 1)}[kind].to("cuda").to(dt)
    got = check_logprob(ft, x, 32)
    assert got["status"][0] == 0
    if kind == "all banned":
        assert (got["entropy"] == 0).all()


@pytest.mark.parametrize("dtype,base,step", [
    ("f32", 0.0, 1e30), ("bf16", 0.0, 1e30), ("f32", 1e9, 64.0), ("f32", -1e9, 64.0), ("f32", 16777216.0, 2.0),
    ("f32", -16777216.0, 2.0), ("f32", 16777216.0, 1e5), ("bf16", 3e9, 1e7), ("bf16", -3e9, 1e7), ("f32", 1e7, 1.0),
    ("bf16", 16777216.0, 65536.0), ("f32", -1e29, 1e22), ("bf16", -2e30, 1e28)])
def test_logprobs_far_from_zero(ft, dtype, base, step):
    """Rows whose values are large beside their differences, on either side of 2^24 too."""
    for T, V in ((3, 20011), (2, 70001), (400, 300)):
        g = torch.Generator(device="cuda").manual_seed(V)
        x = (base + torch.randn((T, V), generator=g, device="cuda", dtype=torch.float64) * step).to(DT[dtype])
        assert check_logprob(ft, x, 5)["status"][0] == 0


def test_logprobs_nan_inf_and_bad_tokens(ft):
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((6, 5003), generator=g, device="cuda").to(torch.bfloat16)
    x[1, 17] = float("nan")
    x[1, 5001] = float("nan")
    x[2, 4000] = float("inf")
    tokens = [3, 4, 5, -1, 5003, 6]
    got = run_logprob(ft, x, tokens, 4)
    assert got["status"][0] == ft.FT_ST_NAN | ft.FT_ST_BAD_TOKEN
    lp, ent, ids, lps = logprob_reference(x[[0, 1, 5]], np.array([3, 4, 6]), 4)
    for key, want in (("logprob", lp), ("entropy", ent), ("lps", lps)):
        close(got[key][[0, 1, 5]], want)
    assert np.array_equal(got["ids"][[0, 1, 5]], ids)
    assert np.isnan(got["logprob"][[2, 3, 4]]).all() and np.isnan(got["entropy"][2]) and np.isnan(got["lps"][2]).all()
    assert got["ids"][2, 0] == 4000
    assert run_logprob(ft, x[3:5], [-1, -100], 1)["status"][0] == 0


def test_logprobs_optional_outputs_and_offsets_past_32_bits(ft):
    g = torch.Generator(device="cuda").manual_seed(4)
    stride = (1 << 32) + 9
    buf = torch.empty(stride + 3000, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (2, 3000), (stride, 1))
    x.copy_(torch.randn((2, 3000), generator=g, device="cuda"))
    check_logprob(ft, x, 6)
    ent = torch.zeros(2, device="cuda")
    ft.ft_token_logprobs(ft.make_logprob_args(logits=at(x), entropy=at(ent), row_stride=stride, dtype=ft.FT_DTYPE_BF16, T=2,
                                              V=3000, top_n=0), stream())
    torch.cuda.synchronize()
    close(ent.cpu().numpy(), logprob_reference(x, [0, 0], 0)[1])


@pytest.mark.parametrize("T,V", [(1, 131072), (40, 30011), (400, 20000), (3, 700)])
@pytest.mark.parametrize("top", [0, 5])
def test_logprobs_nan_is_reported_wherever_it_lies(ft, T, V, top):
    """One NaN in one row, at places that fall to every warp of every CTA of a row, and in the ragged ends."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((T, V + 3), generator=g, device="cuda").to(torch.bfloat16)[:, 1:V + 1]  # not on 16 bytes
    logprob, tok, ids = torch.zeros(T, device="cuda"), dev([0] * T), dev([0] * (T * 5))
    lps = torch.zeros(T * 5, device="cuda")
    places = sorted({0, 6, 7, V - 1, V // 2} | set(range(100, V, max(256, V // 40 // 8 * 8 + 8))))
    status = dev([0] * len(places))
    for i, p in enumerate(places):
        x[i % T, p] = float("nan")
        ft.ft_token_logprobs(ft.make_logprob_args(logits=at(x), tokens=at(tok), logprob=at(logprob), top_ids=at(ids),
                                                  top_logprobs=at(lps), status=at(status) + 4 * i, row_stride=x.stride(0),
                                                  dtype=ft.FT_DTYPE_BF16, T=T, V=V, top_n=top), stream())
        x[i % T, p] = 0
    torch.cuda.synchronize()
    assert status.tolist() == [ft.FT_ST_NAN] * len(places)


def test_plan_columns_past_the_table_take_no_page(ft):
    """A request longer than its row of the table takes pages for the columns there are; the others keep theirs."""
    P = 16
    table = np.array([[0, 1, 2], [-1, -1, -1]], dtype=np.int32)
    r = run_plan(ft, [40, 0], [20, 5], None, [3, 4], table, P, 25)
    assert r["status"][0] == ft.FT_ST_NO_ROOM and r["left"][0] == 1
    assert r["table"].tolist() == [[0, 1, 2], [4, -1, -1]]
    assert r["slots"].tolist() == [2 * 16 + 8 + i for i in range(8)] + [-1] * 12 + [4 * 16 + i for i in range(5)]
    # the overrun begins a page of the table, then two past it; a context that is itself past the table
    table = np.array([[7, -1], [8, 9], [-1, -1]], dtype=np.int32)
    r = run_plan(ft, [10, 70, 3], [50, 30, 14], None, [1, 2, 3, 4], np.concatenate([table[:2], [[5, -1]]]).astype(np.int32),
                 P, 100)
    assert r["status"][0] == ft.FT_ST_NO_ROOM and r["left"][0] == 2
    assert r["table"].tolist() == [[7, 4], [8, 9], [5, 3]]
    assert r["slots"].tolist() == [7 * 16 + 10 + i for i in range(6)] + [4 * 16 + i for i in range(16)] + [-1] * 28 + \
        [-1] * 30 + [5 * 16 + 3 + i for i in range(13)] + [3 * 16] + [-1] * 6


def test_attention_f16_long_tail_beside_one_large_score(ft):
    """One key far above all others whose value is 0: the output is the others' 2^-25.5 each.  As many requests and
    heads as a GPU has SMs, so that a CTA goes through thousands of keys beside the large one.

    Probabilities are held in f16 as 2^11 of their share of the row's largest, so those below 2^-25 of it have a
    fixed spacing of 2^-35: 2^-36 |v| a key, over the softmax sum."""
    B, n_keys = 40, 16385
    a = Attn(ft, [n_keys - 1] * B, [1] * B, 4, 4, 64, "f16", 64, mask="chain", seed=30, scale=1.0)
    a.q.zero_()
    a.q[:, :, 3] = 4.0
    for page, row in a.rows:
        k, v = torch.zeros((n_keys, 4, 64), device="cuda").half(), 1 + torch.rand((n_keys, 4, 64), device="cuda").half()
        k[900, :, 3] = 25.5 * math.log(2) / 4
        v[900] = 0
        a.k[page, row], a.v[page, row] = k, v
    a.run()
    out, lse, mag, top = gpu_reference(a)
    u = U["f16"]
    tol = u * mag + u * np.abs(out) + 2.0 ** -16 * mag + 2.0 ** -36 * 2 * n_keys
    got = a.out.double().cpu().numpy()
    assert out.min() > 2e-4
    assert (np.abs(got - out) <= tol).all(), np.max(np.abs(got - out) / tol)
    assert (np.abs(a.lse.double().cpu().numpy() - lse) <= 2.0 ** -16 * top).all()


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,dtype", [
    ([20000], [1], 8, 1, 128, "bf16"),            # parts of one and two key tiles, joined by the second kernel
    ([9000, 3000], [3, 40], 8, 2, 64, "f16"),
    ([300] * 200, [1] * 200, 8, 2, 128, "bf16"),  # two key tiles of one stream, one of the other
])
def test_attention_equal_scores_far_from_zero(ft, ctx, new, Hq, Hkv, D, dtype):
    """All scores 2^26 (q.k 2^22 in f16, times 16): the output is the mean of what a row sees, however its keys are
    split.  A sum held as one fp32 logarithm would round to a multiple of 8 there."""
    a = Attn(ft, ctx, new, Hq, Hkv, D, dtype, 16, mask="chain", seed=31, scale=16.0)
    a.q.zero_()
    a.q[:, :, 1] = 1024.0
    for rows in a.rows:
        k = torch.zeros((len(rows[0]), Hkv, D), device="cuda", dtype=a.k.dtype)
        k[:, :, 1] = 4096.0
        a.k[rows] = k
        tile = (torch.arange(len(rows[0]), device="cuda") // 128)[:, None, None]
        a.v[rows] = a.v[rows].abs() * (1 + tile % 3)
    a.run()
    out, lse, mag, top = gpu_reference(a)
    got, u = a.out.double().cpu().numpy(), U[dtype]
    bad = np.abs(got - out) / (u * mag + u * np.abs(out) + 2.0 ** -16 * mag)
    assert bad.max() <= 1, bad.max()
    assert (np.abs(a.lse.double().cpu().numpy() - lse) <= 2.0 ** -16 * top).all()


def test_attention_of_a_request_does_not_depend_on_its_neighbours_numbers(ft):
    """The next request's queries lie in the same tile of rows: whatever they are, this request's bits stay."""
    n = 24
    a = Attn(ft, [500, 30] * n, [1, 3] * n, 8, 1, 64, "bf16", 16, mask="chain", seed=32)
    a.run()
    out, lse = a.out.clone(), a.lse.clone()
    mine = torch.arange(a.T, device="cuda") % 4 == 0
    q = a.q.clone()
    for value in (2.0e6, float("inf"), float("nan")):
        a.q.copy_(torch.where(mine[:, None, None], q, q * value))
        a.run()
        assert torch.equal(a.out[mine], out[mine]) and torch.equal(a.lse[mine], lse[mine]), value


@pytest.mark.parametrize("scale", [0.0, 1e-36])
def test_attention_tiny_scales_of_large_products(ft, scale):
    """Products of 1e33 times a scale of 0 or 1e-36 are scores near 0: every seen key counts alike."""
    a = Attn(ft, [700, 33], [5, 20], 8, 2, 128, "bf16", 16, mask="tree", seed=33, scale=scale)
    a.q.mul_(1e16)
    a.k.mul_(1e16)
    a.run().check()


def far_apart(got, out, tol):
    return np.abs(got - out) / tol


LONG = [([33000, 128, 700], [17, 1, 5], 16, 2, 128, "bf16", 16, "token"),
        ([30003], [3], 10, 2, 64, "f16", 64, "head"),
        ([16000, 9000], [40, 1], 32, 4, 128, "f16", 128, "token"),
        ([8000] * 6, [1, 33, 1, 64, 2, 1], 8, 1, 64, "bf16", 32, "head")]


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,dtype,P,layout", LONG)
def test_attention_every_value_tile_in_its_place(ft, ctx, new, Hq, Hkv, D, dtype, P, layout):
    """A tile of 128 keys has values in a column of its own (tiles D apart share one), so that an output is the weight
    of one or a few tiles and a tile left out or exchanged shows; the rows' values rise by half within a tile.

    Tolerance: u = half spacing; every probability and the output are rounded once, u (sum p|v| + |o|), plus 2^-16
    for scores and exponentials, plus in f16 2^-36 |v| a key over the softmax sum, and 2^-25 for an output below the
    type's normal numbers."""
    a = Attn(ft, ctx, new, Hq, Hkv, D, dtype, P, layout, mask="tree", seed=34)
    values = []
    for rows in a.rows:
        key = torch.arange(len(rows[0]), device="cuda")
        v = torch.zeros((len(key), Hkv, D), device="cuda", dtype=a.v.dtype)
        v[key, :, (key // 128) % D] = (1 + (key % 128) / 256).to(a.v.dtype)[:, None]
        a.v[rows] = v
        values.append(v)
    a.run()
    out, lse, mag, top = gpu_reference(a)
    got, u = a.out.double().cpu().numpy(), U[dtype]
    tol = u * mag + u * np.abs(out) + 2.0 ** -16 * mag + 1e-30
    if dtype == "f16":
        keys = np.repeat([c + n for c, n in zip(ctx, new)], new)
        total = np.exp(lse - top_scores(a))  # the softmax sum, its largest term 1
        tol = tol + (2.0 ** -36 * 1.5 * keys[:, None] / total)[:, :, None] + 2.0 ** -25
    bad = far_apart(got, out, tol)
    assert bad.max() <= 1, (bad.max(), np.unravel_index(bad.argmax(), bad.shape))
    assert (np.abs(a.lse.double().cpu().numpy() - lse) <= 2.0 ** -16 * top).all()
    # the same check refuses a reference with one tile of values lost, or those of another
    b = int(np.argmax(ctx))
    t0, rows = a.start[b], a.rows[b]
    tiles = (ctx[b] + new[b]) // 128
    for tile in (0, 1, tiles // 2, tiles - 1):
        for other in (None, tile - 1 if tile else 1):
            wrong = values[b].clone()
            wrong[tile * 128:tile * 128 + 128] = 0 if other is None else values[b][other * 128:other * 128 + 128]
            a.v[rows] = wrong
            moved = gpu_reference(a)[0]
            assert far_apart(got, moved, tol)[t0:t0 + new[b]].max(axis=(1, 2)).min() > 1, (tile, other)
    a.v[rows] = values[b]


def top_scores(a):
    """The largest seen score of every row and head."""
    out = np.zeros((a.T, a.Hq))
    for b, (c, n) in enumerate(zip(a.ctx, a.new)):
        k = a.k[a.rows[b]].double()
        hidden = torch.zeros((n, c + n), dtype=torch.bool, device="cuda")
        hidden[:, c:] = torch.from_numpy(~a.seen[b]).cuda()
        t = slice(a.start[b], a.start[b] + n)
        for h in range(a.Hq):
            s = a.q[t, h].double() @ k[:, h * a.Hkv // a.Hq].T * a.scale
            out[t, h] = s.masked_fill(hidden, -math.inf).amax(1).cpu().numpy()
    return out


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,dtype,P,layout", LONG)
def test_attention_long_contexts_error_is_that_of_its_roundings(ft, ctx, new, Hq, Hkv, D, dtype, P, layout):
    """Random values: the mean square error of a request's rows of one key head is that of independent roundings.

    A rounding is at most u |x| and uniform, a mean square of u^2 x^2 / 3 or less: with e^2 = u^2 (sum p^2 v^2 + o^2) / 3
    the mean of (err / e)^2 stays below 1; 1.15^2 leaves room for the spread of 1000 outputs and the fp32 steps.  A
    tile of values lost or exchanged among 258 moves an output by 6 % of its size, 19 e and more."""
    a = Attn(ft, ctx, new, Hq, Hkv, D, dtype, P, layout, mask="tree", seed=35).run()
    out = gpu_reference(a)[0]
    got, u, G = a.out.double().cpu().numpy(), U[dtype], Hq // Hkv
    for b, (c, n) in enumerate(zip(ctx, new)):
        if c < 1000:
            continue
        k, v = (x[a.rows[b]].double() for x in (a.k, a.v))
        hidden = torch.zeros((n, c + n), dtype=torch.bool, device="cuda")
        hidden[:, c:] = torch.from_numpy(~a.seen[b]).cuda()
        t = slice(a.start[b], a.start[b] + n)
        for g in range(Hkv):
            ratio = []
            for h in range(g * G, g * G + G):
                s = (a.q[t, h].double() @ k[:, g].T * a.scale).masked_fill(hidden, -math.inf)
                pv = torch.softmax(s, 1) ** 2 @ v[:, g] ** 2
                e2 = u * u * (pv.cpu().numpy() + out[t, h] ** 2) / 3
                ratio.append((got[t, h] - out[t, h]) ** 2 / e2)
            assert np.mean(ratio) <= 1.15 ** 2, (b, g, np.mean(ratio))


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,dtype,P", [
    ([0], [1500], 8, 2, 128, "bf16", 16), ([700], [1031], 4, 1, 64, "f16", 64), ([0, 129, 3], [513, 700, 2], 8, 8, 128, "f16", 128)])
def test_attention_of_prompts(ft, ctx, new, Hq, Hkv, D, dtype, P):
    """Without a mask: new tokens one after another, over several blocks of rows."""
    a = Attn(ft, ctx, new, Hq, Hkv, D, dtype, P, mask="chain", seed=36).run()
    a.reference = lambda: gpu_reference(a)
    a.check()
    assert a.status.item() == 0


@pytest.mark.parametrize("base", [0, 2 ** 8, 2 ** 12, 2 ** 16, 2 ** 19, -2 ** 17])
@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,dtype", [
    ([9000, 3000, 260], [3, 40, 1], 8, 2, 64, "f16"), ([20000], [1], 8, 1, 128, "f16"), ([700] * 160, [2] * 160, 8, 1, 128, "bf16")])
def test_attention_small_differences_of_large_scores(ft, ctx, new, Hq, Hkv, D, dtype, base):
    """Scores base + whole numbers of -16 .. 16, exact in fp32: what the base is changes nothing.

    Keys are weighed against one another across rescalings, streams and parts; the tolerance is that of any scores."""
    a = Attn(ft, ctx, new, Hq, Hkv, D, dtype, 16, mask="tree", seed=37, scale=1.0)
    g = torch.Generator(device="cuda").manual_seed(38)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(a.q.dtype)
    half = 2 ** (max(1, abs(base)).bit_length() // 2)
    a.q.zero_()
    a.q[:, :, 0], a.q[:, :, 1:5] = base / half, whole(a.T, Hq, 4)
    for rows in a.rows:
        k = torch.zeros((len(rows[0]), Hkv, D), device="cuda", dtype=a.k.dtype)
        k[:, :, 0], k[:, :, 1:5] = half, whole(len(rows[0]), Hkv, 4)
        a.k[rows] = k
    a.run()
    out, lse, mag, top = gpu_reference(a)
    got, u = a.out.double().cpu().numpy(), U[dtype]
    tol = u * mag + u * np.abs(out) + 2.0 ** -16 * mag
    if dtype == "f16":  # values are below 6; the softmax sum is 1 and more
        tol = tol + 2.0 ** -25 + 2.0 ** -36 * 6 * (max(ctx) + max(new))
    bad = np.abs(got - out) / tol
    assert bad.max() <= 1, (bad.max(), np.unravel_index(bad.argmax(), bad.shape))
    assert (np.abs(a.lse.double().cpu().numpy() - lse) <= 2.0 ** -16 * top).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [9, 5003, 40000])
def test_logprobs_stay_at_or_below_zero_and_entropies_at_or_above(ft, dtype, V):
    """One logit far above all others, of every size: a probability is at most 1, whatever the sums' rounding."""
    T = 500
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((T, V), generator=g, device="cuda")
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda").cpu().numpy()
    size = torch.linspace(-900, 900, T, device="cuda") + torch.rand(T, generator=g, device="cuda")
    x = x - 60 + size[:, None]
    x[torch.arange(T), torch.from_numpy(tokens).cuda()] = size
    x = x.to(DT[dtype])
    got = run_logprob(ft, x, tokens, 3)
    lp, ent, ids, lps = logprob_reference(x, tokens, 3)
    for key, want in (("logprob", lp), ("entropy", ent), ("lps", lps)):
        close(got[key], want)
    assert got["logprob"].max() <= 0 and got["lps"].max() <= 0 and got["entropy"].min() >= 0
