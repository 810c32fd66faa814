"""Attention over the 8-bit paged cache against a plain 64-bit implementation.

The reference takes the cache's numbers, code * 2^(e-127), as they are.
Tolerances, from the arithmetic (u = 2^-8 for bf16, 2^-11 for f16, the half
spacing of the type; sums in fp32): every probability is rounded to the type (u
each) and the output once: |err| <= u sum p |v| + u |o|, plus 2^-16 sum p |v| for
the scores' fp32 sums and exponentials; f16 probabilities have a least spacing:
sum over keys of 2^-25 |v|.  lse: 2^-16 max(1, largest |score|).  The cache's
numbers are exact in bf16, and in f16 but for those below 2^-14, rounded to
multiples of 2^-24 (the caches here hold numbers of scales 2^-8 .. 2^6, whose
least code is 2^-17).
"""
import math

import numpy as np
import pytest

import kv8_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module")
def ft():
    from expert_cache_host_gb300 import build as ftbuild
    ftbuild.build()
    import expert_cache_host_gb300 as lib
    lib.load()
    return lib


def at(t):
    return 0 if t is None else t.data_ptr()


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def stream():
    return torch.cuda.current_stream().cuda_stream


class Attn:
    """A batch of requests over a paged cache whose unused rows hold NaN codes and whose unused blocks have bytes of 255."""

    def __init__(self, ft, ctx, new, Hq, Hkv, D, dtype, P, block, layout="token", mask="tree", seed=0, scale=None, spare=3,
                 bias=0.0, max_new=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ft, self.ctx, self.new, self.D, self.P, self.dtype, self.block = ft, list(ctx), list(new), D, P, dtype, block
        self.Hq, self.Hkv = Hq, Hkv
        held = [-(-(c + n) // P) for c, n in zip(ctx, new)]
        pages = sum(held) + spare
        shape = (pages, P, Hkv, D) if layout == "token" else (pages, Hkv, P, D)
        self.codes = [torch.full(shape, 0x7F, device="cuda", dtype=torch.uint8) for _ in range(2)]
        if layout == "head":
            self.codes = [c.transpose(1, 2) for c in self.codes]
        self.bytes = [torch.full((pages, P // block, Hkv), 255, device="cuda", dtype=torch.uint8) for _ in range(2)]
        ids = rng.permutation(pages)
        self.width = max(held + [1]) + 2
        table = np.full((len(ctx), self.width), -1, dtype=np.int32)
        self.rows = []  # each request's (page, row) of every key
        for b, h in enumerate(held):
            table[b, :h], ids = ids[:h], ids[h:]
            idx = np.arange(ctx[b] + new[b])
            page, row = torch.from_numpy(table[b, idx // P].astype(np.int64)).cuda(), torch.from_numpy(idx % P).cuda()
            self.rows.append((page, row))
            for kv in range(2):
                x = torch.randn((len(idx), Hkv, D), generator=g, device="cuda") * 100 + bias * 100
                self.codes[kv][page, row] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                e = torch.randint(-2, 3, (pages, P // block, Hkv), generator=g, device="cuda") + 127 - 7  # about 100 / 2^7
                self.bytes[kv][page, row // block] = e[page, row // block].to(torch.uint8)
        self.table = dev(table)
        self.T = sum(new)
        self.q = torch.randn((max(1, self.T), Hq, D), generator=g, device="cuda").to(DT[dtype])
        self.start = np.concatenate([[0], np.cumsum(new)]).tolist()
        self.seen = []  # [n, n] of each request
        words = (max(list(new) + [1]) + 31) // 32
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
            self.seen.append(s)
            for i in range(n):
                for j in np.nonzero(s[i])[0]:
                    m[self.start[b] + i, j >> 5] |= np.uint32(1 << (j & 31))
        self.mask = None if mask == "chain" else torch.from_numpy(m.view(np.int32)).cuda()
        self.words = 0 if mask == "chain" else words
        self.scale = 0.5 * D ** -0.5 if scale is None else scale
        self.out = torch.full((max(1, self.T), Hq, D), 5.0, device="cuda", dtype=DT[dtype])
        self.lse = torch.full((max(1, self.T), Hq), 5.0, device="cuda")
        self.status = dev([0])
        self.d_start, self.d_ctx = dev(self.start), dev(ctx if len(ctx) else [0])
        self.args = ft.make_kv8_attn_args(
            q=at(self.q), out=at(self.out), lse=at(self.lse), q_start=at(self.d_start), ctx_len=at(self.d_ctx),
            block_table=at(self.table), mask=at(self.mask), status=at(self.status), q_stride=Hq * D, out_stride=Hq * D,
            dtype=ft.FT_DTYPE_BF16 if dtype == "bf16" else ft.FT_DTYPE_F16, max_tokens=self.T,
            max_new=max(new) if max_new is None else max_new, num_reqs=len(ctx), q_heads=Hq, table_width=self.width,
            mask_words=self.words, scale=self.scale, cache=self.cache())
        self.ws = torch.zeros(ft.ft_kv8_attention_workspace(self.args), dtype=torch.uint8, device="cuda")
        self.args.workspace, self.args.workspace_bytes = at(self.ws), self.ws.numel()

    def cache(self):
        k, v = self.codes
        return self.ft.make_kv8_cache(
            k=at(k), v=at(v), k_scale=at(self.bytes[0]), v_scale=at(self.bytes[1]), num_pages=k.shape[0], page_size=self.P,
            block_size=self.block, kv_heads=self.Hkv, head_dim=self.D, k_page_stride=k.stride(0),
            k_token_stride=k.stride(1), k_head_stride=k.stride(2), v_page_stride=v.stride(0), v_token_stride=v.stride(1),
            v_head_stride=v.stride(2))

    def values(self, kv, b):
        """Request b's keys or values in 64 bits, [key, head, D]."""
        page, row = self.rows[b]
        e = self.bytes[kv][page, row // self.block].double()
        table = torch.from_numpy(ref.VALUE).cuda()
        return table[self.codes[kv][page, row].long()] * torch.exp2(e - 127)[:, :, None]

    def run(self, st=None):
        self.ft.ft_kv8_attention(self.args, stream() if st is None else st)
        torch.cuda.synchronize()
        return self

    def reference(self):
        """(out, lse, sum p|v|, largest |score|) in 64 bits; rows that see nothing: 0, -inf."""
        T, Hq, D, G = self.T, self.Hq, self.D, self.Hq // self.Hkv
        out, mag = (torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda") for _ in range(2))
        lse, top = (torch.full((T, Hq), v, dtype=torch.float64, device="cuda") for v in (-math.inf, 1.0))
        for b, (c, n) in enumerate(zip(self.ctx, self.new)):
            if n == 0 or c + n == 0:
                continue
            k, v = self.values(0, b), self.values(1, b)
            hidden = torch.zeros((n, c + n), dtype=torch.bool, device="cuda")
            hidden[:, c:] = torch.from_numpy(~self.seen[b]).cuda()
            t = slice(self.start[b], self.start[b] + n)
            for h in range(Hq):
                s = (self.q[t, h].double() @ k[:, h // G].T * self.scale).masked_fill(hidden, -math.inf)
                top[t, h] = s.masked_fill(hidden, 0).abs().amax(1).clamp(min=1)
                m = s.amax(1, keepdim=True).clamp(min=-1e300)
                p = torch.exp(s - m)
                total = p.sum(1, keepdim=True)
                lse[t, h] = (m + torch.log(total))[:, 0]
                p = torch.where(total > 0, p / total, 0.0)
                out[t, h], mag[t, h] = p @ v[:, h // G], p @ v[:, h // G].abs()
        return tuple(x.cpu().numpy() for x in (out, lse, mag, top))

    def check(self, where=""):
        out, lse, mag, top = self.reference()
        got = self.out.double().cpu().numpy()[:self.T]
        u = U[self.dtype]
        tol = u * mag + u * np.abs(out) + 2.0 ** -16 * mag + 1e-30
        if self.dtype == "f16":
            tol = tol + 2.0 ** -25 * (max(c + n for c, n in zip(self.ctx, self.new)) * 16.0)
        assert np.isfinite(got).all(), where
        bad = np.abs(got - out) / tol
        assert bad.max(initial=0) <= 1, (where, bad.max(), np.unravel_index(bad.argmax(), bad.shape))
        got_lse = self.lse.double().cpu().numpy()[:self.T]
        empty = np.isinf(lse)
        assert np.array_equal(np.isinf(got_lse), empty), where
        err = np.abs(got_lse[~empty] - lse[~empty]) / (2.0 ** -16 * top[~empty])
        assert err.max(initial=0) <= 1, (where, err.max())


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,dtype,P,block,layout,mask", [
    ([0], [1], 1, 1, 64, "bf16", 16, 16, "token", "chain"), ([1], [1], 8, 1, 128, "bf16", 16, 16, "token", "chain"),
    ([127], [1], 32, 4, 128, "bf16", 16, 16, "token", "chain"), ([128], [1], 32, 4, 128, "f16", 32, 16, "head", "chain"),
    ([1000], [1], 16, 2, 64, "f16", 64, 64, "token", "chain"), ([3000], [1], 32, 4, 128, "bf16", 16, 16, "token", "tree"),
    ([5, 0, 260, 77], [1, 1, 1, 1], 8, 2, 128, "bf16", 16, 16, "head", "chain"),
    ([5, 0, 1260, 77], [2, 2, 1, 0], 16, 2, 64, "bf16", 128, 32, "head", "tree"),
    ([100, 0, 300, 7], [17, 5, 0, 33], 8, 2, 128, "bf16", 32, 32, "token", "tree"),
    ([100, 0, 300, 7], [17, 5, 0, 33], 10, 2, 64, "f16", 32, 16, "head", "tree"),
    ([250, 511], [64, 64], 16, 2, 128, "bf16", 128, 128, "token", "tree"),
    ([40], [100], 8, 1, 128, "bf16", 16, 16, "token", "random"),
    ([0, 130], [40, 70], 3, 3, 64, "bf16", 256, 64, "head", "random"),
    ([900, 10], [31, 2], 7, 1, 128, "f16", 16, 16, "token", "chain"), ([0], [300], 4, 2, 128, "bf16", 64, 16, "token", "chain"),
    ([2000], [40], 128, 1, 64, "bf16", 512, 128, "token", "tree"), ([129, 1], [200, 1], 5, 5, 64, "f16", 16, 16, "head", "chain"),
    ([4000, 3, 1200, 0, 640], [2, 3, 9, 1, 16], 48, 8, 128, "bf16", 32, 16, "token", "tree"),
    ([700, 90, 3, 64], [1, 2, 1, 2], 8, 8, 128, "f16", 64, 32, "token", "chain"),
    ([700, 90, 3, 64], [3, 2, 1, 4], 4, 2, 64, "bf16", 64, 32, "token", "random")])
def test_attention(ft, ctx, new, Hq, Hkv, D, dtype, P, block, layout, mask):
    for max_new in (max(new), 0):  # with and without the hint
        a = Attn(ft, ctx, new, Hq, Hkv, D, dtype, P, block, layout, mask, seed=len(ctx) + D + P, max_new=max_new).run()
        a.check()
        assert a.status.item() == 0


def test_rows_that_see_nothing(ft):
    """An empty context and an empty mask: zeros and -inf, beside rows of other requests that see keys."""
    for new in ([3, 3, 20], [1, 1, 1]):
        a = Attn(ft, [0, 50, 0], new, 8, 2, 128, "bf16", 16, 16, mask="none", seed=3).run()
        a.check()
        one, two = new[0], new[0] + new[1]
        assert bool((a.out[:one] == 0).all()) and bool((a.out[two:] == 0).all()) and bool((a.out[one:two] != 0).any())


@pytest.mark.parametrize("new", [[9, 1, 40], [1, 1, 1]])
def test_without_lse_and_twice(ft, new):
    """The workspace is ready again after every call; results repeat bit by bit."""
    a = Attn(ft, [3000, 20, 900], new, 32, 4, 128, "bf16", 16, 16, seed=4).run()
    first, lse = a.out.clone(), a.lse.clone()
    for _ in range(3):
        a.out.fill_(1)
        a.ws.random_()
        a.run()
        assert torch.equal(a.out, first) and torch.equal(a.lse, lse)
    a.args.lse = None
    a.out.fill_(1)
    a.lse.fill_(9)
    a.run()
    assert torch.equal(a.out, first) and bool((a.lse == 9).all())


@pytest.mark.parametrize("scale,bias", [(3.0, 0.0), (-0.5, 0.0), (0.0, 0.0), (1.0, 1.0)])
@pytest.mark.parametrize("new", [[5, 12], [1, 1]])
def test_scales(ft, scale, bias, new):
    """Sharp, reversed and flat softmax, and scores that are all large."""
    Attn(ft, [700, 90], new, 16, 4, 64, "bf16", 16, 16, seed=5, scale=scale, bias=bias).run().check()


@pytest.mark.parametrize("new", [3, 1])
def test_growing_scores(ft, new):
    """Each key's score above the one before it: the running maximum moves at every step."""
    a = Attn(ft, [600], [new], 8, 1, 128, "bf16", 16, 16, seed=6, scale=1.0)
    a.codes[0][a.rows[0]] = 0
    a.q.zero_()
    a.q[:, :, :3] = 1
    n = 600 + new
    rise = torch.arange(n, device="cuda")
    c = torch.zeros((n, 1, 128), device="cuda")
    c[:, :, 0] = (rise // 64 * 8).clamp(max=448)[:, None]
    c[:, :, 1] = (rise % 64 // 8)[:, None]
    c[:, :, 2] = (rise % 8)[:, None] / 8.0
    a.codes[0][a.rows[0]] = c.to(torch.float8_e4m3fn).view(torch.uint8)
    a.bytes[0][a.bytes[0] != 255] = 127
    a.run().check()


@pytest.mark.parametrize("dtype,byte", [("bf16", 0), ("bf16", 20), ("bf16", 100), ("bf16", 140), ("bf16", 160), ("f16", 110),
                                        ("f16", 130), ("f16", 134)])
@pytest.mark.parametrize("new", [[6, 3], [1, 1]])
def test_values_of_any_scale(ft, dtype, byte, new):
    """Scale bytes far from 1, of keys with a softmax scale that makes up for it, and of values; blocks beside each other
    differ by up to four binades."""
    a = Attn(ft, [300, 70], new, 8, 2, 128, dtype, 32, 16, seed=byte)
    for kv in range(2):
        keep = a.bytes[kv] != 255
        a.bytes[kv][keep] = (byte + (a.bytes[kv][keep].int() - 118) % 5).to(torch.uint8)
    a.scale = a.args.scale = float(np.float32(min(1e30, 0.01 * 2.0 ** (127 - byte))))
    out, lse, mag, top = a.run().reference()
    got = a.out.double().cpu().numpy()
    most = max(float(a.values(1, b).abs().max()) for b in range(2))
    if dtype == "f16" and most > 65504:
        # bytes up to 138 and codes up to 448: 448 * 2^11 is past f16 and may count as infinite
        assert a.status.item() == 0
        return
    # Below its least normal number the type's spacing is fixed: half of it on every value and on the output; f16
    # probabilities are off by 2^-36 of a row's largest.
    floor = 2.0 ** -25 if dtype == "f16" else 2.0 ** -134
    tol = U[dtype] * (mag + np.abs(out)) + 2.0 ** -16 * mag + 2 * floor + (2.0 ** -36 * 310 * most if dtype == "f16" else 0)
    # Keys rounded to the type move a score by half a spacing times sum |q| (128 of size 4 at most), and a probability
    # by a factor of e^(2 shift), below 1 + 2.3 shift up to shift = 0.1; at byte 0 keys are below the type's spacing.
    shift = floor * 128 * 4 * a.scale
    if byte:
        assert shift < 0.1
        assert (np.abs(got - out) <= tol + 2.3 * shift * mag).all(), np.max(np.abs(got - out) / tol)
    assert np.isfinite(got).all()


@pytest.mark.parametrize("code,byte", [(0x7F, None), (0xFF, None), (0x7E, None), (0xFE, 254), (None, 255)])
def test_unseen_keys_take_no_part(ft, code, byte):
    """Unusual codes and scale bytes in new keys and values that a row does not see, and past the request's end; the
    rows that see one are left out of the comparison.  (The byte's block holds new tokens only, all unseen.)"""
    a = Attn(ft, [128, 32], [12, 40], 8, 2, 128, "bf16", 16, 16, mask="tree", seed=7)
    first = {0: 8, 1: 16}  # these new tokens on are seen by nobody before them
    for b, j in first.items():
        a.seen[b][:j, j:] = False
    a.run()
    clean = a.out.clone()
    a.check()
    for b, j in first.items():
        lo = a.ctx[b] + (j if byte is None else 16 if b else 12)
        hi = lo + (1 if byte is None else 16)
        sel = range(lo, min(hi, a.ctx[b] + a.new[b]))
        for key in sel:
            page, row = a.rows[b][0][key], a.rows[b][1][key]
            for kv in range(2):
                if code is not None:
                    a.codes[kv][page, row] = code
                if byte is not None:
                    a.bytes[kv][page, row // 16] = byte
    a.run()
    for b, j in first.items():
        for i in range(j):
            assert torch.equal(a.out[a.start[b] + i], clean[a.start[b] + i]), (b, i)


@pytest.mark.parametrize("new", [6, 2])
def test_seen_nan_reaches_the_output(ft, new):
    a = Attn(ft, [130], [new], 8, 2, 128, "bf16", 16, 16, mask="chain", seed=8)
    page, row = a.rows[0][0][131], a.rows[0][1][131]  # new token 1
    a.codes[1][page, row, 0, 5] = 0x7F
    a.codes[1][page, row, 1, 7] = 0xFF
    a.run()
    got = a.out.float().cpu().numpy()
    assert np.isfinite(got[:1]).all()
    assert np.isnan(got[1:, :4, 5]).all() and np.isnan(got[1:, 4:, 7]).all()
    got[1:, :4, 5] = got[1:, 4:, 7] = 0
    assert np.isfinite(got).all()
    # a context value is seen by every row, and a key's NaN is every number's
    a.codes[1][page, row] = 0
    a.codes[1][a.rows[0][0][40], a.rows[0][1][40], 0, 9] = 0x7F
    a.codes[0][a.rows[0][0][41], a.rows[0][1][41], 1, 9] = 0x7F
    a.run()
    got = a.out.float().cpu().numpy()
    assert np.isnan(got[:, :4, 9]).all() and np.isnan(got[:, 4:]).all()
    got[:, :4, 9] = got[:, 4:] = 0
    assert np.isfinite(got).all()


def test_strided_rows_and_shared_buffer(ft):
    """Keys and values interleaved in one buffer, q and out as slices of wider rows."""
    for new in ([3, 9], [1, 1]):
        a = Attn(ft, [200, 5], new, 8, 2, 128, "bf16", 16, 16, seed=9)
        both = torch.full((a.codes[0].shape[0], 16, 2, 2, 128), 0x7F, device="cuda", dtype=torch.uint8)
        both[:, :, 0], both[:, :, 1] = a.codes
        a.codes = [both[:, :, 0], both[:, :, 1]]
        wide_q = torch.zeros((a.T, 8 * 128 + 24), device="cuda", dtype=a.q.dtype)
        wide_q[:, 8:8 + 1024] = a.q.view(a.T, -1)
        wide_o = torch.full((a.T, 8 * 128 + 40), 2.0, device="cuda", dtype=a.q.dtype)
        a.args.cache = a.cache()
        a.args.q, a.args.q_stride = at(wide_q) + 16, wide_q.stride(0)
        a.args.out, a.args.out_stride = at(wide_o) + 32, wide_o.stride(0)
        a.run()
        a.out = wide_o[:, 16:16 + 1024].unflatten(1, (8, 128))
        a.check()
        assert bool((wide_o[:, :16] == 2).all()) and bool((wide_o[:, 1040:] == 2).all())


@pytest.mark.parametrize("new", [4, 1])
def test_bad_pages_are_reported_and_absent(ft, new):
    a = Attn(ft, [100, 40], [new, new], 8, 2, 128, "bf16", 16, 16, mask="chain", seed=10)
    a.table[0, 2] = a.codes[0].shape[0]  # keys 32..47 of request 0
    a.table[1, 1] = -1                   # keys 16..31 of request 1
    a.run()
    assert a.status.item() == ft.FT_ST_BAD_SLOT
    for b, lo in ((0, 32), (1, 16)):  # the same as requests without those keys
        keep = [i for i in range(a.ctx[b] + a.new[b]) if not lo <= i < lo + 16]
        a.rows[b] = tuple(x[keep] for x in a.rows[b])
        a.ctx[b] -= 16
    a.check()


def test_columns_past_the_table_are_absent(ft):
    for new in (20, 1):
        a = Attn(ft, [200], [new], 8, 2, 64, "f16", 32, 32, mask="chain", seed=10)
        a.args.table_width = 3
        a.run()
        assert a.status.item() == ft.FT_ST_BAD_SLOT
        a.rows[0] = tuple(x[:96] for x in a.rows[0])
        a.ctx[0], a.seen[0] = 96, np.zeros((new, 0), dtype=bool)
        k, v = a.values(0, 0), a.values(1, 0)
        for h in range(8):
            p = torch.softmax(a.q[:, h].double() @ k[:, h // 4].T * a.scale, 1)
            err = (a.out[:, h].double() - p @ v[:, h // 4]).abs()
            assert bool((err <= 2.0 ** -9 * (p @ v[:, h // 4].abs())).all())


@pytest.mark.parametrize("ctx", [(1 << 31) - 1, (1 << 31) - 256])
@pytest.mark.parametrize("new", [[4, 3, 5], [1, 1, 1]])
def test_request_of_too_many_keys_is_reported_and_left(ft, ctx, new):
    a = Attn(ft, [100, 20, 300], new, 8, 2, 128, "bf16", 16, 16, mask="chain", seed=16)
    a.d_ctx[1] = ctx
    a.run()
    one, two = new[0], new[0] + new[1]
    assert a.status.item() == ft.FT_ST_BAD_SLOT
    assert bool((a.out[one:two] == 5).all()) and bool((a.lse[one:two] == 5).all())
    got = a.out.clone()
    a.d_ctx[1] = 20
    a.status.zero_()
    a.run()
    a.check()
    for rows in (slice(0, one), slice(two, None)):  # split elsewhere, so close and not the same
        assert bool(torch.allclose(got[rows].float(), a.out[rows].float(), atol=2.0 ** -6, rtol=2.0 ** -6))


@pytest.mark.parametrize("most", [2, 1])
def test_request_of_more_than_max_new_is_reported_and_left(ft, most):
    a = Attn(ft, [100, 20, 30], [1, most + 1, most], 8, 2, 128, "bf16", 16, 16, mask="chain", seed=16, max_new=most)
    a.run()
    assert a.status.item() == ft.FT_ST_NO_ROOM
    assert bool((a.out[1:2 + most] == 5).all()) and bool((a.lse[1:2 + most] == 5).all())
    out, lse, mag, top = a.reference()
    got = a.out.double().cpu().numpy()
    for rows in (slice(0, 1), slice(2 + most, None)):
        assert (np.abs(got[rows] - out[rows]) <= 2.0 ** -7 * (mag[rows] + np.abs(out[rows]))).all()


def test_rows_past_the_last_request_stay(ft):
    for new in ([3, 2], [1, 2]):
        a = Attn(ft, [60, 10], new, 4, 1, 64, "f16", 16, 16, seed=11)
        last = sum(new) - 1
        a.d_start[2] = last  # the second request's last token is not part of the step
        a.run()
        assert bool((a.out[last] == 5).all()) and bool((a.lse[last] == 5).all())
        assert bool((a.out[:last] != 5).any(2).any(1).all())


@pytest.mark.parametrize("new", [2, 1])
def test_offsets_past_32_bits(ft, new):
    """Pages more than 2^32 bytes apart."""
    stride = (1 << 32) + 16 * 64
    D, P, Hkv = 64, 16, 1
    buf = torch.empty(stride + 4 * P * D, dtype=torch.uint8, device="cuda")
    a = Attn(ft, [20], [new], 4, Hkv, D, "bf16", P, 16, seed=12, spare=0)
    assert a.codes[0].shape[0] == 2
    far = [torch.as_strided(buf, (2, P, Hkv, D), (stride, D, D, 1), i * P * D) for i in range(2)]
    for f, c in zip(far, a.codes):
        f.copy_(c)
    a.codes = far
    a.args.cache = a.cache()
    a.run().check()


@pytest.mark.parametrize("new", [[6, 1], [1, 1]])
def test_on_another_stream_and_in_a_graph(ft, new):
    a = Attn(ft, [700, 33], new, 32, 4, 128, "bf16", 16, 16, seed=13)
    want = a.run().out.clone()
    side = torch.cuda.Stream()
    a.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    a.run(side.cuda_stream)
    assert torch.equal(a.out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ft.ft_kv8_attention(a.args, stream())
    for _ in range(2):
        a.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, want)


@pytest.mark.parametrize("most", [3, 1])
def test_many_requests(ft, most):
    rng = np.random.default_rng(14)
    ctx = rng.integers(0, 60, 700).tolist()
    new = rng.integers(0, most + 1, 700).tolist()
    Attn(ft, ctx, new, 4, 2, 64, "bf16", 16, 16, seed=14).run().check()


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,dtype,P,block,layout", [
    # many tiles to a CTA, one and two row tiles side by side
    ([21000, 300, 9000, 33000, 5], [32, 1, 17, 5, 40], 32, 4, 128, "bf16", 16, 16, "token"),
    ([30000, 17000, 128, 4097], [3, 50, 1, 64], 40, 8, 64, "f16", 64, 32, "head"),
    ([5000] * 40 + [100] * 40, [1, 20] * 40, 16, 2, 128, "f16", 128, 128, "token"),
    ([21000, 300, 9000, 33000, 5], [1] * 5, 32, 4, 128, "bf16", 16, 16, "token"),
    ([30000, 17000, 128, 4097], [2, 1, 2, 1], 16, 2, 64, "f16", 64, 32, "head"),
    ([5000] * 40 + [100] * 40, [1] * 80, 16, 2, 128, "f16", 128, 128, "token")])
def test_long_contexts(ft, ctx, new, Hq, Hkv, D, dtype, P, block, layout):
    a = Attn(ft, ctx, new, Hq, Hkv, D, dtype, P, block, layout, seed=sum(new)).run()
    a.check()
    assert a.status.item() == 0


@pytest.mark.parametrize("new", [[20, 1, 5], [1, 1, 1]])
def test_back_to_back(ft, new):
    """Calls of several batches one after another without a pause, each with the result it has alone."""
    batch = [Attn(ft, [9000, 60, 3000], new, 32, 4, 128, "bf16", 16, 16, seed=20 + i) for i in range(3)]
    want = []
    for a in batch:
        a.run()
        want.append((a.out.clone(), a.lse.clone()))
        a.out.zero_()
    for _ in range(20):
        for a in batch:
            ft.ft_kv8_attention(a.args, stream())
    torch.cuda.synchronize()
    for a, (out, lse) in zip(batch, want):
        assert torch.equal(a.out, out) and torch.equal(a.lse, lse) and a.status.item() == 0


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,dtype,P,block", [
    # up to 16 rows a key head: 2 x 8, 1 x 16, 5 x 3, 1 x 9, 16 x 1
    ([2000, 40, 0], [2, 1, 2], 32, 4, 128, "bf16", 16, 16), ([700, 17], [1, 1], 32, 2, 128, "f16", 64, 32),
    ([1300, 3], [5, 4], 6, 2, 128, "bf16", 32, 16), ([130], [1], 9, 1, 64, "bf16", 16, 16),
    ([400, 5, 64], [16, 3, 16], 2, 2, 128, "f16", 128, 128), ([9000], [2], 64, 8, 64, "f16", 64, 64)])
@pytest.mark.parametrize("mask", ["chain", "random"])
def test_rows_up_to_sixteen(ft, ctx, new, Hq, Hkv, D, dtype, P, block, mask):
    a = Attn(ft, ctx, new, Hq, Hkv, D, dtype, P, block, mask=mask, seed=Hq + D).run()
    a.check()
    assert a.status.item() == 0


@pytest.mark.parametrize("code,byte", [(0x7F, 127), (0x7E, 254), (0xFE, 200), (0x38, 255), (0xFF, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq", [4, 16, 32])
def test_a_later_token_in_a_block_of_its_own(ft, code, byte, dtype, Hq):
    """Whatever its codes and scales, the rows before it do not see it: with 4, 16 and 32 rows a key head."""
    a = Attn(ft, [15, 47], [2, 2], Hq, 2, 128, dtype, 32, 16, mask="chain", seed=3).run()
    a.check()
    clean = a.out.clone()
    for b in range(2):
        page, row = a.rows[b][0][a.ctx[b] + 1], a.rows[b][1][a.ctx[b] + 1]
        for kv in range(2):
            a.codes[kv][page, row] = code
            a.bytes[kv][page, row // 16] = byte
    a.run()
    assert torch.equal(a.out[[0, 2]], clean[[0, 2]])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new", [[1, 1], [3, 9]])
def test_blocks_of_zeros_and_blocks_far_larger(ft, dtype, new):
    """Keys or values all zero with byte 0, and values 2^12 larger than the others' with next to no weight: the scores'
    share of both stays."""
    a = Attn(ft, [500, 70], new, 8, 2, 128, dtype, 16, 16, mask="chain", seed=21)
    for b in range(2):
        page = a.rows[b][0][:64:16]  # the request's first four blocks
        a.codes[1][page[0]], a.bytes[1][page[0]] = 0, 0
        a.codes[0][page[1]], a.bytes[0][page[1]] = 0, 0
        a.bytes[1][page[2]] += 12
        # scores near -40: keys along minus the queries' sum, which is what every row shares here
        a.q[a.start[b]:a.start[b + 1]] = a.q[a.start[b], 0]
        away = -a.q[a.start[b], 0].float()
        x = away * (40.0 / a.scale / float((away * away).sum()))
        e = int(torch.ceil(torch.log2(x.abs().max() / 448)).item())
        a.codes[0][page[2]] = (x * 2.0 ** -e).to(torch.float8_e4m3fn).view(torch.uint8)
        a.bytes[0][page[2]] = 127 + e
    a.run().check()


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,dtype,P,block", [
    ([33000] * 8, [1] * 8, 16, 8, 128, "bf16", 16, 16), ([40000] * 7 + [13], [2] * 8, 8, 8, 64, "f16", 128, 64),
    ([33000] * 6 + [17], [3] * 7, 64, 8, 128, "bf16", 64, 32)])
def test_many_tiles_to_a_cta(ft, ctx, new, Hq, Hkv, D, dtype, P, block):
    """More tiles than a window of pages holds, one and two windows on."""
    a = Attn(ft, ctx, new, Hq, Hkv, D, dtype, P, block, seed=D).run()
    a.check()
    a.table[1, 1000 // (P // 16)] = -1  # a page missing far inside
    a.status.zero_()
    clean = a.out.clone()
    a.run()
    assert a.status.item() == ft.FT_ST_BAD_SLOT
    lo = 1000 // (P // 16) * P
    keep = [i for i in range(a.ctx[1] + a.new[1]) if not lo <= i < lo + P]
    a.rows[1] = tuple(x[keep] for x in a.rows[1])
    a.ctx[1] -= P
    a.check()
    first = a.start[1]
    assert torch.equal(a.out[:first], clean[:first])
