"""The 8-bit paged cache against a plain 64-bit implementation.

Codes and scale bytes are equal: x 2^(127-e) is exact (a power of two), so the
one rounding is to the nearest code, ties to even, on both sides.  Rows read
back are code * 2^(e-127) rounded once to the 16-bit type: equal too.
"""
import numpy as np
import pytest

import kv8_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


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


def code_of(ft, dtype):
    return ft.FT_DTYPE_BF16 if dtype == "bf16" else ft.FT_DTYPE_F16


class Device:
    """A cache on the GPU beside its reference, every byte random at first."""

    def __init__(self, ft, pages, P, block, heads, D, layout="token", seed=0, shared=False):
        rng = np.random.default_rng(seed)
        self.ft, self.P, self.block, self.heads, self.D, self.pages = ft, P, block, heads, D, pages
        codes = [rng.integers(0, 256, (pages, P, heads, D)).astype(np.uint8) for _ in range(2)]
        for c in codes:
            c[(c & 127) == 127] = 3  # no NaN among what is there
        scale = [rng.integers(110, 135, (pages, P // block, heads)).astype(np.uint8) for _ in range(2)]
        self.ref = ref.Cache(codes, scale, block)
        if shared:  # keys and values beside each other in one buffer
            both = torch.zeros((pages, P, heads, 2, D), dtype=torch.uint8, device="cuda")
            self.codes = [both[..., 0, :], both[..., 1, :]]
        else:
            shape = (pages, P, heads, D) if layout == "token" else (pages, heads, P, D)
            self.codes = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
            if layout == "head":
                self.codes = [c.transpose(1, 2) for c in self.codes]
        for d, c in zip(self.codes, codes):
            d.copy_(torch.from_numpy(c))
        self.scale = [torch.from_numpy(s).cuda() for s in scale]

    def cache(self):
        k, v = self.codes
        return self.ft.make_kv8_cache(
            k=at(k), v=at(v), k_scale=at(self.scale[0]), v_scale=at(self.scale[1]), num_pages=self.pages, page_size=self.P,
            block_size=self.block, kv_heads=self.heads, head_dim=self.D, k_page_stride=k.stride(0),
            k_token_stride=k.stride(1), k_head_stride=k.stride(2), v_page_stride=v.stride(0), v_token_stride=v.stride(1),
            v_head_stride=v.stride(2))

    def store(self, rows, dtype, ctx, new, table, max_tokens=None, check=True):
        """rows: [T, 2, heads, D + pad] 16-bit tensor."""
        T = sum(new) if max_tokens is None else max_tokens
        t = dict(ctx=dev(ctx), start=dev(np.concatenate([[0], np.cumsum(new)])), table=dev(table), status=dev([0]))
        k, v = rows[:, 0], rows[:, 1]
        args = self.ft.make_kv8_store_args(k=at(k), v=at(v), q_start=at(t["start"]), ctx_len=at(t["ctx"]),
                                           block_table=at(t["table"]), status=at(t["status"]), k_stride=rows.stride(0),
                                           v_stride=rows.stride(0), dtype=code_of(self.ft, dtype), max_tokens=T,
                                           num_reqs=len(ctx), table_width=np.asarray(table).shape[1], cache=self.cache())
        self.ft.ft_kv8_store(args, stream())
        said = self.ref.store([x.double().cpu().numpy() for x in (k, v)], dtype, ctx, new, table)
        if check:
            torch.cuda.synchronize()
            want = (self.ft.FT_ST_BAD_SLOT if "slot" in said else 0) | (self.ft.FT_ST_NAN if "nan" in said else 0)
            assert t["status"].item() == want
            self.check()
        return args, t

    def check(self):
        for name, d, c in zip(("k", "v"), self.codes, self.ref.codes):
            assert np.array_equal(d.cpu().numpy(), c), name
        for name, d, c in zip(("k", "v"), self.scale, self.ref.scale):
            assert np.array_equal(d.cpu().numpy(), c), name + " scale"


def tables(rng, ctx, new, P, pages, spare=2):
    held = [-(-(c + n) // P) for c, n in zip(ctx, new)]
    ids = rng.permutation(pages)
    table, k = np.full((len(ctx), max(held + [1]) + spare), -1, dtype=np.int64), 0
    for b, h in enumerate(held):
        table[b, :h] = ids[k:k + h]
        k += h
    assert k <= pages
    return table


def random_rows(T, heads, D, dtype, seed, pad=0, spread=6.0):
    """Heads and tokens of sizes a few binades apart, zeros among them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.zeros((max(1, T), 2 * heads * D + pad), dtype=DT[dtype], device="cuda")
    rows = buf[:, :2 * heads * D].view(max(1, T), -1).unflatten(1, (2, heads, D))
    x = torch.randn((max(1, T), 2, heads, D), generator=g, device="cuda")
    x *= torch.exp2(spread * torch.rand((max(1, T), 2, heads, 1), generator=g, device="cuda") - 3)
    x *= torch.rand((max(1, T), 2, heads, D), generator=g, device="cuda") > 0.1
    rows.copy_(x)
    return rows


@pytest.mark.parametrize("ctx,new,P,block,heads,D,dtype,layout,pad", [
    ([0], [1], 16, 16, 1, 64, "bf16", "token", 0), ([15], [1], 16, 16, 2, 128, "f16", "token", 8),
    ([16], [1], 16, 16, 2, 128, "bf16", "head", 0), ([7, 0, 31, 5], [1, 1, 1, 0], 32, 16, 4, 128, "bf16", "token", 0),
    ([3, 40, 0], [37, 0, 130], 64, 32, 8, 64, "f16", "head", 24), ([100, 1, 63], [200, 64, 66], 64, 64, 3, 128, "bf16", "token", 40),
    ([0, 130], [300, 5], 128, 128, 2, 128, "f16", "head", 0), ([250, 10], [7, 300], 256, 128, 2, 64, "bf16", "token", 0),
    ([4090], [20], 4096, 16, 1, 128, "bf16", "token", 0), ([i % 50 for i in range(300)], [i % 3 for i in range(300)], 16, 16, 1, 64, "f16", "token", 0),
    ([11], [2000], 64, 64, 8, 128, "bf16", "token", 0)])
def test_store(ft, ctx, new, P, block, heads, D, dtype, layout, pad):
    rng = np.random.default_rng(sum(new) + P)
    pages = sum(-(-(c + n) // P) for c, n in zip(ctx, new)) + 3
    d = Device(ft, pages, P, block, heads, D, layout, seed=P)
    d.store(random_rows(sum(new), heads, D, dtype, seed=D + P, pad=pad), dtype, ctx, new, tables(rng, ctx, new, P, pages))


def test_keys_and_values_in_one_buffer(ft):
    rng = np.random.default_rng(3)
    d = Device(ft, 6, 32, 16, 2, 64, shared=True)
    d.store(random_rows(50, 2, 64, "bf16", 1), "bf16", [9, 30], [20, 30], tables(rng, [9, 30], [20, 30], 32, 6))


@pytest.mark.parametrize("dtype,block", [("bf16", 16), ("f16", 32), ("bf16", 128)])
def test_a_cache_filled_token_by_token(ft, dtype, block):
    """Scales that grow by many binades on the way, and blocks that start anew."""
    rng = np.random.default_rng(5)
    n, heads, D, P = 2 * block + 9, 2, 64, 128
    d = Device(ft, 4, P, block, heads, D, seed=1)
    table = tables(rng, [n], [0], P, 4)
    rows = random_rows(n, heads, D, dtype, 7, spread=12.0)
    for i in range(n):
        d.store(rows[i:i + 1], dtype, [i], [1], table, check=i % 8 == 0 or i + 1 == n)
    torch.cuda.synchronize()
    d.check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_extreme_numbers(ft, dtype):
    """Every finite pattern of the type, 64 to a row, each row in a block of its own scale or beside others."""
    bits = np.arange(65536, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).cuda().view(DT[dtype])
    x = torch.where(x.isfinite(), x, torch.ones_like(x)).view(-1, 1, 1, 64).expand(-1, 2, -1, -1).contiguous()
    T = x.shape[0]
    for per in (1, 16):  # rows of a request: a block each, or sixteen to a block
        new = [per] * (T // per)
        d = Device(ft, len(new), 16, 16, 1, 64)
        d.store(x, dtype, [0] * len(new), new, np.arange(len(new))[:, None])
    # beside tokens that are already there with a large scale
    new = [1] * T
    d = Device(ft, T, 16, 16, 1, 64, seed=9)
    d.store(x, dtype, [5] * T, new, np.arange(T)[:, None])


def test_infinities_and_nan(ft):
    for dtype in ("bf16", "f16"):
        rows = random_rows(40, 2, 128, dtype, 3)
        rows[3, 0, 1, 5] = float("inf")
        rows[4, 1, 0, 127] = float("-inf")
        rows[20, 0] = float("nan")
        rows[21, 1, 1, ::7] = float("nan")
        d = Device(ft, 4, 32, 32, 2, 128)
        d.store(rows, dtype, [10], [40], np.array([[2, 0, 1]]))
        d.store(rows[20:21], dtype, [50], [1], np.array([[2, 0, 1]]))  # nothing finite beside what is there


def test_zeros_leave_the_scale_free(ft):
    rows = torch.zeros((3, 2, 1, 64), dtype=torch.bfloat16, device="cuda")
    rows[1] = 1e-20
    rows[2] = 5.0
    d = Device(ft, 1, 16, 16, 1, 64)
    for i in range(3):
        d.store(rows[i:i + 1], "bf16", [i], [1], np.array([[0]]))
    assert d.ref.scale[0][0, 0, 0] == 127 - 6


def test_missing_pages_and_bytes_of_255(ft):
    rows = random_rows(100, 2, 64, "f16", 2)
    d = Device(ft, 3, 16, 16, 2, 64)
    d.store(rows, "f16", [20, 0], [40, 60], np.array([[0, 3, -1, 1], [2, 100, -7, -1]]))  # 2: one row of 16 left
    d = Device(ft, 3, 16, 16, 2, 64)
    d.store(rows[:30], "f16", [0], [30], np.array([[1]]))  # past the table
    d = Device(ft, 2, 16, 16, 2, 64)
    d.scale[1][1, 0, 1] = 255
    d.ref.scale[1][1, 0, 1] = 255
    d.store(rows[:4], "f16", [3], [4], np.array([[1]]))


def test_rows_past_max_tokens_and_negative_lengths(ft):
    rows = random_rows(40, 2, 64, "bf16", 4)
    d = Device(ft, 4, 16, 16, 2, 64)
    t = dict(ctx=dev([0, -3, 2]), start=dev([0, 10, 10, 40]), table=dev([[0], [1], [2]]))
    args = ft.make_kv8_store_args(k=at(rows[:, 0]), v=at(rows[:, 1]), q_start=at(t["start"]), ctx_len=at(t["ctx"]),
                                  block_table=at(t["table"]), k_stride=rows.stride(0), v_stride=rows.stride(0),
                                  dtype=ft.FT_DTYPE_BF16, max_tokens=15, num_reqs=3, table_width=1, cache=d.cache())
    ft.ft_kv8_store(args, stream())
    torch.cuda.synchronize()
    x = rows.double().cpu().numpy()
    d.ref.store([x[:15, 0], x[:15, 1]], "bf16", [0, 0, 2], [10, 0, 5], [[0], [1], [2]])
    d.check()


@pytest.mark.parametrize("T,heads,D,dtype,P,block,layout", [
    (1, 1, 64, "bf16", 16, 16, "token"), (77, 4, 128, "f16", 64, 32, "head"), (1000, 3, 64, "bf16", 32, 16, "token"),
    (4099, 2, 128, "f16", 4096, 128, "token"), (5, 8, 128, "bf16", 128, 64, "head")])
def test_load(ft, T, heads, D, dtype, P, block, layout):
    rng = np.random.default_rng(T)
    pages = max(3, T // P)
    d = Device(ft, pages, P, block, heads, D, layout, seed=T)
    # any scale byte and any code
    for s, r, c, rc in zip(d.scale, d.ref.scale, d.codes, d.ref.codes):
        r[:] = rng.integers(0, 256, r.shape)
        rc[:] = rng.integers(0, 256, rc.shape)
        s.copy_(torch.from_numpy(r))
        c.copy_(torch.from_numpy(rc))
    slots = rng.integers(0, pages * P, T)
    slots[rng.random(T) < 0.1] = -1
    out = [torch.full((T, heads * D + 8), 3.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    status, s = dev([0]), dev(slots, torch.int64)
    args = ft.make_kv8_load_args(k=at(out[0]), v=at(out[1]), slots=at(s), status=at(status), k_stride=heads * D + 8,
                                 v_stride=heads * D + 8, dtype=code_of(ft, dtype), T=T, cache=d.cache())
    ft.ft_kv8_load(args, stream())
    torch.cuda.synchronize()
    assert status.item() == 0
    for kv in range(2):
        want = d.ref.values(kv)[slots // P, slots % P]
        want[slots < 0] = 0
        want = torch.from_numpy(want).to(DT[dtype])
        got = out[kv][:, :heads * D].unflatten(1, (heads, D)).cpu()
        assert torch.equal(torch.nan_to_num(got, 7.0, 9.0, -9.0), torch.nan_to_num(want, 7.0, 9.0, -9.0))
        assert bool((out[kv][:, heads * D:] == 3).all())


def test_load_past_the_cache(ft):
    d = Device(ft, 2, 16, 16, 1, 64)
    out = torch.full((2, 3, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    status, s = dev([0]), dev([31, 32, 1 << 40], torch.int64)
    ft.ft_kv8_load(ft.make_kv8_load_args(k=at(out[0]), v=at(out[1]), slots=at(s), status=at(status), k_stride=64, v_stride=64,
                                         dtype=ft.FT_DTYPE_BF16, T=3, cache=d.cache()), stream())
    torch.cuda.synchronize()
    assert status.item() == ft.FT_ST_BAD_SLOT
    assert bool((out[:, 1:] == 0).all()) and bool((out[:, 0] != 3).any())


def test_tokens_moved_together(ft):
    """Rows read back and stored at other places are what they were: power-of-two scales lose nothing but subnormals."""
    rng = np.random.default_rng(8)
    heads, D, P = 2, 64, 32
    d = Device(ft, 3, P, 16, heads, D)
    rows = random_rows(40, heads, D, "bf16", 5, spread=1.0)
    d.store(rows, "bf16", [9], [40], np.array([[1, 0, -1]]))
    keep = [9, 12, 13, 30, 44]  # positions of accepted tokens
    slots = dev([[1, 0][p // P] * P + p % P for p in keep], torch.int64)
    out = torch.zeros((len(keep), 2, heads, D), dtype=torch.bfloat16, device="cuda")
    ft.ft_kv8_load(ft.make_kv8_load_args(k=at(out[:, 0]), v=at(out[:, 1]), slots=at(slots), k_stride=out.stride(0),
                                         v_stride=out.stride(0), dtype=ft.FT_DTYPE_BF16, T=len(keep), cache=d.cache()), stream())
    before = [d.ref.values(kv)[[[1, 0][p // P] for p in keep], [p % P for p in keep]] for kv in range(2)]
    d.store(out, "bf16", [9], [len(keep)], np.array([[1, 0, -1]]))
    for kv in range(2):
        after = d.ref.values(kv)[1, 9:9 + len(keep)]
        scale = 2.0 ** (d.ref.scale[kv][1, 0:1].astype(float) - 127)  # tokens 9 .. 13: one block
        assert (np.abs(after - before[kv]) <= 2.0 ** -10 * scale[..., None]).all()


def test_captured_and_replayed_on_another_stream(ft):
    heads, D, P = 2, 128, 64
    rng = np.random.default_rng(2)
    d = Device(ft, 8, P, 32, heads, D)
    ctx, new = [3, 60], [10, 100]
    table = tables(rng, ctx, new, P, 8)
    rows = random_rows(110, heads, D, "bf16", 6)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        args, t = d.store(rows, "bf16", ctx, new, table)
        slots = dev(np.arange(P), torch.int64)
        out = torch.zeros((P, 2, heads, D), dtype=torch.bfloat16, device="cuda")
        load = ft.make_kv8_load_args(k=at(out[:, 0]), v=at(out[:, 1]), slots=at(slots), k_stride=out.stride(0),
                                     v_stride=out.stride(0), dtype=ft.FT_DTYPE_BF16, T=P, cache=d.cache())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ft.ft_kv8_store(args, stream())
            ft.ft_kv8_load(load, stream())
        for i in range(3):
            rows.copy_(random_rows(110, heads, D, "bf16", 20 + i, spread=6.0 + i))
            graph.replay()
            torch.cuda.synchronize()
            x = rows.double().cpu().numpy()
            d.ref.store([x[:, 0], x[:, 1]], "bf16", ctx, new, table)
            d.check()
            for kv in range(2):
                want = torch.from_numpy(d.ref.values(kv)[0]).to(torch.bfloat16)
                assert torch.equal(out[:, kv].cpu(), want)
