"""Verification of drafted tokens against a plain 64-bit implementation.

Results are whole numbers and equal: the library's entries are rounded to
multiples of 2^-45, sums over a row are off by 2^-46 sqrt(V) or so, and no random
number here lies that near a border (but in the test that puts them there with
exact sums).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ft():
    from expert_cache_host_gb300 import build as ftbuild
    ftbuild.build()
    import expert_cache_host_gb300 as lib
    lib.load()
    return lib


def reference(p, q, tokens, parents, u, draw_u, start):
    """p, q: float64 [T, V] (q None: drafts without a choice)."""
    accepted, counts, following = -np.ones(len(tokens), dtype=np.int64), [], []
    V = p.shape[1]
    p = np.where((p >= 0) & (p <= 2), p, 0)
    if q is not None:
        q = np.where((q >= 0) & (q <= 2), q, 0)
    for b in range(len(start) - 1):
        t0, n = start[b], start[b + 1] - start[b]
        if n == 0:
            counts.append(0)
            following.append(-1)
            continue
        at, count = 0, 0
        a, A = p[t0].copy(), 1.0
        for i in range(1, n):  # (a child's row comes after its parent's)
            parent = i - 1 if parents is None else parents[t0 + i]
            x = tokens[t0 + i]
            if parent != at or not 0 <= x < V:
                continue
            row = np.eye(1, V, x)[0] if q is None else q[t0 + at]
            if u[t0 + i] * row[x] * A < a[x]:
                accepted[t0 + count] = at = i
                count += 1
                a, A = p[t0 + at].copy(), 1.0
            else:
                a = np.maximum(a - A * row, 0)
                A = a.sum()
        if a.sum() == 0:
            a = p[t0 + at]
        counts.append(count)
        c = np.cumsum(a)
        following.append(int(np.searchsorted(c, draw_u[b] * c[-1], side="right")) if c[-1] > 0 else -1)
    return accepted, np.array(counts), np.array(following)


class Case:
    def __init__(self, ft, new, V, dtype, tree, draft, pad=0, draft_pad=None, seed=0, sharp=2.0, iid=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.ft, self.V, self.dtype = ft, V, dtype
        T, self.T = max(1, sum(new)), sum(new)
        self.start = np.concatenate([[0], np.cumsum(new)])
        draft_pad = pad if draft_pad is None else draft_pad
        x = torch.randn((T, V), generator=g, device="cuda") * sharp
        self.p = torch.full((T, V + pad), float("nan"), device="cuda", dtype=DT[dtype])[:, :V]
        self.p.copy_(torch.softmax(x, 1))
        self.q = None
        if draft:
            self.q = torch.full((T, V + draft_pad), float("nan"), device="cuda", dtype=DT[dtype])[:, :V]
            self.q.copy_(torch.softmax(x + torch.randn((T, V), generator=g, device="cuda") * 0.7, 1))
        self.parents = None
        if tree:
            self.parents = np.concatenate([[-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, n)] for n in new if n] or
                                          [[]]).astype(np.int32)
        self.tokens = np.zeros(T, dtype=np.int64)
        for b, n in enumerate(new):
            for i in range(1, n):
                row = self.start[b] + (self.parents[self.start[b] + i] if tree else i - 1)
                w = (self.q if draft else self.p)[row].double().cpu().numpy()
                self.tokens[self.start[b] + i] = rng.choice(V, p=w / w.sum())
        self.u = torch.rand(T, generator=g, device="cuda")
        self.draw = torch.rand(max(1, len(new)), generator=g, device="cuda")
        self.B = len(new)

    def args(self):
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
        self.d = dict(tokens=i32(self.tokens), parents=None if self.parents is None else i32(self.parents),
                      start=i32(self.start), accepted=i32([-7] * (max(1, self.T) + 3)), n=i32([-7] * (self.B + 1)),
                      token=i32([-7] * (self.B + 1)), status=i32([0]))
        at = lambda t: 0 if t is None else t.data_ptr()
        d = self.d
        code = {"bf16": self.ft.FT_DTYPE_BF16, "f16": self.ft.FT_DTYPE_F16, "f32": self.ft.FT_DTYPE_F32}[self.dtype]
        return self.ft.make_verify_args(
            probs=at(self.p), draft_probs=at(self.q), tokens=at(d["tokens"]), parents=at(d["parents"]), accept_u=at(self.u),
            draw_u=at(self.draw), q_start=at(d["start"]), accepted=at(d["accepted"]), n_accepted=at(d["n"]),
            next_token=at(d["token"]), status=at(d["status"]), probs_stride=self.p.stride(0),
            draft_stride=0 if self.q is None else self.q.stride(0), dtype=code, max_tokens=self.T + 3, num_reqs=self.B, V=self.V)

    def want(self):
        wide = lambda t: None if t is None else t.double().cpu().numpy()
        return reference(wide(self.p), wide(self.q), self.tokens, self.parents, wide(self.u), wide(self.draw), self.start)

    def check(self, status=0):
        torch.cuda.synchronize()
        accepted, counts, following = self.want()
        assert self.d["status"].item() == status
        assert np.array_equal(self.d["n"].cpu().numpy()[:self.B], counts)
        assert np.array_equal(self.d["accepted"].cpu().numpy()[:self.T], accepted[:self.T])
        assert np.array_equal(self.d["token"].cpu().numpy()[:self.B], following)
        assert (self.d["accepted"].cpu().numpy()[max(1, self.T):] == -7).all()
        assert self.d["n"][-1].item() == -7 and self.d["token"][-1].item() == -7
        return counts

    def run(self, status=0):
        self.ft.ft_verify_drafts(self.args(), torch.cuda.current_stream().cuda_stream)
        return self.check(status)


@pytest.mark.parametrize("new,V,dtype,tree,draft,pad", [
    ([1], 1, "f32", False, True, 0), ([5], 131072, "f32", False, True, 0), ([5], 131072, "bf16", True, True, 0),
    ([3, 0, 1, 9], 50021, "bf16", True, False, 27), ([17] * 20, 32000, "f32", True, True, 0), ([4, 2], 7, "f16", False, False, 1),
    ([2] * 400, 1000, "f32", False, True, 3), ([33, 1, 20], 5003, "f16", True, True, 5), ([8] * 700, 257, "f32", True, True, 0),
    ([6] * 3, 262147, "bf16", True, True, 2), ([1] * 9, 3000, "f32", True, False, 0)])
def test_verify(ft, new, V, dtype, tree, draft, pad):
    for seed in range(3):
        Case(ft, new, V, dtype, tree, draft, pad, seed=seed + V).run()


def test_rows_of_other_alignment(ft):
    """Rows of the target and of the draft that never lie on 16-byte boundaries together."""
    for dtype, pads in (("f32", (1, 2)), ("bf16", (0, 3)), ("f16", (5, 8))):
        Case(ft, [9, 4, 17], 9001, dtype, True, True, pads[0], pads[1], seed=4).run()


def test_flat_and_peaked_rows(ft):
    for sharp in (0.0, 12.0):
        for draft in (False, True):
            Case(ft, [12] * 30, 8192, "f32", True, draft, seed=5, sharp=sharp).run()


@pytest.mark.parametrize("V", [3001, 50021, 131071, 200003])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_equal_probabilities(ft, V, dtype):
    """Every entry the same, no multiple of a power of two: what is left of the entries at any level adds up."""
    for draft in (False, True):
        c = Case(ft, [1] * 30 + [2] * 30, V, dtype, False, draft, seed=V, sharp=0.0)
        c.p.fill_(1.0 / V)
        c.u.fill_(0.999)
        if draft:
            c.q.fill_(0.4 / V)
            c.q[:, ::2] = 1.5 / V
        c.run()


def test_many_rows_and_many_children(ft):
    """More rows than are gathered ahead, and a row with many children that are all rejected."""
    c = Case(ft, [900, 60], 500, "f32", True, True, seed=6)
    c.parents[600] = 0  # a child of the first row, far behind
    c.run()
    c = Case(ft, [1300], 400, "f32", False, False, seed=6, sharp=0.0)
    c.u.zero_()  # every one accepted
    assert c.run()[0] == 1299
    for draft in (False, True):
        c = Case(ft, [64, 30], 3000, "f32", True, draft, seed=7)
        c.parents[:] = 0
        c.parents[[0, 64]] = -1
        c.u.fill_(0.99999)
        c.tokens[5] = c.tokens[2]  # the same token twice
        c.run()


def test_more_rejected_children_than_are_kept(ft):
    c = Case(ft, [90], 1000, "f32", True, False, seed=8)
    c.parents[:] = 0
    c.parents[0] = -1
    c.tokens[:] = np.arange(90)
    c.u.fill_(0.99999)
    args = c.args()
    ft.ft_verify_drafts(args, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert c.d["status"].item() == ft.FT_ST_BAD_TREE and c.d["n"][0].item() == 0
    a = c.p[0].double().cpu().numpy()
    a[1:65] = 0  # rows 1 .. 64
    s = np.cumsum(a)
    assert c.d["token"][0].item() == np.searchsorted(s, c.draw[0].item() * s[-1], side="right")


def test_borders(ft):
    """Sums of powers of two: a number on a border belongs to the token after it, and does not accept."""
    c = Case(ft, [2] * 6, 4, "f32", False, False, seed=1)
    c.p.copy_(torch.tensor([0.25, 0.0, 0.5, 0.25], device="cuda").expand(12, 4))
    c.tokens[:] = 2
    c.u.copy_(torch.tensor([0, 0.5, 0, 0.5 - 2.0 ** -25, 0, 0.75, 0, 0.75, 0, 0.75, 0, 0.75], device="cuda"))
    # accepted or not; then the draw: from (1/4, 0, 0, 1/4) where token 2 was rejected
    c.draw.copy_(torch.tensor([0.5, 0.75, 0.5 - 2.0 ** -25, 0.0, 0.49, 1 - 2.0 ** -24], device="cuda"))
    counts = c.run()
    assert counts.tolist() == [0, 1, 0, 0, 0, 0]
    assert c.d["token"].tolist()[:6] == [3, 3, 0, 0, 0, 3]


def test_nothing_left_after_a_rejection(ft):
    """The draft's probabilities cover the target's: the draw is from the target's."""
    c = Case(ft, [2] * 50, 64, "f32", False, True, seed=2)
    c.q.copy_(c.p * 1.5)
    c.u.fill_(0.9)
    c.run()


def test_random_numbers_out_of_range(ft):
    c = Case(ft, [2] * 4, 100, "f32", False, True, seed=3)
    c.u.copy_(torch.tensor([0, 1.5, 0, float("nan"), 0, -3.0, 0, float("inf")], device="cuda"))
    c.draw.copy_(torch.tensor([1.0, float("nan"), -1.0, 7.0], device="cuda"))
    ft.ft_verify_drafts(c.args(), torch.cuda.current_stream().cuda_stream)
    top = 1 - 2.0 ** -24
    c.u.copy_(torch.tensor([0, top, 0, 0, 0, 0, 0, top], device="cuda"))
    c.draw.copy_(torch.tensor([top, 0, 0, top], device="cuda"))
    c.check()


def test_bad_entries_and_tokens(ft):
    c = Case(ft, [3, 3], 5000, "f32", False, True, seed=4)
    c.p[:, 100:200] = float("nan")
    c.p[:, 300] = -1.0
    c.p[:, 301] = float("inf")
    c.run(ft.FT_ST_NAN)
    c = Case(ft, [3, 3], 5000, "f32", True, True, seed=4)
    c.parents[:] = [-1, 0, 0, -1, 0, 0]
    c.tokens[1], c.tokens[4] = 5000, -1
    c.run(ft.FT_ST_BAD_TOKEN)
    for value in (0.0, float("nan"), 1.0):  # nothing to draw from; a sum of 5000
        c = Case(ft, [1, 2], 5000, "f32", False, False, seed=5)
        c.p[0] = value
        ft.ft_verify_drafts(c.args(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert c.d["status"].item() == ft.FT_ST_NAN
        assert c.d["token"].tolist()[0] == -1 and c.d["token"].tolist()[1] >= 0 and c.d["n"].tolist()[0] == 0


def test_bad_parents_take_no_part(ft):
    c = Case(ft, [6], 300, "f32", True, False, seed=4)
    c.parents[:] = [-1, -1, 2, 9, -5, 4]
    assert c.run()[0] == 0


@pytest.mark.parametrize("tree,draft", [(False, True), (True, True), (True, False)])
def test_what_is_said_is_distributed_as_the_target(ft, tree, draft):
    """The first token told after row 0 (accepted or drawn) over many requests: within 5 standard deviations."""
    B, V, n = 40000, 6, 4
    g = torch.Generator(device="cuda").manual_seed(11)
    p1 = torch.softmax(torch.randn(V, generator=g, device="cuda"), 0)
    q1 = torch.softmax(torch.randn(V, generator=g, device="cuda"), 0)
    c = Case(ft, [1], V, "f32", False, draft, seed=1)
    c.T, c.B, c.start = B * n, B, np.arange(B + 1) * n
    c.p = p1.expand(B * n, V).contiguous()
    c.q = q1.expand(B * n, V).contiguous() if draft else None
    if draft:
        c.tokens = torch.multinomial(q1, B * n, replacement=True, generator=g).cpu().numpy()
    else:
        c.tokens = np.tile(np.array([0, 3, 1, 4]), B)
    c.parents = np.tile(np.array([-1, 0, 0, 0]), B) if tree else None
    c.u, c.draw = torch.rand(B * n, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    ft.ft_verify_drafts(c.args(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    first = c.d["accepted"].cpu().numpy()[:B * n:n]
    said = np.where(first > 0, c.tokens[np.arange(B) * n + np.maximum(first, 0)], c.d["token"].cpu().numpy()[:B])
    share = np.bincount(said, minlength=V) / B
    want = p1.double().cpu().numpy()
    assert (np.abs(share - want) < 5 * np.sqrt(want * (1 - want) / B)).all()


def test_captured_and_replayed_on_another_stream(ft):
    c = Case(ft, [9] * 12, 20000, "bf16", True, True, seed=3)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        args = c.args()
        ft.ft_verify_drafts(args, side.cuda_stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ft.ft_verify_drafts(args, torch.cuda.current_stream().cuda_stream)
        for _ in range(3):
            c.u.uniform_()
            c.draw.uniform_()
            graph.replay()
            c.check()
