"""Sums of what is left after rejections with draft probabilities, against exact fractions.

Draws and acceptances lie on both sides of a border, as near to it as a 32-bit
random number comes (some 2^-25 of it; the library's sums are multiples of 2^-44
and V is small, so 2^-36 is far beyond what they can be off by: asserted here of
every input).  An entry that is off by 2^-25 puts some of them on the wrong side.
"""
from fractions import Fraction

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_verify import DT, ft  # noqa: E402, F401

MARGIN = Fraction(1, 2 ** 36)
ONE = np.float32(1 - 2.0 ** -24)


def held(x, dtype):
    """x rounded to the type, as numpy float64."""
    return torch.tensor(np.asarray(x, dtype=np.float64)).to(DT[dtype]).double().numpy()


def fractions(row):
    return [Fraction(float(x)) for x in row]


def after(p, q, k):
    """a and A after k rejections."""
    a, A = list(p), Fraction(1)
    for _ in range(k):
        a = [max(x - A * y, Fraction(0)) for x, y in zip(a, q)]
        A = sum(a)
    return a, A


def around(x):
    """The 32-bit numbers next to a fraction in (0, 1), below and above."""
    f = np.float32(float(x))
    if Fraction(float(f)) > x:
        return np.nextafter(f, np.float32(0)), f
    return f, np.nextafter(f, np.float32(2))


def rejected(p, q, k):
    """k tokens, one after another, that a random number next to 1 rejects; None where there are none."""
    out = []
    for j in range(k):
        a, A = after(p, q, j)
        x = max(range(len(p)), key=lambda i: q[i] * A - a[i])
        if not Fraction(float(ONE)) * q[x] * A >= a[x]:
            return None
        out.append(x)
    return out


def least(a, u):
    """The least i with a_0 + .. + a_i > u sum a, which no sum comes near to."""
    point, run, token = Fraction(float(u)) * sum(a), Fraction(0), None
    for i, x in enumerate(a):
        run += x
        assert abs(run - point) > MARGIN or x == 0 or u == 0
        if token is None and run > point:
            token = i
    return token


class Batch:
    """Requests of a first row and children of it, every one of k + `extra` tokens."""

    def __init__(self, dtype, V, draft=True):
        self.dtype, self.V, self.draft = dtype, V, draft
        self.p, self.q, self.tokens, self.u, self.draw, self.n, self.want = [], [], [], [], [], [], []

    def add(self, p, q, tokens, u, draw, accepted, token):
        self.p += [p] * (1 + len(tokens))
        self.q += [q] * (1 + len(tokens))
        self.tokens += [0] + list(tokens)
        self.u += [0.0] + list(u)
        self.draw.append(draw)
        self.n.append(1 + len(tokens))
        self.want.append((accepted, token))

    def check(self, ft):
        start = np.concatenate([[0], np.cumsum(self.n)])
        dev = lambda x, t: torch.tensor(np.asarray(x), dtype=t, device="cuda")
        i32 = torch.int32
        p, q = dev(self.p, DT[self.dtype]), dev(self.q, DT[self.dtype])
        parents = np.concatenate([[-1] + [0] * (n - 1) for n in self.n])
        d = [dev(self.tokens, i32), dev(parents, i32), dev(self.u, torch.float32), dev(self.draw, torch.float32), dev(start, i32)]
        T, B = len(self.tokens), len(self.n)
        accepted, count, token, status = (torch.full((n,), v, dtype=i32, device="cuda") for n, v in ((T, -7), (B, -7), (B, -7), (1, 0)))
        code = {"bf16": ft.FT_DTYPE_BF16, "f16": ft.FT_DTYPE_F16, "f32": ft.FT_DTYPE_F32}[self.dtype]
        ft.ft_verify_drafts(ft.make_verify_args(
            probs=p.data_ptr(), draft_probs=q.data_ptr() if self.draft else 0, tokens=d[0].data_ptr(), parents=d[1].data_ptr(),
            accept_u=d[2].data_ptr(), draw_u=d[3].data_ptr(), q_start=d[4].data_ptr(), accepted=accepted.data_ptr(),
            n_accepted=count.data_ptr(), next_token=token.data_ptr(), status=status.data_ptr(), probs_stride=self.V,
            draft_stride=self.V, dtype=code, max_tokens=T, num_reqs=B, V=self.V), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert status.item() == 0
        first = accepted[dev(start[:-1], torch.int64)].tolist()
        wrong = [(b, got, want) for b, (got, want) in enumerate(zip(zip(first, token.tolist()), self.want))
                 if got[0] != want[0] or (want[1] is not None and got[1] != want[1])]
        assert not wrong, (len(wrong), len(self.want), wrong[:5])


@pytest.mark.parametrize("excess,other", [(2.0 ** -25, 66), (2.0 ** -25, 87), (2.0 ** -22 - 2.0 ** -25, 65), (2.0 ** -22 - 2.0 ** -25, 81)])
def test_a_residual_between_two_numbers(ft, excess, other):
    """What is left of an entry is 0.5 + 2^-23 and some more, which 32 bits do not hold; beside `other` 1024ths a draw lies
    within 2^-26 of the border."""
    left, other = Fraction(1, 2) + Fraction(1, 2 ** 23) + Fraction(excess), Fraction(other, 1024)
    p, q = [0.75, float(other), 0.125], [float(Fraction(3, 4) - left), 0.0, 0.75]
    a, _ = after(fractions(p), fractions(held(q, "f32")), 1)
    assert a == [left, other, 0]
    b = Batch("f32", 3)
    for u in around(left / sum(a)):
        b.add(p, q, [2], [ONE], u, -1, least(a, u))
    assert {w[1] for w in b.want} == {0, 1}
    b.check(ft)


@pytest.mark.parametrize("p0,q0,other", [("0x1.d1c91cp+0", "0x1.77cf84p-1", 54), ("0x1.fb4dccp+0", "0x1.4550f4p-1", 298),
                                         ("0x1.fec008p+0", "0x1.56f14cp-1", 199)])
def test_a_residual_of_an_entry_above_one(ft, p0, q0, other):
    """The same after two rejections, where what 32 bits do not hold is up to 2^-22."""
    p, q = [float.fromhex(p0), other / 1024, 0.125], [float.fromhex(q0), 0.0, 0.75]
    a, A = after(fractions(p), fractions(q), 2)
    b = Batch("f32", 3)
    for u in around(a[0] / A):
        b.add(p, q, [2, 2], [ONE, ONE], u, -1, least(a, u))
    assert {w[1] for w in b.want} == {0, 1}
    b.check(ft)


def rows(rng, V, dtype, most):
    """A pair of rows; most > 1: entries up to it."""
    p, q = rng.dirichlet(np.full(V, 0.5)), rng.dirichlet(np.full(V, 0.5))
    if rng.random() < 0.5:
        q = 0.5 * p + 0.5 * q
    if most > 1:
        p = rng.random(V) * most
        q = rng.random(V) * most / 3
    return held(p, dtype), held(q, dtype)


@pytest.mark.parametrize("k", [1, 2, 3])
@pytest.mark.parametrize("V,dtype,most", [(3, "f32", 1), (5, "f32", 1), (12, "f32", 1), (4, "f32", 2), (5, "bf16", 1), (12, "f16", 1)])
def test_draws_on_both_sides_of_borders(ft, k, V, dtype, most):
    rng = np.random.default_rng(1000 * k + V)
    b = Batch(dtype, V)
    for _ in range(400):
        p, q = rows(rng, V, dtype, most)
        fp, fq = fractions(p), fractions(q)
        tokens = rejected(fp, fq, k)
        a, A = after(fp, fq, k)
        if tokens is None or A < Fraction(1, 64):
            continue
        i = int(rng.integers(V))
        border = sum(a[:i + 1]) / A
        for u in around(border) if 0 < border < 1 else []:
            if abs(border - Fraction(float(u))) * A > 2 * MARGIN and u < 1:
                b.add(p, q, tokens, [ONE] * k, u, -1, least(a, u))
    assert len(b.n) > 40, len(b.n)
    b.check(ft)


@pytest.mark.parametrize("k", [1, 2, 3])
@pytest.mark.parametrize("V,dtype,most", [(5, "f32", 1), (12, "f32", 1), (4, "f32", 2)])
def test_later_children_on_both_sides_of_acceptance(ft, k, V, dtype, most):
    """After k rejections one more child: accepted where accept_u q(x) A < a(x)."""
    rng = np.random.default_rng(2000 * k + V)
    b = Batch(dtype, V)
    for _ in range(3000):
        p, q = rows(rng, V, dtype, most)
        fp, fq = fractions(p), fractions(q)
        tokens = rejected(fp, fq, k)
        a, A = after(fp, fq, k)
        x = int(rng.integers(V))
        if tokens is None or A < Fraction(1, 64) or q[x] < 1e-3:
            continue
        border = a[x] / (fq[x] * A)
        for u in around(border) if 0 < border < 1 else []:
            off = Fraction(float(u)) - border
            if abs(off) * fq[x] * A > 2 * MARGIN and u < 1:
                b.add(p, q, tokens + [x], [ONE] * k + [u], 0.0, k + 1 if off < 0 else -1, None)
    assert len(b.n) > 30, len(b.n)
    b.check(ft)


def whole(x):
    """x rounded to a multiple of 2^-44, ties to even."""
    return Fraction(round(x * 2 ** 44), 2 ** 44)


@pytest.mark.parametrize("removed,x,other,u", [
    (["0x1.36f676p-24", "0x1.6f0368p-24", "0x1.3d9c18p-27"], "0x1.0f21dep-24", "0x1.fb17c4p-27", "0x1.9efbaap-1"),
    (["0x1.24ede6p-24", "0x1.922766p-25", "0x1.1a61dcp-25"], "0x1.5f5572p-24", "0x1.6c99c8p-24", "0x1.f68324p-2"),
    (["0x1.907a70p-25", "0x1.7f1506p-27", "0x1.c6f878p-27"], "0x1.95e762p-23", "0x1.7242a6p-25", "0x1.a0ec18p-1"),
    (["0x1.3f98e2p-25", "0x1.b2f14cp-25", "0x1.14f474p-26"], "0x1.867348p-23", "0x1.7579dap-24", "0x1.5a5a36p-1"),
    (["0x1.49b64ap-24", "0x1.1e3990p-27", "0x1.2a3af4p-26"], "0x1.26e876p-23", "0x1.afd1b2p-25", "0x1.76ccbcp-1")])
def test_little_left_without_draft_probabilities(ft, removed, x, other, u):
    """Nearly all of a row is rejected, then three of the small entries: what is left is the sum of the other entries,
    each rounded, not what the removed ones as they are leave of the sum before."""
    removed, x, other = [float.fromhex(r) for r in removed], float.fromhex(x), float.fromhex(other)
    p, u = [0.99, *removed, x, other], np.float32(float.fromhex(u))
    a, left = [Fraction(y) for y in p], Fraction(0)
    for j in range(4):  # tokens 0 .. 3 are rejected
        A = sum(whole(y) for y in a[j:]) if j else Fraction(1)
        assert Fraction(float(ONE)) * A > a[j]
    A = whole(a[4]) + whole(a[5])
    b = Batch("f32", 6, draft=False)
    for v in (u, np.nextafter(u, np.float32(0)), np.nextafter(u, np.float32(1))):
        b.add(p, p, [0, 1, 2, 3, 4], [ONE] * 4 + [v], 0.0, 5 if Fraction(float(v)) * A < a[4] else -1, None)
    assert {w[0] for w in b.want} == {5, -1}
    b.check(ft)
