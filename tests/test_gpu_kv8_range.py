"""Attention over the 8-bit cache at the ends of the types' ranges, against a plain
64-bit implementation: the largest numbers f16 holds, the smallest scale bytes, and
queries whose numbers lie far apart.

Tolerances as in test_gpu_kv8_attention.py: u (sum p |v| + |o|) + 2^-16 sum p |v|
(u = 2^-8 for bf16, 2^-11 for f16), half the least spacing of the type for a value
and for the output, f16 probabilities off by 2^-36 of a row's largest.  A score that
is off by s moves a probability by a factor of e^(2 s) at most and lse by s.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_kv8_attention import DT, U, Attn, ft  # noqa: E402, F401

HALF_SPACING = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}


class Rounded(Attn):
    """The cache's numbers as the type of the rows holds them."""

    def values(self, kv, b):
        return super().values(kv, b).float().to(DT[self.dtype]).double()


def compare(a, shift=0.0, most=0.0):
    """shift: how far a score may be off, [T, Hq] or a number; most: the largest value's size."""
    out, lse, mag, top = a.run().reference()
    got, got_lse = a.out.double().cpu().numpy()[:a.T], a.lse.double().cpu().numpy()[:a.T]
    moved = np.expm1(2 * np.broadcast_to(np.asarray(shift, dtype=np.float64), lse.shape))[:, :, None]
    tol = U[a.dtype] * (mag + np.abs(out)) + 2.0 ** -16 * mag + moved * mag + 2 * HALF_SPACING[a.dtype]
    if most:
        tol = tol + 2.0 ** -36 * most * (max(a.ctx) + max(a.new))
    assert np.isfinite(got).all() and a.status.item() == 0
    bad = np.abs(got - out) / tol
    assert bad.max() <= 1, (bad.max(), np.unravel_index(bad.argmax(), bad.shape))
    err = np.abs(got_lse - lse) / (2.0 ** -16 * top + shift)
    assert err.max() <= 1, err.max()


def set_bytes(a, byte, span):
    """Scale bytes byte .. byte + span - 1 for the blocks in use, as their old ones say."""
    for kv in range(2):
        keep = a.bytes[kv] != 255
        a.bytes[kv][keep] = (byte + a.bytes[kv][keep].int() % span).to(torch.uint8)


@pytest.mark.parametrize("new", [[6, 3], [1, 1], [2, 2]])
@pytest.mark.parametrize("Hq,D", [(8, 128), (16, 64)])
def test_numbers_up_to_the_largest_of_f16(ft, new, Hq, D):
    """Bytes of 134 to 138, codes as large as f16 has room for, so that none is past 65504."""
    a = Attn(ft, [300, 70], new, Hq, 2, D, "f16", 32, 16, seed=134)
    set_bytes(a, 134, 5)
    for b in range(2):
        page, row = a.rows[b]
        for kv in range(2):
            x = a.codes[kv][page, row].view(torch.float8_e4m3fn).float()
            room = 65504.0 * torch.exp2(127.0 - a.bytes[kv][page, row // 16].float())[:, :, None]
            x = torch.where(x.abs() > room, x.sign() * room, x)
            # (towards 0: a code above `room` would be past f16)
            c = x.to(torch.float8_e4m3fn)
            over = c.float().abs() > room
            c = torch.where(over, c.view(torch.uint8) - 1, c.view(torch.uint8))
            a.codes[kv][page, row] = c
    most = max(float(a.values(kv, b).abs().max()) for kv in range(2) for b in range(2))
    assert 60000 < most <= 65504
    a.scale = a.args.scale = float(np.float32(0.01 * 2.0 ** -7))
    compare(a, most=most)


@pytest.mark.parametrize("new", [[6, 3], [1, 1], [2, 2]])
@pytest.mark.parametrize("Hq,D", [(8, 128), (16, 64)])
def test_the_smallest_scale_bytes(ft, new, Hq, D):
    """Bytes of 0 to 4 in bf16, below whose spacing the lowest codes are, and a softmax scale that makes up for it."""
    few = max(new) * Hq // 2 <= 16  # these are not rounded to the type
    a = (Attn if few else Rounded)(ft, [300, 70], new, Hq, 2, D, "bf16", 32, 16, seed=5)
    set_bytes(a, 0, 5)
    a.scale = a.args.scale = float(np.float32(0.005 * 2.0 ** 123))
    compare(a)


def spread(a, low, high, seed):
    """Queries of one large number and others 2^-high .. 2^-low of it; keys are 0 where it is."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    big = torch.randint(0, a.D, (a.T, a.Hq), generator=g, device="cuda")
    big[:] = big[0, 0]  # every query's in one place, where all keys can be 0
    e = -low - (high - low) * torch.rand(a.q.shape, generator=g, device="cuda")
    sign = torch.randint(0, 2, a.q.shape, generator=g, device="cuda") * 2 - 1
    q = (sign * 1000.0 * torch.exp2(e)).to(a.q.dtype)
    q[:, :, big[0, 0]] = torch.where(sign[:, :, 0] > 0, 1000.0, 1999.0 / 2).to(a.q.dtype)
    a.q.copy_(q)
    for b in range(len(a.ctx)):
        page, row = a.rows[b]
        x = a.codes[0][page, row]
        x[:, :, big[0, 0]] = 0
        a.codes[0][page, row] = x
    return q


@pytest.mark.parametrize("new,Hq,Hkv,D", [([1, 1], 8, 1, 128), ([2, 2], 32, 4, 128), ([1, 2], 8, 2, 64), ([3, 9], 16, 2, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_queries_that_lie_far_apart(ft, new, Hq, Hkv, D, dtype):
    """Down to 2^-26 of the largest every number of a bf16 query has its say (f16: as far as its own range goes)."""
    low, high = (16.0, 26.0) if dtype == "bf16" else (12.0, 20.0)
    a = Attn(ft, [300, 70], new, Hq, Hkv, D, dtype, 32, 16, seed=9)
    spread(a, low, high, 3)
    a.scale = a.args.scale = float(np.float32(0.1 * 2.0 ** (low - 10)))
    compare(a, most=448 / 8 if dtype == "f16" else 0.0)


@pytest.mark.parametrize("high", [28, 30, 32])
@pytest.mark.parametrize("new,Hq,Hkv,D", [([1, 1], 8, 1, 128), ([2, 2], 32, 4, 128), ([1, 2], 8, 2, 64)])
def test_queries_further_apart(ft, high, new, Hq, Hkv, D):
    """Few rows take bf16 queries as f16 times a power of two: numbers below 2^-27 of the row's largest become multiples
    of at most 2^-34 of it, so a score is off by scale sum 2^-35 max |q| |k| over them."""
    a = Attn(ft, [300, 70], new, Hq, Hkv, D, "bf16", 32, 16, seed=9)
    spread(a, high - 0.5, high, 4)
    a.scale = 1.0
    weight = max(float(a.values(0, b).abs().sum(2).max()) for b in range(2))  # the largest sum |k|
    shift = 0.25  # of the worst score
    a.scale = a.args.scale = float(np.float32(shift / (weight * 2.0 ** -35 * 1000.0)))
    largest = a.q.float().abs().amax(2).double().cpu().numpy()
    compare(a, shift=a.scale * weight * 2.0 ** -35 * largest)
