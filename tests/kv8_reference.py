"""The 8-bit paged cache in plain numpy, 64 bits, one block after another."""
import numpy as np

# the largest number of the 16-bit types
MOST = {"bf16": (2 - 2.0 ** -7) * 2.0 ** 127, "f16": 65504.0}


def decode_table():
    t = np.zeros(256)
    for c in range(256):
        s, e, m = (-1.0 if c & 128 else 1.0), (c >> 3) & 15, c & 7
        t[c] = np.nan if (c & 127) == 127 else s * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return t


VALUE = decode_table()


def encode(y):
    """Codes of the numbers y (|y| <= 448), nearest, ties to even; not finite: 0x7F."""
    y = np.asarray(y, dtype=np.float64)
    fin = np.isfinite(y)
    a = np.where(fin, np.abs(y), 0.0)
    ex = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6)
    n = np.rint(a / 2.0 ** (ex - 3)).astype(np.int64)  # eighths of the binade; 16 carries into the next one
    code = np.where(n >= 8, ((ex + 7).astype(np.int64) << 3) + (n - 8), n)
    assert (code[fin] <= 126).all()
    code = code | np.where(np.signbit(y), 128, 0)
    return np.where(fin, code, 127).astype(np.uint8)


def power(e):
    return 2.0 ** (float(e) - 127.0)


def least_byte(most):
    e = 0
    while most > 448.0 * power(e):
        e += 1
    return e


class Cache:
    """codes [page, row, head, D], scale [page, block, head] of keys and of values."""

    def __init__(self, codes, scale, block):
        self.codes, self.scale, self.block = [c.copy() for c in codes], [s.copy() for s in scale], block

    def store(self, rows, dtype, ctx, new, table):
        """rows: two [T, head, D] arrays; returns the status bits' names."""
        said = set()
        pages, P, heads, _ = self.codes[0].shape
        t0 = 0
        for b, (c, n) in enumerate(zip(ctx, new)):
            at = c
            while at < c + n:
                first = at // self.block * self.block
                end = min(c + n, first + self.block)
                page = table[b][at // P] if at // P < len(table[b]) else -1
                if not 0 <= page < pages:
                    said.add("slot")
                    at = end
                    continue
                j, r0 = first % P // self.block, first % P
                for kv in range(2):
                    for h in range(heads):
                        x = rows[kv][t0 + at - c:t0 + end - c, h]
                        fin = np.abs(x[np.isfinite(x)])
                        need = least_byte(fin.max() if fin.size else 0.0)
                        codes = self.codes[kv][page, :, h]
                        was = int(self.scale[kv][page, j, h])
                        e = need
                        if at > first:
                            old = codes[r0:r0 + at - first]
                            if was == 255:
                                said.add("nan")
                                old[:] = 127
                            else:
                                e = max(was, need)
                                if e != was:
                                    old[:] = encode(VALUE[old] * 2.0 ** (was - e))
                        y = x * 2.0 ** (127.0 - e)
                        if 256 * power(e) > MOST[dtype]:
                            y = np.where(np.isfinite(y), np.clip(y, -240, 240), y)
                        codes[at % P:at % P + end - at] = encode(y)
                        self.scale[kv][page, j, h] = e
                at = end
            t0 += n
        return said

    def values(self, kv):
        """[page, row, head, D] numbers."""
        s = np.where(self.scale[kv] == 255, np.nan, 2.0 ** (self.scale[kv].astype(np.float64) - 127))
        return VALUE[self.codes[kv]] * np.repeat(s, self.block, axis=1)[..., None]
