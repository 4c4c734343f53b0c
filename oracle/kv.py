"""Plain statement of the 8-bit key-value cache in numpy, 64-bit arithmetic.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  A cache is kept as
bytes in the layout of include/nf4.h, so results compare byte for byte; every
operation is a loop over tokens, rows or pages with the definition in it.

Page cited: the vibevoice.c README (the KV cache in FP8 and in pages); the
block format and the pool's rules are the library's own.
"""
from __future__ import annotations

import numpy as np

BLOCK = 16
EXP_MIN, EXP_MAX = -40, 100


def e4m3_values() -> np.ndarray:
    """The 256 values: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        out[c] = np.nan if (c & 127) == 127 else x
        if c >= 128:
            out[c] = -out[c]
    return out


VALUES = e4m3_values()


def encode(x) -> np.ndarray:
    """Codes nearest to x, ties to the even code; past +-448 as +-448, NaN as
    0x7F with x's sign dropped."""
    x = np.asarray(x, np.float64)
    top = VALUES[:127]  # ascending, code = index
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0)), 448.0)
    hi = np.clip(np.searchsorted(top, a), 1, 126)
    lo = hi - 1
    dl, dh = a - top[lo], top[hi] - a  # exact: few bits each
    code = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    code = code | (np.signbit(x) * 128)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def exponent(amax: float) -> int:
    """The least e with amax <= 448 2^e, held to the format's range."""
    e = EXP_MIN
    while e < EXP_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


class Cache:
    """Bytes of a cache; k [L][P][H][page][D], v [L][P][H][page/4][D][4]."""

    def __init__(self, layers, pages, kv_heads, page, dim, rng=None):
        self.page, self.dim, self.kv_heads, self.pages, self.layers = page, dim, kv_heads, pages, layers
        lead = (layers, pages, kv_heads)
        if rng is None:
            self.k = np.zeros(lead + (page, dim), np.uint8)
            self.v = np.zeros(lead + (page // 4, dim, 4), np.uint8)
            self.ks = np.zeros(lead + (page // BLOCK,), np.float32)
            self.vs = np.zeros(lead + (page // BLOCK,), np.float32)
        else:
            self.k = rng.integers(0, 256, lead + (page, dim), dtype=np.uint8)
            self.v = rng.integers(0, 256, lead + (page // 4, dim, 4), dtype=np.uint8)
            self.ks = (2.0 ** rng.integers(-9, -5, lead + (page // BLOCK,))).astype(np.float32)
            self.vs = (2.0 ** rng.integers(-9, -5, lead + (page // BLOCK,))).astype(np.float32)

    def arrays(self):
        return {"k": self.k, "v": self.v, "k_scale": self.ks, "v_scale": self.vs}

    def codes(self, kv, layer, page, head, token):
        """View of one token's codes."""
        if kv == 0:
            return self.k[layer, page, head, token]
        return self.v[layer, page, head, token // 4, :, token % 4]

    def dense(self, kv, layer, head, table_row, n):
        """The values [n][D] of a sequence's first n tokens, and which are holes."""
        out = np.zeros((n, self.dim))
        hole = np.zeros(n, bool)
        scale = self.vs if kv else self.ks
        for t in range(n):
            p = int(table_row[t // self.page])
            if not 0 <= p < self.pages:
                hole[t] = True
                continue
            u = t % self.page
            out[t] = VALUES[self.codes(kv, layer, p, head, u)] * float(scale[layer, p, head, u // BLOCK])
        return out, hole


def append(c: Cache, layer, table, row_start, kv_len, k, v):
    """k, v: float64 [rows][kv_heads][D]."""
    for s in range(len(kv_len)):
        r0, r1 = int(row_start[s]), int(row_start[s + 1])
        begin = int(kv_len[s]) - (r1 - r0)
        new = [t for t in range(max(begin, 0), int(kv_len[s]))]
        for b in sorted({t // BLOCK for t in new}):
            toks = [t for t in new if t // BLOCK == b]
            p = int(table[s][b * BLOCK // c.page])
            if not 0 <= p < c.pages:
                continue
            blk = b * BLOCK % c.page // BLOCK
            kept = range(b * BLOCK, toks[0])
            for h in range(c.kv_heads):
                for kv, x, scale in ((0, k, c.ks), (1, v, c.vs)):
                    rows = np.stack([x[r0 + t - begin, h] for t in toks])
                    fin = np.abs(rows[np.isfinite(rows)])
                    e = exponent(fin.max() if fin.size else 0.0)
                    if len(kept):
                        was = int(np.log2(float(scale[layer, p, h, blk])))
                        e = max(e, was)
                        if e != was:
                            for t in kept:
                                old = c.codes(kv, layer, p, h, t % c.page)
                                old[:] = encode(VALUES[old] * 2.0 ** (was - e))
                    for t, row in zip(toks, rows):
                        c.codes(kv, layer, p, h, t % c.page)[:] = encode(row * 2.0 ** -e)
                    scale[layer, p, h, blk] = 2.0 ** e


def attention(c: Cache, layer, table, row_start, kv_len, q, scale, window, sinks):
    """q: float64 [rows][heads][D].  Returns out, lse and, for the error
    bounds, sum w |v| / l, max_j sum_d |q k| scale, and the number of keys."""
    rows, heads, dim = q.shape
    group = heads // c.kv_heads
    out = np.zeros((rows, heads, dim))
    lse = np.full((rows, heads), -np.inf)
    mag, big = np.zeros((rows, heads, dim)), np.zeros((rows, heads))
    for s in range(len(kv_len)):
        n, r0, r1 = int(kv_len[s]), int(row_start[s]), int(row_start[s + 1])
        if n == 0 or r1 == r0:
            continue
        t = np.arange(n)
        for h in range(c.kv_heads):
            k, hole = c.dense(0, layer, h, table[s], n)
            v, _ = c.dense(1, layer, h, table[s], n)
            for r in range(r0, r1):
                at = n - (r1 - r0) + r - r0
                see = (t <= at) & ~hole
                if window:
                    see &= (t > at - window) | (t < sinks)
                if not see.any():
                    continue
                for i in range(h * group, (h + 1) * group):
                    x = k[see] @ q[r, i] * scale
                    m = x.max()
                    w = np.exp(x - m)
                    out[r, i] = w @ v[see] / w.sum()
                    lse[r, i] = m + np.log(w.sum())
                    mag[r, i] = w @ np.abs(v[see]) / w.sum()
                    big[r, i] = (np.abs(k[see]) @ np.abs(q[r, i])).max() * scale
    return out, lse, mag, big


class Pool:
    """Page ownership as lists."""

    def __init__(self, pages, rows, stride, page):
        self.refs = np.zeros(pages, np.int32)
        self.table = np.full((rows, stride), -1, np.int32)
        self.len = np.zeros(rows, np.int32)
        self.page, self.missing = page, 0

    def _take(self):
        for p, r in enumerate(self.refs):
            if r == 0:
                self.refs[p] = 1
                return p
        self.missing += 1
        return -1

    def reserve(self, add):
        self.missing = 0
        for r, more in enumerate(add):
            if more <= 0:
                continue
            for e in range(-(-int(self.len[r]) // self.page), -(-int(self.len[r] + more) // self.page)):
                if e >= self.table.shape[1]:
                    self.missing += 1
                else:
                    self.table[r, e] = self._take()
            self.len[r] += more

    def fork(self, src, dst, caches=()):
        self.missing = 0
        pairs = [(a, d) for a, d in zip(src, dst)
                 if 0 <= a < len(self.table) and 0 <= d < len(self.table)]
        for a, d in pairs:
            n = int(self.len[a])
            full = n // self.page
            self.table[d] = -1
            if n % self.page and full < self.table.shape[1] and self.table[a, full] >= 0:
                p = self.table[d, full] = self._take()
                for c in caches:
                    if p >= 0:
                        for x in c.arrays().values():
                            x[:, p] = x[:, self.table[a, full]]
            self.len[d] = n
        for a, d in pairs:
            for e in range(int(self.len[a]) // self.page):
                self.table[d, e] = self.table[a, e]
                if self.table[a, e] >= 0:
                    self.refs[self.table[a, e]] += 1

    def release(self, rows):
        for r in rows:
            if not 0 <= r < len(self.table):
                continue
            for e in range(self.table.shape[1]):
                if self.table[r, e] >= 0:
                    self.refs[self.table[r, e]] -= 1
            self.table[r] = -1
            self.len[r] = 0

    def compact(self, caches=()):
        n = int((self.refs > 0).sum())
        src = [p for p in range(n, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(n) if self.refs[p] <= 0]
        for a, b in zip(src, dst):
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.table[self.table == a] = b
            for c in caches:
                for x in c.arrays().values():
                    x[:, b] = x[:, a]
