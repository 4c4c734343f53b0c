"""The 8-bit key-value cache on the GPU against the plain one (oracle/kv.py):
codes and page tables byte for byte, attention within bounds derived from its
roundings."""
import numpy as np
import pytest

from oracle import kv

from gpu_helpers import Side, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def side():
    return Side()


def bf16(x):
    """x rounded to bfloat16 (to even), as float32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def device_cache(side, c):
    d = {n: side.to_dev(a) for n, a in c.arrays().items()}
    return side.nf4.KVCache(c.layers, c.pages, c.kv_heads, c.page, c.dim, **d)


def i32(side, a):
    return side.to_dev(np.ascontiguousarray(a, np.int32))


def device_batch(side, table, kv_len, row_start, **kw):
    counts = np.diff(row_start)
    kw = dict(rows=max(1, int(row_start[-1])), max_rows=max(1, int(counts.max())),
              max_len=int(max(kv_len))) | kw
    return side.nf4.KVBatch(i32(side, kv_len), i32(side, table), row_start=i32(side, row_start), **kw)


def rows_dev(side, x, pad, f32):
    """Rows of x [rows][width] as a strided slice of a wider device tensor
    filled with NaN, in bfloat16 or fp32."""
    t = side.torch
    w = t.full((x.shape[0], x.shape[1] + 2 * pad), float("nan"),
               dtype=t.float32 if f32 else t.bfloat16, device="cuda")
    w[:, pad:pad + x.shape[1]] = side.to_dev(np.asarray(x, np.float32))
    return w[:, pad:pad + x.shape[1]]


def same_cache(c, d):
    """Byte for byte, NaN codes of either sign alike."""
    for n, a in c.arrays().items():
        got = getattr(d, n).cpu().numpy()
        if a.dtype == np.uint8:
            a, got = (np.where(z & 127 == 127, 127, z) for z in (a, got))
        bad = np.argwhere(a != got)
        assert not len(bad), f"{n}: {len(bad)} differ, first at {bad[0]}: {got[tuple(bad[0])]} for {a[tuple(bad[0])]}"


def pages_for(rng, kv_len, page, extra=2, stride_more=1):
    need = [-(-max(int(n), 0) // page) for n in kv_len]
    pages = max(1, sum(need)) + extra
    order = rng.permutation(pages)
    table = np.full((len(kv_len), max(1, max(need)) + stride_more), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return pages, table


# ---------------------------------------------------------------- append
# (lengths after the call, new rows of each)
APPENDS = [([1], [1]), ([17], [1]), ([16], [16]), ([31], [30]), ([40, 0, 5], [3, 0, 5]),
           ([129, 64, 65, 200], [128, 1, 2, 77])]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, 3), (128, 64, 1), (128, 16, 2), (64, 256, 2)])
@pytest.mark.parametrize("kv_len,count", APPENDS)
def test_append(side, f32, dim, page, heads, kv_len, count):
    rng = np.random.default_rng(dim + page + len(kv_len) + kv_len[0])
    pages, table = pages_for(rng, kv_len, page)
    c = kv.Cache(2, pages, heads, page, dim, rng)
    d = device_cache(side, c)
    start = np.concatenate([[0], np.cumsum(count)])
    x = [rng.normal(size=(start[-1], heads * dim)) * 2.0 ** rng.integers(-6, 7, (start[-1], 1))
         for _ in range(2)]
    x = [(z.astype(np.float32) if f32 else bf16(z)) for z in x]
    say(f"[kv append] f32={f32} dim={dim} page={page} {kv_len} {count}")
    b = device_batch(side, table, kv_len, start)
    k, v = rows_dev(side, x[0], 8, f32), rows_dev(side, x[1], 16, f32)
    side.stream.wait_stream(side.torch.cuda.current_stream())
    side.nf4.nf4_kv_append(d, 1, b, k, k.stride(0), v, v.stride(0), int(f32), stream=side.stream)
    side.sync()
    kv.append(c, 1, table, start, kv_len, *(z.reshape(-1, heads, dim).astype(np.float64) for z in x))
    same_cache(c, d)


def test_append_token_by_token_and_special_values(side):
    """40 single tokens whose sizes grow and shrink by powers of two, zeros,
    infinities, NaN, subnormals and the largest floats among them."""
    rng = np.random.default_rng(5)
    dim, heads, page, n = 64, 2, 16, 40
    pages, table = pages_for(rng, [n], page)
    c = kv.Cache(1, pages, heads, page, dim, rng)
    d = device_cache(side, c)
    x = rng.normal(size=(n, heads * dim)) * 2.0 ** rng.integers(-30, 30, (n, 1))
    x[3], x[17, :64], x[18] = 0.0, 0.0, 1e-45
    x[5, 7], x[6, 9], x[9, 70], x[21, 0] = np.nan, np.inf, -np.inf, 3.4e38
    x[25] = np.nan
    x[30, :] = 448.0 * 2.0 ** 5
    x[31, ::2] = 2.0 ** -10 * 2.0 ** 5
    x[33] = -2.0 ** -140
    x = x.astype(np.float32)
    for t in range(n):
        b = device_batch(side, table, [t + 1], [0, 1])
        r = side.to_dev(x[t:t + 1])
        side.nf4.nf4_kv_append(d, 0, b, r, heads * dim, r, heads * dim, side.nf4.NF4_KV_F32,
                               stream=side.stream)
        side.sync()
        y = x[t:t + 1].reshape(1, heads, dim).astype(np.float64)
        kv.append(c, 0, table, [0, 1], [t + 1], y, y)
    same_cache(c, d)


def test_append_leaves_holes_and_what_is_no_token(side):
    """Holes and ids past the pool in the table, more rows than tokens, more
    rows than max_rows, more tokens than max_len or than the table holds:
    nothing is written there."""
    rng = np.random.default_rng(6)
    dim, heads, page = 128, 1, 16
    table = np.array([[0, -1, 2], [3, 900, 4], [5, 6, 7], [8, 9, 10]], np.int32)
    c = kv.Cache(1, 12, heads, page, dim, rng)
    d = device_cache(side, c)
    kv_len, count = [48, 40, 5, 48], [48, 40, 9, 20]
    start = np.concatenate([[0], np.cumsum(count)])
    x = rng.normal(size=(start[-1], heads * dim)).astype(np.float32)
    b = device_batch(side, table, kv_len, start)
    r = side.to_dev(x)
    side.nf4.nf4_kv_append(d, 0, b, r, dim, r, dim, 1, stream=side.stream)
    side.sync()
    y = x.reshape(-1, heads, dim).astype(np.float64)
    kv.append(c, 0, table, start, kv_len, y, y)
    same_cache(c, d)
    # bounds of the host's that are too small cut off what lies past them
    b = device_batch(side, table, [60, 40, 5, 48], start, max_rows=7, max_len=41)
    side.nf4.nf4_kv_append(d, 0, b, r, dim, r, dim, 1, stream=side.stream)
    side.sync()
    for s, n in enumerate([41, 40, 5, 41]):
        begin = n - count[s]
        lo = max(begin, 0)
        hi = min(n, begin + 7)
        if hi > lo:
            kv.append(c, 0, table[s:s + 1], [0, hi - lo], [hi], y[start[s] + lo - begin:start[s] + hi - begin],
                      y[start[s] + lo - begin:start[s] + hi - begin])
    same_cache(c, d)


# ------------------------------------------------------------- attention
def bounds(dim, keys, out, lse, mag, big):
    """What the roundings may add up to.  A weight w = 2^(t - m + e): t is an
    fp32 sum of `dim` exact products (each partial sum within `big` in natural
    units, twice 2^-24 of it per addition covers a scaled and fused form), a
    few fp32 operations on |t| <= big log2(e) follow, and exp2 is good to
    2^-21.  The weights are rounded to bf16 and so is the result: 8 significant
    bits, half a unit in the last place is up to 2^-8 of the value (1 + 2^-8
    becomes 1).  Sums over the keys are fp32 in pieces of 16 or more, joined in
    up to a hundred steps more."""
    delta = 2.0 ** -24 * (2 * dim + 16) * big + 2.0 ** -21
    sums = (keys / 8 + 200) * 2.0 ** -24
    tol = mag * (2.0 ** -8 + 2 * delta[..., None] + 2 * sums) * 1.01 + np.abs(out) * 2.0 ** -8 * 1.01 + 1e-30
    with np.errstate(invalid="ignore"):
        tol_lse = delta + sums + np.abs(np.where(np.isfinite(lse), lse, 0)) * 2.0 ** -21
    return tol, tol_lse


class Case:
    def __init__(self, side, seed, dim, page, heads, kv_heads, kv_len, count, layers=1, stride_more=1):
        self.side, self.dim, self.page, self.heads, self.kv_heads = side, dim, page, heads, kv_heads
        self.kv_len, self.count = list(kv_len), list(count)
        self.rng = rng = np.random.default_rng(seed)
        self.pages, self.table = pages_for(rng, kv_len, page, stride_more=stride_more)
        # random codes everywhere, NaN among them; the sequences' own tokens are finite
        self.c = kv.Cache(layers, self.pages, kv_heads, page, dim, rng)
        self.start = np.concatenate([[0], np.cumsum(count)])
        for s, n in enumerate(kv_len):
            for t in range(n):
                for h in range(kv_heads):
                    for w in (0, 1):
                        code = self.c.codes(w, layers - 1, self.table[s, t // page], h, t % page)
                        code[code & 127 == 127] = 0x30
        rows = max(1, int(self.start[-1]))
        self.q = bf16(rng.normal(size=(rows, heads * dim)) * 4)

    def tokens(self, s, ts, kind, value, heads=None):
        """Set the codes of tokens of a sequence."""
        for t in ts:
            for h in range(self.kv_heads) if heads is None else heads:
                self.c.codes(kind, self.c.layers - 1, self.table[s, t // self.page], h, t % self.page)[:] = value

    def run(self, window=0, sinks=0, scale=0.09, check=True, lse=True, stream=None, d=None, pad=8, **kw):
        side, t = self.side, self.side.torch
        d = d or device_cache(side, self.c)
        b = device_batch(side, self.table, self.kv_len, self.start, **kw)
        q = rows_dev(side, self.q, pad, False)
        rows = self.q.shape[0]
        out = t.full((rows, self.heads * self.dim), 7.0, dtype=t.bfloat16, device="cuda")
        z = t.full((rows, self.heads), 7.0, dtype=t.float32, device="cuda") if lse else None
        n = side.nf4.nf4_kv_attention_workspace_bytes(d, b, self.heads, window, sinks)
        ws = t.full((max(n, 16),), 0xAB, dtype=t.uint8, device="cuda")
        stream = stream or side.stream
        stream.wait_stream(t.cuda.current_stream())
        say(f"[kv attention] dim={self.dim} page={self.page} heads={self.heads}/{self.kv_heads} "
            f"len={self.kv_len[:6]} rows={self.count[:6]} window={window} sinks={sinks} ws={n}")
        side.nf4.nf4_kv_attention(d, self.c.layers - 1, b, q, q.stride(0), self.heads, scale, window,
                                  sinks, out, z, ws, n, stream=stream)
        stream.synchronize()
        out = out.float().cpu().numpy().reshape(rows, self.heads, self.dim)
        z = z.cpu().numpy() if lse else None
        if check:
            self.check(out, z, window, sinks, scale)
        return out, z

    def check(self, out, z, window, sinks, scale):
        q = self.q.reshape(-1, self.heads, self.dim).astype(np.float64)
        scale = float(np.float32(scale))
        want, lse, mag, big = kv.attention(self.c, self.c.layers - 1, self.table, self.start,
                                           self.kv_len, q, scale, window, sinks)
        n = int(self.start[-1])
        tol, tol_lse = bounds(self.dim, max(self.kv_len), want, lse, mag, big)
        nan = np.isnan(want[:n])
        assert np.array_equal(np.isnan(out[:n]), nan)
        bad = ~nan & (np.abs(out[:n] - want[:n]) > tol[:n])
        assert not bad.any(), f"{bad.sum()} past the bound, worst {np.nanmax(np.abs(out[:n] - want[:n]) / tol[:n])}"
        if z is not None:
            empty = np.isneginf(lse[:n])
            assert np.array_equal(np.isneginf(z[:n]), empty)
            ok = ~empty & ~np.isnan(lse[:n])
            assert (np.abs(z[:n][ok] - lse[:n][ok]) <= tol_lse[:n][ok]).all()


SHAPES = [(128, 16, 4, 4), (64, 64, 7, 1), (128, 32, 8, 2), (64, 16, 14, 2), (128, 128, 20, 1)]


@pytest.mark.parametrize("dim,page,heads,kv_heads", SHAPES)
@pytest.mark.parametrize("kv_len", [[1], [15, 16, 17], [31, 33, 0, 64, 65, 1], [500, 2, 129]])
def test_single_tokens(side, dim, page, heads, kv_heads, kv_len):
    c = Case(side, 1, dim, page, heads, kv_heads, kv_len, [1 if n else 0 for n in kv_len])
    c.run()


@pytest.mark.parametrize("dim,page,heads,kv_heads", SHAPES)
@pytest.mark.parametrize("kv_len,count", [([5], [5]), ([33, 64], [33, 3]), ([130, 0, 70, 16], [130, 0, 66, 16]),
                                          ([300], [41]), ([257], [257])])
def test_prompts_and_chunks(side, dim, page, heads, kv_heads, kv_len, count):
    Case(side, 2, dim, page, heads, kv_heads, kv_len, count).run()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 0), (64, 70), (100, 33), (1 << 40, 3),
                                          (5, 1 << 40)])
@pytest.mark.parametrize("kv_len,count", [([400, 31], [1, 1]), ([400, 90], [150, 90])])
def test_windows(side, window, sinks, kv_len, count):
    for dim, page, heads, kv_heads in ((128, 64, 7, 1), (64, 16, 8, 2)):
        Case(side, 3, dim, page, heads, kv_heads, kv_len, count).run(window, sinks)


def test_window_far_into_a_long_cache(side):
    """Rows near the end of 5000 tokens that see a window and first tokens:
    the pages between them may be gone."""
    for count in (1, 40):
        c = Case(side, 4, 64, 16, 4, 2, [5000], [count])
        c.table[0, 3:290] = -1
        c.run(200, 20)


def test_rows_that_see_nothing(side):
    # more rows than tokens: the first ones stand before the sequence
    for kv_len, count in (([3], [7]), ([0], [1]), ([2, 0, 40], [40, 3, 64])):
        c = Case(side, 5, 128, 16, 4, 2, kv_len, count)
        out, z = c.run()
        assert np.isneginf(z[0]).all() and not out[0].any()
    # every page a hole
    c = Case(side, 6, 64, 16, 4, 2, [100], [30])
    c.table[:] = -1
    out, z = c.run()
    assert np.isneginf(z).all() and not out.any()
    # a hole in the middle, an id past the pool
    for count in (1, 60):
        c = Case(side, 7, 64, 16, 4, 2, [100], [count])
        c.table[0, 2], c.table[0, 4] = -1, c.pages
        c.run()


@pytest.mark.parametrize("count", [1, 50])
def test_nan_and_infinity_stay_where_they_are_seen(side, count):
    """NaN codes in keys and values of tokens outside a window, after a row,
    and inside: only the rows that see them are NaN (a value's NaN only in
    its own element)."""
    c = Case(side, 8, 128, 16, 6, 2, [200], [count])
    c.tokens(0, [20, 90], 0, 0x7F)
    c.tokens(0, [30, 95], 1, 0xFF)
    out, _ = c.run(60, 4)
    assert not np.isnan(out[-1]).any()
    c.tokens(0, [198], 0, 0xFF, heads=[1])
    out, z = c.run(60, 4)
    assert np.isnan(out[-1, 3:]).all() and not np.isnan(out[-1, :3]).any()
    c = Case(side, 9, 64, 32, 2, 2, [200], [count])
    c.c.codes(1, 0, c.table[0, 198 // 32], 0, 198 % 32)[5] = 0x7F
    out, z = c.run()
    assert np.isnan(out[-1, 0, 5]) and not np.isnan(out[-1, 1]).any() and not np.isnan(z).any()
    assert np.isnan(out[-1, 0]).sum() == 1 and (count == 1 or not np.isnan(out[:-2]).any())


def test_scales_at_the_ends_of_their_range(side):
    """Blocks of zeros (the least scale) beside blocks of ordinary and of huge
    values: every key keeps its weight in the sum."""
    for count in (1, 40):
        c = Case(side, 10, 128, 16, 4, 2, [150], [count])
        c.c.k[:], c.c.ks[:] = c.c.k & 0x3F, 2.0 ** -8
        for t in range(0, 150, 48):
            p = c.table[0, t // 16]
            c.c.vs[0, p], c.c.v[0, p] = 2.0 ** -40, 0
            c.c.ks[0, p], c.c.k[0, p] = 2.0 ** -40, 0
        c.run()
        c.c.vs[0, c.table[0, 2]] = 2.0 ** 60
        c.run()


def test_large_scores(side):
    """Scores of several hundreds, growing and falling along the keys."""
    for count in (1, 70):
        c = Case(side, 11, 64, 64, 4, 1, [700], [count])
        c.c.ks[:] = 2.0 ** -3
        c.run(scale=0.2)


def test_strides_streams_lse_and_layers(side):
    t = side.torch
    c = Case(side, 12, 128, 64, 8, 2, [300, 70], [1, 1], layers=3, stride_more=5)
    a, z = c.run(pad=64)
    b, _ = c.run(lse=False, pad=0, stream=t.cuda.Stream())
    assert np.array_equal(a, b)
    for _ in range(3):
        x, y = c.run(check=False)
        assert np.array_equal(a, x) and np.array_equal(z, y)
    # bounds above what the sequences have change nothing but the launch
    x, y = c.run(max_len=4000)
    c = Case(side, 13, 64, 16, 4, 2, [90, 33], [64, 33])
    c.run()
    c.run(max_rows=97, max_len=1 << 30)


def test_more_rows_and_tokens_than_the_bounds(side):
    c = Case(side, 14, 64, 16, 4, 2, [90, 33], [64, 33])
    full, _ = c.run()
    x, _ = c.run(check=False, max_rows=20)
    assert np.array_equal(np.abs(x[:20] - full[:20]) <= 2.0 ** -6 * np.abs(full[:20]) + 1e-2, np.ones_like(x[:20], bool))
    assert (x[20:64] == 7.0).all() and (x[84:] == 7.0).all()
    x, _ = c.run(check=False, max_len=80)
    c.kv_len = [80, 33]
    c.check(x, None, 0, 0, 0.09)


def test_long_sequence_and_split(side):
    """One and three rows against 9001 tokens, a heavy key near the start, the
    middle and the end."""
    for heads, kv_heads, count in ((7, 1, [1, 1]), (4, 1, [3, 1]), (16, 2, [1, 2]), (8, 1, [5, 5])):
        c = Case(side, 15, 64, 64, heads, kv_heads, [9001, 40], count)
        for tok in (3, 4500, 8990):
            c.tokens(0, [tok], 0, 0x50)
        c.run()
    Case(side, 16, 128, 16, 4, 1, [3001, 700, 1500], [33, 64, 1]).run()


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64)])
def test_more_tiles_than_compute_units(side, dim, page):
    """320 tiles of rows: one team of waves each, the keys unsplit; with a
    window, holes and NaN in unseen places."""
    kv_len = [1 + (37 * i) % 90 for i in range(40)]
    count = [min(n, 1 + (23 * i) % 50) for i, n in enumerate(kv_len)]
    c = Case(side, 21, dim, page, 8, 8, kv_len, count)
    c.run()
    c.run(20, 3)
    c.tokens(4, [1, kv_len[4] - 1], 1, 0x7F)
    c.table[7, 0] = -1
    c.run(20, 1)
    Case(side, 22, dim, page, 6, 3, [300] * 90, [17] * 90).run()


@pytest.mark.parametrize("dim,page,heads,kv_heads", [(128, 32, 2, 2), (64, 16, 7, 1)])
def test_rows_that_end_inside_tiles(side, dim, page, heads, kv_heads):
    """Sequences of one to several tiles that end in any part of the last one."""
    count = [64, 65, 128, 129, 192, 193, 300, 1, 0, 33]
    c = Case(side, 24, dim, page, heads, kv_heads,
             [n + (41 * i) % 130 for i, n in enumerate(count)], count)
    c.run()
    c.run(70, 2)
    c.table[5, 1] = c.table[6, 7] = -1
    c.run()


def test_many_short_sequences(side):
    """4800 (sequence, head) pairs of single tokens, some without a token."""
    kv_len = [(7 * i) % 45 for i in range(600)]
    c = Case(side, 23, 64, 16, 8, 8, kv_len, [1 if n else 0 for n in kv_len])
    c.run()


def test_offsets_past_32_bits(side):
    """A cache whose codes pass 4 GiB: pages at its end are read and written."""
    t = side.torch
    dim, page, heads = 128, 256, 8
    pages = (1 << 32) // (page * dim * heads) + 40
    d = side.nf4.KVCache(1, pages, heads, page, dim)
    n = 600
    table = np.array([[pages - 1, 5, pages - 7]], np.int32)
    rng = np.random.default_rng(17)
    x = [bf16(rng.normal(size=(n, heads * dim))) for _ in range(2)]
    k, v = (side.to_dev(z).to(t.bfloat16) for z in x)
    side.stream.wait_stream(t.cuda.current_stream())
    b = device_batch(side, table, [n], [0, n])
    side.nf4.nf4_kv_append(d, 0, b, k, heads * dim, v, heads * dim, 0, stream=side.stream)
    side.sync()
    # a small cache with the same three pages
    c = kv.Cache(1, 3, heads, page, dim)
    small = np.array([[0, 1, 2]], np.int32)
    idx = t.from_numpy(table[0].astype(np.int64)).cuda()
    for name, a in c.arrays().items():
        a[0] = getattr(d, name)[0].index_select(0, idx).cpu().numpy()
    want = kv.Cache(1, 3, heads, page, dim)
    kv.append(want, 0, small, [0, n], [n], *(z.reshape(n, heads, dim).astype(np.float64) for z in x))
    for name, a in want.arrays().items():
        assert np.array_equal(a, c.arrays()[name]), name
    case = Case(side, 18, dim, page, heads, heads, [n], [1])
    case.c, case.table = c, small
    ref, z_ref = case.run()
    case.table = table
    got, z = case.run(check=False, d=d)
    assert np.array_equal(ref, got) and np.array_equal(z_ref, z)


def test_attention_in_a_replayed_graph(side):
    """Append and attention captured once: the lengths live on the device, so
    every replay takes the next token."""
    t, nf4 = side.torch, side.nf4
    c = Case(side, 19, 128, 16, 8, 2, [2000], [1])
    d, b = device_cache(side, c.c), device_batch(side, c.table, [1990], [0, 1], max_len=2000)
    k = t.zeros(1, 256, dtype=t.bfloat16, device="cuda")
    q, out = t.zeros(1, 1024, dtype=t.bfloat16, device="cuda"), t.zeros(1, 1024, dtype=t.bfloat16, device="cuda")
    n = nf4.nf4_kv_attention_workspace_bytes(d, b, 8)
    ws = t.zeros(max(n, 16), dtype=t.uint8, device="cuda")

    def step():
        nf4.nf4_kv_append(d, 0, b, k, 256, k, 256, nf4.NF4_KV_BF16, stream=side.stream)
        nf4.nf4_kv_attention(d, 0, b, q, 1024, 8, 0.09, 0, 0, out, None, ws, n, stream=side.stream)

    side.stream.wait_stream(t.cuda.current_stream())
    side.sync()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=side.stream):
        step()
    side.sync()
    rng = np.random.default_rng(20)
    for length in range(1990, 1994):
        x, y = (bf16(rng.normal(size=(1, w))) for w in (256, 1024))
        with t.cuda.stream(side.stream):
            k.copy_(side.to_dev(x))
            q.copy_(side.to_dev(y))
            b.kv_len.fill_(length)
            out.zero_()
            g.replay()
        side.sync()
        got = out.float().cpu().numpy()
        kv.append(c.c, 0, c.table, [0, 1], [length], *(x.reshape(1, 2, 128).astype(np.float64),) * 2)
        c.kv_len, c.q = [length], y
        c.check(got.reshape(1, 8, 128), None, 0, 0, 0.09)
        same_cache(c.c, d)
        with t.cuda.stream(side.stream):
            step()
        side.sync()
        assert np.array_equal(got, out.float().cpu().numpy())


# ------------------------------------------------------------------ pool
class PoolCase:
    def __init__(self, side, pages, rows, stride, page=16, layers=2, kv_heads=1, dim=64, seed=0):
        self.side = side
        self.rng = np.random.default_rng(seed)
        self.c = kv.Cache(layers, pages, kv_heads, page, dim, self.rng)
        self.p = kv.Pool(pages, rows, stride, page)
        self.d = device_cache(side, self.c)
        self.pool = side.nf4.KVPool(i32(side, self.p.refs), i32(side, self.p.table),
                                    i32(side, self.p.len), i32(side, [0]))
        self.ws = side.torch.full((side.nf4.nf4_kv_compact_workspace_bytes(self.d),), 0xAB,
                                  dtype=side.torch.uint8, device="cuda")

    def do(self, op, *a):
        nf4, side = self.side.nf4, self.side
        dev = [i32(side, x) for x in a]
        side.stream.wait_stream(side.torch.cuda.current_stream())
        if op == "reserve":
            nf4.nf4_kv_reserve(self.d, self.pool, *dev, stream=side.stream)
            self.p.reserve(*a)
        elif op == "fork":
            nf4.nf4_kv_fork(self.d, self.pool, *dev, len(a[0]), stream=side.stream)
            self.p.fork(*a, caches=[self.c])
        elif op == "release":
            nf4.nf4_kv_release(self.d, self.pool, *dev, len(a[0]), stream=side.stream)
            self.p.release(*a)
        else:
            nf4.nf4_kv_compact(self.d, self.pool, self.pool.refs, self.pool.table, self.ws,
                               self.ws.numel(), stream=side.stream)
            self.p.compact([self.c])
        side.sync()
        for name in ("refs", "table"):
            got = getattr(self.pool, name).cpu().numpy()
            assert np.array_equal(got, getattr(self.p, name)), (op, a, name)
        assert np.array_equal(self.pool.length.cpu().numpy(), self.p.len), (op, a)
        if op in ("reserve", "fork"):
            assert int(self.pool.missing) == self.p.missing, (op, a)
        same_cache(self.c, self.d)


@pytest.mark.parametrize("pages,rows,stride,page", [(1, 1, 1, 16), (40, 6, 8, 16), (33, 12, 5, 64),
                                                    (70, 9, 20, 32)])
def test_pool_random_steps(side, pages, rows, stride, page):
    c = PoolCase(side, pages, rows, stride, page, seed=pages)
    rng = c.rng
    for step in range(40):
        say(f"[kv pool] pages={pages} step {step}")
        op = rng.choice(["reserve", "reserve", "fork", "release", "compact"])
        empty = [r for r in range(rows) if c.p.len[r] == 0]
        full = [r for r in range(rows) if c.p.len[r]]
        if op == "reserve":
            c.do(op, np.where(rng.random(rows) < 0.5, rng.integers(-3, 3 * page, rows), 0))
        elif op == "fork" and empty and full:
            n = int(rng.integers(1, len(empty) + 1))
            c.do(op, [int(rng.choice(full)) for _ in range(n)], [int(x) for x in rng.permutation(empty)[:n]])
        elif op == "release" and full:
            n = int(rng.integers(1, len(full) + 1))
            c.do(op, [int(x) for x in rng.permutation(full)[:n]])
        elif op == "compact":
            c.do(op)


def test_pool_rows_outside_the_table_and_named_twice(side):
    c = PoolCase(side, 20, 5, 4, seed=1)
    c.do("reserve", [20, 33, 16, 0, 0])
    c.do("fork", [0, 7, 1, -1], [3, 4, 9, 2])
    c.do("release", [3, 8, -2])
    # the plain pool takes a row's second mention as the empty row it then is
    c.do("release", [1, 1, 0])


def test_pool_of_many_pages_and_rows(side):
    """More than one pass of the planning workgroup over rows and over pages."""
    rng = np.random.default_rng(3)
    c = PoolCase(side, 40000, 2600, 20, page=16, layers=1, seed=2)
    c.do("reserve", rng.integers(0, 320, 2600))
    c.do("release", rng.permutation(2600)[:1500])
    c.do("fork", list(np.nonzero(c.p.len)[0][:1050]), list(np.nonzero(c.p.len == 0)[0][:1050]))
    c.do("compact")
    c.do("reserve", rng.integers(0, 100, 2600))


def test_copy_pages(side):
    t = side.torch
    rng = np.random.default_rng(4)
    for page, heads, dim, layers in ((16, 1, 64, 1), (256, 3, 128, 3)):
        c = kv.Cache(layers, 12, heads, page, dim, rng)
        d = device_cache(side, c)
        src, dst = [3, 4, -1, 5, 12, 3], [0, 11, 2, 99, 6, 7]
        side.nf4.nf4_kv_copy_pages(d, i32(side, src), i32(side, dst), 6, stream=side.stream)
        side.sync()
        for a, b in ((3, 0), (4, 11), (3, 7)):
            for x in c.arrays().values():
                x[:, b] = x[:, a]
        same_cache(c, d)


def test_compact_out_of_place_leaves_the_pool(side):
    c = PoolCase(side, 30, 4, 8, seed=5)
    c.do("reserve", [100, 90, 33, 64])
    c.do("release", [0, 2])
    refs, table = (x.clone() for x in (c.pool.refs, c.pool.table))
    r, tb = side.torch.empty_like(refs), side.torch.empty_like(table)
    side.stream.wait_stream(side.torch.cuda.current_stream())
    for _ in range(2):  # the sources are kept, so again gives the same
        side.nf4.nf4_kv_compact(c.d, c.pool, r, tb, c.ws, c.ws.numel(), stream=side.stream)
    side.sync()
    assert side.torch.equal(refs, c.pool.refs) and side.torch.equal(table, c.pool.table)
    c.p.compact([c.c])
    assert np.array_equal(r.cpu().numpy(), c.p.refs) and np.array_equal(tb.cpu().numpy(), c.p.table)
    same_cache(c.c, c.d)
