"""Attention of batches whose sequences share their first tokens
(nf4_kv_attention_shared) against the plain one, sequence by sequence, within the
bounds of test_gpu_kv.py: the parts of a row's keys are summed apart and joined, which
those bounds' sums cover."""
import numpy as np
import pytest

from oracle import kv

from gpu_helpers import Side, say
from test_gpu_kv import SHAPES, Case, device_batch, device_cache, i32, rows_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def side():
    return Side()


SAVED = 64 << 20  # bytes of cache that taking the shared tokens apart has to save, by the bounds


class Shared(Case):
    """A Case whose sequences first[g] .. first[g + 1] - 1 have the same first
    prefix[g] tokens: whole pages shared, a page in part copied.  Its table has room for so
    many tokens that the shared ones are taken apart (`apart`: whether they can be)."""

    def __init__(self, side, seed, dim, page, heads, kv_heads, kv_len, count, first, prefix, roomy=True,
                 **kw):
        group = heads // kv_heads
        of = [sum(count[a:b]) for a, b in zip(first, first[1:])]
        self.most = max([1] + of)
        tiles = len(kv_len) * -(-max(count) * group // 16) - len(prefix) * -(-self.most * group // 64)
        self.tiles, self.apart = tiles, roomy and tiles > 0 and max(count) * group <= 128
        if self.apart:
            kw = {"stride_more": SAVED // (tiles * kv_heads * 2 * dim) // page + 2} | kw
        super().__init__(side, seed, dim, page, heads, kv_heads, kv_len, count, **kw)
        self.first, self.prefix = first, prefix
        for g, n in enumerate(prefix):
            a = first[g]
            for s in range(a + 1, first[g + 1]):
                own = min(n, self.kv_len[s], self.kv_len[a])  # what both have
                whole = own // page
                self.table[s, :whole] = self.table[a, :whole]
                for b in range(whole * page, own):  # the rest in copies, with their scales
                    p, q = self.table[a, b // page], self.table[s, b // page]
                    u = b % page
                    self.c.k[:, q, :, u] = self.c.k[:, p, :, u]
                    self.c.v[:, q, :, u // 4, :, u % 4] = self.c.v[:, p, :, u // 4, :, u % 4]
                    for x in (self.c.ks, self.c.vs):
                        x[:, q, :, u // 16] = x[:, p, :, u // 16]

    def run(self, window=0, sinks=0, scale=0.09, check=True, lse=True, stream=None, d=None, pad=8,
            max_rows=None, max_prefix=None, groups=None, **kw):
        side, t = self.side, self.side.torch
        d = d or device_cache(side, self.c)
        b = device_batch(side, self.table, self.kv_len, self.start,
                         **(({"max_len": 1 << 30} if self.apart else {}) | kw))
        g = groups or side.nf4.KVGroups(i32(side, self.prefix), i32(side, self.first),
                                        max_rows=self.most if max_rows is None else max_rows,
                                        max_prefix=max_prefix)
        q = rows_dev(side, self.q, pad, False)
        rows = self.q.shape[0]
        out = t.full((rows + 2, self.heads * self.dim), 7.0, dtype=t.bfloat16, device="cuda")
        z = t.full((rows + 2, self.heads), 7.0, dtype=t.float32, device="cuda") if lse else None
        n = side.nf4.nf4_kv_attention_shared_workspace_bytes(d, b, g, self.heads, window, sinks)
        # a slot of every part holds the sums of all rows and heads
        slots, rest = divmod(n, rows * self.heads * (self.dim + 2) * 4)
        alone = side.nf4.nf4_kv_attention_workspace_bytes(d, b, self.heads, window, sinks)
        seen = min(self.table.shape[1] * self.page, window or 1 << 30)
        if max_prefix is None and max_rows is None and "max_len" not in kw:
            if self.apart and seen > SAVED // (self.tiles * self.kv_heads * 2 * self.dim):
                assert rest == 0 and slots >= 2 and n != alone, "not taken apart"
            else:
                assert n == alone
        ws = t.full((max(n, 16) + 64,), 0xAB, dtype=t.uint8, device="cuda")
        stream = stream or side.stream
        stream.wait_stream(t.cuda.current_stream())
        say(f"[kv shared] dim={self.dim} page={self.page} heads={self.heads}/{self.kv_heads} "
            f"len={self.kv_len[:6]} rows={self.count[:6]} first={self.first} prefix={self.prefix} "
            f"window={window} sinks={sinks} apart={self.apart} ws={n}")
        side.nf4.nf4_kv_attention_shared(d, self.c.layers - 1, b, g, q, q.stride(0), self.heads, scale,
                                         window, sinks, out, z, ws, n, stream=stream)
        stream.synchronize()
        assert bool((ws[-64:] == 0xAB).all()) and bool((out[rows:] == 7).all())
        out = out[:rows].float().cpu().numpy().reshape(rows, self.heads, self.dim)
        z = z[:rows].cpu().numpy() if lse else None
        if check:
            self.check(out, z, window, sinks, scale)
        return out, z


# (lengths, groups' first sequences, shared tokens)
BATCHES = [([20, 21], [0, 2], [16]), ([40, 33, 64], [0, 3], [33]), ([1, 2, 3, 4], [0, 4], [1]),
           ([70, 130, 65, 64, 200, 90], [0, 2, 3, 6], [64, 10, 50]),
           ([300, 301, 280, 290, 5], [1, 3, 5], [250, 300])]


@pytest.mark.parametrize("dim,page,heads,kv_heads", SHAPES)
@pytest.mark.parametrize("kv_len,first,prefix", BATCHES)
def test_single_tokens(side, dim, page, heads, kv_heads, kv_len, first, prefix):
    Shared(side, 1, dim, page, heads, kv_heads, kv_len, [1] * len(kv_len), first, prefix).run()


@pytest.mark.parametrize("dim,page,heads,kv_heads", SHAPES)
@pytest.mark.parametrize("count", [[5, 5, 5, 5, 5, 5], [1, 0, 7, 3, 30, 2], [0, 16, 1, 16, 0, 17]])
def test_ragged_rows(side, dim, page, heads, kv_heads, count):
    """Few and many rows in a group and in a sequence, none in some."""
    Shared(side, 2, dim, page, heads, kv_heads, [150, 130, 165, 140, 200, 190], count, [0, 3, 6], [128, 101]).run()


@pytest.mark.parametrize("rows", [1, 4])
def test_many_rows_of_a_group(side, rows):
    """Groups over several tiles, the last ones in part; tokens that tiles end inside of."""
    rng = np.random.default_rng(3)
    n = 45
    kv_len = [int(x) for x in 100 + rng.integers(4, 60, n)]
    Shared(side, 3, 64, 16, 7, 1, kv_len, [rows] * n, [0, 40, 45], [97, 100]).run()


@pytest.mark.parametrize("count", [[1, 1, 1, 1], [5, 5, 5, 5], [40, 1, 3, 36]])
def test_rows_among_the_shared_tokens(side, count):
    """Sequences that are no longer than what they share, or end inside it: a row
    sees nothing past its position."""
    Shared(side, 4, 128, 16, 4, 2, [64, 40, 100, 65], count, [0, 4], [64]).run()
    Shared(side, 4, 128, 16, 4, 2, [64, 64, 64, 64], count, [0, 4], [64]).run()
    # longer than any sequence
    Shared(side, 4, 64, 16, 4, 2, [64, 64, 64, 64], count, [0, 4], [100]).run()


def test_nothing_shared_and_no_group(side):
    """Lengths of zero and less, sequences outside every group, groups without sequences."""
    for first, prefix in (([0, 5], [0]), ([0, 5], [-3]), ([2, 4], [30]), ([0, 0, 3, 3, 5], [10, 20, 5, 17]),
                          ([5, 5], [64]), ([0, 1, 2, 3, 4, 5], [64, 0, 64, 1, 16])):
        Shared(side, 5, 64, 16, 4, 2, [70, 80, 64, 65, 90], [1, 2, 1, 1, 3], first, prefix).run()


def test_first_tokens_of_all(side):
    """Without `first`: one group of all sequences; one row each without row_start."""
    c = Shared(side, 6, 128, 16, 8, 2, [90, 100, 110], [1, 1, 1], [0, 3], [80])
    g = side.nf4.KVGroups(i32(side, [80]))
    a, za = c.run(groups=g)
    b, zb = c.run()
    assert np.array_equal(a, b) and np.array_equal(za, zb)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 0), (64, 70), (100, 33), (150, 5),
                                          (1 << 40, 3), (5, 1 << 40), (40, 210)])
@pytest.mark.parametrize("count", [[1, 1, 1, 1], [3, 20, 1, 40]])
def test_windows(side, window, sinks, count):
    """Windows that end past, in and before what is shared, first tokens that pass it."""
    for dim, page, heads, kv_heads in ((128, 64, 7, 1), (64, 16, 8, 2)):
        Shared(side, 7, dim, page, heads, kv_heads, [260, 230, 400, 201], count, [0, 3, 4], [200, 64]).run(window, sinks)


@pytest.fixture(scope="module")
def long(side):
    """33 sequences of some 1400 tokens, all but one behind 1200 shared ones."""
    rng = np.random.default_rng(20)
    kv_len = [int(x) for x in 1201 + rng.integers(0, 250, 33)]
    count = [1, 3, 2] * 11
    c = Shared(side, 20, 128, 64, 16, 8, kv_len, count, [0, 32], [1200], stride_more=0)
    assert c.apart and SAVED // (c.tiles * 8 * 2 * 128) < 1100
    return c


@pytest.mark.parametrize("window,sinks", [(1 << 31, 0), (1100, 0), (1103, 1), (1150, 64), (1200, 70), (1201, 1300),
                                          (1300, 1199), (1400, 5)])
def test_windows_over_what_is_taken_apart(long, window, sinks):
    """Windows long enough for it, that begin in what is shared or before it."""
    long.run(window, sinks)


def test_bounds_as_they_are_taken_apart(long):
    """The parts of a call whose bounds are the lengths themselves."""
    long.run(max_len=max(long.kv_len), max_prefix=1200)


@pytest.mark.parametrize("count", [1, 9])
def test_long_prefix_in_parts(side, count):
    """A prefix over many parts, groups of few rows of a head and of many."""
    kv_len = [5200, 5101, 5300, 5111, 5105, 5106, 5120]
    Shared(side, 8, 64, 64, 4, 1, kv_len, [count] * 7, [0, 7], [5099]).run()
    Shared(side, 8, 64, 16, 1, 1, kv_len[:3], [count] * 3, [0, 3], [5099]).run(3000, 3)


@pytest.mark.parametrize("count", [1, 12])
def test_nan_and_infinity_stay_where_they_are_seen(side, count):
    """NaN among the shared tokens reaches the rows that see it, and only those; so do
    scores of infinity."""
    kv_len = [120, 100, 40, 119]
    for t, kind, seen in ((30, 1, True), (50, 0, True), (95, 1, True), (5, 0, False), (5, 1, False)):
        c = Shared(side, 9, 64, 16, 4, 2, kv_len, [count] * 4, [0, 4], [97])
        for s in range(4):
            if t < kv_len[s]:
                c.tokens(s, [t], kind, 0x7F, heads=[1])
        window = 0 if seen else 20
        out, z = c.run(window=window, check=False)
        at = np.concatenate([np.arange(n - count, n) for n in kv_len])
        hit = (at >= t) & ((at < t + window) if window else True)
        assert np.isnan(out[hit][:, 2:]).all() and not np.isnan(out[~hit]).any()
        assert not np.isnan(out[:, :2]).any()
        assert np.isnan(z[hit][:, 2:]).all() == (kind == 0) or not hit.any()


def test_holes_and_unwritten_scales(side):
    """Pages that are gone from the shared part and from the rest; scales that were never
    written, in places that no row sees."""
    c = Shared(side, 10, 128, 16, 8, 2, [100, 120, 90], [1, 3, 1], [0, 3], [80])
    c.table[:, 2] = -1
    c.table[1, 6] = 1000
    c.run()
    for bad in (np.nan, np.inf, -1.0, 0.0):
        c = Shared(side, 11, 128, 16, 8, 2, [101, 120, 90], [1, 3, 1], [0, 3], [81])
        for s, n in ((0, 101), (1, 120), (2, 90)):
            p = c.table[s, n // 16] if n % 16 == 0 else -1
            if p >= 0:
                c.c.ks[0, p] = c.c.vs[0, p] = bad
        c.run()


def test_scales_at_the_ends_of_their_range(side):
    """Values of the largest scale in the shared part, in the rest, in both: the parts'
    sums meet in range."""
    for where in ("shared", "rest", "both"):
        c = Shared(side, 12, 64, 16, 2, 1, [200, 180], [1, 2], [0, 2], [160])
        for s in (0, 1):
            for t in range(0, c.kv_len[s], 16):
                if (t < 160 and where != "rest") or (t >= 160 and where != "shared"):
                    c.c.vs[0, c.table[s, t // 16], :] = np.float32(2.0 ** 100)
                else:
                    c.c.vs[0, c.table[s, t // 16], :] = np.float32(2.0 ** -40)
        c.run(scale=0.05)


def test_large_scores(side):
    """Scores of thousands: what is shared outweighs the rest, and the other way round."""
    c = Shared(side, 13, 64, 16, 4, 2, [90, 100], [1, 1], [0, 2], [64])
    c.c.ks[:] = 2.0 ** -2
    c.run(scale=0.5)


@pytest.mark.parametrize("count,first,prefix", [([33, 70], [0, 2], [100]), ([1, 1], [0, 2], [100]),
                                                ([1, 1], [0, 1, 2], [100, 100])])
def test_as_without_sharing(side, count, first, prefix):
    """Sequences whose own rows fill tiles, and what saves little, go as without sharing."""
    c = Shared(side, 14, 64, 16, 4, 1, [140, 170], count, first, prefix, roomy=count[0] > 1)
    a, za = c.run()
    b, zb = Case.run(c)
    assert not c.apart and np.array_equal(a, b) and np.array_equal(za, zb)


@pytest.mark.parametrize("dim,page,heads,kv_heads", SHAPES)
def test_small_calls(side, dim, page, heads, kv_heads):
    for kv_len, first, prefix in BATCHES:
        Shared(side, 1, dim, page, heads, kv_heads, kv_len, [1] * len(kv_len), first, prefix, roomy=False).run()


def test_bounds_of_the_host(side):
    """max_prefix below a length cuts it; exact bounds change nothing but the order of
    sums; rows past max_rows do not see what is shared."""
    c = Shared(side, 15, 128, 16, 4, 2, [150, 140, 160], [1, 1, 1], [0, 3], [128])
    for m in (None, 128, 100, 17, 1, 0):
        c.run(max_prefix=m)
    for m in (3, 1000):
        c.run(max_rows=m)
    out, z = c.run(max_rows=2, check=False)
    full, zf = c.run()
    assert np.allclose(out[:2], full[:2], rtol=2.0 ** -6, atol=1e-2) and not np.allclose(z[2], zf[2], atol=1e-3)


def test_more_tokens_than_the_table(side):
    """Shared lengths past the table and past max_len."""
    c = Shared(side, 16, 64, 16, 4, 2, [64, 60], [1, 1], [0, 2], [1 << 30], stride_more=0)
    c.run()
    c.run(max_len=1 << 30)


def test_reproducible_and_without_lse(side):
    c = Shared(side, 17, 128, 64, 28, 4, [1100, 1030, 1050, 1026], [1, 1, 1, 1], [0, 4], [1024], layers=3)
    d = device_cache(side, c.c)
    runs = [c.run(d=d)[0] for _ in range(3)] + [c.run(d=d, lse=False, pad=64)[0]]
    for r in runs[1:]:
        assert np.array_equal(runs[0], r)


def test_in_a_replayed_graph(side):
    """Lengths, tables and what is shared change between replays; two graphs share a
    workspace, one after the other."""
    t, nf4 = side.torch, side.nf4
    c = Shared(side, 18, 128, 16, 8, 2, [150, 140, 160, 155], [1] * 4, [0, 4], [128],
               stride_more=SAVED // (2 * 2 * 2 * 128) // 16 + 2)
    d = device_cache(side, c.c)
    lens, table = i32(side, c.kv_len), i32(side, c.table)
    first, prefix = i32(side, [0, 4, 4]), i32(side, [128, 0])
    b = nf4.KVBatch(lens, table)
    g = nf4.KVGroups(prefix, first)
    q = side.to_dev(c.q).bfloat16()
    n = nf4.nf4_kv_attention_shared_workspace_bytes(d, b, g, 8)
    assert n != nf4.nf4_kv_attention_workspace_bytes(d, b, 8), "not taken apart"
    ws = t.full((n,), 0xFF, dtype=t.uint8, device="cuda")
    outs = [t.zeros(4, 8 * 128, dtype=t.bfloat16, device="cuda") for _ in range(3)]
    zs = [t.zeros(4, 8, device="cuda") for _ in range(3)]

    def step(i, scale, ws=ws):
        nf4.nf4_kv_attention_shared(d, 0, b, g, q, 1024, 8, scale, 0, 0, outs[i], zs[i], ws, n)
    graphs = [t.cuda.CUDAGraph() for _ in range(2)]
    t.cuda.synchronize()
    for i, graph in enumerate(graphs):
        with t.cuda.graph(graph):
            step(i, 0.09 * (i + 1))
    other = t.empty(n, dtype=t.uint8, device="cuda")
    for change in (lambda: None, lambda: prefix.copy_(i32(side, [100, 0])), lambda: lens.sub_(3),
                   lambda: first.copy_(i32(side, [0, 2, 4])), lambda: prefix.copy_(i32(side, [128, 64]))):
        change()
        q.mul_(1.0625)
        for i, graph in enumerate(graphs):
            graph.replay()
            t.cuda.synchronize()
            step(2, 0.09 * (i + 1), other)
            t.cuda.synchronize()
            assert t.equal(outs[i], outs[2]) and t.equal(zs[i], zs[2])


def test_forked_sequences(side):
    """A prompt forked into four that go on by a token each: what nf4_kv_attention says."""
    t, nf4 = side.torch, side.nf4
    rng = np.random.default_rng(19)
    kvh, dim, page, heads, n = 2, 64, 16, 8, 75
    cache = nf4.KVCache(1, 40, kvh, page, dim)
    i = lambda *a: t.tensor(a, dtype=t.int32, device="cuda")  # noqa: E731
    pool = nf4.KVPool(t.zeros(40, dtype=t.int32, device="cuda"),
                      t.full((5, 8), -1, dtype=t.int32, device="cuda"),
                      t.zeros(5, dtype=t.int32, device="cuda"), i(0))
    x = lambda r, w: side.to_dev(rng.normal(size=(r, w)).astype(np.float32))  # noqa: E731
    k, v = x(n, kvh * dim), x(n, kvh * dim)
    nf4.nf4_kv_reserve(cache, pool, i(n, 0, 0, 0, 0))
    one = nf4.KVBatch(pool.length[:1], pool.table[:1], row_start=i(0, n), rows=n, max_rows=n, max_len=n)
    nf4.nf4_kv_append(cache, 0, one, k, kvh * dim, v, kvh * dim, nf4.NF4_KV_F32)
    shared = pool.length[:1].clone()
    nf4.nf4_kv_fork(cache, pool, i(0, 0, 0, 0), i(1, 2, 3, 4), 4)
    nf4.nf4_kv_release(cache, pool, i(0), 1)
    b = nf4.KVBatch(pool.length[1:], pool.table[1:], max_len=128)
    g = nf4.KVGroups(shared)
    for step in range(20):
        nf4.nf4_kv_reserve(cache, pool, i(0, 1, 1, 1, 1))
        k, v, q = x(4, kvh * dim), x(4, kvh * dim), x(4, heads * dim).bfloat16()
        nf4.nf4_kv_append(cache, 0, b, k, kvh * dim, v, kvh * dim, nf4.NF4_KV_F32)
        res = []
        for f, size, more in ((nf4.nf4_kv_attention, nf4.nf4_kv_attention_workspace_bytes, ()),
                              (nf4.nf4_kv_attention_shared, nf4.nf4_kv_attention_shared_workspace_bytes, (g,))):
            ws_bytes = size(cache, b, *more, heads)
            ws = t.empty(max(16, ws_bytes), dtype=t.uint8, device="cuda")
            out, z = t.empty_like(q), t.empty(4, heads, device="cuda")
            f(cache, 0, b, *more, q, heads * dim, heads, 0.125, 0, 0, out, z, ws, ws_bytes)
            res.append((out.float(), z))
        t.cuda.synchronize()
        # both round weights and results to bf16: twice two half steps of values of up to 6
        assert float((res[0][0] - res[1][0]).abs().max()) <= 4 * 2.0 ** -8 * 6
        assert float((res[0][1] - res[1][1]).abs().max()) <= 1e-4


@pytest.mark.parametrize("dim,heads,kv_heads,count", [(128, 7, 1, [1] * 8), (64, 14, 2, [2] * 6),
                                                      (64, 4, 1, [12, 9, 12]), (128, 8, 2, [20, 1, 17])])
def test_weights_of_many_rows_keep_two_terms(side, dim, heads, kv_heads, count):
    """Groups and sequences of more than 32 rows of a kv head: as exact as few rows.  A result
    is within half a step of bf16 of a sum whose weights are within 2^-16 of theirs (each of
    the two roundings keeps 2^-8 of what it is given), its scores and sums as in `bounds`:
    with weights of one bf16 term a fifth of the results and more are not."""
    n = len(count)
    c = Shared(side, 21, dim, 16, heads, kv_heads, [300 + 7 * s + count[s] for s in range(n)], count, [0, n], [300])
    assert c.apart
    c.c.ks[:], c.c.vs[:] = 2.0 ** -8, 2.0 ** -6
    scale = float(np.float32(0.02))
    out, z = c.run(scale=scale)
    want, lse, mag, big = kv.attention(c.c, 0, c.table, c.start, c.kv_len,
                                       c.q.reshape(-1, heads, dim).astype(np.float64), scale, 0, 0)
    delta = 2.0 ** -24 * (2 * dim + 16) * big + 2.0 ** -21
    sums = (max(c.kv_len) / 8 + 200) * 2.0 ** -24
    off = mag * (2.0 ** -16 + 2 * delta[..., None] + 2 * sums) * 1.01
    assert off.max() < 2.0 ** -12 * mag.max()  # so that one term shows
    half = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(out), 2.0 ** -100))) - 8)
    bad = np.abs(out - want) > half + off
    assert not bad.any(), f"{bad.sum()} of {bad.size} past the bound"


def shorter(c, s, n):
    """Sequence s of a case has n tokens left, and pages for no more."""
    c.kv_len[s] = n
    c.table[s, -(-n // c.page):] = -1


@pytest.mark.parametrize("window,sinks", [(0, 0), (1 << 40, 3)])
@pytest.mark.parametrize("dim,heads,kv_heads,count", [(128, 4, 2, 1), (64, 7, 1, 2), (64, 4, 1, 12)])
@pytest.mark.parametrize("left", [[(0, 0)], [(0, 0), (1, 0), (2, 40)], [(0, 40)], [(0, 0), (4, 17), (5, 0)],
                                  [(s, n) for s, n in enumerate((50, 0, 90, 90, 17, 90))]])
def test_groups_whose_first_sequence_ended(side, left, dim, heads, kv_heads, count, window, sinks):
    """Released sequences stay in the batch with no tokens, others fall behind: the rest see
    what they share all the same, from the pages of one that has it, or most of it."""
    c = Shared(side, 22, dim, 16, heads, kv_heads, [130, 140, 133, 150, 120, 125], [count] * 6, [0, 4, 6], [100, 101])
    for s, n in left:
        shorter(c, s, n)
    c.run(window, sinks)


@pytest.mark.parametrize("count", [1, 3])
def test_many_sequences_ended(side, count):
    """More of them than lanes before the first that is left; none that has all of it."""
    for last in (90, 60):
        c = Shared(side, 23, 64, 16, 2, 1, [90 + count] * 140, [count] * 140, [0, 140], [90])
        for s in range(140):
            shorter(c, s, 0 if s < 133 else 30 if s % 2 else last)
        c.run()


def test_first_sequence_released_between_replays(side):
    """A captured step goes on after a fork's first branch is released."""
    t, nf4 = side.torch, side.nf4
    c = Shared(side, 24, 128, 16, 8, 2, [150, 140, 160, 155], [1] * 4, [0, 4], [128],
               stride_more=SAVED // (2 * 2 * 2 * 128) // 16 + 2)
    d = device_cache(side, c.c)
    lens, table = i32(side, c.kv_len), i32(side, c.table)
    b, g = nf4.KVBatch(lens, table), nf4.KVGroups(i32(side, [128]), i32(side, [0, 4]))
    q = side.to_dev(c.q).bfloat16()
    n = nf4.nf4_kv_attention_shared_workspace_bytes(d, b, g, 8)
    assert n != nf4.nf4_kv_attention_workspace_bytes(d, b, 8), "not taken apart"
    ws = t.full((n,), 0xFF, dtype=t.uint8, device="cuda")
    out, z = t.zeros(4, 8 * 128, dtype=t.bfloat16, device="cuda"), t.zeros(4, 8, device="cuda")
    graph = t.cuda.CUDAGraph()
    t.cuda.synchronize()
    with t.cuda.graph(graph):
        nf4.nf4_kv_attention_shared(d, 0, b, g, q, 1024, 8, 0.09, 0, 0, out, z, ws, n)
    for s in (None, 0, 1):
        if s is not None:
            shorter(c, s, 0)
            lens[s], table[s] = 0, -1
        graph.replay()
        t.cuda.synchronize()
        c.check(out.float().cpu().numpy().reshape(4, 8, 128), z.cpu().numpy(), 0, 0, 0.09)
