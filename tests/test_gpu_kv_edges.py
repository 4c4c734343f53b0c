"""The 8-bit key-value cache where it holds little or unusual things."""
import numpy as np
import pytest

from oracle import kv

from gpu_helpers import say
from test_gpu_kv import Case, PoolCase, bf16, bounds, device_batch, device_cache, i32, same_cache, side  # noqa: F401

pytestmark = pytest.mark.gpu


def move_page(c, page, to):
    """The case's pages `page` and `to` change places."""
    if page != to:
        for a in c.c.arrays().values():
            a[:, [page, to]] = a[:, [to, page]]
        was = c.table.copy()
        c.table[was == page], c.table[was == to] = to, page


def never_written(c, value):
    """Blocks that no token of the case's sequences lies in get the scale
    `value`."""
    written = np.zeros((c.pages, c.page // kv.BLOCK), bool)
    for s, n in enumerate(c.kv_len):
        for t in range(0, n, kv.BLOCK):
            written[c.table[s, t // c.page], t % c.page // kv.BLOCK] = True
    for a in (c.c.ks, c.c.vs):
        a[:] = np.where(written[None, :, None], a, np.float32(value))


# (heads, kv heads, lengths, rows): two teams of waves, with the keys split, one team
FORMS = [(14, 2, [40, 100], [40, 100]), (7, 1, [10], [10]), (4, 1, [1100, 3], [40, 3]),
         (8, 8, [40 + i for i in range(40)], [33] * 40)]


@pytest.mark.parametrize("value", [0.0, np.nan, -1.0, np.inf])
@pytest.mark.parametrize("dim,page", [(128, 64), (64, 256)])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_scales_of_blocks_that_were_never_written(side, form, dim, page, value):
    """Page 0 in use but not full, page 0 in nobody's use, and holes."""
    heads, kv_heads, kv_len, count = FORMS[form]
    c = Case(side, 30, dim, page, heads, kv_heads, kv_len, count)
    last = (kv_len[0] - 1) // page
    move_page(c, c.table[0, last], 0)
    never_written(c, value)
    say(f"[kv never written] page 0 in part, scale {value}")
    c.run()
    c.run(20, 3)
    free = next(p for p in range(c.pages) if p not in c.table)
    move_page(c, 0, free)
    say(f"[kv never written] page 0 free, scale {value}")
    c.run()
    c.run(20, 3)
    c.table[0, 0] = -1
    c.run()


def test_a_prompt_on_a_new_cache(side):
    """As a first call meets it: a cache filled with zeros, 40 tokens in 64-token
    pages, appended and attended to."""
    t, nf4 = side.torch, side.nf4
    rng = np.random.default_rng(31)
    heads, kv_heads, dim, page, n = 28, 4, 128, 64, 40
    c, d = kv.Cache(1, 3, kv_heads, page, dim), nf4.KVCache(1, 3, kv_heads, page, dim)
    table = np.array([[0]], np.int32)
    x = [bf16(rng.normal(size=(n, kv_heads * dim))) for _ in range(2)]
    k, v = (side.to_dev(z).to(t.bfloat16) for z in x)
    side.stream.wait_stream(t.cuda.current_stream())
    nf4.nf4_kv_append(d, 0, device_batch(side, table, [n], [0, n]), k, kv_heads * dim, v,
                      kv_heads * dim, nf4.NF4_KV_BF16, stream=side.stream)
    side.sync()
    kv.append(c, 0, table, [0, n], [n], *(z.reshape(n, kv_heads, dim).astype(np.float64) for z in x))
    same_cache(c, d)
    case = Case(side, 32, dim, page, heads, kv_heads, [n], [n])
    case.c, case.table = c, table
    case.run(d=d)


# -------------------------------------------------- NaN in all that a row sees
def run_nan(c, *a, **kw):
    """The case's check, and lse NaN just where the plain one is."""
    out, z = c.run(*a, **kw)
    q = c.q.reshape(-1, c.heads, c.dim).astype(np.float64)
    with np.errstate(invalid="ignore"):
        lse = kv.attention(c.c, 0, c.table, c.start, c.kv_len, q, float(np.float32(0.09)), *(a or (0, 0)))[1]
    assert np.array_equal(np.isnan(z), np.isnan(lse))
    return out, z


# one wave, single tokens, single tokens over split keys, two teams, split, one team
NAN_FORMS = [(4, 2, [20], [1]), (4, 2, [200, 64], [1, 1]), (4, 1, [5001], [2]), (8, 2, [200, 70], [50, 70]),
             (4, 1, [1500], [40]), (8, 8, [40] * 40, [33] * 40)]


@pytest.mark.filterwarnings("ignore:invalid value")
@pytest.mark.parametrize("form", range(len(NAN_FORMS)))
@pytest.mark.parametrize("dim", [64, 128])
def test_rows_whose_scores_are_all_nan(side, form, dim):
    """A query with NaN in it, and one whose scores are all -infinity, come out
    as NaN, lse too, however the call is split."""
    heads, kv_heads, kv_len, count = NAN_FORMS[form]
    c = Case(side, 33, dim, 64, heads, kv_heads, kv_len, count)
    c.q.reshape(-1, heads, dim)[-1, 1, 3] = np.nan
    out, z = run_nan(c)
    assert np.isnan(out[-1, 1]).all() and np.isnan(z[-1, 1]) and not np.isnan(z[-1, 0])
    run_nan(c, 25, 2)
    c = Case(side, 34, dim, 64, heads, kv_heads, kv_len, count)
    c.c.k[..., 5] = c.c.k[..., 5] & 0x7F | 0x08  # positive and not 0
    c.c.k[c.c.k == 127] = 0x38
    row = c.q.reshape(-1, heads, dim)[-1, 1]
    row[:] = 0.0
    row[5] = -np.inf
    out, z = run_nan(c)
    assert np.isnan(out[-1, 1]).all() and np.isnan(z[-1, 1]) and not np.isnan(z[-1, 0])


@pytest.mark.filterwarnings("ignore:invalid value")
@pytest.mark.parametrize("form", range(len(NAN_FORMS)))
def test_keys_that_are_all_nan_in_a_part(side, form):
    """NaN keys wherever one wave, one team or one part of split keys looks:
    the rows that see them are NaN, lse too."""
    heads, kv_heads, kv_len, count = NAN_FORMS[form]
    c = Case(side, 35, 64, 64, heads, kv_heads, kv_len, count)
    n = kv_len[0]
    for lo, hi in ((0, 1), (0, 32), (32, 64), (64, 128), (0, 2048), (2048, 5001), (0, n)):
        if lo >= n:
            continue
        was = c.c.k.copy()
        c.tokens(0, range(lo, min(hi, n)), 0, 0x7F, heads=[0])
        out, z = run_nan(c)
        assert np.isnan(z[count[0] - 1, 0])
        run_nan(c, 16, 1)
        c.c.k[:] = was


def test_one_token_whose_key_is_nan(side):
    c = Case(side, 36, 64, 16, 4, 2, [1], [1])
    c.tokens(0, [0], 0, 0xFF)
    out, z = run_nan(c)
    assert np.isnan(out).all() and np.isnan(z).all()


# ------------------------------------------- sequences longer than their tables
def with_holes(table, entries):
    """The table with entries that name no page after its own."""
    return np.concatenate([table, np.full((len(table), entries), -1, np.int32)], 1)


@pytest.mark.parametrize("kv_len,count", [([49, 40], [1, 1]), ([60, 48], [20, 7]), ([48, 200], [48, 40]),
                                          ([100, 49], [100, 49])])
@pytest.mark.parametrize("max_len", [None, 48, 1000])
def test_sequences_longer_than_their_tables(side, kv_len, count, max_len):
    """Tokens past the table are dropped as in a hole, and every row keeps its
    position."""
    rng = np.random.default_rng(40)
    dim, heads, page = 64, 2, 16
    table = np.array([[4, 1, 6], [0, 5, 2]], np.int32)
    c = kv.Cache(1, 8, heads, page, dim, rng)
    start = np.concatenate([[0], np.cumsum(count)])
    x = bf16(rng.normal(size=(start[-1], heads * dim)))
    d = device_cache(side, c)
    b = device_batch(side, table, kv_len, start, max_len=max_len)
    r = side.to_dev(x)
    side.stream.wait_stream(side.torch.cuda.current_stream())
    side.nf4.nf4_kv_append(d, 0, b, r, heads * dim, r, heads * dim, 1, stream=side.stream)
    side.sync()
    y = x.reshape(-1, heads, dim).astype(np.float64)
    kv.append(c, 0, with_holes(table, 20), start, kv_len, y, y)
    same_cache(c, d)
    for a in (c.k, c.v):
        a[a & 127 == 127] = 0x30
    for group in (1, 8, 24):
        case = Case(side, 41, dim, page, heads * group, heads, kv_len, count)
        case.c, case.pages = c, 8
        for window, sinks in ((0, 0), (5, 0), (9, 40), (30, 3)):
            case.table = table
            out, z = case.run(window, sinks, check=False, max_len=max_len)
            case.table = with_holes(table, 20)
            case.check(out, z, window, sinks, 0.09)


def test_a_long_sequence_past_its_table(side):
    """Keys in parts, the window past what the table holds."""
    for count in (1, 40):
        for length in (4097, 9000):
            c = Case(side, 42, 64, 64, 4, 1, [4096], [1], stride_more=0)
            c.kv_len, c.count, c.start = [length], [count], np.array([0, count])
            c.q = bf16(c.rng.normal(size=(count, 4 * 64)) * 4)
            table = c.table
            for window, sinks in ((0, 0), (300, 5), (4950, 0), (100, 1 << 40)):
                c.table = table
                out, z = c.run(window, sinks, check=False, max_len=None)
                c.table = with_holes(table, 80)
                c.check(out, z, window, sinks, 0.09)


def test_fork_and_go_on_past_a_full_table(side):
    """Both rows of a fork whose pages are all shared outgrow the table: no code
    of the shared pages changes."""
    c = PoolCase(side, 12, 3, 3, page=16, layers=1, seed=6)
    c.do("reserve", [48, 20, 0])
    c.do("fork", [0], [2])
    c.do("reserve", [1, 1, 1])
    assert c.p.missing == 2 and c.p.len.tolist() == [49, 21, 49]
    t = side.torch
    for max_len in (1 << 30, 48):
        b = side.nf4.KVBatch(c.pool.length, c.pool.table, max_len=max_len)
        x = t.randn(3, 64, device="cuda")
        side.stream.wait_stream(t.cuda.current_stream())
        side.nf4.nf4_kv_append(c.d, 0, b, x, 64, x, 64, side.nf4.NF4_KV_F32, stream=side.stream)
        side.sync()
        y = x.double().cpu().numpy().reshape(3, 1, 64)
        kv.append(c.c, 0, with_holes(c.p.table, 2), [0, 1, 2, 3], c.p.len, y, y)
        same_cache(c.c, c.d)


# ------------------------------------------------------------ the largest scale
@pytest.mark.parametrize("heads,kv_heads,kv_len,count,low", [
    (1, 1, [8192], [1], 512),                          # single token, the keys split
    (1, 1, [9000], [40], 512),                         # two teams, split
    (8, 8, [6000] + [9] * 19, [33] + [9] * 19, 10000),  # two teams, not split
    (8, 8, [6000] + [9] * 39, [33] + [9] * 39, 10000)])  # one team
def test_largest_values_over_many_keys(side, heads, kv_heads, kv_len, count, low):
    """Values of 448 * 2^100 under thousands of equal weights, the first keys of
    every `low` of them 2^-7.9 as heavy: the result is as large as the values,
    and no sum on the way overflows."""
    c = Case(side, 37, 64, 64, heads, kv_heads, kv_len, count)
    c.q[:] = 0.0
    c.q.reshape(-1, heads, 64)[..., 0] = 1.0
    n = kv_len[0]
    for page in c.table[0, :-(-n // 64)]:
        c.c.k[0, page], c.c.v[0, page] = 0, 0x7E
        c.c.ks[0, page], c.c.vs[0, page] = 1.0, 2.0 ** 100
    for t in range(n):
        if t % low >= 128:
            for h in range(kv_heads):
                c.c.codes(0, 0, c.table[0, t // 64], h, t % 64)[0] = 0x38
    out, z = c.run(scale=7.9 * np.log(2))
    assert np.isfinite(out).all() and np.isfinite(z).all()


@pytest.mark.parametrize("columns", [slice(0, 3), slice(2, 5), slice(6, 9)])
def test_tables_that_are_columns_of_wider_ones(side, columns):
    """Entries beside the view are other things' pages: sequences end with the view."""
    rng = np.random.default_rng(60)
    dim, heads, page = 64, 2, 16
    wide = rng.permutation(27).reshape(3, 9).astype(np.int32)
    kv_len, count = [48, 61, 200], [1, 20, 1]
    c = kv.Cache(1, 27, heads, page, dim, rng)
    d, t = device_cache(side, c), side.torch
    start = np.concatenate([[0], np.cumsum(count)])
    x = bf16(rng.normal(size=(start[-1], heads * dim)))
    r, view = side.to_dev(x), i32(side, wide)[:, columns]
    side.stream.wait_stream(t.cuda.current_stream())
    b = side.nf4.KVBatch(i32(side, kv_len), view, row_start=i32(side, start), rows=int(start[-1]), max_rows=20)
    side.stream.wait_stream(t.cuda.current_stream())
    side.nf4.nf4_kv_append(d, 0, b, r, heads * dim, r, heads * dim, 1, stream=side.stream)
    side.sync()
    table = with_holes(wide[:, columns], 20)
    y = x.reshape(-1, heads, dim).astype(np.float64)
    kv.append(c, 0, table, start, kv_len, y, y)
    same_cache(c, d)
    for a in (c.k, c.v):
        a[a & 127 == 127] = 0x30
    d = device_cache(side, c)
    for group in (1, 8):
        h = heads * group
        case = Case(side, 61, dim, page, h, heads, kv_len, count)
        case.c, case.table, case.pages = c, table, 27
        q = side.to_dev(case.q).bfloat16()
        out, lse = t.empty_like(q), t.empty(len(q), h, dtype=t.float32, device="cuda")
        n = side.nf4.nf4_kv_attention_workspace_bytes(d, b, h)
        ws = t.empty(max(n, 16), dtype=t.uint8, device="cuda")
        side.stream.wait_stream(t.cuda.current_stream())
        say(f"[kv columns] {columns} group {group}")
        side.nf4.nf4_kv_attention(d, 0, b, q, h * dim, h, 0.09, 0, 0, out, lse, ws, n, stream=side.stream)
        side.sync()
        case.check(out.float().cpu().numpy().reshape(-1, h, dim), lse.cpu().numpy(), 0, 0, 0.09)


def test_one_long_prompt_among_many_short_sequences(side):
    """A batch whose bound on rows makes many tiles, most of them empty."""
    t, nf4 = side.torch, side.nf4
    rng = np.random.default_rng(50)
    heads, kv_heads, dim, page, n, others = 128, 8, 64, 64, 2000, 63
    pages = -(-n // page) + others
    c = kv.Cache(1, pages, kv_heads, page, dim, rng)
    for a in (c.k, c.v):
        a[a & 127 == 127] = 0x30
    table = np.full((1 + others, -(-n // page)), -1, np.int32)
    table[0] = np.arange(others, pages)
    table[1:, 0] = np.arange(others)
    d = device_cache(side, c)
    q = side.to_dev(rng.normal(size=(n + others, heads * dim)).astype(np.float32)).bfloat16()

    def run(rows, kv_len, start):
        b = device_batch(side, table[rows], kv_len, start)
        qs = q[:start[-1]]
        out = t.empty_like(qs)
        ws_bytes = nf4.nf4_kv_attention_workspace_bytes(d, b, heads)
        ws = t.empty(max(ws_bytes, 16), dtype=t.uint8, device="cuda")
        side.stream.wait_stream(t.cuda.current_stream())
        say(f"[kv ragged] sequences={len(kv_len)} rows={start[-1]} ws={ws_bytes}")
        nf4.nf4_kv_attention(d, 0, b, qs, qs.stride(0), heads, 0.1, 0, 0, out, None, ws, ws_bytes,
                             stream=side.stream)
        side.sync()
        return out
    short = [1 + i % page for i in range(others)]
    both = run(slice(0, 1 + others), [n] + short, np.concatenate([[0], n + np.arange(1 + others)]))
    alone = run(slice(0, 1), [n], np.array([0, n]))
    assert t.equal(both[:n], alone)
    case = Case(side, 51, dim, page, heads, kv_heads, short, [1] * others)
    case.c, case.table, case.pages = c, table[1:], pages
    case.q = q[n:].float().cpu().numpy()
    case.check(both[n:].float().cpu().numpy().reshape(others, heads, dim), None, 0, 0, 0.1)


def test_reserve_counts_past_31_bits(side):
    """Rows that ask for far more than there is: lengths and the count of
    missing pages stop at 2^31 - 1."""
    t, nf4 = side.torch, side.nf4
    d = nf4.KVCache(1, 8, 1, 16, 64)
    rows, top = 40, 2 ** 31 - 1
    pool = nf4.KVPool(i32(side, np.zeros(8)), i32(side, np.full((rows, 2), -1)),
                      i32(side, np.arange(rows)), i32(side, [5]))
    add = i32(side, np.full(rows, top))
    side.stream.wait_stream(t.cuda.current_stream())
    for _ in range(2):
        nf4.nf4_kv_reserve(d, pool, add, stream=side.stream)
        side.sync()
        assert pool.length.tolist() == [top] * rows
        assert int(pool.missing) == top
    assert pool.refs.tolist() == [1] * 8
    # row 0 has no token yet, the others one page that this call did not have to give
    assert pool.table.flatten().tolist()[:6] == [0, 1, -1, 2, -1, 3]


@pytest.mark.parametrize("window,sinks", [(0, 0), (1 << 40, 0), (1 << 31, 3), (1, 1 << 40)])
def test_lengths_at_the_end_of_their_type(side, window, sinks):
    """Rows at positions past 2^30 see what the table holds, and nothing is
    written there."""
    rng = np.random.default_rng(70)
    dim, heads, page = 64, 2, 16
    table = np.array([[4, 1, 6], [0, 5, 2]], np.int32)
    for group, count in ((1, 1), (24, 2)):
        case = Case(side, 71, dim, page, heads * group, heads, [48, 48], [count, count])
        case.c, case.table, case.pages = kv.Cache(1, 8, heads, page, dim, rng), table, 8
        for a in (case.c.k, case.c.v):
            a[a & 127 == 127] = 0x30
        case.kv_len = [2 ** 31 - 1, 2 ** 30 + 5]
        out, z = case.run(window, sinks, check=False, max_len=None)
        case.kv_len, case.table = [48 + count] * 2, with_holes(table, 3)
        case.check(out, z, 0, 0, 0.09)  # as rows just past the table that see it all
        d = device_cache(side, case.c)
        x = side.to_dev(np.ones((2 * count, heads * dim), np.float32))
        b = device_batch(side, table, [2 ** 31 - 1, 2 ** 30 + 5], case.start, max_len=None)
        side.stream.wait_stream(side.torch.cuda.current_stream())
        side.nf4.nf4_kv_append(d, 0, b, x, heads * dim, x, heads * dim, 1, stream=side.stream)
        side.sync()
        same_cache(case.c, d)


@pytest.mark.parametrize("form", range(len(NAN_FORMS)))
@pytest.mark.parametrize("first", [True, False])
def test_scores_past_the_least_float_have_no_weight(side, form, first):
    """Keys whose scores are under -2^128 (-infinity in 32 bits), before or
    after all others: the rest of the keys make the result."""
    heads, kv_heads, kv_len, count = NAN_FORMS[form]
    page = 16
    n = kv_len[0]
    c = Case(side, 38, 64, page, heads, kv_heads, kv_len, count)
    c.c.k[..., 5] = 0
    c.q.reshape(-1, heads, 64)[..., 5] = -2.0 ** 33
    # (the last row of sequence 0 sees other keys in either case)
    entries = range(0, max(1, n // 3 // page)) if first else range((n - 1) // page - max(0, n // 3 // page), (n - 1) // page)
    for e in entries:
        p = c.table[0, e]
        c.c.k[0, p], c.c.ks[0, p] = 0, 2.0 ** 100
        c.c.k[0, p, :, :, 5] = 0x7E
    out, z = c.run(check=False)
    rows = count[0]
    c.table[0, entries.start:entries.stop] = -1  # as if they were not there
    q = c.q.reshape(-1, heads, 64).astype(np.float64)
    want, lse, mag, big = kv.attention(c.c, 0, c.table, c.start, c.kv_len, q, float(np.float32(0.09)), 0, 0)
    ok = ~np.isneginf(lse[:rows])  # rows that see nothing else are 0 / 0
    tol, tol_lse = bounds(64, n, want, lse, mag, big)
    assert ok[-1].all()
    assert (np.abs(out - want) <= tol)[:rows][ok].all()
    assert (np.abs(z - lse) <= tol_lse)[:rows][ok].all()
