"""Rotary positions, norms of heads, the append that does both, and reading the cache
back, against 64-bit arithmetic (oracle/rotary.py, oracle/kv.py).

Bounds.  A turned value is a c - b s (or a s + b c) with c and s rounded to fp32
from sums that are right to 2^-28, a product and a sum rounded to fp32: at most
(|a| + |b|) gain 2^-24 for each of c and s, as much for the product and for the sum,
4 in all with room for the 2^-28 (each of the three products' errors has |c| or |s|
under 1).  The norm before it is 1/sqrt of a sum in 64 bits rounded to fp32 (half
a rounding in the root), a root good to 1.5 roundings, and two products: 4 more.
The result is rounded to its type: half a step of it."""
import numpy as np
import pytest

from oracle import kv
from oracle import rotary as plain

from gpu_helpers import Side, say
from test_gpu_kv import bf16, device_batch, device_cache, i32, pages_for, rows_dev, same_cache

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def side():
    return Side()


def near(got, want, mag, normed, bf):
    """Within the bounds above; what is not finite is the same."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    # values that do not turn keep their bits without a norm, and 4 roundings with one
    turns = mag > 0
    bound = np.where(turns, (8 if normed else 4) * U * mag, 4 * U * np.abs(want) if normed else 0.0)
    with np.errstate(invalid="ignore"):  # infinities, which are not `fine`
        bound = bound + (np.abs(want) + bound) * (2.0 ** -8 if bf else 0.0) + 2.0 ** -148
        bad = fine & (np.abs(got - want) > bound)
    assert not bad.any(), f"{bad.sum()} off, first at {np.argwhere(bad)[0]}: " \
        f"{got[bad][0]} for {want[bad][0]}, bound {bound[bad][0]}"


def turned(x, at, f, layout, gain, weight):
    """x [rows][heads][D] in 64 bits, normed and turned, and the pairs' magnitudes."""
    if weight is not None:
        x = plain.norm(x, weight.astype(np.float64), EPS)
    return plain.rotate(x, at, f, layout, gain)


def values(rng, rows, heads, dim, f32):
    x = rng.normal(size=(rows, heads * dim)) * 2.0 ** rng.integers(-4, 5, (rows, heads)).repeat(dim, 1)
    return x.astype(np.float32) if f32 else bf16(x)


def weights(side, rng, dim, on):
    w = (1 + 0.3 * rng.normal(size=dim)).astype(np.float32) if on else None
    return w, side.to_dev(w) if on else None


def rotate(side, r, x, f32, at, heads, dim, w, to32, pad=16):
    t = side.torch
    xd = rows_dev(side, x, pad, f32)
    rows = len(x)
    y = t.full((rows, heads * dim + 32), 7.0, dtype=t.float32 if to32 else t.bfloat16, device="cuda")
    out = y[:, 16:16 + heads * dim]
    pos = i32(side, at)
    side.stream.wait_stream(t.cuda.current_stream())
    side.nf4.nf4_rotate(r, xd, xd.stride(0), int(f32), pos, rows, heads, dim, w, EPS, out, out.stride(0),
                        int(to32), stream=side.stream)
    side.sync()
    assert bool((y[:, :16] == 7).all()) and bool((y[:, -16:] == 7).all())  # beside the rows: as it was
    return out.float().cpu().numpy()


# (head_dim, dims): whole heads, halves, odd numbers of pairs, none, one pair
SHAPES = [(128, 128), (128, 64), (128, 96), (128, 50), (128, 2), (128, 0), (64, 64), (64, 32), (64, 8), (64, 62)]


@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("layout", [plain.HALVES, plain.PAIRS])
@pytest.mark.parametrize("dim,dims", SHAPES)
def test_rotate(side, dim, dims, layout, normed):
    rng = np.random.default_rng(dim + 3 * dims + layout)
    f = plain.frequencies(dims, 1e4)
    r = side.nf4.Rotary(dims, layout, frequencies=f, gain=1.25)
    for rows, heads, f32, to32 in ((1, 5, True, False), (17, 3, False, False), (33, 1, True, True),
                                   (16, 13, False, True)):
        say(f"[rotate] dim={dim} dims={dims} layout={layout} norm={normed} {rows} x {heads} {f32} {to32}")
        x = values(rng, rows, heads, dim, f32)
        at = rng.integers(-50, 20000, rows)
        w, wd = weights(side, rng, dim, normed)
        got = rotate(side, r, x, f32, at, heads, dim, wd, to32)
        want, mag = turned(x.reshape(rows, heads, dim).astype(np.float64), at, f, layout, 1.25, w)
        near(got.reshape(want.shape), want, mag, normed, not to32)


@pytest.mark.parametrize("rows,heads", [(1, 1), (2, 32), (300, 7), (1025, 28)])
def test_rotate_many_rows(side, rows, heads):
    """Few and many workgroups, the last ones in part: one head and three of a wave."""
    rng = np.random.default_rng(rows)
    f = plain.frequencies(128, 1e6)
    r = side.nf4.Rotary(128, base=1e6)
    x = values(rng, rows, heads, 128, True)
    at = np.arange(rows) + 14449
    got = rotate(side, r, x, True, at, heads, 128, None, True)
    want, mag = turned(x.reshape(rows, heads, 128).astype(np.float64), at, f, 0, 1.0, None)
    near(got.reshape(want.shape), want, mag, False, False)


def test_rotate_far_positions(side):
    """Positions to the ends of 32 bits: the turns of every frequency to 2^-34."""
    rng = np.random.default_rng(1)
    at = np.array([0, 1, -1, 2 ** 20 + 7, 2 ** 30 + 8388607, 2 ** 31 - 1, -2 ** 31, 123456789])
    f = plain.frequencies(64, 5e5)
    r = side.nf4.Rotary(64, base=5e5)
    x = values(rng, len(at), 4, 64, True)
    got = rotate(side, r, x, True, at, 4, 64, None, True)
    want, mag = turned(x.reshape(-1, 4, 64).astype(np.float64), at, f, 0, 1.0, None)
    near(got.reshape(want.shape), want, mag, False, False)
    # position 0 turns nothing, exactly
    assert np.array_equal(got[0], x[0])


def test_rotate_back_and_composed(side):
    """Turning by p and by -p gives the values back, by p then q what p + q does;
    lengths stay (the rotation is orthogonal)."""
    rng = np.random.default_rng(2)
    r = side.nf4.Rotary(96, plain.PAIRS)
    p, q = rng.integers(0, 100000, 40), rng.integers(0, 1000, 40)
    x = values(rng, 40, 3, 128, True)
    once = rotate(side, r, x, True, p, 3, 128, None, True)
    size = np.abs(x).max(1, keepdims=True) * 2
    # two turns, each within 4 roundings of a pair's magnitude, and the first one's
    # error turned by the second (at most sqrt 2 times as large)
    assert np.all(np.abs(rotate(side, r, once, True, -p, 3, 128, None, True) - x) <= 16 * U * size)
    twice = rotate(side, r, once, True, q, 3, 128, None, True)
    both = rotate(side, r, x, True, p + q, 3, 128, None, True)
    assert np.all(np.abs(twice - both) <= 16 * U * size)


def test_gradient_is_the_turn_back(side):
    """The gradient of <g, rotate(x, p)> with respect to x is rotate(g, -p) (gain
    included): against the formula's in 64 bits and against differences."""
    rng = np.random.default_rng(3)
    f = plain.frequencies(50, 1e4)
    r = side.nf4.Rotary(50, frequencies=f, gain=1.5)
    at = rng.integers(0, 5000, 6)
    x, g = (values(rng, 6, 2, 64, True) for _ in range(2))
    got = rotate(side, r, g, True, -at, 2, 64, None, True).reshape(6, 2, 64)
    want, mag = plain.rotate(g.reshape(6, 2, 64).astype(np.float64), -at, f, 0, 1.5)
    near(got, want, mag, False, False)
    x64, g64 = (z.reshape(6, 2, 64).astype(np.float64) for z in (x, g))
    for i in rng.integers(0, x64.size, 20):
        e = np.zeros(x64.size)
        e[i] = 0.5
        e = e.reshape(x64.shape)
        hi, lo = (plain.rotate(x64 + d, at, f, 0, 1.5)[0] for d in (e, -e))
        # linear: the difference is the derivative, but for 64-bit roundings
        assert abs(((hi - lo) * g64).sum() - got.reshape(-1)[i]) <= 8 * U * np.abs(g64).max() * 3


@pytest.mark.parametrize("f32", [False, True])
def test_rotate_in_place_and_on_streams(side, f32):
    t, rng = side.torch, np.random.default_rng(4)
    r = side.nf4.Rotary(128)
    x = values(rng, 70, 6, 128, f32)
    at = rng.integers(0, 9999, 70)
    want = rotate(side, r, x, f32, at, 6, 128, None, f32)
    d = rows_dev(side, x, 8, f32)
    pos = i32(side, at)
    side.stream.wait_stream(t.cuda.current_stream())
    side.nf4.nf4_rotate(r, d, d.stride(0), int(f32), pos, 70, 6, 128, None, 0.0, d, d.stride(0), int(f32),
                        stream=side.stream)
    side.sync()
    assert np.array_equal(d.float().cpu().numpy(), want)
    # the current stream of torch
    d2 = rows_dev(side, x, 8, f32)
    with t.cuda.stream(side.stream):
        side.stream.wait_stream(t.cuda.default_stream())
        side.nf4.nf4_rotate(r, d2, d2.stride(0), int(f32), pos, 70, 6, 128, None, 0.0, d2, d2.stride(0), int(f32))
    side.sync()
    assert np.array_equal(d2.float().cpu().numpy(), want)


def test_rotate_special_values(side):
    """Infinities and NaN reach their own pair, zeros and values that do not turn keep
    their bits, the norm's sum passes neither end of fp32, heads do not mix."""
    rng = np.random.default_rng(5)
    f = plain.frequencies(64, 1e4)
    at = np.array([3, 100, 7, 7, 9, 11])
    x = values(rng, 6, 4, 128, True)
    x[0, 5], x[0, 40], x[1, 130], x[2, 300] = np.inf, np.nan, -np.inf, 3e38
    x[3, :128] = 0.0
    x[3, 100:128] = -0.0
    r = side.nf4.Rotary(64)
    got = rotate(side, r, x, True, at, 4, 128, None, True).reshape(6, 4, 128)
    want, mag = turned(x.reshape(6, 4, 128).astype(np.float64), at, f, 0, 1.0, None)
    want[np.abs(want) > 3.4e38] = np.sign(want[np.abs(want) > 3.4e38]) * np.inf
    near(got, want, mag, False, False)
    passed = x.reshape(6, 4, 128)[..., 64:]
    assert np.array_equal(got[..., 64:].view(np.uint32), passed.view(np.uint32))
    # norms: heads of the largest and of tiny values, zeros, a NaN and an infinity in one head
    x = values(rng, 6, 4, 128, True)
    x[0, :128] *= np.float32(2.0 ** 115)
    x[1, :128] *= np.float32(2.0 ** -120)
    x[2, :128] = 0.0
    x[3, 7], x[4, 7] = np.nan, np.inf
    x[5, :128] = 3.4e38
    w, wd = weights(side, rng, 128, True)
    got = rotate(side, r, x, True, at, 4, 128, wd, True).reshape(6, 4, 128)
    x64 = x.reshape(6, 4, 128).astype(np.float64)
    with np.errstate(all="ignore"):
        want, mag = turned(x64, at, f, 0, 1.0, w)
    # an infinity's own pair is NaN, the rest of its head 0
    near(got, want, np.nan_to_num(mag), True, False)


# ---------------------------------------------------------------- append
# (lengths after the call, new rows of each)
BATCHES = [([1], [1]), ([17], [1]), ([31], [30]), ([40, 0, 5, 33], [3, 0, 5, 0]),
           ([129, 64, 65, 200], [128, 1, 2, 77]), ([3, 20, 2], [5, 20, 19])]


@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("dim,dims,layout,page,kvh,group", [
    (128, 128, 0, 64, 2, 7), (128, 96, 1, 16, 1, 4), (64, 50, 0, 16, 3, 1), (64, 64, 1, 256, 2, 2)])
@pytest.mark.parametrize("kv_len,count", BATCHES)
def test_append_rotated(side, normed, f32, dim, dims, layout, page, kvh, group, kv_len, count):
    """Queries within the bounds of the definition; keys and values byte for byte
    what turning to fp32 and then appending those gives; rows that are no tokens zeros."""
    t, nf4 = side.torch, side.nf4
    rng = np.random.default_rng(dim + dims + len(kv_len) + kv_len[0])
    heads = kvh * group
    pages, table = pages_for(rng, kv_len, page)
    c = kv.Cache(2, pages, kvh, page, dim, rng)
    d, e = device_cache(side, c), device_cache(side, c)
    start = np.concatenate([[0], np.cumsum(count)])
    rows = int(start[-1])
    q, k, v = (values(rng, rows, h, dim, f32) for h in (heads, kvh, kvh))
    qd, kd, vd = (rows_dev(side, z, p, f32) for z, p in ((q, 8), (k, 16), (v, 24)))
    (qw, qwd), (kw, kwd) = (weights(side, rng, dim, normed) for _ in range(2))
    f = plain.frequencies(dims, 1e4)
    r = nf4.Rotary(dims, layout, frequencies=f, gain=0.9)
    b = device_batch(side, table, kv_len, start)
    out = t.full((rows + 3, heads * dim), 7.0, dtype=t.bfloat16, device="cuda")
    at = np.concatenate([np.arange(n - m, n) for n, m in zip(kv_len, count)])
    pos, turned_k = i32(side, at), t.empty(rows, kvh * dim, device="cuda")
    say(f"[append rotated] {dim}/{dims} {layout} page={page} f32={f32} norm={normed} {kv_len} {count}")
    side.stream.wait_stream(t.cuda.current_stream())
    nf4.nf4_kv_append_rotated(d, 1, b, r, qd, qd.stride(0), heads, qwd, kd, kd.stride(0), kwd, vd,
                              vd.stride(0), int(f32), EPS, out, stream=side.stream)
    nf4.nf4_rotate(r, kd, kd.stride(0), int(f32), pos, rows, kvh, dim, kwd, EPS, turned_k, kvh * dim,
                   nf4.NF4_KV_F32, stream=side.stream)
    v32 = vd.float().contiguous()
    side.stream.wait_stream(t.cuda.current_stream())
    nf4.nf4_kv_append(e, 1, b, turned_k, kvh * dim, v32, kvh * dim, nf4.NF4_KV_F32, stream=side.stream)
    side.sync()
    got = out.float().cpu().numpy()
    assert (got[rows:] == 7).all()  # behind the last sequence: as it was
    want, mag = turned(q.reshape(rows, heads, dim).astype(np.float64), at, f, layout, 0.9, qw)
    want[at < 0], mag[at < 0] = 0.0, 0.0
    near(got[:rows].reshape(want.shape), want, mag, normed, True)
    for name in ("k", "v", "k_scale", "v_scale"):
        assert t.equal(getattr(d, name), getattr(e, name)), name
    # and that is what the plain cache gets from the turned keys
    kv.append(c, 1, table, start, kv_len, turned_k.double().cpu().numpy().reshape(rows, kvh, dim),
              v.reshape(rows, kvh, dim).astype(np.float64))
    same_cache(c, d)


def test_append_rotated_leaves_what_has_no_place(side):
    """Holes, ids past the pool, rows past max_rows, tokens past the table and past
    max_len: the keys as nf4_kv_append leaves them, the queries turned all the same."""
    t, nf4 = side.torch, side.nf4
    rng = np.random.default_rng(6)
    dim, kvh, heads, page = 128, 1, 3, 16
    table = np.array([[0, -1, 2], [3, 900, 4], [5, 6, 7], [8, 9, 10], [11, 11, 11]], np.int32)
    kv_len, count = [48, 40, 5, 60, 70], [48, 40, 9, 20, 2]
    start = np.concatenate([[0], np.cumsum(count)])
    rows = int(start[-1])
    f = plain.frequencies(128, 1e4)
    r = nf4.Rotary(128)
    for bounds in ({}, {"max_rows": 40}, {"max_len": 45}):
        c = kv.Cache(1, 12, kvh, page, dim, rng)
        d, e = device_cache(side, c), device_cache(side, c)
        q, k, v = (values(rng, rows, h, dim, True) for h in (heads, kvh, kvh))
        qd, kd, vd = (side.to_dev(z) for z in (q, k, v))
        b = device_batch(side, table, kv_len, start, **({"max_len": 100} | bounds))
        held = [min(n, bounds.get("max_len", 10 ** 9)) for n in kv_len]
        at = np.concatenate([np.arange(n - m, n) for n, m in zip(held, count)])
        out = t.full((rows, heads * dim), 7.0, dtype=t.bfloat16, device="cuda")
        turned_k = t.empty(rows, kvh * dim, device="cuda")
        say(f"[append rotated] no place, {bounds}")
        side.stream.wait_stream(t.cuda.current_stream())
        nf4.nf4_kv_append_rotated(d, 0, b, r, qd, heads * dim, heads, None, kd, dim, None, vd, dim,
                                  nf4.NF4_KV_F32, 0.0, out, stream=side.stream)
        nf4.nf4_rotate(r, kd, dim, nf4.NF4_KV_F32, i32(side, at), rows, kvh, dim, None, 0.0, turned_k,
                       dim, nf4.NF4_KV_F32, stream=side.stream)
        nf4.nf4_kv_append(e, 0, b, turned_k, dim, vd, dim, nf4.NF4_KV_F32, stream=side.stream)
        side.sync()
        for name in ("k", "v", "k_scale", "v_scale"):
            assert t.equal(getattr(d, name), getattr(e, name)), (name, bounds)
        want, mag = turned(q.reshape(rows, heads, dim).astype(np.float64), at, f, 0, 1.0, None)
        got = out.float().cpu().numpy().reshape(want.shape)
        own = np.concatenate([np.arange(m) for m in count])
        done = own < bounds.get("max_rows", 10 ** 9)
        assert (got[~done] == 7).all()
        want[at < 0], mag[at < 0] = 0.0, 0.0
        near(got[done], want[done], mag[done], False, True)


def test_append_rotated_in_place(side):
    """bf16 queries of their own tensor turn where they lie."""
    t, nf4 = side.torch, side.nf4
    rng = np.random.default_rng(8)
    table = np.arange(4, dtype=np.int32)[None]
    c = kv.Cache(1, 5, 2, 16, 64, rng)
    q, k = bf16(rng.normal(size=(37, 8 * 64))), bf16(rng.normal(size=(37, 2 * 64)))
    qd, kd = (side.to_dev(z).bfloat16() for z in (q, k))
    out, b, r = t.empty_like(qd), device_batch(side, table, [50], [0, 37]), nf4.Rotary(64)
    for to in (out, qd):
        d = device_cache(side, c)
        t.cuda.synchronize()
        nf4.nf4_kv_append_rotated(d, 0, b, r, qd, 512, 8, None, kd, 128, None, kd, 128, nf4.NF4_KV_BF16,
                                  0.0, to, stream=side.stream)
        side.sync()
    assert t.equal(out, qd)


def test_append_rotated_in_a_graph(side):
    """Captured once and replayed as the sequences grow, eager work in between."""
    t, nf4 = side.torch, side.nf4
    rng = np.random.default_rng(9)
    table = rng.permutation(12).astype(np.int32).reshape(3, 4)
    c = kv.Cache(1, 12, 2, 16, 128, rng)
    d, e = device_cache(side, c), device_cache(side, c)
    r = nf4.Rotary(128)
    lens = i32(side, [5, 17, 30])
    b = nf4.KVBatch(lens, i32(side, table), max_len=64)
    x = t.zeros(3, 8 * 128, device="cuda")
    out, ref = (t.zeros(3, 4 * 128, dtype=t.bfloat16, device="cuda") for _ in range(2))

    def step(cache, to):
        nf4.nf4_kv_append_rotated(cache, 0, b, r, x, 1024, 4, None, x[:, 512:], 1024, None, x[:, 768:],
                                  1024, nf4.NF4_KV_F32, 0.0, to)
    g = t.cuda.CUDAGraph()
    t.cuda.synchronize()
    with t.cuda.graph(g):
        step(d, out)
    for i in range(5):
        x.copy_(t.from_numpy(rng.normal(size=(3, 1024)).astype(np.float32)))
        lens.add_(1)
        g.replay()
        step(e, ref)
        t.cuda.synchronize()
        assert t.equal(out, ref) and t.equal(d.k, e.k) and t.equal(d.v, e.v) and t.equal(d.k_scale, e.k_scale)


# ---------------------------------------------------------------- read
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, 3), (128, 64, 1), (128, 16, 2), (64, 256, 2)])
@pytest.mark.parametrize("kv_len,count", BATCHES)
def test_read(side, f32, dim, page, heads, kv_len, count):
    t = side.torch
    rng = np.random.default_rng(dim + page + len(kv_len) + kv_len[0])
    pages, table = pages_for(rng, kv_len, page)
    c = kv.Cache(2, pages, heads, page, dim, rng)
    d = device_cache(side, c)
    start = np.concatenate([[0], np.cumsum(count)])
    rows = int(start[-1])
    b = device_batch(side, table, kv_len, start)
    kind = t.float32 if f32 else t.bfloat16
    k, v = (t.full((rows + 2, heads * dim + p), 7.0, dtype=kind, device="cuda") for p in (16, 8))
    say(f"[kv read] f32={f32} dim={dim} page={page} {kv_len} {count}")
    side.stream.wait_stream(t.cuda.current_stream())
    side.nf4.nf4_kv_read(d, 1, b, k, k.stride(0), v, v.stride(0), int(f32), stream=side.stream)
    side.sync()
    for which, y in ((0, k), (1, v)):
        got = y.double().cpu().numpy()
        assert (got[rows:] == 7).all() and (got[:, heads * dim:] == 7).all()
        for s, (n, m) in enumerate(zip(kv_len, count)):
            for h in range(heads):
                dense, _ = c.dense(which, 1, h, table[s], n)
                want = np.zeros((m, dim))
                want[max(m - n, 0):] = dense[max(n - m, 0):]
                mine = got[start[s]:start[s + 1], h * dim:(h + 1) * dim]
                assert np.array_equal(mine, want, equal_nan=True), (which, s, h)


def test_read_of_holes_and_bounds(side):
    t, nf4 = side.torch, side.nf4
    rng = np.random.default_rng(7)
    table = np.array([[0, -1, 2], [3, 900, 1]], np.int32)
    c = kv.Cache(1, 4, 2, 16, 64, rng)
    d = device_cache(side, c)
    b = device_batch(side, table, [60, 40], [0, 60, 100], max_len=100, max_rows=50)
    y = t.full((2, 100, 128), 7.0, device="cuda")
    side.sync()
    t.cuda.synchronize()
    nf4.nf4_kv_read(d, 0, b, y[0], 128, y[1], 128, nf4.NF4_KV_F32, stream=side.stream)
    side.sync()
    for which in (0, 1):
        got = y[which].double().cpu().numpy().reshape(100, 2, 64)
        assert (got[50:60] == 7).all()  # past max_rows
        for s, (r0, n, rows) in enumerate(((0, 60, 50), (60, 40, 40))):
            for h in range(2):
                dense, hole = c.dense(which, 0, h, table[s], min(n, 48))
                want = np.zeros((n, 64))
                want[:len(dense)] = np.where(hole[:, None], 0.0, dense)
                assert np.array_equal(got[r0:r0 + rows, h], want[:rows], equal_nan=True)


def test_read_gives_back_what_was_appended(side):
    """Rows of e4m3 values times powers of two come back as they were; read with
    another page size and appended again, the codes are the same."""
    t, nf4 = side.torch, side.nf4
    rng = np.random.default_rng(10)
    n, kvh, dim = 100, 2, 64
    x = kv.VALUES[rng.integers(0, 127, (2, n, kvh * dim))] * 2.0 ** 5
    x[:, ::16, ::dim] = 448.0 * 2.0 ** 5  # every block's largest: the scale is 2^5
    x = [side.to_dev(z.astype(np.float32)) for z in x]
    caches = []
    for page in (16, 64):
        d = nf4.KVCache(1, 8, kvh, page, dim)
        b = device_batch(side, np.arange(7, dtype=np.int32)[None], [n], [0, n])
        y = t.empty(2, n, kvh * dim, device="cuda")
        t.cuda.synchronize()
        nf4.nf4_kv_append(d, 0, b, x[0], kvh * dim, x[1], kvh * dim, nf4.NF4_KV_F32, stream=side.stream)
        nf4.nf4_kv_read(d, 0, b, y[0], kvh * dim, y[1], kvh * dim, nf4.NF4_KV_F32, stream=side.stream)
        side.sync()
        assert t.equal(y[0], x[0]) and t.equal(y[1], x[1])
        x = [y[0].clone(), y[1].clone()]
        caches.append(d)


def test_rotate_refuses_fewer_positions_than_rows(side):
    t, nf4 = side.torch, side.nf4
    x, r = t.zeros(5, 128, device="cuda"), nf4.Rotary(64)
    with pytest.raises(nf4.NF4Error, match="one for each row"):
        nf4.nf4_rotate(r, x, 128, nf4.NF4_KV_F32, i32(side, range(4)), 5, 2, 64, None, 0.0, x, 128,
                       nf4.NF4_KV_F32)


@pytest.mark.parametrize("dim", [64, 128])
def test_large_rows_leave_their_neighbours_alone(side, dim):
    """A row whose squares pass 32 bits is normed in 64; the rows beside it are not."""
    t, nf4 = side.torch, side.nf4
    rng = np.random.default_rng(41)
    heads, rows = 5, 19
    x = side.to_dev(rng.normal(size=(rows, heads * dim)).astype(np.float32))
    y = x.clone()
    y[3, dim:2 * dim] *= 2.0 ** 90
    y[12] *= 2.0 ** 70
    w = side.to_dev((1 + 0.3 * rng.normal(size=dim)).astype(np.float32))
    out = []
    for z in (x, y):
        out.append(t.zeros(rows, heads * dim, dtype=t.bfloat16, device="cuda"))
        nf4.nf4_rotate(nf4.Rotary(dim), z, heads * dim, nf4.NF4_KV_F32, i32(side, range(rows)), rows, heads, dim,
                       w, EPS, out[-1], heads * dim, nf4.NF4_KV_BF16)
    t.cuda.synchronize()
    same = (out[0] == out[1]).reshape(rows, heads, dim).all(-1)
    for r in range(rows):
        for h in range(heads):
            if not (r == 12 or (r == 3 and h == 1)):
                assert bool(same[r, h]), (r, h)
    # scaled by a power of two, and eps far below both: the same up to the roundings
    assert float((out[0].float() - out[1].float()).abs().max()) <= float(out[0].float().abs().max()) * 2.0 ** -7


def half_step(x):
    """Half a step of fp32 at x."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 24)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("layout", [plain.HALVES, plain.PAIRS])
@pytest.mark.parametrize("dim,dims", [(128, 128), (128, 50), (64, 64)])
def test_fp32_results_are_rounded_once(side, dim, dims, layout, f32):
    """Half a step of the exact value and what 64 bits leave: the sine's sum stops before
    x^13 / 13! of the angle x that a quarter turn leaves, each pair's turns a token are 2^-65 of a
    turn off, sines and cosines are kept to 2^-48 and products are good to 2^-52 (2^-46 for
    all of that), 80 bits of the oracle's angle are 2^-61 of its radians.  Slow pairs at small
    positions, and pairs of which one value is 0, show the sine by itself."""
    rng = np.random.default_rng(51)
    f = plain.frequencies(dims, 1e6)
    at = np.array([0, 1, -1, 2, 5, 17, -100, 1000, 14449, 2 ** 20 + 7, -2 ** 20 - 7])
    rows = len(at)
    x = values(rng, rows, 4, dim, f32).reshape(rows, 4, dim)
    a, b = plain.pair_indexes(dims, layout)
    x[:, 1, a], x[:, 1, b], x[:, 2, a], x[:, 2, b] = 0.0, 1.0, 1.0, 0.0
    x = x.reshape(rows, 4 * dim)
    got = rotate(side, side.nf4.Rotary(dims, layout, frequencies=f), x, f32, at, 4, dim, None, True)
    got = got.reshape(rows, 4, dim).astype(np.float64)
    want, mag = turned(x.reshape(rows, 4, dim).astype(np.float64), at, f, layout, 1.0, None)
    angle = np.abs(at)[:, None] * f
    left = np.abs(angle - np.rint(angle / (np.pi / 2)) * (np.pi / 2))
    off = left ** 13 / 6227020800 + 2 * np.pi * 2.0 ** -65 * np.abs(at)[:, None] + angle * 2.0 ** -61
    c, s = np.abs(np.cos(angle))[:, None], np.abs(np.sin(angle))[:, None]
    p, q = (np.abs(x.reshape(rows, 4, dim)[..., i]) for i in (a, b))
    bound = half_step(want)
    bound[..., a] += off[:, None] * mag[..., a] + 2.0 ** -46 * (p * c + q * s)
    bound[..., b] += off[:, None] * mag[..., b] + 2.0 ** -46 * (p * s + q * c)
    bad = np.abs(got - want) > bound
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
        f"{got[bad][0]} for {want[bad][0]}"
    # a turn back is the negative angle, to the bit
    for i, j in ((1, 2), (9, 10)):
        assert np.array_equal(got[i, 1, a], -got[j, 1, a]) and np.array_equal(got[i, 2, b], -got[j, 2, b])
        assert np.array_equal(got[i, 1, b], got[j, 1, b])


@pytest.mark.parametrize("f32", [False, True])
def test_norm_of_small_rows_under_large_weights(side, f32):
    """Rows of zeros stay zeros and tiny ones come out finite, whatever 1 / sqrt(eps) times a
    weight is."""
    t, nf4 = side.torch, side.nf4
    rng = np.random.default_rng(61)
    x = bf16(rng.normal(size=(3, 2 * 64)))
    x[0] = 0.0
    x[1] *= np.float32(2.0 ** -60)
    eps, w = 2.0 ** -100, np.full(64, 2.0 ** 100, np.float32)
    f = plain.frequencies(64, 1e4)
    xd = side.to_dev(x) if f32 else side.to_dev(x).bfloat16()
    for to in (t.bfloat16, t.float32):
        y = t.empty(3, 128, dtype=to, device="cuda")
        nf4.nf4_rotate(nf4.Rotary(64, frequencies=f), xd, 128, int(f32), i32(side, [0, 1, 2]), 3, 2, 64,
                       side.to_dev(w), eps, y, 128, int(to is t.float32))
        t.cuda.synchronize()
        x64 = x.reshape(3, 2, 64).astype(np.float64)
        z = x64 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + eps) * 2.0 ** 100
        want, mag = plain.rotate(z, [0, 1, 2], f, 0)
        near(y.double().cpu().numpy().reshape(want.shape), want, mag, True, to is t.bfloat16)
