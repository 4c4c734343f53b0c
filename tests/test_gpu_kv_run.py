"""The cache's operators as a server runs them: a prompt in chunks, branches that share
it, and steps of a token each in a captured graph, where queries and keys are normed,
turned and appended, attended to with the shared tokens read once, and read back."""
import numpy as np
import pytest

from oracle import kv
from oracle import rotary as plain

from gpu_helpers import Side, say
from test_gpu_kv import bf16, bounds, i32
from test_gpu_kv_shared import SAVED
from test_gpu_rotary import EPS, near, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def side():
    return Side()


def host_cache(d, c):
    """The device's cache as the oracle's."""
    h = kv.Cache(c.layers, c.pages, c.kv_heads, c.page_tokens, c.head_dim)
    h.k, h.v = (np.array(x.cpu().numpy()).reshape(y.shape) for x, y in ((d.k, h.k), (d.v, h.v)))
    h.ks, h.vs = (np.array(x.cpu().numpy()).reshape(y.shape) for x, y in ((d.k_scale, h.ks), (d.v_scale, h.vs)))
    return h


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("dim,dims,layout,heads,kvh,branches,window,sinks",
                         [(64, 64, plain.HALVES, 8, 2, 24, 0, 0), (128, 64, plain.PAIRS, 4, 1, 30, 150, 8)])
def test_prompt_branches_and_steps(side, dim, dims, layout, heads, kvh, branches, window, sinks, f32):
    t, nf4 = side.torch, side.nf4
    rng = np.random.default_rng(31 + dim)
    page, prompt, steps = 16, 203, 6
    # tables with room for so many tokens that the shared ones are taken apart, but for a
    # window, which keeps few of them
    tiles = branches - -(-branches * heads // kvh // 64)
    width = 60 if window else SAVED // (tiles * kvh * 2 * dim) // page + 2
    pages = 20 + 3 * branches
    make = lambda: nf4.KVCache(1, pages, kvh, page, dim)  # noqa: E731
    cache, other = make(), make()
    scale = float(np.float32(dim ** -0.5))
    rot = nf4.Rotary(dims, layout, 10000.0, nf4.NF4_SCALING_RAMP, 4.0, 128, 1.0, 32.0, gain=1.1)
    freq = plain.frequencies(dims, 10000.0, "ramp", 4.0, 128, 1.0, 32.0)
    wq, wk = ((1 + 0.2 * rng.normal(size=dim)).astype(np.float32) for _ in range(2))
    dq, dk = side.to_dev(wq), side.to_dev(wk)
    type = nf4.NF4_KV_F32 if f32 else nf4.NF4_KV_BF16
    fused = (heads + 2 * kvh) * dim
    cut = lambda x: (x[:, :heads * dim], x[:, heads * dim:(heads + kvh) * dim], x[:, (heads + kvh) * dim:])  # noqa: E731

    def rows(n):
        x = rng.normal(size=(n, fused))
        return x.astype(np.float32) if f32 else bf16(x)

    def dev(x):
        return side.to_dev(x) if f32 else side.to_dev(x).bfloat16()
    pool = nf4.KVPool(t.zeros(pages, dtype=t.int32, device="cuda"),
                      t.full((branches + 1, width), -1, dtype=t.int32, device="cuda"),
                      t.zeros(branches + 1, dtype=t.int32, device="cuda"), i32(side, [0]))

    def append(c, b, x, out):
        q, k, v = cut(x)
        nf4.nf4_kv_append_rotated(c, 0, b, rot, q, fused, heads, dq, k, fused, dk, v, fused, type, EPS, out)

    # the prompt in two chunks
    x = rows(prompt)
    for lo, hi in ((0, 120), (120, prompt)):
        add = i32(side, [hi - lo] + [0] * branches)
        nf4.nf4_kv_reserve(cache, pool, add)
        b = nf4.KVBatch(pool.length[:1], pool.table[:1], row_start=i32(side, [0, hi - lo]), rows=hi - lo,
                        max_rows=hi - lo, max_len=width * page)
        out = t.empty(hi - lo, heads * dim, dtype=t.bfloat16, device="cuda")
        for c in (cache, other):
            append(c, b, dev(x[lo:hi]), out)
        got = out.double().cpu().numpy().reshape(-1, heads, dim)
        q = cut(x[lo:hi])[0].astype(np.float64).reshape(-1, heads, dim)
        want, mag = turned(q, np.arange(lo, hi), freq, layout, 1.1, wq)
        near(got, want, mag, True, True)
    shared = pool.length[:1].clone()
    sources, targets = i32(side, [0] * branches), i32(side, range(1, branches + 1))
    twin = nf4.KVPool(pool.refs.clone(), pool.table.clone(), pool.length.clone(), i32(side, [0]))
    for c, p in ((cache, pool), (other, twin)):  # the page in part is copied in both
        nf4.nf4_kv_fork(c, p, sources, targets, branches)
    assert t.equal(twin.table, pool.table) and t.equal(twin.refs, pool.refs)
    nf4.nf4_kv_release(cache, pool, i32(side, [0]), 1)

    # steps of a token each, captured; the second cache goes the single operators' way
    batch = nf4.KVBatch(pool.length[1:], pool.table[1:], max_len=1 << 30)
    groups = nf4.KVGroups(shared, max_rows=branches)
    n = nf4.nf4_kv_attention_shared_workspace_bytes(cache, batch, groups, heads, window, sinks)
    alone = nf4.nf4_kv_attention_workspace_bytes(cache, batch, heads, window, sinks)
    assert (n != alone) == (window == 0), "taken apart without the window"
    ws, ws2 = (t.full((max(m, 16),), 0xFF, dtype=t.uint8, device="cuda") for m in (n, alone))
    one = i32(side, [0] + [1] * branches)
    xd = dev(rows(branches))
    new = lambda *s: t.zeros(*s, device="cuda")  # noqa: E731
    q, out = (new(branches, heads * dim).bfloat16() for _ in range(2))
    z, kb, vb = new(branches, heads), new(branches, kvh * dim), new(branches, kvh * dim)
    missing = i32(side, [0])

    def step():
        nf4.nf4_kv_reserve(cache, pool, one)
        missing.add_(pool.missing)
        append(cache, batch, xd, q)
        nf4.nf4_kv_attention_shared(cache, 0, batch, groups, q, heads * dim, heads, scale, window, sinks,
                                    out, z, ws, n)
        nf4.nf4_kv_read(cache, 0, batch, kb, kvh * dim, vb, kvh * dim, nf4.NF4_KV_F32)
    graph = t.cuda.CUDAGraph()
    t.cuda.synchronize()
    with t.cuda.graph(graph):
        step()
    for i in range(steps):
        x = rows(branches)
        xd.copy_(dev(x))
        graph.replay()
        at = prompt + i
        say(f"[kv run] dim={dim} branches={branches} window={window} at={at} ws={n}")
        # apart: the keys turned to fp32 and appended, the queries turned, plain attention
        qx, kx, vx = cut(xd)
        pos = pool.length[1:] - 1
        k2, q2, out2, z2 = new(branches, kvh * dim), t.empty_like(q), t.empty_like(out), t.empty_like(z)
        nf4.nf4_rotate(rot, kx, fused, type, pos, branches, kvh, dim, dk, EPS, k2, kvh * dim, nf4.NF4_KV_F32)
        nf4.nf4_rotate(rot, qx, fused, type, pos, branches, heads, dim, dq, EPS, q2, heads * dim, nf4.NF4_KV_BF16)
        v2 = vx.float().contiguous()
        nf4.nf4_kv_append(other, 0, batch, k2, kvh * dim, v2, kvh * dim, nf4.NF4_KV_F32)
        nf4.nf4_kv_attention(other, 0, batch, q2, heads * dim, heads, scale, window, sinks, out2, z2, ws2, alone)
        t.cuda.synchronize()
        assert t.equal(q, q2) and t.equal(cache.k, other.k) and t.equal(cache.v, other.v)
        assert t.equal(cache.k_scale, other.k_scale) and t.equal(cache.v_scale, other.v_scale)
        # in 64 bits: the new rows, and attention over what the cache holds
        for got, w, wt, hs in ((q, cut(x)[0], wq, heads), (k2, cut(x)[1], wk, kvh)):
            want, mag = turned(w.astype(np.float64).reshape(branches, hs, dim), [at] * branches, freq, layout, 1.1, wt)
            near(got.double().cpu().numpy().reshape(want.shape), want, mag, True, got is q)
        h = host_cache(cache, cache.struct)
        table, lens = pool.table[1:].cpu().numpy(), [at + 1] * branches
        ref = kv.attention(h, 0, table, list(range(branches + 1)), lens,
                           q.double().cpu().numpy().reshape(branches, heads, dim), scale, window, sinks)
        tol, tol_lse = bounds(dim, at + 1, *ref)
        for o, zz in ((out, z), (out2, z2)):
            o, zz = o.double().cpu().numpy().reshape(ref[0].shape), zz.cpu().numpy()
            assert (np.abs(o - ref[0]) <= tol).all() and (np.abs(zz - ref[1]) <= tol_lse).all()
        # what was read back: the codes' values; within half a step of e4m3 of what went in
        for got, w, kind in ((kb, k2, 0), (vb, v2, 1)):
            got, w = got.cpu().numpy().reshape(branches, kvh, dim), w.cpu().numpy().reshape(branches, kvh, dim)
            for b in range(branches):
                p, u = table[b, at // page], at % page // kv.BLOCK
                for head in range(kvh):
                    assert np.array_equal(got[b, head], h.dense(kind, 0, head, table[b], at + 1)[0][at])
                    half = 2.0 ** -10 * (h.vs if kind else h.ks)[0, p, head, u]
                    off = np.abs(got[b, head].astype(np.float64) - w[b, head])
                    assert (off <= np.abs(w[b, head]) * 2.0 ** -4 + half).all()
    assert int(missing) == 0


def branches_of(side, cache, pages, seqs, width, n, seed):
    """`seqs` sequences over the same n tokens in the given pages, one more token in a page
    of its own each: the batch, its groups and what one step appends."""
    t, nf4 = side.torch, side.nf4
    page, kvh, dim = cache.struct.page_tokens, cache.struct.kv_heads, cache.struct.head_dim
    table = np.full((seqs, width), -1, np.int32)
    table[:, :n // page] = pages[:n // page]
    table[:, n // page] = pages[n // page:n // page + seqs]
    g = t.Generator(device="cuda").manual_seed(seed)
    rows = lambda r, h: t.randn(r, (h + 2 * kvh) * dim, generator=g, device="cuda")  # noqa: E731
    first, one = rows(n, 0), rows(seqs, 4 * kvh)
    b = nf4.KVBatch(i32(side, [n]), i32(side, table[:1]), row_start=i32(side, [0, n]), rows=n, max_rows=n, max_len=n)
    nf4.nf4_kv_append(cache, 0, b, first, 2 * kvh * dim, first[:, kvh * dim:], 2 * kvh * dim, nf4.NF4_KV_F32)
    return (nf4.KVBatch(i32(side, [n + 1] * seqs), i32(side, table), max_len=1 << 30),
            nf4.KVGroups(i32(side, [n]), max_rows=seqs), one)


def step(side, cache, b, g, x, ws, out, stream=None):
    """Appends a token to each sequence, attends and reads the new rows back."""
    nf4, (seqs, width) = side.nf4, x.shape
    kvh, dim = cache.struct.kv_heads, cache.struct.head_dim
    h, kv_at = 4 * kvh, 4 * kvh * dim
    q, o, z, k, v = out
    nf4.nf4_kv_append_rotated(cache, 0, b, nf4.Rotary(dim), x, width, h, None, x[:, kv_at:], width, None,
                              x[:, kv_at + kvh * dim:], width, nf4.NF4_KV_F32, 0.0, q, stream=stream)
    nf4.nf4_kv_attention_shared(cache, 0, b, g, q, h * dim, h, 0.1, 0, 0, o, z, ws, ws.numel(), stream=stream)
    nf4.nf4_kv_read(cache, 0, b, k, kvh * dim, v, kvh * dim, nf4.NF4_KV_F32, stream=stream)


def outputs(side, cache, seqs):
    t, kvh, dim = side.torch, cache.struct.kv_heads, cache.struct.head_dim
    full = lambda w, d: t.full((seqs, w), 7.0, dtype=d, device="cuda")  # noqa: E731
    return (full(4 * kvh * dim, t.bfloat16), full(4 * kvh * dim, t.bfloat16), full(4 * kvh, t.float32),
            full(kvh * dim, t.float32), full(kvh * dim, t.float32))


def test_pages_past_32_bits(side):
    """The last pages of a cache whose codes pass 2^32 bytes: what the first pages give."""
    t, nf4 = side.torch, side.nf4
    pages, page, kvh, dim, seqs, n = 17000, 256, 8, 128, 20, 512
    cache = nf4.KVCache(1, pages, kvh, page, dim)
    assert cache.k.numel() > 1 << 32
    width = SAVED // ((seqs - 2) * kvh * 2 * dim) // page + 2
    res = []
    for at in (0, pages - 2 - seqs):
        b, g, x = branches_of(side, cache, at + np.arange(2 + seqs), seqs, width, n, 3)
        need = nf4.nf4_kv_attention_shared_workspace_bytes(cache, b, g, 4 * kvh)
        assert need != nf4.nf4_kv_attention_workspace_bytes(cache, b, 4 * kvh), "not taken apart"
        ws = t.full((need,), 0xFF, dtype=t.uint8, device="cuda")
        res.append(outputs(side, cache, seqs))
        step(side, cache, b, g, x, ws, res[-1])
        t.cuda.synchronize()
    for a, b in zip(*res):
        assert t.equal(a, b) and not bool((a == 7).all(-1).any())


def test_two_at_once(side):
    """Two runs on two streams, each with its own cache, workspace and outputs."""
    t, nf4 = side.torch, side.nf4
    runs = []
    for seed, (dim, kvh, seqs) in ((4, (128, 2, 40)), (5, (64, 4, 24))):
        cache = nf4.KVCache(1, 200, kvh, 16, dim)
        width = SAVED // ((seqs - 3) * kvh * 2 * dim) // 16 + 2
        b, g, x = branches_of(side, cache, np.arange(200), seqs, width, 960, seed)
        need = nf4.nf4_kv_attention_shared_workspace_bytes(cache, b, g, 4 * kvh)
        assert need != nf4.nf4_kv_attention_workspace_bytes(cache, b, 4 * kvh), "not taken apart"
        want = outputs(side, cache, seqs)
        ws = t.empty(need, dtype=t.uint8, device="cuda")
        step(side, cache, b, g, x, ws, want)
        runs.append((cache, b, g, x, ws, want, outputs(side, cache, seqs), t.cuda.Stream()))
    t.cuda.synchronize()
    for _ in range(10):
        for cache, b, g, x, ws, _, got, stream in runs:
            step(side, cache, b, g, x, ws, got, stream)
        t.cuda.synchronize()
        for *_, want, got, _ in runs:
            assert all(t.equal(a, b) for a, b in zip(want, got))
            for a in got:
                a.fill_(7.0)


def test_two_at_once_each_after_its_fill(side):
    """As test_two_at_once, with every run's stream behind the fills of what it writes: those are
    the current stream's, which streams of torch do not wait for by themselves."""
    t, nf4 = side.torch, side.nf4
    runs = []
    for seed, (dim, kvh, seqs) in ((4, (128, 2, 40)), (5, (64, 4, 24))):
        cache = nf4.KVCache(1, 200, kvh, 16, dim)
        width = SAVED // ((seqs - 3) * kvh * 2 * dim) // 16 + 2
        b, g, x = branches_of(side, cache, np.arange(200), seqs, width, 960, seed)
        need = nf4.nf4_kv_attention_shared_workspace_bytes(cache, b, g, 4 * kvh)
        want = outputs(side, cache, seqs)
        ws = t.empty(need, dtype=t.uint8, device="cuda")
        step(side, cache, b, g, x, ws, want)
        runs.append((cache, b, g, x, ws, want, outputs(side, cache, seqs), t.cuda.Stream()))
    t.cuda.synchronize()
    for _ in range(10):
        for cache, b, g, x, ws, _, got, stream in runs:
            for a in got:
                a.fill_(7.0)
            stream.wait_stream(t.cuda.current_stream())
            step(side, cache, b, g, x, ws, got, stream)
        t.cuda.synchronize()
        for *_, want, got, _ in runs:
            assert all(t.equal(a, b) for a, b in zip(want, got))
