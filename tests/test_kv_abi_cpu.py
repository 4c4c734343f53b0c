"""The key-value cache's entry points without a GPU: size queries, and bad
arguments refused on the host before any HIP call."""
import ctypes

import pytest

from bit_weight_only_amd import nf4

A = 1 << 20  # a 16-byte aligned stand-in address; never dereferenced


def cache(**kw):
    v = dict(k=A, v=A, k_scale=A, v_scale=A, layers=2, pages=10, kv_heads=4, page_tokens=64,
             head_dim=128) | kw
    return ctypes.pointer(nf4._KVCache(**v))


def batch(**kw):
    v = dict(seqs=2, rows=5, max_rows=4, max_len=100, row_start=A, kv_len=A, table=A,
             table_stride=3) | kw
    return ctypes.pointer(nf4._KVBatch(**v))


def pool(**kw):
    v = dict(refs=A, table=A, table_rows=3, table_stride=3, len=A, missing=None) | kw
    return ctypes.pointer(nf4._KVPool(**v))


BAD_SHAPES = [dict(layers=0), dict(pages=0), dict(pages=(1 << 24) + 1), dict(kv_heads=0),
              dict(kv_heads=1025), dict(page_tokens=0), dict(page_tokens=48), dict(page_tokens=8),
              dict(page_tokens=512), dict(head_dim=96), dict(head_dim=0), dict(layers=1 << 22, pages=1 << 24)]


@pytest.mark.parametrize("dim,page,heads", [(64, 16, 1), (128, 64, 4), (128, 256, 8)])
def test_sizes(dim, page, heads):
    c = cache(head_dim=dim, page_tokens=page, kv_heads=heads)
    assert nf4.lib().nf4_kv_code_bytes(c) == 2 * 10 * heads * page * dim
    assert nf4.lib().nf4_kv_scale_bytes(c) == 2 * 10 * heads * page // 16 * 4
    assert nf4.lib().nf4_kv_compact_workspace_bytes(c) >= 3 * 4 * 10


@pytest.mark.parametrize("bad", BAD_SHAPES)
def test_cache_shapes_refused(bad):
    L, c = nf4.lib(), cache(**bad)
    assert L.nf4_kv_code_bytes(c) == L.nf4_kv_scale_bytes(c) == L.nf4_kv_compact_workspace_bytes(c) == 0
    assert L.nf4_kv_append(c, 0, batch(), A, 1 << 17, A, 1 << 17, 0, None) == nf4.NF4_ERR_SHAPE
    assert L.nf4_kv_copy_pages(c, A, A, 1, None) == nf4.NF4_ERR_SHAPE
    assert L.nf4_kv_reserve(c, pool(), A, None) == nf4.NF4_ERR_SHAPE


BAD_BATCHES = [(dict(kv_len=None), nf4.NF4_ERR_NULL), (dict(table=None), nf4.NF4_ERR_NULL),
               (dict(row_start=None), nf4.NF4_ERR_NULL), (dict(seqs=0), nf4.NF4_ERR_SHAPE),
               (dict(rows=0), nf4.NF4_ERR_SHAPE), (dict(max_rows=0), nf4.NF4_ERR_SHAPE),
               (dict(max_rows=6), nf4.NF4_ERR_SHAPE), (dict(max_len=-1), nf4.NF4_ERR_SHAPE),
               (dict(max_len=(1 << 30) + 1), nf4.NF4_ERR_SHAPE), (dict(table_stride=0), nf4.NF4_ERR_SHAPE),
               (dict(rows=(1 << 23) + 1), nf4.NF4_ERR_SHAPE), (dict(kv_len=A + 2), nf4.NF4_ERR_ALIGN),
               (dict(table=A + 1), nf4.NF4_ERR_ALIGN), (dict(row_start=A + 2), nf4.NF4_ERR_ALIGN)]


@pytest.mark.parametrize("bad,status", BAD_BATCHES)
def test_batches_refused(bad, status):
    b = batch(**bad)
    assert nf4.lib().nf4_kv_append(cache(), 0, b, A, 512, A, 512, 0, None) == status
    assert nf4.lib().nf4_kv_attention(cache(), 0, b, A, 1024, 8, 0.1, 0, 0, A, None, None, 0,
                                      None) == status


def test_append_refusals():
    f = nf4.lib().nf4_kv_append
    ok = [cache(), 0, batch(), A, 512, A, 512, 0, None]

    def status(i, v):
        a = list(ok)
        a[i] = v
        return f(*a)
    for i in (0, 2, 3, 5):
        assert status(i, None) == nf4.NF4_ERR_NULL
    for name in ("k", "v", "k_scale", "v_scale"):
        assert status(0, cache(**{name: None})) == nf4.NF4_ERR_NULL
        assert status(0, cache(**{name: A + 8})) == nf4.NF4_ERR_ALIGN
    for i, v in ((1, -1), (1, 2), (4, 504), (6, 511), (7, 2), (7, -1)):
        assert status(i, v) == nf4.NF4_ERR_SHAPE, (i, v)
    for i, v in ((3, A + 8), (5, A + 2), (4, 516), (6, 513)):
        assert status(i, v) == nf4.NF4_ERR_ALIGN, (i, v)


def test_attention_refusals():
    f = nf4.lib().nf4_kv_attention
    ok = [cache(), 0, batch(), A, 1024, 8, 0.1, 0, 0, A, None, A, 1 << 30, None]

    def status(i, v):
        a = list(ok)
        a[i] = v
        return f(*a)
    for i in (0, 2, 3, 9):
        assert status(i, None) == nf4.NF4_ERR_NULL
    for i, v in ((1, 2), (4, 1016), (5, 0), (5, 6), (5, -4), (6, 0.0), (6, -1.0), (6, float("nan")),
                 (6, float("inf")), (7, -1), (8, -1)):
        assert status(i, v) == nf4.NF4_ERR_SHAPE, (i, v)
    for i, v in ((3, A + 8), (4, 1028), (9, A + 4), (10, A + 2)):
        assert status(i, v) == nf4.NF4_ERR_ALIGN, (i, v)


def test_attention_workspace():
    """A long batch of few rows is summed in parts that meet in the workspace."""
    size = nf4.lib().nf4_kv_attention_workspace_bytes
    b = batch(seqs=1, rows=1, max_rows=1, max_len=1 << 20, table_stride=1 << 20)
    need = size(cache(), b, 28, 0, 0)
    f = nf4.lib().nf4_kv_attention
    if need:
        assert f(cache(), 0, b, A, 3584, 28, 0.1, 0, 0, A, None, None, 0, None) == nf4.NF4_ERR_NULL
        assert f(cache(), 0, b, A, 3584, 28, 0.1, 0, 0, A, None, A, need - 1,
                 None) == nf4.NF4_ERR_WORKSPACE
        assert f(cache(), 0, b, A, 3584, 28, 0.1, 0, 0, A, None, A + 8, need,
                 None) == nf4.NF4_ERR_ALIGN
    assert size(cache(head_dim=96), b, 28, 0, 0) == 0
    assert size(cache(), b, 27, 0, 0) == 0
    assert size(cache(), b, 28, -1, 0) == 0
    assert size(cache(), batch(seqs=0), 28, 0, 0) == 0


def test_pool_refusals():
    L = nf4.lib()
    calls = {"reserve": lambda c, p: L.nf4_kv_reserve(c, p, A, None),
             "fork": lambda c, p: L.nf4_kv_fork(c, p, A, A, 1, None),
             "release": lambda c, p: L.nf4_kv_release(c, p, A, 1, None),
             "compact": lambda c, p: L.nf4_kv_compact(c, p, A, A, A, 1 << 20, None)}
    for name, f in calls.items():
        assert f(None, pool()) == f(cache(), None) == nf4.NF4_ERR_NULL, name
        for field in ("refs", "table", "len"):
            assert f(cache(), pool(**{field: None})) == nf4.NF4_ERR_NULL, name
        for bad in (dict(table_rows=0), dict(table_stride=0), dict(table_rows=1 << 23, table_stride=1 << 30)):
            assert f(cache(), pool(**bad)) == nf4.NF4_ERR_SHAPE, name
        for bad in (dict(refs=A + 4), dict(table=A + 2), dict(len=A + 1), dict(missing=A + 2)):
            assert f(cache(), pool(**bad)) == nf4.NF4_ERR_ALIGN, name
    for n in (0, 4, -1):  # more than the table has rows
        assert L.nf4_kv_fork(cache(), pool(), A, A, n, None) == nf4.NF4_ERR_SHAPE
        assert L.nf4_kv_release(cache(), pool(), A, n, None) == nf4.NF4_ERR_SHAPE
    assert L.nf4_kv_fork(cache(), pool(), None, A, 1, None) == nf4.NF4_ERR_NULL
    assert L.nf4_kv_copy_pages(cache(), A, None, 1, None) == nf4.NF4_ERR_NULL
    assert L.nf4_kv_copy_pages(cache(), A, A, 0, None) == nf4.NF4_ERR_SHAPE
    assert L.nf4_kv_copy_pages(cache(), A + 2, A, 1, None) == nf4.NF4_ERR_ALIGN
    need = L.nf4_kv_compact_workspace_bytes(cache())
    assert L.nf4_kv_compact(cache(), pool(), A, A, A, need - 1, None) == nf4.NF4_ERR_WORKSPACE
    assert L.nf4_kv_compact(cache(), pool(), A, A, None, need, None) == nf4.NF4_ERR_NULL
    assert L.nf4_kv_compact(cache(), pool(), A + 4, A, A, need, None) == nf4.NF4_ERR_ALIGN
    assert L.nf4_kv_compact(cache(), pool(), A, A, A + 4, need, None) == nf4.NF4_ERR_ALIGN


def test_python_structures_refuse_wrong_tensors():
    torch = pytest.importorskip("torch")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(nf4.NF4Error):
        nf4.KVCache(1, 4, 2, 48, 128, device="cpu")
    with pytest.raises(nf4.NF4Error):
        nf4.KVCache(1, 4, 2, 16, 64, device="cpu", k=torch.zeros(5, dtype=torch.uint8))
    c = nf4.KVCache(1, 4, 2, 16, 64, device="cpu")
    assert c.v.shape == (1, 4, 2, 4, 64, 4) and c.k_scale.shape == (1, 4, 2, 1)
    with pytest.raises(nf4.NF4Error):
        nf4.KVBatch(i(3), i(2, 4))
    with pytest.raises(nf4.NF4Error):
        nf4.KVBatch(i(3).long(), i(3, 4))
    with pytest.raises(nf4.NF4Error):
        nf4.KVBatch(i(3), i(3, 4), row_start=i(3))
    with pytest.raises(nf4.NF4Error):
        nf4.KVPool(i(4), i(3, 4), i(2))
    # a table of one row may carry any stride, a slice of a wider one its own
    assert nf4.KVBatch(i(1), i(5).as_strided((1, 5), (0, 1))).struct.table_stride == 5
    assert nf4.KVBatch(i(2), i(3, 9)[:, :4]).struct.table_stride == 9
