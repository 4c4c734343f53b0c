"""What the Python structures of the key-value cache tell the library, and what
they refuse, without a GPU."""
import ctypes

import pytest

from bit_weight_only_amd import nf4
from test_kv_abi_cpu import A, batch, cache

torch = pytest.importorskip("torch")


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_a_table_of_columns_has_its_own_entries():
    wide = i32(3, 9)
    for view, stride, entries in ((wide, 9, 9), (wide[:, :4], 9, 4), (wide[:, 5:], 9, 4),
                                  (wide[1:, 8:], 9, 1), (i32(1, 5).expand(3, 5)[:1], 5, 5)):
        b = nf4.KVBatch(i32(len(view)), view)
        assert (b.struct.table_stride, b.struct.table_entries) == (stride, entries)
        # the last entry that may be read lies in the tensor
        last = view.storage_offset() + (len(view) - 1) * stride + entries
        assert last <= view.untyped_storage().nbytes() // 4


def test_tables_that_are_no_rows_of_entries_are_refused():
    for bad in (i32(1, 5).expand(3, 5), i32(20).as_strided((3, 5), (4, 1)), i32(3, 0), i32(3, 9)[:, :0],
                i32(5, 3).T):
        with pytest.raises(nf4.NF4Error) as e:
            nf4.KVBatch(i32(3), bad)
        assert e.value.status == nf4.NF4_ERR_SHAPE


@pytest.mark.parametrize("entries", [-1, 4])
def test_entries_outside_the_stride_are_refused(entries):
    b = batch(table_entries=entries)
    f = nf4.lib()
    assert f.nf4_kv_append(cache(), 0, b, A, 512, A, 512, 0, None) == nf4.NF4_ERR_SHAPE
    assert f.nf4_kv_attention(cache(), 0, b, A, 1024, 8, 0.1, 0, 0, A, None, None, 0,
                              None) == nf4.NF4_ERR_SHAPE
    assert f.nf4_kv_attention_workspace_bytes(cache(), b, 8, 0, 0) == 0


def test_fewer_entries_need_less_workspace():
    size = nf4.lib().nf4_kv_attention_workspace_bytes
    need = [size(cache(), batch(seqs=1, rows=1, max_rows=1, max_len=1 << 20, table_stride=1 << 15,
                                table_entries=n), 28, 0, 0) for n in (0, 1 << 15, 1 << 10, 1)]
    assert need[0] == need[1] > need[2] > need[3] == 0
    assert ctypes.sizeof(nf4._KVBatch) == 9 * 8


def test_caches_of_other_types_are_refused():
    n = 4 * 2 * 16 * 64
    codes, scales = torch.zeros(n, dtype=torch.uint8), torch.zeros(8)
    new = lambda **kw: nf4.KVCache(1, 4, 2, 16, 64, device="cpu", **kw)  # noqa: E731
    for kw in (dict(k=codes), dict(v=codes.view(torch.float8_e4m3fn)), dict(k_scale=scales),
               dict(v_scale=scales.view(torch.uint8))):
        new(**kw)
    for kw in (dict(k=codes.view(torch.float32)), dict(v=codes.view(torch.bfloat16)),
               dict(k_scale=scales.int()), dict(v_scale=torch.zeros(4, dtype=torch.float64))):
        with pytest.raises(nf4.NF4Error) as e:
            new(**kw)
        assert e.value.status == nf4.NF4_ERR_SHAPE


def test_structures_on_the_host_are_refused():
    """Every call that would launch a kernel on a host address."""
    c, b = nf4.KVCache(1, 4, 2, 16, 64, device="cpu"), nf4.KVBatch(i32(2), i32(2, 4))
    p, x = nf4.KVPool(i32(4), i32(2, 4), i32(2)), torch.zeros(2, 128)
    calls = [lambda: nf4.nf4_kv_append(c, 0, b, x, 128, x, 128, nf4.NF4_KV_F32, stream=0),
             lambda: nf4.nf4_kv_attention(c, 0, b, x, 128, 2, 0.1, 0, 0, x, stream=0),
             lambda: nf4.nf4_kv_copy_pages(c, i32(1), i32(1), 1, stream=0),
             lambda: nf4.nf4_kv_reserve(c, p, i32(2), stream=0),
             lambda: nf4.nf4_kv_fork(c, p, i32(1), i32(1), 1, stream=0),
             lambda: nf4.nf4_kv_release(c, p, i32(1), 1, stream=0),
             lambda: nf4.nf4_kv_compact(c, p, i32(4), i32(2, 4), x, 1024, stream=0)]
    for call in calls:
        with pytest.raises(nf4.NF4Error) as e:
            call()
        assert e.value.status == nf4.NF4_ERR_SHAPE


def test_tensors_of_several_devices_are_no_gpus():
    class T:
        def __init__(self, index):
            self.is_cuda, self.device = index is not None, torch.device("cpu" if index is None else f"cuda:{index}")
    assert nf4._gpu(T(0), None, T(0)) == 0 and nf4._gpu(T(1)) == 1
    assert nf4._gpu(T(0), T(1)) == nf4._gpu(T(0), T(None)) == nf4._gpu(T(None)) == -1


def test_a_pool_with_too_few_counts_is_refused():
    """Checked as for a pool on a GPU, which this one is made out to be."""
    c, p = nf4.KVCache(1, 4, 2, 16, 64, device="cpu"), nf4.KVPool(i32(3), i32(2, 4), i32(2))
    c.gpu = p.gpu = 0
    for call in (lambda: nf4.nf4_kv_reserve(c, p, i32(2), stream=0),
                 lambda: nf4.nf4_kv_fork(c, p, i32(1), i32(1), 1, stream=0),
                 lambda: nf4.nf4_kv_release(c, p, i32(1), 1, stream=0),
                 lambda: nf4.nf4_kv_compact(c, p, i32(4), i32(2, 4), i32(300), 1200, stream=0)):
        with pytest.raises(nf4.NF4Error, match="fewer counts than pages") as e:
            call()
        assert e.value.status == nf4.NF4_ERR_SHAPE


@pytest.mark.parametrize("there", [True, False])
def test_current_stream_with_and_without_the_raw_handle(monkeypatch, there):
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: type("S", (), {"cuda_stream": 0x40})())
    if there:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0x30 + d, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert nf4._stream(None) == (0x33 if there else 0x40)
