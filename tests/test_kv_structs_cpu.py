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
