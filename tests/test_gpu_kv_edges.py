"""The 8-bit key-value cache where it holds little or unusual things."""
import numpy as np
import pytest

from oracle import kv

from gpu_helpers import say
from test_gpu_kv import Case, bf16, device_batch, same_cache, side  # noqa: F401

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
