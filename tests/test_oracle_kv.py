"""The plain key-value cache that the GPU tests compare with, pinned on its
own: the code table and its rounding against torch's e4m3 type, scales at the
ends of their range, what appending token by token may change, and attention
against a softmax written another way."""
import numpy as np
import pytest

from oracle import kv


def test_values_and_rounding_are_e4m3():
    torch = pytest.importorskip("torch")
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(kv.VALUES, want.astype(np.float64), equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 4000), rng.normal(0, 1e-2, 4000),
                        (kv.VALUES[:126] + kv.VALUES[1:127]) / 2,  # every tie
                        kv.VALUES[:127], [0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10]]).astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv.encode(x), got)
    assert list(kv.encode([np.nan, np.inf, -np.inf, 1e9])) == [127, 126, 254, 126]


@pytest.mark.parametrize("amax,e", [(0.0, -40), (448.0, 0), (448.0001, 1), (447.0, 0), (224.0, -1),
                                    (2.0 ** -60, -40), (448 * 2.0 ** 100, 100), (3e38, 100)])
def test_exponent(amax, e):
    assert kv.exponent(amax) == e


def test_token_by_token_differs_from_at_once_by_subnormals_only():
    rng = np.random.default_rng(1)
    n, table = 40, np.array([[2, 0, 1]])
    x = rng.normal(0, 1, (n, 1, 8)) * 2.0 ** rng.integers(-3, 4, (n, 1, 1))
    one, all_ = kv.Cache(1, 3, 1, 16, 8), kv.Cache(1, 3, 1, 16, 8)
    kv.append(all_, 0, table, [0, n], [n], x, x)
    for t in range(n):
        kv.append(one, 0, table, [0, 1], [t + 1], x[t:t + 1], x[t:t + 1])
    assert np.array_equal(one.ks, all_.ks) and np.array_equal(one.vs, all_.vs)
    a, b = one.dense(0, 0, 0, table[0], n)[0], all_.dense(0, 0, 0, table[0], n)[0]
    scale = np.repeat(all_.ks[0, table[0], 0, 0], 16)[:n, None].astype(np.float64)
    normal = np.abs(b) >= scale * 2.0 ** -6
    assert np.array_equal(a[normal], b[normal])
    assert np.max(np.abs(a - b) / scale) <= 2.0 ** -9


def test_attention_against_a_softmax_in_another_order():
    rng = np.random.default_rng(2)
    c = kv.Cache(1, 4, 2, 16, 8)
    table, n = np.array([[3, 1, 0, 2]]), 50
    kv.append(c, 0, table, [0, n], [n], rng.normal(size=(n, 2, 8)), rng.normal(size=(n, 2, 8)))
    q = rng.normal(size=(5, 4, 8))
    out, lse, _, _ = kv.attention(c, 0, table, [0, 5], [n], q, 0.3, 10, 2)
    for r in range(5):
        at = n - 5 + r
        for i in range(4):
            k, v = (c.dense(x, 0, i // 2, table[0], n)[0] for x in (0, 1))
            num, den = np.zeros(8), 0.0
            for j in list(range(2)) + list(range(at - 9, at + 1)):
                w = np.exp(0.3 * float(q[r, i] @ k[j]))
                num, den = num + w * v[j], den + w
            assert np.allclose(out[r, i], num / den, rtol=1e-12)
            assert np.isclose(lse[r, i], np.log(den), rtol=1e-12)


def test_pool_keeps_its_counts():
    p = kv.Pool(8, 4, 6, 16)
    p.reserve([40, 0, 16, 0])
    assert p.table[0, :3].tolist() == [0, 1, 2] and p.table[2, 0] == 3 and p.missing == 0
    p.fork([0, 2], [1, 3])
    assert p.table[1, :3].tolist() == [0, 1, 4] and p.refs[:5].tolist() == [2, 2, 1, 2, 1]
    p.reserve([200, 0, 0, 0])
    assert p.missing == 15 - 6 and p.len[0] == 240
    p.release([0])
    assert p.refs.tolist() == [1, 1, 0, 2, 1, 0, 0, 0]
    p.compact()
    assert p.refs.tolist() == [1, 1, 1, 2, 0, 0, 0, 0] and p.table[1, :3].tolist() == [0, 1, 2]
