"""Rotary positions and reading the cache without a GPU: the frequencies and the
turns that the host works out, and bad arguments refused before any HIP call."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from bit_weight_only_amd import nf4
from oracle import rotary as plain
from test_kv_abi_cpu import A, BAD_BATCHES, BAD_SHAPES, batch, cache

SCALED = [("plain", {}), ("linear", dict(factor=2.5)), ("base", dict(factor=3.0)),
          ("ramp", dict(factor=4.0, original=4096.0, low=1.0, high=32.0)),
          ("ramp", dict(factor=16.0, original=100.0, low=1.0, high=1.5)),
          ("smooth", dict(factor=8.0, original=8192.0, low=1.0, high=4.0))]
# pi to 50 digits
PI = Fraction("3.14159265358979323846264338327950288419716939937511")


def scaling(name):
    return getattr(nf4, "NF4_SCALING_" + name.upper())


@pytest.mark.parametrize("dims", [0, 2, 4, 50, 64, 96, 128])
@pytest.mark.parametrize("base", [1e4, 1e6])
@pytest.mark.parametrize("name,kw", SCALED)
def test_frequencies(dims, base, name, kw):
    got = nf4.nf4_rotary_frequencies(dims, base, scaling(name), **kw)
    want = plain.frequencies(dims, base, name, **kw)
    # a power, a logarithm and a few products in 64 bits
    np.testing.assert_allclose(got, want, rtol=2.0 ** -45)
    assert len(got) == dims // 2


def test_frequencies_scaled_for_longer_contexts():
    """The ends of the scalings: fast pairs stay, slow ones are divided, and a
    pair in between lies between."""
    f = nf4.nf4_rotary_frequencies(128, 1e4)
    for name, kw in SCALED[3:4] + SCALED[5:]:
        r = nf4.nf4_rotary_frequencies(128, 1e4, scaling(name), **kw) / f
        assert r[0] == 1.0 and abs(r[-1] * kw["factor"] - 1) < 1e-12
        assert np.all(np.diff(r) <= 1e-15) and len(set(np.round(r, 9))) > 4
    # BASE divides the slowest pair by the factor and leaves the fastest
    r = nf4.nf4_rotary_frequencies(128, 1e4, nf4.NF4_SCALING_BASE, 3.0) / f
    assert r[0] == 1.0 and abs(r[-1] * 3 - 1) < 1e-12


BAD_FREQUENCIES = [(1, 1e4, 0, 1, 0, 0, 0), (130, 1e4, 0, 1, 0, 0, 0), (-2, 1e4, 0, 1, 0, 0, 0),
                   (64, 1.0, 0, 1, 0, 0, 0), (64, math.inf, 0, 1, 0, 0, 0), (64, math.nan, 0, 1, 0, 0, 0),
                   (64, 1e4, -1, 1, 0, 0, 0), (64, 1e4, 5, 1, 0, 0, 0), (64, 1e4, 1, 0, 0, 0, 0),
                   (64, 1e4, 1, math.nan, 0, 0, 0), (64, 1e4, 2, -1, 0, 0, 0), (64, 1e4, 2, 1e-9, 0, 0, 0),
                   (64, 1e4, 3, 2, 0, 1, 4), (64, 1e4, 3, 2, 4096, 4, 4), (64, 1e4, 4, 2, 4096, 0, 4),
                   (64, 1e4, 4, 2, math.inf, 1, 4)]


@pytest.mark.parametrize("bad", BAD_FREQUENCIES)
def test_bad_frequencies(bad):
    out = (ctypes.c_double * 64)(*[7.0] * 64)
    assert nf4.lib().nf4_rotary_frequencies(*bad, out) == nf4.NF4_ERR_SHAPE
    assert list(out) == [7.0] * 64
    assert nf4.lib().nf4_rotary_frequencies(*bad, None) == nf4.NF4_ERR_NULL


def test_turns():
    """2^64 times the part of a turn past the last whole one, to 80 bits' rounding."""
    f = [0.0, 1.0, -1.0, 1e-6, 0.333, 7.0, -123.456, 2.0 ** 20, 2.0 * math.pi, 1e-30, -1e-30]
    r = nf4._Rotary()
    nf4.nf4_rotary_init(r, 2 * len(f), nf4.NF4_ROTARY_PAIRS, f, 1.5)
    assert (r.dims, r.layout, r.gain) == (2 * len(f), 1, 1.5) and not any(r.turns[len(f):])
    for x, got in zip(f, r.turns):
        turn = Fraction(x) / (2 * PI)
        want = (turn - math.floor(turn)) * 2 ** 64
        off = abs(want - got)
        off = min(off, 2 ** 64 - off)
        # the 80-bit quotient is right to 2^-64 of itself, pi to as much, and half a unit
        assert off <= 0.5 + 2 * abs(turn) + 1e-9, (x, got, float(off))
    assert ctypes.sizeof(nf4._Rotary) == 24 + 64 * 8


def test_init_refusals():
    r, f = nf4._Rotary(), (ctypes.c_double * 64)()
    init = nf4.lib().nf4_rotary_init
    assert init(ctypes.byref(r), 128, 0, f, 1.0) == init(ctypes.byref(r), 0, 0, None, 1.0) == nf4.NF4_OK
    assert init(None, 128, 0, f, 1.0) == init(ctypes.byref(r), 2, 0, None, 1.0) == nf4.NF4_ERR_NULL
    for dims, layout, gain in ((130, 0, 1.0), (3, 0, 1.0), (-2, 0, 1.0), (64, 2, 1.0), (64, -1, 1.0),
                               (64, 0, math.nan), (64, 0, math.inf)):
        assert init(ctypes.byref(r), dims, layout, f, gain) == nf4.NF4_ERR_SHAPE
    for x in (math.nan, math.inf, -2.0 ** 21):
        f[3] = x
        assert init(ctypes.byref(r), 128, 0, f, 1.0) == nf4.NF4_ERR_SHAPE
        assert init(ctypes.byref(r), 6, 0, f, 1.0) == nf4.NF4_OK  # not looked at
    with pytest.raises(nf4.NF4Error):
        nf4.Rotary(64, frequencies=[1.0] * 31)
    with pytest.raises(nf4.NF4Error):
        nf4.Rotary(63)


def rotary(**kw):
    r = nf4.Rotary(64).struct
    for k, v in kw.items():
        setattr(r, k, v)
    return ctypes.pointer(r)


BAD_ROTARY = [dict(dims=130), dict(dims=3), dict(dims=-2), dict(layout=2), dict(gain=math.nan)]


def test_rotate_refusals():
    f = nf4.lib().nf4_rotate
    ok = [rotary(), A, 1024, 0, A, 5, 8, 128, A, 1e-6, 2 * A, 1024, 0, None]

    def status(*changes):
        a = list(ok)
        for i, v in changes:
            a[i] = v
        return f(*a)
    for i in (0, 1, 4, 10):
        assert status((i, None)) == nf4.NF4_ERR_NULL
    for bad in BAD_ROTARY:
        assert status((0, rotary(**bad))) == nf4.NF4_ERR_SHAPE
    for i, v in ((2, 1016), (3, 2), (5, 0), (5, (1 << 23) + 1), (6, 0), (6, 65537), (7, 96), (7, 0),
                 (9, 0.0), (9, math.nan), (9, math.inf), (9, -1.0), (9, 2.0 ** -101), (11, 1016), (12, -1)):
        assert status((i, v)) == nf4.NF4_ERR_SHAPE, (i, v)
    assert status((0, rotary(dims=66)), (7, 64), (6, 16)) == nf4.NF4_ERR_SHAPE  # more than the head
    for i, v in ((1, A + 8), (2, 1028), (4, A + 2), (8, A + 4), (10, 2 * A + 8), (11, 1028)):
        assert status((i, v)) == nf4.NF4_ERR_ALIGN, (i, v)
    wide = (1 << 24) + 8  # rows further apart than the kernels go
    assert status((2, wide)) == status((11, wide)) == nf4.NF4_ERR_SHAPE
    # in place with another type or stride
    assert status((10, A), (12, 1)) == status((10, A), (11, 1032)) == nf4.NF4_ERR_SHAPE


def test_append_rotated_refusals():
    f = nf4.lib().nf4_kv_append_rotated
    ok = [cache(), 0, batch(), rotary(), A, 1024, 8, A, A, 512, A, A, 512, 0, 1e-6, 2 * A, None]

    def status(*changes):
        a = list(ok)
        for i, v in changes:
            a[i] = v
        return f(*a)
    for i in (0, 2, 3, 4, 8, 11, 15):
        assert status((i, None)) == nf4.NF4_ERR_NULL
    for bad in BAD_SHAPES:
        assert status((0, cache(**bad))) == nf4.NF4_ERR_SHAPE
    for bad, want in BAD_BATCHES:
        assert status((2, batch(**bad))) == want
    for bad in BAD_ROTARY:
        assert status((3, rotary(**bad))) == nf4.NF4_ERR_SHAPE
    for i, v in ((1, -1), (1, 2), (5, 1016), (6, 0), (6, 6), (6, -4), (9, 504), (12, 504), (13, 2),
                 (14, 0.0), (14, math.nan)):
        assert status((i, v)) == nf4.NF4_ERR_SHAPE, (i, v)
    for i, v in ((4, A + 8), (5, 1028), (7, A + 4), (8, A + 2), (9, 516), (10, A + 8), (11, A + 8),
                 (12, 513), (15, A + 2)):
        assert status((i, v)) == nf4.NF4_ERR_ALIGN, (i, v)
    assert status((15, A), (13, 1)) == status((15, A), (5, 1032)) == nf4.NF4_ERR_SHAPE
    wide = (1 << 24) + 8  # rows further apart than the kernels go
    assert status((5, wide)) == status((9, wide)) == status((12, wide)) == nf4.NF4_ERR_SHAPE


def test_read_refusals():
    f = nf4.lib().nf4_kv_read
    ok = [cache(), 0, batch(), A, 512, 2 * A, 512, 0, None]

    def status(i, v):
        a = list(ok)
        a[i] = v
        return f(*a)
    for i in (0, 2, 3, 5):
        assert status(i, None) == nf4.NF4_ERR_NULL
    for bad in BAD_SHAPES:
        assert status(0, cache(**bad)) == nf4.NF4_ERR_SHAPE
    for bad, want in BAD_BATCHES:
        assert status(2, batch(**bad)) == want
    wide = (1 << 24) + 8  # rows further apart than the kernels go
    for i, v in ((1, -1), (1, 2), (4, 504), (6, 511), (7, 2), (7, -1), (5, A), (4, wide), (6, wide)):
        assert status(i, v) == nf4.NF4_ERR_SHAPE, (i, v)
    for i, v in ((3, A + 8), (5, A + 2), (4, 516), (6, 513)):
        assert status(i, v) == nf4.NF4_ERR_ALIGN, (i, v)


def groups(**kw):
    v = dict(groups=2, max_rows=0, max_prefix=64, first=A, prefix_len=A) | kw
    return ctypes.pointer(nf4._KVGroups(**v))


def test_shared_attention_refusals():
    f, size = nf4.lib().nf4_kv_attention_shared, nf4.lib().nf4_kv_attention_shared_workspace_bytes
    # 64 sequences that share so much that it is taken apart, through the workspace
    big = dict(seqs=64, rows=64, max_rows=1, max_len=1 << 20, table_stride=1 << 15)
    ok = [cache(), 0, batch(**big), groups(max_prefix=4096), A, 1024, 8, 0.1, 0, 0, A, None, A, 1 << 30, None]

    def status(*changes):
        a = list(ok)
        for i, v in changes:
            a[i] = v
        return f(*a)
    for i in (0, 2, 3, 4, 10):
        assert status((i, None)) == nf4.NF4_ERR_NULL
    assert status((3, groups(prefix_len=None))) == nf4.NF4_ERR_NULL
    for bad in (dict(groups=0), dict(groups=65), dict(groups=-1), dict(first=None), dict(max_rows=-1),
                dict(max_prefix=-1), dict(max_prefix=(1 << 30) + 1)):
        assert status((3, groups(**bad))) == nf4.NF4_ERR_SHAPE, bad
        assert size(cache(), batch(**big), groups(**bad), 8, 0, 0) == 0
    for bad in (dict(first=A + 2), dict(prefix_len=A + 1)):
        assert status((3, groups(**bad))) == nf4.NF4_ERR_ALIGN
    for bad, want in BAD_BATCHES:
        assert status((2, batch(**bad))) == want
    for bad in BAD_SHAPES:
        assert status((0, cache(**bad))) == nf4.NF4_ERR_SHAPE
        assert size(cache(**bad), batch(**big), groups(), 8, 0, 0) == 0
    for i, v in ((1, 2), (5, 1016), (6, 0), (6, 6), (7, 0.0), (7, math.nan), (8, -1), (9, -1)):
        assert status((i, v)) == nf4.NF4_ERR_SHAPE, (i, v)
    for i, v in ((4, A + 8), (5, 1028), (10, A + 4), (11, A + 2)):
        assert status((i, v)) == nf4.NF4_ERR_ALIGN, (i, v)
    need = size(cache(), batch(**big), groups(max_prefix=4096), 8, 0, 0)
    # slots of every row and head's sums
    assert need > 0 and need % (64 * 8 * (128 + 2) * 4) == 0
    assert status((12, None)) == nf4.NF4_ERR_NULL
    assert status((13, need - 1)) == nf4.NF4_ERR_WORKSPACE
    assert status((12, A + 8)) == nf4.NF4_ERR_ALIGN
    # nothing shared, and rows that fill tiles by themselves: as without groups
    plain_size = nf4.lib().nf4_kv_attention_workspace_bytes
    assert size(cache(), batch(), groups(max_prefix=0), 8, 0, 0) == plain_size(cache(), batch(), 8, 0, 0)
    many = batch(seqs=2, rows=400, max_rows=200, max_len=60000, table_stride=1000)
    assert size(cache(), many, groups(), 8, 0, 0) == plain_size(cache(), many, 8, 0, 0) > 0


def test_python_groups():
    torch = pytest.importorskip("torch")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for bad in ((i(2),), (i(2), i(2)), (i(0), i(1)), (i(1).long(),), (i(2), i(3).long()), (i(2), i(6)[::2])):
        with pytest.raises(nf4.NF4Error) as e:
            nf4.KVGroups(*bad)
        assert e.value.status == nf4.NF4_ERR_SHAPE
    g = nf4.KVGroups(i(2), i(3), max_rows=5)
    assert (g.struct.groups, g.struct.max_rows, g.struct.max_prefix, g.gpu) == (2, 5, 1 << 30, -1)
    assert nf4.KVGroups(i(1)).struct.first is None and ctypes.sizeof(nf4._KVGroups) == 40


def test_tensors_on_the_host_are_refused():
    torch = pytest.importorskip("torch")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    c, b = nf4.KVCache(1, 4, 2, 16, 64, device="cpu"), nf4.KVBatch(i32(2), i32(2, 4))
    x, r = torch.zeros(2, 128), nf4.Rotary(64)
    out = torch.zeros(2, 128, dtype=torch.bfloat16)
    calls = [lambda: nf4.nf4_kv_read(c, 0, b, x, 128, x, 128, nf4.NF4_KV_F32, stream=0),
             lambda: nf4.nf4_kv_append_rotated(c, 0, b, r, x, 128, 2, None, x, 128, None, x, 128,
                                               nf4.NF4_KV_F32, 1e-6, out, stream=0),
             lambda: nf4.nf4_rotate(r, x, 128, nf4.NF4_KV_F32, i32(2), 2, 2, 64, None, 0.0, x, 128,
                                    nf4.NF4_KV_F32, stream=0)]
    for call in calls:
        with pytest.raises(nf4.NF4Error) as e:
            call()
        assert e.value.status == nf4.NF4_ERR_SHAPE
    with pytest.raises(nf4.NF4Error, match="not on one GPU"):
        nf4.nf4_kv_attention_shared(c, 0, b, nf4.KVGroups(i32(1)), out, 128, 2, 0.1, 0, 0, out, stream=0)
    c.gpu = b.gpu = 0  # structures made out to be on a GPU, rows that are not
    for call in calls[:2]:
        with pytest.raises(nf4.NF4Error, match="not on one GPU"):
            call()


def test_streams_of_another_gpu_are_refused(monkeypatch):
    torch = pytest.importorskip("torch")

    class Stream:
        def __init__(self, index):
            self.device, self.cuda_stream = torch.device(f"cuda:{index}"), 0x50 + index
    monkeypatch.setattr(nf4, "_kinds", {})
    monkeypatch.setattr(nf4, "_current_device", lambda: 1, raising=False)
    monkeypatch.setattr(nf4, "_raw_stream", lambda gpu: 0x76 + gpu, raising=False)
    assert nf4._stream_on("f", 1, None) == 0x77
    assert nf4._stream_on("f", 0, 0x60) == 0x60
    assert nf4._stream_on("f", 2, Stream(2)) == 0x52
    for gpu, stream in ((0, None), (0, Stream(1)), (1, Stream(0))):
        with pytest.raises(nf4.NF4Error) as e:
            nf4._stream_on("f", gpu, stream)
        assert e.value.status == nf4.NF4_ERR_SHAPE


def test_parts_that_take_too_much_room_are_not_taken_apart():
    shared = nf4.lib().nf4_kv_attention_shared_workspace_bytes
    plain = nf4.lib().nf4_kv_attention_workspace_bytes
    for rows, apart in ((1000, True), (1 << 20, False)):
        b = batch(seqs=rows, rows=rows, max_rows=1, max_len=20000, table_stride=400)
        need = shared(cache(), b, groups(groups=1, max_prefix=16000), 8, 0, 0)
        assert (need != plain(cache(), b, 8, 0, 0)) == apart and need <= 2 << 30


def test_turns_of_large_frequencies():
    """Half a unit of 2^-64 of a turn over the whole range, and what 128 bits of 1 / (2 pi) leave."""
    rng = np.random.default_rng(0)
    f = np.concatenate([rng.uniform(-1, 1, 40) * 2.0 ** rng.integers(-60, 21, 40),
                        [2.0 ** 20, -2.0 ** 20, np.nextafter(2.0 ** 20, 0), 2.0 * math.pi, 3e5 * math.pi, 5e-324,
                         -5e-324, 2.0 ** -61, 2.0 ** -63, -2.0 ** -62, 1e-19, 0.0, -0.0, 1.0]])
    r = nf4._Rotary()
    nf4.nf4_rotary_init(r, 2 * len(f), nf4.NF4_ROTARY_HALVES, f)
    for x, got in zip(f, r.turns):
        turn = Fraction(float(x)) / (2 * PI)
        off = abs((turn - math.floor(turn)) * 2 ** 64 - got)
        assert min(off, 2 ** 64 - off) <= 0.5 + 2.0 ** -31, (x, got)


@pytest.mark.parametrize("gain,ok", [(0.0, True), (2.0 ** -100, True), (-2.0 ** 100, True), (1e300, False),
                                     (-2.0 ** 101, False), (2.0 ** -101, False), (1e-45, False)])
def test_gains_past_what_the_kernels_hold(gain, ok):
    """Sines and cosines times the gain are two fp32 terms: 2^128 would make them infinite,
    2^-140 leave them a few bits."""
    r, f = nf4._Rotary(), (ctypes.c_double * 64)()
    assert nf4.lib().nf4_rotary_init(ctypes.byref(r), 128, 0, f, gain) == (nf4.NF4_OK if ok else nf4.NF4_ERR_SHAPE)
    # the structure's own; what is accepted is refused by its y, which is not aligned
    status = nf4.lib().nf4_rotate(rotary(gain=gain), A, 1024, 0, A, 5, 8, 128, A, 1e-6, 2 * A + 2, 1024, 0, None)
    assert status == (nf4.NF4_ERR_ALIGN if ok else nf4.NF4_ERR_SHAPE)


def test_workspaces_of_the_host_or_too_small_are_refused(monkeypatch):
    """The kernels would take a host address as the GPU's, and write as many bytes as said."""
    torch = pytest.importorskip("torch")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    c, b = nf4.KVCache(1, 4, 2, 16, 64, device="cpu"), nf4.KVBatch(i32(2), i32(2, 4))
    g, out = nf4.KVGroups(i32(1)), torch.zeros(2, 128, dtype=torch.bfloat16)
    ws = torch.zeros(64, dtype=torch.float32)

    def call(workspace, ws_bytes):
        nf4.nf4_kv_attention_shared(c, 0, b, g, out, 128, 2, 0.1, 0, 0, out, None, workspace, ws_bytes, stream=0)
    reached = []
    monkeypatch.setattr(nf4, "_operands", lambda *a: None)  # rows as if on the GPU
    monkeypatch.setattr(nf4, "_on_gpu", lambda *a: None)
    monkeypatch.setattr(nf4, "_check", lambda *a: reached.append(a))
    monkeypatch.setattr(nf4, "lib", lambda: type("L", (), {"nf4_kv_attention_shared": lambda *a: 0,
                                                           "nf4_status_string": lambda s: b"refused"}))
    c.gpu = 0
    with pytest.raises(nf4.NF4Error, match="not on one GPU"):
        call(ws, 256)
    c.gpu = -1  # where the host's tensors are
    for bad, n in ((ws, 257), (ws[::2], 128)):
        with pytest.raises(nf4.NF4Error) as e:
            call(bad, n)
        assert e.value.status == nf4.NF4_ERR_WORKSPACE
    assert not reached
    for fine, n in ((ws, 256), (ws, 16), (None, 0), (0x1000, 1 << 40)):
        call(fine, n)
    assert len(reached) == 4
