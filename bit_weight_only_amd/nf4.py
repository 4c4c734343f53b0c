"""ctypes binding of libnf4.so with the same entry-point names as include/nf4.h.

Argument marshalling only: every step of the layer runs in the HIP kernels.
Tensors supply device pointers; the stream defaults to torch's current
stream.  A missing library is an error, never a fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnf4.so")

NF4_OK, NF4_ERR_NULL, NF4_ERR_SHAPE, NF4_ERR_ALIGN, NF4_ERR_CODEBOOK, NF4_ERR_WORKSPACE, \
    NF4_ERR_HIP, NF4_ERR_SCRATCH = range(8)

EXPORTS = ("nf4_status_string", "nf4_codebook", "nf4_qweight_bytes", "nf4_absmax_bytes", "nf4_workspace_bytes",
           "nf4_pack", "nf4_dequant", "nf4_repack", "nf4_unpack", "nf4_gemv", "nf4_gemm",
           "nf4_gemv_argmax_workspace_bytes", "nf4_gemv_argmax", "nf4_gemv_argmax_noalloc",
           "nf4_gemv_prefetch",
           "nf4_awq_params_bytes", "nf4_awq_workspace_bytes", "nf4_awq_pack", "nf4_awq_repack",
           "nf4_awq_unpack", "nf4_awq_dequant", "nf4_gather_columns", "nf4_awq_gemv_prefetch", "nf4_awq_gemv", "nf4_awq_gemm",
           "nf4_kv_code_bytes", "nf4_kv_scale_bytes", "nf4_kv_append",
           "nf4_kv_attention_workspace_bytes", "nf4_kv_attention", "nf4_kv_copy_pages",
           "nf4_kv_reserve", "nf4_kv_fork", "nf4_kv_release", "nf4_kv_compact_workspace_bytes",
           "nf4_kv_compact")

NF4_KV_BF16, NF4_KV_F32 = range(2)

_lib = None


class _KVCache(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in ("k", "v", "k_scale", "v_scale")] + \
               [(f, ctypes.c_int64) for f in ("layers", "pages", "kv_heads", "page_tokens",
                                              "head_dim")]


class _KVBatch(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in ("seqs", "rows", "max_rows", "max_len")] + \
               [(f, ctypes.c_void_p) for f in ("row_start", "kv_len", "table")] + \
               [("table_stride", ctypes.c_int64), ("table_entries", ctypes.c_int64)]


class _KVPool(ctypes.Structure):
    _fields_ = [("refs", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_rows", ctypes.c_int64), ("table_stride", ctypes.c_int64),
                ("len", ctypes.c_void_p), ("missing", ctypes.c_void_p)]


class NF4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {nf4_status_string(status)}")


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m bit_weight_only_amd.build` (no fallback path exists)")
        L = ctypes.CDLL(LIB_PATH)
        i64, vp, sz, st = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        fp = ctypes.POINTER(ctypes.c_float)
        L.nf4_status_string.restype = ctypes.c_char_p
        L.nf4_status_string.argtypes = [st]
        L.nf4_codebook.restype = st
        L.nf4_codebook.argtypes = [ctypes.c_double, fp]
        for f in (L.nf4_qweight_bytes, L.nf4_absmax_bytes):
            f.restype = sz
            f.argtypes = [i64, i64]
        L.nf4_workspace_bytes.restype = sz
        L.nf4_workspace_bytes.argtypes = [i64, i64, i64]
        L.nf4_pack.restype = st
        L.nf4_pack.argtypes = [vp, i64, i64, fp, vp, vp, vp]
        L.nf4_dequant.restype = st
        L.nf4_dequant.argtypes = [vp, vp, fp, i64, i64, vp, vp]
        L.nf4_repack.restype = st
        L.nf4_repack.argtypes = [vp, vp, i64, i64, vp, vp, vp]
        L.nf4_unpack.restype = st
        L.nf4_unpack.argtypes = [vp, vp, i64, i64, vp, vp, vp]
        for f in (L.nf4_gemv, L.nf4_gemm):
            f.restype = st
            f.argtypes = [vp, i64, vp, vp, fp, i64, i64, vp, vp, sz, vp]
        L.nf4_gemv_argmax_workspace_bytes.restype = sz
        L.nf4_gemv_argmax_workspace_bytes.argtypes = [i64, i64, i64]
        L.nf4_gemv_argmax.restype = st
        L.nf4_gemv_argmax.argtypes = [vp, i64, vp, vp, fp, i64, i64, vp, vp, vp, sz, vp]
        L.nf4_gemv_argmax_noalloc.restype = st
        L.nf4_gemv_argmax_noalloc.argtypes = [vp, i64, vp, vp, fp, i64, i64, vp, vp, vp]
        L.nf4_gemv_prefetch.restype = st
        L.nf4_gemv_prefetch.argtypes = [vp, i64, vp, vp, fp, i64, i64, vp, vp, sz, vp, vp, i64,
                                        i64, vp]
        L.nf4_awq_params_bytes.restype = sz
        L.nf4_awq_params_bytes.argtypes = [i64, i64]
        L.nf4_awq_workspace_bytes.restype = sz
        L.nf4_awq_workspace_bytes.argtypes = [i64, i64, i64]
        L.nf4_awq_pack.restype = st
        L.nf4_awq_pack.argtypes = [vp, i64, i64, vp, vp, vp]
        L.nf4_awq_repack.restype = st
        L.nf4_awq_repack.argtypes = [vp, vp, vp, i64, i64, vp, vp, vp]
        L.nf4_awq_unpack.restype = st
        L.nf4_awq_unpack.argtypes = [vp, vp, i64, i64, vp, vp, vp, vp]
        L.nf4_awq_dequant.restype = st
        L.nf4_awq_dequant.argtypes = [vp, vp, i64, i64, vp, vp]
        L.nf4_awq_gemv_prefetch.restype = st
        L.nf4_awq_gemv_prefetch.argtypes = [vp, i64, vp, vp, i64, i64, vp, vp, sz, vp, vp, i64,
                                            i64, vp]
        L.nf4_gather_columns.restype = st
        L.nf4_gather_columns.argtypes = [vp, i64, i64, vp, vp, vp]
        for f in (L.nf4_awq_gemv, L.nf4_awq_gemm):
            f.restype = st
            f.argtypes = [vp, i64, vp, vp, i64, i64, vp, vp, sz, vp]
        cache, batch, pool = (ctypes.POINTER(t) for t in (_KVCache, _KVBatch, _KVPool))
        for f in (L.nf4_kv_code_bytes, L.nf4_kv_scale_bytes, L.nf4_kv_compact_workspace_bytes):
            f.restype = sz
            f.argtypes = [cache]
        L.nf4_kv_append.restype = st
        L.nf4_kv_append.argtypes = [cache, i64, batch, vp, i64, vp, i64, st, vp]
        L.nf4_kv_attention_workspace_bytes.restype = sz
        L.nf4_kv_attention_workspace_bytes.argtypes = [cache, batch, i64, i64, i64]
        L.nf4_kv_attention.restype = st
        L.nf4_kv_attention.argtypes = [cache, i64, batch, vp, i64, i64, ctypes.c_float, i64, i64,
                                       vp, vp, vp, sz, vp]
        L.nf4_kv_copy_pages.restype = st
        L.nf4_kv_copy_pages.argtypes = [cache, vp, vp, i64, vp]
        L.nf4_kv_reserve.restype = st
        L.nf4_kv_reserve.argtypes = [cache, pool, vp, vp]
        L.nf4_kv_fork.restype = st
        L.nf4_kv_fork.argtypes = [cache, pool, vp, vp, i64, vp]
        L.nf4_kv_release.restype = st
        L.nf4_kv_release.argtypes = [cache, pool, vp, i64, vp]
        L.nf4_kv_compact.restype = st
        L.nf4_kv_compact.argtypes = [cache, pool, vp, vp, vp, sz, vp]
        _lib = L
    return _lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        # the raw handle, where this torch gives it: a Stream object first costs
        # 2.9 us of a 6.5 us call
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None and torch.cuda.is_initialized():
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _codebook(cb) -> ctypes.Array:
    a = np.ascontiguousarray(np.asarray(cb, dtype=np.float32).reshape(16))
    return (ctypes.c_float * 16)(*a.tolist())


def _check(status: int, where: str) -> None:
    if status != NF4_OK:
        raise NF4Error(status, where)


def nf4_status_string(status: int) -> str:
    return lib().nf4_status_string(int(status)).decode()


DEFAULT_DELTA = 0.9677083  # tail probability of the default codebook


def nf4_codebook(delta: float = DEFAULT_DELTA) -> np.ndarray:
    """The library's default 16-entry codebook (host computation): normal
    quantiles normalised to [-1, 1] with an exact zero, each a bfloat16 value."""
    out = (ctypes.c_float * 16)()
    _check(lib().nf4_codebook(float(delta), out), "nf4_codebook")
    return np.array(out[:], dtype=np.float32)


def nf4_qweight_bytes(N: int, K: int) -> int:
    return lib().nf4_qweight_bytes(N, K)


def nf4_absmax_bytes(N: int, K: int) -> int:
    return lib().nf4_absmax_bytes(N, K)


def nf4_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib().nf4_workspace_bytes(M, N, K)


def nf4_pack(W, N: int, K: int, codebook, qweight, absmax, stream=None) -> None:
    _check(lib().nf4_pack(_ptr(W), N, K, _codebook(codebook), _ptr(qweight), _ptr(absmax),
                          _stream(stream)), "nf4_pack")


def nf4_dequant(qweight, absmax, codebook, N: int, K: int, W_out, stream=None) -> None:
    _check(lib().nf4_dequant(_ptr(qweight), _ptr(absmax), _codebook(codebook), N, K,
                             _ptr(W_out), _stream(stream)), "nf4_dequant")


def nf4_repack(codes, scales, N: int, K: int, qweight, absmax, stream=None) -> None:
    _check(lib().nf4_repack(_ptr(codes), _ptr(scales), N, K, _ptr(qweight), _ptr(absmax),
                            _stream(stream)), "nf4_repack")


def nf4_unpack(qweight, absmax, N: int, K: int, codes, scales, stream=None) -> None:
    _check(lib().nf4_unpack(_ptr(qweight), _ptr(absmax), N, K, _ptr(codes), _ptr(scales),
                            _stream(stream)), "nf4_unpack")


def nf4_gemv(x, M: int, qweight, absmax, codebook, N: int, K: int, y, workspace=None,
             ws_bytes: int = 0, stream=None) -> None:
    _check(lib().nf4_gemv(_ptr(x), M, _ptr(qweight), _ptr(absmax), _codebook(codebook), N, K,
                          _ptr(y), _ptr(workspace), ws_bytes, _stream(stream)), "nf4_gemv")


def nf4_gemv_prefetch(x, M: int, qweight, absmax, codebook, N: int, K: int, y, workspace=None,
                      ws_bytes: int = 0, next_qweight=None, next_absmax=None, next_N: int = 0,
                      next_K: int = 0, stream=None) -> None:
    _check(lib().nf4_gemv_prefetch(_ptr(x), M, _ptr(qweight), _ptr(absmax), _codebook(codebook),
                                   N, K, _ptr(y), _ptr(workspace), ws_bytes, _ptr(next_qweight),
                                   _ptr(next_absmax), next_N, next_K, _stream(stream)),
           "nf4_gemv_prefetch")


def nf4_gemm(x, M: int, qweight, absmax, codebook, N: int, K: int, y, workspace=None,
             ws_bytes: int = 0, stream=None) -> None:
    _check(lib().nf4_gemm(_ptr(x), M, _ptr(qweight), _ptr(absmax), _codebook(codebook), N, K,
                          _ptr(y), _ptr(workspace), ws_bytes, _stream(stream)), "nf4_gemm")


def nf4_gemv_argmax_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib().nf4_gemv_argmax_workspace_bytes(M, N, K)


def nf4_gemv_argmax(x, M: int, qweight, absmax, codebook, N: int, K: int, y, index, workspace,
                    ws_bytes: int, stream=None) -> None:
    _check(lib().nf4_gemv_argmax(_ptr(x), M, _ptr(qweight), _ptr(absmax), _codebook(codebook),
                                 N, K, _ptr(y), _ptr(index), _ptr(workspace), ws_bytes,
                                 _stream(stream)), "nf4_gemv_argmax")


def nf4_gemv_argmax_noalloc(x, M: int, qweight, absmax, codebook, N: int, K: int, y, index,
                            stream=None) -> None:
    _check(lib().nf4_gemv_argmax_noalloc(_ptr(x), M, _ptr(qweight), _ptr(absmax),
                                         _codebook(codebook), N, K, _ptr(y), _ptr(index),
                                         _stream(stream)), "nf4_gemv_argmax_noalloc")


def nf4_awq_params_bytes(N: int, K: int) -> int:
    return lib().nf4_awq_params_bytes(N, K)


def nf4_awq_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib().nf4_awq_workspace_bytes(M, N, K)


def nf4_awq_pack(W, N: int, K: int, qweight, params, stream=None) -> None:
    _check(lib().nf4_awq_pack(_ptr(W), N, K, _ptr(qweight), _ptr(params), _stream(stream)),
           "nf4_awq_pack")


def nf4_awq_repack(codes, scales, zeros, N: int, K: int, qweight, params, stream=None) -> None:
    _check(lib().nf4_awq_repack(_ptr(codes), _ptr(scales), _ptr(zeros), N, K, _ptr(qweight),
                                _ptr(params), _stream(stream)), "nf4_awq_repack")


def nf4_awq_unpack(qweight, params, N: int, K: int, codes, scales, zeros, stream=None) -> None:
    _check(lib().nf4_awq_unpack(_ptr(qweight), _ptr(params), N, K, _ptr(codes), _ptr(scales),
                                _ptr(zeros), _stream(stream)), "nf4_awq_unpack")


def nf4_awq_dequant(qweight, params, N: int, K: int, W_out, stream=None) -> None:
    _check(lib().nf4_awq_dequant(_ptr(qweight), _ptr(params), N, K, _ptr(W_out),
                                 _stream(stream)), "nf4_awq_dequant")


def nf4_gather_columns(x, M: int, K: int, perm, x_out, stream=None) -> None:
    _check(lib().nf4_gather_columns(_ptr(x), M, K, _ptr(perm), _ptr(x_out), _stream(stream)),
           "nf4_gather_columns")


def nf4_awq_gemv(x, M: int, qweight, params, N: int, K: int, y, workspace=None,
                 ws_bytes: int = 0, stream=None) -> None:
    _check(lib().nf4_awq_gemv(_ptr(x), M, _ptr(qweight), _ptr(params), N, K, _ptr(y),
                              _ptr(workspace), ws_bytes, _stream(stream)), "nf4_awq_gemv")


def nf4_awq_gemv_prefetch(x, M: int, qweight, params, N: int, K: int, y, workspace=None,
                          ws_bytes: int = 0, next_qweight=None, next_params=None,
                          next_N: int = 0, next_K: int = 0, stream=None) -> None:
    _check(lib().nf4_awq_gemv_prefetch(_ptr(x), M, _ptr(qweight), _ptr(params), N, K, _ptr(y),
                                       _ptr(workspace), ws_bytes, _ptr(next_qweight),
                                       _ptr(next_params), next_N, next_K, _stream(stream)),
           "nf4_awq_gemv_prefetch")


def nf4_awq_gemm(x, M: int, qweight, params, N: int, K: int, y, workspace=None,
                 ws_bytes: int = 0, stream=None) -> None:
    _check(lib().nf4_awq_gemm(_ptr(x), M, _ptr(qweight), _ptr(params), N, K, _ptr(y),
                              _ptr(workspace), ws_bytes, _stream(stream)), "nf4_awq_gemm")


def nf4_kv_code_bytes(cache) -> int:
    return lib().nf4_kv_code_bytes(cache.arg)


def nf4_kv_scale_bytes(cache) -> int:
    return lib().nf4_kv_scale_bytes(cache.arg)


def _gpu(*tensors) -> int:
    """The GPU that all the tensors lie on (None is left out), -1 if they do not."""
    at = {t.device.index if t.is_cuda else -1 for t in tensors if t is not None}
    return at.pop() if len(at) == 1 else -1


def _on_gpu(where: str, *gpus: int) -> None:
    """A kernel would take a host address as one of the GPU's."""
    if gpus[0] < 0 or gpus[0] != gpus[-1]:
        raise NF4Error(NF4_ERR_SHAPE, f"{where}: tensors that are not on one GPU")


def _counted(where: str, cache, pool) -> None:
    """The kernels go over the counts of all of the cache's pages."""
    if pool.refs.numel() < cache.struct.pages:
        raise NF4Error(NF4_ERR_SHAPE, f"{where}: fewer counts than pages")


def nf4_kv_append(cache, layer: int, batch, k, k_stride: int, v, v_stride: int, type: int,
                  stream=None) -> None:
    _on_gpu("nf4_kv_append", cache.gpu, batch.gpu)
    _check(lib().nf4_kv_append(cache.arg, layer, batch.arg, _ptr(k), k_stride, _ptr(v), v_stride,
                               type, _stream(stream)), "nf4_kv_append")


def nf4_kv_attention_workspace_bytes(cache, batch, heads: int, window: int = 0,
                                     sinks: int = 0) -> int:
    return lib().nf4_kv_attention_workspace_bytes(cache.arg, batch.arg, heads, window, sinks)


def nf4_kv_attention(cache, layer: int, batch, q, q_stride: int, heads: int, scale: float,
                     window: int, sinks: int, out, lse=None, workspace=None, ws_bytes: int = 0,
                     stream=None) -> None:
    _on_gpu("nf4_kv_attention", cache.gpu, batch.gpu)
    _check(lib().nf4_kv_attention(cache.arg, layer, batch.arg, _ptr(q), q_stride, heads, scale,
                                  window, sinks, _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
                                  _stream(stream)), "nf4_kv_attention")


def nf4_kv_copy_pages(cache, src, dst, n: int, stream=None) -> None:
    _on_gpu("nf4_kv_copy_pages", cache.gpu)
    _check(lib().nf4_kv_copy_pages(cache.arg, _ptr(src), _ptr(dst), n, _stream(stream)),
           "nf4_kv_copy_pages")


def nf4_kv_reserve(cache, pool, add, stream=None) -> None:
    _on_gpu("nf4_kv_reserve", pool.gpu)
    _counted("nf4_kv_reserve", cache, pool)
    _check(lib().nf4_kv_reserve(cache.arg, pool.arg, _ptr(add), _stream(stream)),
           "nf4_kv_reserve")


def nf4_kv_fork(cache, pool, src, dst, n: int, stream=None) -> None:
    _on_gpu("nf4_kv_fork", cache.gpu, pool.gpu)
    _counted("nf4_kv_fork", cache, pool)
    _check(lib().nf4_kv_fork(cache.arg, pool.arg, _ptr(src), _ptr(dst), n, _stream(stream)),
           "nf4_kv_fork")


def nf4_kv_release(cache, pool, rows, n: int, stream=None) -> None:
    _on_gpu("nf4_kv_release", pool.gpu)
    _counted("nf4_kv_release", cache, pool)
    _check(lib().nf4_kv_release(cache.arg, pool.arg, _ptr(rows), n, _stream(stream)),
           "nf4_kv_release")


def nf4_kv_compact_workspace_bytes(cache) -> int:
    return lib().nf4_kv_compact_workspace_bytes(cache.arg)


def nf4_kv_compact(cache, pool, refs_out, table_out, workspace, ws_bytes: int,
                   stream=None) -> None:
    _on_gpu("nf4_kv_compact", cache.gpu, pool.gpu)
    _counted("nf4_kv_compact", cache, pool)
    _check(lib().nf4_kv_compact(cache.arg, pool.arg, _ptr(refs_out), _ptr(table_out),
                                _ptr(workspace), ws_bytes, _stream(stream)), "nf4_kv_compact")


# ------------------------------------------------------------ conveniences
class PackedWeight:
    """Device-layout codes and scales of one N x K weight (torch uint8/fp32)."""

    def __init__(self, N: int, K: int, device="cuda"):
        import torch
        qb, ab = nf4_qweight_bytes(N, K), nf4_absmax_bytes(N, K)
        if qb == 0:
            raise NF4Error(NF4_ERR_SHAPE, "PackedWeight")
        self.N, self.K = N, K
        self.qweight = torch.empty(qb, dtype=torch.uint8, device=device)
        self.absmax = torch.empty(ab // 4, dtype=torch.float32, device=device)

    @property
    def nbytes(self) -> int:
        """Algorithmic bytes a full read moves: 4-bit codes plus fp32 scales."""
        return self.N * self.K // 2 + 4 * self.N * (self.K // 64)

    def rows(self, n0: int, n1: int) -> "PackedWeight":
        """Rows [n0, n1) as a view of this weight's buffers (one part of a
        matrix fused along N; n0, n1 multiples of 16).  The device layout keeps
        each group of 16 rows contiguous, so the part is itself a weight in
        the device layout."""
        if n0 % 16 or n1 % 16 or not 0 <= n0 < n1 <= self.N:
            raise NF4Error(NF4_ERR_SHAPE, "PackedWeight.rows")
        v = PackedWeight.__new__(PackedWeight)
        v.N, v.K = n1 - n0, self.K
        per_q = self.qweight.numel() // (self.N // 16)
        per_a = self.absmax.numel() // (self.N // 16)
        v.qweight = self.qweight[n0 // 16 * per_q:n1 // 16 * per_q]
        v.absmax = self.absmax[n0 // 16 * per_a:n1 // 16 * per_a]
        return v


def pack_weight(W, codebook, stream=None) -> PackedWeight:
    """Quantize a device fp32 [N, K] tensor into a new PackedWeight."""
    N, K = W.shape
    pw = PackedWeight(N, K, device=W.device)
    nf4_pack(W, N, K, codebook, pw.qweight, pw.absmax, stream)
    return pw


class AwqWeight:
    """Device-layout codes and (s, z) params (int32 dwords) of one N x K int4 weight."""

    def __init__(self, N: int, K: int, device="cuda"):
        import torch
        qb, pb = nf4_qweight_bytes(N, K), nf4_awq_params_bytes(N, K)
        if qb == 0 or pb == 0:
            raise NF4Error(NF4_ERR_SHAPE, "AwqWeight")
        self.N, self.K = N, K
        self.qweight = torch.empty(qb, dtype=torch.uint8, device=device)
        self.params = torch.empty(pb // 4, dtype=torch.int32, device=device)

    @property
    def nbytes(self) -> int:
        """Algorithmic bytes a full read moves: 4-bit codes plus one 4-byte (s, z) per group."""
        return self.N * self.K // 2 + 4 * self.N * (self.K // 128)


def awq_pack_weight(W, stream=None) -> AwqWeight:
    """Quantize a device fp32 [N, K] tensor into a new AwqWeight."""
    N, K = W.shape
    aw = AwqWeight(N, K, device=W.device)
    nf4_awq_pack(W, N, K, aw.qweight, aw.params, stream)
    return aw


class KVCache:
    """A key-value cache's tensors (allocated zero-filled here, or given, as the
    codes' bytes and the float32 scales or as plain bytes) and the structure
    that names them to the library."""

    def __init__(self, layers: int, pages: int, kv_heads: int, page_tokens: int, head_dim: int,
                 device="cuda", k=None, v=None, k_scale=None, v_scale=None):
        self.struct = _KVCache(None, None, None, None, layers, pages, kv_heads, page_tokens,
                               head_dim)
        self.arg = ctypes.pointer(self.struct)
        codes, scales = nf4_kv_code_bytes(self), nf4_kv_scale_bytes(self)
        if codes == 0:
            raise NF4Error(NF4_ERR_SHAPE, "KVCache")
        for name, size, given, width in (("k", codes, k, 1), ("v", codes, v, 1),
                                         ("k_scale", scales, k_scale, 4),
                                         ("v_scale", scales, v_scale, 4)):
            if given is None:
                import torch
                lead = (layers, pages, kv_heads)
                if width == 4:
                    given = torch.zeros(lead + (page_tokens // 16,), dtype=torch.float32,
                                        device=device)
                else:
                    shape = (page_tokens, head_dim) if name == "k" else \
                        (page_tokens // 4, head_dim, 4)
                    given = torch.zeros(lead + shape, dtype=torch.uint8, device=device)
            elif given.numel() * given.element_size() != size or not given.is_contiguous() or \
                    (given.element_size() != 1 and (width == 1 or not _is_float32(given))):
                raise NF4Error(NF4_ERR_SHAPE, "KVCache")
            setattr(self, name, given)
            setattr(self.struct, name, given.data_ptr())
        self.gpu = _gpu(self.k, self.v, self.k_scale, self.v_scale)


class KVBatch:
    """The new rows of a step: int32 device tensors kv_len [seqs] and table
    [seqs][entries] (rows or columns of a wider one, too), row_start [seqs + 1]
    where sequences have other than one row each, and the host's bounds on
    rows (in all, by default one for each sequence, and of one sequence, by
    default 1) and lengths: rows past them are not processed."""

    def __init__(self, kv_len, table, row_start=None, rows=None, max_rows: int = 1, max_len=None):
        seqs = kv_len.numel()
        if table.dim() != 2 or table.shape[1] < 1 or table.stride(1) != 1 or \
                table.shape[0] < seqs or (seqs > 1 and table.stride(0) < table.shape[1]) or \
                (row_start is not None and row_start.numel() != seqs + 1):
            raise NF4Error(NF4_ERR_SHAPE, "KVBatch")
        self.kv_len, self.table, self.row_start = _int32(kv_len), table, row_start
        _int32(table[:1])
        self.struct = _KVBatch(seqs, seqs if rows is None else rows, max_rows,
                               (1 << 30) if max_len is None else max_len,
                               None if row_start is None else _int32(row_start).data_ptr(),
                               kv_len.data_ptr(), table.data_ptr(),
                               max(table.stride(0), table.shape[1]),  # one row: any stride
                               table.shape[1])
        self.arg = ctypes.pointer(self.struct)
        self.gpu = _gpu(kv_len, table, row_start)


class KVPool:
    """Who owns which page: int32 device tensors refs [pages], table
    [rows][entries], length [rows] and, if wanted, missing [1]."""

    def __init__(self, refs, table, length, missing=None):
        if table.dim() != 2 or length.numel() != table.shape[0]:
            raise NF4Error(NF4_ERR_SHAPE, "KVPool")
        self.refs, self.table, self.length, self.missing = refs, table, length, missing
        self.struct = _KVPool(_int32(refs).data_ptr(), _int32(table).data_ptr(), *table.shape,
                              _int32(length).data_ptr(),
                              None if missing is None else _int32(missing).data_ptr())
        self.arg = ctypes.pointer(self.struct)
        self.gpu = _gpu(refs, table, length, missing)


def _is_float32(t) -> bool:
    import torch
    return t.dtype == torch.float32


def _int32(t):
    import torch
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise NF4Error(NF4_ERR_SHAPE, "int32 tensor")
    return t
