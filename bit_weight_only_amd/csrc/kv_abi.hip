// kv_abi.hip -- the exported entry points of the key-value cache (the last
// part of include/nf4.h): host-side validation and launch on the caller's
// stream, under the conventions that nf4_abi.hip states.
#include <math.h>

#include "../../include/nf4.h"
#include "kv_internal.h"

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxPages = int64_t(1) << 24;
constexpr int64_t kMaxRows = int64_t(1) << 23;
constexpr int64_t kMaxLen = int64_t(1) << 30;
constexpr int64_t kMaxHeads = 1024;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

nf4_status from_hip(hipError_t e) {
  // a grid past the launch limits is a matter of the arguments' sizes
  return e == hipSuccess ? NF4_OK : e == hipErrorInvalidConfiguration ? NF4_ERR_SHAPE : NF4_ERR_HIP;
}

bool shape_ok(const nf4_kv_cache &c, nf4::KvCache &out) {
  if (c.layers < 1 || c.layers > kMaxRows || c.pages < 1 || c.pages > kMaxPages) return false;
  if (c.kv_heads < 1 || c.kv_heads > kMaxHeads) return false;
  if (c.head_dim != 64 && c.head_dim != 128) return false;
  int shift = 0;
  for (int s = 4; s <= 8; ++s)
    if (c.page_tokens == int64_t(1) << s) shift = s;
  if (shift == 0) return false;
  if (c.layers * c.pages > kMaxElems / (c.kv_heads * c.page_tokens * c.head_dim)) return false;
  out = nf4::KvCache{c.k, c.v, c.k_scale, c.v_scale, c.layers, c.pages, (int)c.kv_heads, shift,
                     (int)c.head_dim};
  return true;
}

nf4_status check_cache(const nf4_kv_cache *c, nf4::KvCache &out) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return NF4_ERR_NULL;
  if (!shape_ok(*c, out)) return NF4_ERR_SHAPE;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) ||
      !aligned(c->v_scale, 16))
    return NF4_ERR_ALIGN;
  return NF4_OK;
}

bool batch_shape_ok(const nf4_kv_batch &b) {
  if (b.seqs < 1 || b.seqs > kMaxRows || b.rows < 1 || b.rows > kMaxRows) return false;
  if (b.max_rows < 1 || b.max_rows > b.rows || b.max_len < 0 || b.max_len > kMaxLen) return false;
  if (b.table_stride < 1 || b.table_stride > kMaxLen) return false;
  return b.table_entries >= 0 && b.table_entries <= b.table_stride;
}

// No key lies past the table: a large max_len costs no launch size.
nf4::KvBatch as_batch(const nf4_kv_batch &b, const nf4::KvCache &c) {
  const int64_t room = (b.table_entries ? b.table_entries : b.table_stride) << c.page_shift;
  const bool held = b.max_len < room;
  return nf4::KvBatch{b.seqs, b.rows, (int)b.max_rows, (int)(held ? b.max_len : room),
                      held ? (int)b.max_len : nf4::kKvLongest,
                      b.row_start, b.kv_len, b.table, b.table_stride};
}

nf4_status check_batch(const nf4_kv_batch *b, const nf4::KvCache &c, nf4::KvBatch &out) {
  if (!b || !b->kv_len || !b->table) return NF4_ERR_NULL;
  if (!batch_shape_ok(*b)) return NF4_ERR_SHAPE;
  // without row_start every sequence has one row
  if (!b->row_start && (b->rows != b->seqs || b->max_rows != 1)) return NF4_ERR_NULL;
  if (!aligned(b->row_start, 4) || !aligned(b->kv_len, 4) || !aligned(b->table, 4))
    return NF4_ERR_ALIGN;
  out = as_batch(*b, c);
  return NF4_OK;
}

nf4_status check_pool(const nf4_kv_cache *c, const nf4_kv_pool *p, nf4::KvCache &cache,
                      nf4::KvPool &out) {
  if (!c || !p || !p->refs || !p->table || !p->len) return NF4_ERR_NULL;
  if (!shape_ok(*c, cache)) return NF4_ERR_SHAPE;
  if (p->table_rows < 1 || p->table_rows > kMaxRows || p->table_stride < 1 ||
      p->table_stride > kMaxLen || p->table_rows > kMaxElems / p->table_stride)
    return NF4_ERR_SHAPE;
  if (!aligned(p->refs, 16) || !aligned(p->table, 4) || !aligned(p->len, 4) ||
      !aligned(p->missing, 4))
    return NF4_ERR_ALIGN;
  out = nf4::KvPool{p->refs, p->table, p->table_rows, p->table_stride, p->len, p->missing};
  return NF4_OK;
}

bool attention_shape_ok(const nf4::KvCache &c, int64_t rows, int64_t heads, int64_t window,
                        int64_t sinks) {
  if (heads < 1 || heads > kMaxHeads * 64 || heads % c.kv_heads != 0) return false;
  if (rows * heads > int64_t(1) << 31) return false;
  return window >= 0 && sinks >= 0;
}

// Windows and first tokens past any position are as good as the longest one.
int held(int64_t v) { return (int)(v > nf4::kKvLongest ? nf4::kKvLongest : v); }
static_assert(nf4::kKvLongest == kMaxLen + kMaxRows, "no row of the longest sequence is held");

}  // namespace

extern "C" {

size_t nf4_kv_code_bytes(const nf4_kv_cache *cache) {
  nf4::KvCache c;
  if (!cache || !shape_ok(*cache, c)) return 0;
  return (size_t)c.layers * (size_t)c.pages * (size_t)c.page_bytes();
}

size_t nf4_kv_scale_bytes(const nf4_kv_cache *cache) {
  nf4::KvCache c;
  if (!cache || !shape_ok(*cache, c)) return 0;
  return (size_t)c.layers * (size_t)c.pages * (size_t)c.page_blocks() * sizeof(float);
}

nf4_status nf4_kv_append(const nf4_kv_cache *cache, int64_t layer, const nf4_kv_batch *batch,
                         const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                         nf4_kv_type type, hipStream_t stream) {
  nf4::KvCache c;
  nf4::KvBatch b;
  if (!k || !v) return NF4_ERR_NULL;
  nf4_status st = check_cache(cache, c);
  if (st != NF4_OK) return st;
  if ((st = check_batch(batch, c, b)) != NF4_OK) return st;
  if (layer < 0 || layer >= c.layers) return NF4_ERR_SHAPE;
  if (type != NF4_KV_BF16 && type != NF4_KV_F32) return NF4_ERR_SHAPE;
  const int64_t width = (int64_t)c.kv_heads * c.head_dim, unit = type == NF4_KV_F32 ? 4 : 8;
  if (k_stride < width || v_stride < width || k_stride > kMaxElems || v_stride > kMaxElems)
    return NF4_ERR_SHAPE;
  if (!aligned(k, 16) || !aligned(v, 16) || k_stride % unit != 0 || v_stride % unit != 0)
    return NF4_ERR_ALIGN;
  return from_hip(nf4::launch_kv_append(c, layer, b, k, k_stride, v, v_stride,
                                        type == NF4_KV_F32, stream));
}

size_t nf4_kv_attention_workspace_bytes(const nf4_kv_cache *cache, const nf4_kv_batch *batch,
                                        int64_t heads, int64_t window, int64_t sinks) {
  nf4::KvCache c;
  if (!cache || !batch || !shape_ok(*cache, c) || !batch_shape_ok(*batch)) return 0;
  if (!attention_shape_ok(c, batch->rows, heads, window, sinks)) return 0;
  return nf4::kv_attention_workspace_bytes(c, as_batch(*batch, c), (int)heads, held(window),
                                           held(sinks));
}

nf4_status nf4_kv_attention(const nf4_kv_cache *cache, int64_t layer, const nf4_kv_batch *batch,
                            const hip_bfloat16 *q, int64_t q_stride, int64_t heads, float scale,
                            int64_t window, int64_t sinks, hip_bfloat16 *out, float *lse,
                            void *workspace, size_t ws_bytes, hipStream_t stream) {
  nf4::KvCache c;
  nf4::KvBatch b;
  if (!q || !out) return NF4_ERR_NULL;
  nf4_status st = check_cache(cache, c);
  if (st != NF4_OK) return st;
  if ((st = check_batch(batch, c, b)) != NF4_OK) return st;
  if (layer < 0 || layer >= c.layers) return NF4_ERR_SHAPE;
  if (!attention_shape_ok(c, b.rows, heads, window, sinks)) return NF4_ERR_SHAPE;
  if (!isfinite(scale) || !(scale > 0.0f)) return NF4_ERR_SHAPE;
  if (q_stride < heads * c.head_dim || q_stride > kMaxElems) return NF4_ERR_SHAPE;
  if (!aligned(q, 16) || q_stride % 8 != 0 || !aligned(out, 16) || !aligned(lse, 4))
    return NF4_ERR_ALIGN;
  const size_t need =
      nf4::kv_attention_workspace_bytes(c, b, (int)heads, held(window), held(sinks));
  if (need > 0 && !workspace) return NF4_ERR_NULL;
  if (need > ws_bytes) return NF4_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 16)) return NF4_ERR_ALIGN;
  const nf4::KvAttention a{reinterpret_cast<const uint16_t *>(q),
                           q_stride,
                           (int)heads,
                           scale,
                           held(window),
                           held(sinks),
                           reinterpret_cast<uint16_t *>(out),
                           lse,
                           workspace};
  return from_hip(nf4::launch_kv_attention(c, layer, b, a, stream));
}

nf4_status nf4_kv_copy_pages(const nf4_kv_cache *cache, const int32_t *src, const int32_t *dst,
                             int64_t n, hipStream_t stream) {
  nf4::KvCache c;
  if (!src || !dst) return NF4_ERR_NULL;
  const nf4_status st = check_cache(cache, c);
  if (st != NF4_OK) return st;
  if (n < 1 || n > kMaxPages) return NF4_ERR_SHAPE;
  if (!aligned(src, 4) || !aligned(dst, 4)) return NF4_ERR_ALIGN;
  return from_hip(nf4::launch_kv_copy_pages(c, src, dst, n, stream));
}

nf4_status nf4_kv_reserve(const nf4_kv_cache *cache, const nf4_kv_pool *pool, const int32_t *add,
                          hipStream_t stream) {
  nf4::KvCache c;
  nf4::KvPool p;
  if (!add) return NF4_ERR_NULL;
  const nf4_status st = check_pool(cache, pool, c, p);
  if (st != NF4_OK) return st;
  if (!aligned(add, 4)) return NF4_ERR_ALIGN;
  return from_hip(nf4::launch_kv_reserve(c, p, add, stream));
}

nf4_status nf4_kv_fork(const nf4_kv_cache *cache, const nf4_kv_pool *pool, const int32_t *src,
                       const int32_t *dst, int64_t n, hipStream_t stream) {
  nf4::KvCache c;
  nf4::KvPool p;
  if (!src || !dst) return NF4_ERR_NULL;
  nf4_status st = check_cache(cache, c);
  if (st != NF4_OK) return st;
  if ((st = check_pool(cache, pool, c, p)) != NF4_OK) return st;
  if (n < 1 || n > p.rows) return NF4_ERR_SHAPE;
  if (!aligned(src, 4) || !aligned(dst, 4)) return NF4_ERR_ALIGN;
  return from_hip(nf4::launch_kv_fork(c, p, src, dst, n, stream));
}

nf4_status nf4_kv_release(const nf4_kv_cache *cache, const nf4_kv_pool *pool, const int32_t *rows,
                          int64_t n, hipStream_t stream) {
  nf4::KvCache c;
  nf4::KvPool p;
  if (!rows) return NF4_ERR_NULL;
  const nf4_status st = check_pool(cache, pool, c, p);
  if (st != NF4_OK) return st;
  if (n < 1 || n > p.rows) return NF4_ERR_SHAPE;
  if (!aligned(rows, 4)) return NF4_ERR_ALIGN;
  return from_hip(nf4::launch_kv_release(c, p, rows, n, stream));
}

size_t nf4_kv_compact_workspace_bytes(const nf4_kv_cache *cache) {
  nf4::KvCache c;
  if (!cache || !shape_ok(*cache, c)) return 0;
  return nf4::kv_compact_workspace_bytes(c);
}

nf4_status nf4_kv_compact(const nf4_kv_cache *cache, const nf4_kv_pool *pool, int32_t *refs_out,
                          int32_t *table_out, void *workspace, size_t ws_bytes,
                          hipStream_t stream) {
  nf4::KvCache c;
  nf4::KvPool p;
  if (!refs_out || !table_out || !workspace) return NF4_ERR_NULL;
  nf4_status st = check_cache(cache, c);
  if (st != NF4_OK) return st;
  if ((st = check_pool(cache, pool, c, p)) != NF4_OK) return st;
  if (!aligned(refs_out, 16) || !aligned(table_out, 4) || !aligned(workspace, 16))
    return NF4_ERR_ALIGN;
  if (nf4::kv_compact_workspace_bytes(c) > ws_bytes) return NF4_ERR_WORKSPACE;
  return from_hip(nf4::launch_kv_compact(c, p, refs_out, table_out, workspace, stream));
}

}  // extern "C"
