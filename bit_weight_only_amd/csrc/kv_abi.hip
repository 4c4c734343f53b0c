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

bool type_ok(int type) { return type == NF4_KV_BF16 || type == NF4_KV_F32; }

// Rows of `width` values: a stride that holds them, in whole 16-byte pieces.
nf4_status check_rows(const void *p, int64_t stride, int64_t width, nf4_kv_type type) {
  if (stride < width || stride > nf4::kKvWidestRows) return NF4_ERR_SHAPE;
  return aligned(p, 16) && stride % (type == NF4_KV_F32 ? 4 : 8) == 0 ? NF4_OK : NF4_ERR_ALIGN;
}

// The norms' eps: what is divided by stays a normal float.
bool eps_ok(float eps) { return isfinite(eps) && eps >= 0x1p-100f; }

// Gains whose products with sines and cosines, held as two fp32 terms, stay in fp32's range.
bool gain_ok(double gain) { return gain == 0.0 || (fabs(gain) >= 0x1p-100 && fabs(gain) <= 0x1p100); }

nf4_status check_rotary(const nf4_rotary *r, int64_t head_dim, nf4::KvRotary &out) {
  if (!r) return NF4_ERR_NULL;
  if (r->dims < 0 || r->dims > head_dim || r->dims % 2 != 0) return NF4_ERR_SHAPE;
  if (r->layout != NF4_ROTARY_HALVES && r->layout != NF4_ROTARY_PAIRS) return NF4_ERR_SHAPE;
  if (!gain_ok(r->gain)) return NF4_ERR_SHAPE;
  out.dims = (int)r->dims;
  out.pairs = r->layout == NF4_ROTARY_PAIRS;
  out.gain = r->gain;
  for (int i = 0; i < 64; ++i) out.turns[i] = r->turns[i];
  return NF4_OK;
}

// 2^64 times the turns of f radians, |f| <= 2^20, modulo 2^64 and rounded to nearest: half a
// unit and 2^-32 of one off.  With |f| = m 2^(e - 53) for a whole m under 2^53, and
// 1 / (2 pi) to 128 bits, what is wanted is m times those bits, shifted right by 117 - e;
// the lowest 64 are left out.
uint64_t turns_of(double f) {
  constexpr uint64_t kHigh = 0x28BE60DB9391054A, kLow = 0x7F09D5F47D4D3770;
  using Wide = unsigned __int128;
  int e;
  const uint64_t m = (uint64_t)ldexp(frexp(fabs(f), &e), 53);
  const Wide high = (Wide)m * kHigh + (uint64_t)((Wide)m * kLow >> 64);  // under 2^118
  const int shift = 53 - e;                                             // 32 or more
  if (shift > 119) return 0;
  const uint64_t t = (uint64_t)((high + ((Wide)1 << (shift - 1))) >> shift);
  return f < 0.0 ? 0 - t : t;
}

// Windows and first tokens past any position are as good as the longest one.
int held(int64_t v) { return (int)(v > nf4::kKvLongest ? nf4::kKvLongest : v); }
static_assert(nf4::kKvLongest == kMaxLen + kMaxRows, "no row of the longest sequence is held");

bool groups_shape_ok(const nf4_kv_groups &g, const nf4_kv_batch &b) {
  if (g.groups < 1 || g.groups > b.seqs || (!g.first && g.groups != 1)) return false;
  return g.max_rows >= 0 && g.max_prefix >= 0 && g.max_prefix <= kMaxLen;
}

nf4::KvGroups as_groups(const nf4_kv_groups &g, const nf4_kv_batch &b) {
  return nf4::KvGroups{(int)g.groups, (int)(g.max_rows == 0 || g.max_rows > b.rows ? b.rows : g.max_rows),
                       (int)g.max_prefix, g.first, g.prefix_len};
}

struct Attention {
  nf4::KvCache c;
  nf4::KvBatch b;
  nf4::KvGroups g;
  nf4::KvAttention a;
};

// What both attentions check; groups: of the one that has them, or null.
nf4_status check_attention(const nf4_kv_cache *cache, int64_t layer, const nf4_kv_batch *batch,
                           const nf4_kv_groups *groups, const hip_bfloat16 *q, int64_t q_stride,
                           int64_t heads, float scale, int64_t window, int64_t sinks,
                           hip_bfloat16 *out, float *lse, void *workspace, size_t ws_bytes,
                           Attention &x) {
  if (!q || !out || (groups && !groups->prefix_len)) return NF4_ERR_NULL;
  nf4_status st = check_cache(cache, x.c);
  if (st != NF4_OK) return st;
  if ((st = check_batch(batch, x.c, x.b)) != NF4_OK) return st;
  if (groups && !groups_shape_ok(*groups, *batch)) return NF4_ERR_SHAPE;
  if (layer < 0 || layer >= x.c.layers) return NF4_ERR_SHAPE;
  if (!attention_shape_ok(x.c, x.b.rows, heads, window, sinks)) return NF4_ERR_SHAPE;
  if (!isfinite(scale) || !(scale > 0.0f)) return NF4_ERR_SHAPE;
  if (q_stride < heads * x.c.head_dim || q_stride > kMaxElems) return NF4_ERR_SHAPE;
  if (!aligned(q, 16) || q_stride % 8 != 0 || !aligned(out, 16) || !aligned(lse, 4))
    return NF4_ERR_ALIGN;
  if (groups && (!aligned(groups->first, 4) || !aligned(groups->prefix_len, 4)))
    return NF4_ERR_ALIGN;
  size_t need;
  if (groups) {
    x.g = as_groups(*groups, *batch);
    need = nf4::kv_attention_shared_workspace_bytes(x.c, x.b, x.g, (int)heads, held(window),
                                                    held(sinks));
  } else {
    need = nf4::kv_attention_workspace_bytes(x.c, x.b, (int)heads, held(window), held(sinks));
  }
  if (need > 0 && !workspace) return NF4_ERR_NULL;
  if (need > ws_bytes) return NF4_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 16)) return NF4_ERR_ALIGN;
  x.a = nf4::KvAttention{reinterpret_cast<const uint16_t *>(q),
                         q_stride,
                         (int)heads,
                         scale,
                         held(window),
                         held(sinks),
                         reinterpret_cast<uint16_t *>(out),
                         lse,
                         workspace};
  return NF4_OK;
}

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

nf4_status nf4_rotary_frequencies(int64_t dims, double base, nf4_rotary_scaling scaling,
                                  double factor, double original, double low, double high,
                                  double *frequency) {
  if (!frequency) return NF4_ERR_NULL;
  if (dims < 0 || dims > 128 || dims % 2 != 0) return NF4_ERR_SHAPE;
  if (!isfinite(base) || !(base > 1.0)) return NF4_ERR_SHAPE;
  if (scaling < NF4_SCALING_PLAIN || scaling > NF4_SCALING_SMOOTH) return NF4_ERR_SHAPE;
  const bool by_turns = scaling == NF4_SCALING_RAMP || scaling == NF4_SCALING_SMOOTH;
  if (scaling != NF4_SCALING_PLAIN && (!isfinite(factor) || !(factor > 0.0))) return NF4_ERR_SHAPE;
  if (by_turns && (!isfinite(original) || !isfinite(high) || !(original > 0.0) || !(low > 0.0) ||
                   !(high > low)))
    return NF4_ERR_SHAPE;
  const double turn = 2.0 * M_PI, n = (double)dims;
  if (scaling == NF4_SCALING_BASE && dims > 2) base *= pow(factor, n / (n - 2.0));
  if (!isfinite(base) || !(base > 1.0)) return NF4_ERR_SHAPE;
  // number of the pair that makes so many turns over the original context
  auto pair = [&](double turns) { return n * log(original / (turns * turn)) / (2.0 * log(base)); };
  double from = 0.0, to = 0.0;
  if (scaling == NF4_SCALING_RAMP) {
    from = fmax(floor(pair(high)), 0.0);
    to = fmin(ceil(pair(low)), n - 1.0);
    if (from == to) to += 0.001;
  }
  for (int64_t i = 0; i < dims / 2; ++i) {
    const double f = pow(base, -2.0 * (double)i / n);
    double kept = 1.0;  // how much of f stays as it is, the rest divided by the factor
    if (scaling == NF4_SCALING_LINEAR) kept = 0.0;
    if (scaling == NF4_SCALING_RAMP) kept = 1.0 - ((double)i - from) / (to - from);
    if (scaling == NF4_SCALING_SMOOTH) kept = (original * f / turn - low) / (high - low);
    kept = fmin(fmax(kept, 0.0), 1.0);
    frequency[i] = kept == 1.0 ? f : f * kept + f / factor * (1.0 - kept);
  }
  return NF4_OK;
}

nf4_status nf4_rotary_init(nf4_rotary *rotary, int64_t dims, nf4_rotary_layout layout,
                           const double *frequency, double gain) {
  if (!rotary || (!frequency && dims > 0)) return NF4_ERR_NULL;
  if (dims < 0 || dims > 128 || dims % 2 != 0 || !gain_ok(gain)) return NF4_ERR_SHAPE;
  if (layout != NF4_ROTARY_HALVES && layout != NF4_ROTARY_PAIRS) return NF4_ERR_SHAPE;
  for (int64_t i = 0; i < dims / 2; ++i)
    if (!(fabs(frequency[i]) <= 0x1p20)) return NF4_ERR_SHAPE;
  rotary->dims = dims;
  rotary->layout = layout;
  rotary->gain = gain;
  for (int64_t i = 0; i < 64; ++i) rotary->turns[i] = i < dims / 2 ? turns_of(frequency[i]) : 0;
  return NF4_OK;
}

nf4_status nf4_rotate(const nf4_rotary *rotary, const void *x, int64_t x_stride,
                      nf4_kv_type x_type, const int32_t *positions, int64_t rows, int64_t heads,
                      int64_t head_dim, const float *weight, float eps, void *y, int64_t y_stride,
                      nf4_kv_type y_type, hipStream_t stream) {
  nf4::KvRotary rot;
  if (!x || !positions || !y) return NF4_ERR_NULL;
  if (head_dim != 64 && head_dim != 128) return NF4_ERR_SHAPE;
  nf4_status st = check_rotary(rotary, head_dim, rot);
  if (st != NF4_OK) return st;
  if (rows < 1 || rows > kMaxRows || heads < 1 || heads > kMaxHeads * 64) return NF4_ERR_SHAPE;
  if (!type_ok(x_type) || !type_ok(y_type) || (weight && !eps_ok(eps))) return NF4_ERR_SHAPE;
  if ((st = check_rows(x, x_stride, heads * head_dim, x_type)) != NF4_OK) return st;
  if ((st = check_rows(y, y_stride, heads * head_dim, y_type)) != NF4_OK) return st;
  // in place each value's reader is its writer only where it stays where it was
  if (x == y && (x_stride != y_stride || x_type != y_type)) return NF4_ERR_SHAPE;
  if (!aligned(positions, 4) || !aligned(weight, 16)) return NF4_ERR_ALIGN;
  return from_hip(nf4::launch_rotate(rot, {const_cast<void *>(x), x_stride, x_type == NF4_KV_F32},
                                     positions, rows, (int)heads, (int)head_dim, weight, eps,
                                     {y, y_stride, y_type == NF4_KV_F32}, stream));
}

nf4_status nf4_kv_append_rotated(const nf4_kv_cache *cache, int64_t layer,
                                 const nf4_kv_batch *batch, const nf4_rotary *rotary, const void *q,
                                 int64_t q_stride, int64_t heads, const float *q_weight,
                                 const void *k, int64_t k_stride, const float *k_weight,
                                 const void *v, int64_t v_stride, nf4_kv_type type, float eps,
                                 hip_bfloat16 *q_out, hipStream_t stream) {
  nf4::KvCache c;
  nf4::KvBatch b;
  nf4::KvRotary rot;
  if (!q || !k || !v || !q_out) return NF4_ERR_NULL;
  nf4_status st = check_cache(cache, c);
  if (st != NF4_OK) return st;
  if ((st = check_batch(batch, c, b)) != NF4_OK) return st;
  if ((st = check_rotary(rotary, c.head_dim, rot)) != NF4_OK) return st;
  if (layer < 0 || layer >= c.layers || !type_ok(type)) return NF4_ERR_SHAPE;
  if (heads < 1 || heads > kMaxHeads * 64 || heads % c.kv_heads != 0 ||
      b.rows * heads > int64_t(1) << 31)
    return NF4_ERR_SHAPE;
  if ((q_weight || k_weight) && !eps_ok(eps)) return NF4_ERR_SHAPE;
  const int64_t width = (int64_t)c.kv_heads * c.head_dim;
  if ((st = check_rows(q, q_stride, heads * c.head_dim, type)) != NF4_OK) return st;
  if ((st = check_rows(k, k_stride, width, type)) != NF4_OK) return st;
  if ((st = check_rows(v, v_stride, width, type)) != NF4_OK) return st;
  if (q == q_out && (type != NF4_KV_BF16 || q_stride != heads * c.head_dim)) return NF4_ERR_SHAPE;
  if (!aligned(q_out, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16)) return NF4_ERR_ALIGN;
  const int64_t size = type == NF4_KV_F32 ? 4 : 2;
  const nf4::KvTurned a{static_cast<const uint8_t *>(q),
                        static_cast<const uint8_t *>(k),
                        static_cast<const uint8_t *>(v),
                        q_stride * size,
                        k_stride * size,
                        v_stride * size,
                        (int)heads,
                        q_weight,
                        k_weight,
                        eps,
                        reinterpret_cast<uint16_t *>(q_out)};
  return from_hip(
      nf4::launch_kv_append_rotated(c, layer, b, rot, a, type == NF4_KV_F32, stream));
}

nf4_status nf4_kv_read(const nf4_kv_cache *cache, int64_t layer, const nf4_kv_batch *batch, void *k,
                       int64_t k_stride, void *v, int64_t v_stride, nf4_kv_type type,
                       hipStream_t stream) {
  nf4::KvCache c;
  nf4::KvBatch b;
  if (!k || !v) return NF4_ERR_NULL;
  nf4_status st = check_cache(cache, c);
  if (st != NF4_OK) return st;
  if ((st = check_batch(batch, c, b)) != NF4_OK) return st;
  if (layer < 0 || layer >= c.layers || !type_ok(type)) return NF4_ERR_SHAPE;
  const int64_t width = (int64_t)c.kv_heads * c.head_dim;
  if ((st = check_rows(k, k_stride, width, type)) != NF4_OK) return st;
  if ((st = check_rows(v, v_stride, width, type)) != NF4_OK) return st;
  if (k == v) return NF4_ERR_SHAPE;
  const bool f32 = type == NF4_KV_F32;
  return from_hip(nf4::launch_kv_read(c, layer, b, {k, k_stride, f32}, {v, v_stride, f32}, stream));
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
  Attention x;
  const nf4_status st = check_attention(cache, layer, batch, nullptr, q, q_stride, heads, scale,
                                        window, sinks, out, lse, workspace, ws_bytes, x);
  if (st != NF4_OK) return st;
  return from_hip(nf4::launch_kv_attention(x.c, layer, x.b, x.a, stream));
}

size_t nf4_kv_attention_shared_workspace_bytes(const nf4_kv_cache *cache,
                                               const nf4_kv_batch *batch,
                                               const nf4_kv_groups *groups, int64_t heads,
                                               int64_t window, int64_t sinks) {
  nf4::KvCache c;
  if (!cache || !batch || !groups || !shape_ok(*cache, c) || !batch_shape_ok(*batch)) return 0;
  if (!groups_shape_ok(*groups, *batch)) return 0;
  if (!attention_shape_ok(c, batch->rows, heads, window, sinks)) return 0;
  return nf4::kv_attention_shared_workspace_bytes(c, as_batch(*batch, c),
                                                  as_groups(*groups, *batch), (int)heads,
                                                  held(window), held(sinks));
}

nf4_status nf4_kv_attention_shared(const nf4_kv_cache *cache, int64_t layer,
                                   const nf4_kv_batch *batch, const nf4_kv_groups *groups,
                                   const hip_bfloat16 *q, int64_t q_stride, int64_t heads,
                                   float scale, int64_t window, int64_t sinks, hip_bfloat16 *out,
                                   float *lse, void *workspace, size_t ws_bytes,
                                   hipStream_t stream) {
  if (!groups) return NF4_ERR_NULL;
  Attention x;
  const nf4_status st = check_attention(cache, layer, batch, groups, q, q_stride, heads, scale,
                                        window, sinks, out, lse, workspace, ws_bytes, x);
  if (st != NF4_OK) return st;
  return from_hip(nf4::launch_kv_attention_shared(x.c, layer, x.b, x.g, x.a, stream));
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
