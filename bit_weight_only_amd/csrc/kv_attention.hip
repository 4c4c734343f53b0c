// kv_attention.hip -- causal attention over the 8-bit key-value cache.
//
// vibevoice.c README ("The kernels that matter"): attention is a streaming
// softmax, prompts on matrix cores, single tokens split over the cache.  The
// mathematics, for one row with keys k_j, values v_j, c = scale log2(e):
//
//   t_j = c q.k_j,  m = max t_j,  l = sum 2^(t_j - m),
//   out = sum 2^(t_j - m) v_j / l,  lse = (m + log2 l) ln 2,
//
// over pieces of the keys: when a piece raises m, l and the sum of values are
// multiplied by 2^(m_old - m_new).  A key block's scale multiplies t after the
// product of codes.  A value block's scale 2^e goes into the exponent of the
// weight, w = 2^(t - m + e), and the block's part of l is 2^-e sum w: no
// multiplication per element, and exact, since both are powers of two.
//
// Both products have the cache as the left operand: S^T = K Q^T gives a lane
// the weights of one query row, in the places where the right operand of
// O^T = V^T W^T wants them.
#include <algorithm>
#include <type_traits>

#include "kv_internal.h"
#include "nf4_internal.h"

namespace nf4 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Eight codes (two dwords) as bf16, exactly.
__device__ inline bf16x8 widen(uint32_t a, uint32_t b) {
  union {
    bf16x8 v;
    bf16x2 p[4];
  } u;
  u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return u.v;
}

// 0x80 in every byte that holds a NaN code (0x7F or 0xFF).
__device__ inline uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// 1 (e4m3 0x38) for every NaN code, else 0; and the codes with 0 for NaN.
__device__ inline uint32_t nan_ones(uint32_t w) { return (nan_bytes(w) >> 7) * 0x38u; }
__device__ inline uint32_t without_nan(uint32_t w) { return w & ~((nan_bytes(w) >> 7) * 0xFFu); }

__device__ inline f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ inline f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// The largest of three, NaN left out.  (fmaxf first quiets its arguments, an
// instruction each.)
__device__ inline float max3(float a, float b, float c) {
  float d;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Exponent of a block's scale, held to what a cache can have.
__device__ inline int kv_scale_exponent(float s) {
  const int e = (int)((__float_as_uint(s) >> 23) & 255u) - 127;
  return e < kKvExpMin ? kKvExpMin : e > kKvExpMax ? kKvExpMax : e;
}

// m only has to be near the maximum: it is raised, and the sums rescaled, when a
// weight would pass 2^8 (as the first key's would).  The 2^30 keys that a
// sequence may have then sum to less than 2^30 * 2^8 * 448 * 2^e, which fp32
// holds up to e = 80.  In steps with a value scale over that, m is kept 27 over
// the maximum: the weights are at most 2^-19, and 2^30 of them times 448 * 2^100
// stay under 2^120.
constexpr float kSlack = 8.0f, kLift = 27.0f;
constexpr int kLiftExp = 80;

// m of a row that saw keys whose scores are all NaN or -inf (past the range of
// 32 bits): NaN ones make its sums NaN, -inf ones have weight 0, and any finite
// score raises m.  So m is -inf for a row that saw no key, and only for that.
constexpr float kLeast = -3.402823466e38f;

// A lane's value as a scalar.
__device__ inline float lane_float(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// The smallest of the lanes' values.
__device__ inline int lanes_min(int v) {
  v = min(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true));   // lane ^ 1
  v = min(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true));   // lane ^ 2
  v = min(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true));  // 7 - lane of 8
  v = min(v, __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true));  // 15 - lane of 16
  return min(min(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
             min(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}

// A number that the host knows and workgroups divide by: n / value for n under 2^31, as
// n factor / 2^shift with factor = 2^shift / value rounded up, shift = 31 + log2 value
// rounded up, so that what rounding adds stays under one part.  (A division by a number that
// is not known beforehand takes some 30 instructions that wait for one another.)
struct Divisor {
  uint32_t value, factor, shift;
  static Divisor of(int64_t value) {
    uint32_t s = 0;
    while ((int64_t(1) << s) < value) ++s;
    return Divisor{(uint32_t)value, (uint32_t)(((uint64_t(1) << (31 + s)) + value - 1) / value), 31 + s};
  }
  __device__ operator uint32_t() const { return value; }
  friend __device__ uint32_t operator/(uint32_t n, const Divisor &d) {
    return (uint32_t)((uint64_t)n * d.factor >> d.shift);
  }
  friend __device__ uint32_t operator%(uint32_t n, const Divisor &d) { return n - n / d * d.value; }
};

// What a workgroup takes of the keys: all that its rows see, or, where sequences share
// their first tokens, those of the shared ones (rows of a whole group at once, its
// keys split at fixed places) or those past them.  The parts of the latter two meet in
// the workspace: slot i holds the i-th part's sums of every row and head, [rows][heads][D],
// the prefix's parts before the suffix's; behind all slots (m, l) of each.  All of it is
// less than 2^32 bytes (kMostPartBytes), so that places are 32 bits past one address.
struct Shared {
  using Number = Divisor;
  KvGroups g;
  uint32_t row_heads;
  int prefix_slots, slots;
  Divisor kv_heads, heads_each;  // heads of keys, and of queries to each
  __device__ Divisor heads(const KvCache &) const { return kv_heads; }
  __device__ Divisor group(const KvCache &, const KvAttention &) const { return heads_each; }
  __device__ f32x4 *sums(void *ws, uint32_t slot, uint32_t row_head, int dim, int d) const {
    return reinterpret_cast<f32x4 *>(static_cast<uint8_t *>(ws) + ((slot * row_heads + row_head) * dim + d) * 4);
  }
  __device__ float2 *ml(void *ws, uint32_t slot, uint32_t row_head, int dim) const {
    return reinterpret_cast<float2 *>(static_cast<uint8_t *>(ws) + (slots * row_heads * dim * 4 + (slot * row_heads + row_head) * 8));
  }
};
struct Whole {
  static constexpr bool kPrefix = false, kSuffix = false;
  using Number = uint32_t;
  __device__ static uint32_t heads(const KvCache &c) { return (uint32_t)c.kv_heads; }
  __device__ static uint32_t group(const KvCache &c, const KvAttention &a) {
    return (uint32_t)a.heads / (uint32_t)c.kv_heads;
  }
};
struct Prefix : Shared {
  static constexpr bool kPrefix = true, kSuffix = false;
};
struct Suffix : Shared {
  static constexpr bool kPrefix = false, kSuffix = true;
};

// The keys of one row: up to its position, inside the window or among the
// first tokens.
template <class S>
struct Visible {
  int window, sinks, shared;  // shared: keys before it are the prefix's
  __device__ bool operator()(int key, int pos) const {
    return (key <= pos) & ((window == 0) | (key > pos - window) | (key < sinks)) &
           (!S::kPrefix | (key < shared)) & (!S::kSuffix | (key >= shared));
  }
  // Bit x: whether the row sees key + x, x = 0 .. 63.
  __device__ uint64_t bits(int key, int pos) const {
    auto upto = [](int t) {  // bits 0 .. t
      return t < 0 ? 0ull : t >= 63 ? ~0ull : ~0ull >> (63 - t);
    };
    uint64_t b = upto(pos - key);
    if (window > 0) b &= ~upto(pos - window - key) | upto(sinks - 1 - key);
    if (S::kPrefix) b &= upto(shared - 1 - key);
    if (S::kSuffix) b &= ~upto(shared - 1 - key);
    return b;
  }
  // Whether every row at p_lo .. p_hi sees all of key .. key + n - 1.
  __device__ bool all(int key, int n, int p_lo, int p_hi) const {
    return key + n - 1 <= p_lo && (window == 0 || key > p_hi - window || key + n <= sinks) &&
           (!S::kPrefix || key + n <= shared) && (!S::kSuffix || key >= shared);
  }
};

// The steps of N keys from step `low` on that rows from p_lo on can see, as a list:
// those with first tokens, then from the start of the lowest row's window to the
// key `last`.
template <int N>
struct Steps {
  int low, sink_steps, from, count;
  __device__ Steps(int low_step, int p_lo, int last, int window, int sinks) {
    low = from = low_step;
    sink_steps = 0;
    const int steps = last < 0 ? 0 : last / N + 1;
    if (window > 0 && p_lo - window + 1 > low * N) {
      from = (p_lo - window + 1) / N;
      const int past = min((int)(((int64_t)sinks + N - 1) / N), steps);
      if (past >= from) from = low;
      else sink_steps = max(past - low, 0);
    }
    count = sink_steps + max(steps - from, 0);
  }
  __device__ int key(int i) const { return (i < sink_steps ? i + low : i - sink_steps + from) * N; }
};

// Most steps of N keys that any N-aligned list above can have, for the host.
int64_t most_steps(int N, const KvBatch &b, int tile_rows, int window, int sinks) {
  const int64_t all = ((int64_t)b.max_len + N - 1) / N;
  if (window == 0) return all < 1 ? 1 : all;
  const int64_t some = ((int64_t)window + tile_rows + N - 2) / N + 1 + ((int64_t)sinks + N - 1) / N;
  const int64_t n = all < some ? all : some;
  return n < 1 ? 1 : n;
}

// Rows of a sequence's tile: query row r of a kv head is token r / group and
// head r % group of its group.
template <class Number>
struct TileOf {
  int64_t row0;
  int all;            // rows of a group, max_rows or no
  Number group;
  uint32_t rows, r0;  // rows of a kv head of one sequence stay under 2^31
  int n, len, end, p_lo, p_hi;
  __device__ TileOf(Number group, const KvBatch &b, const KvBatch::Raw &seq, uint32_t tile, uint32_t width)
      : group(group) {
    b.sequence(seq, row0, n, len, end);
    rows = (uint32_t)(n < b.max_rows ? n : b.max_rows) * group;
    r0 = tile * width;
    const uint32_t last = r0 + width < rows ? r0 + width - 1 : rows - 1;
    p_lo = len - n + (int)(r0 / group);
    p_hi = len - n + (int)(last / group);
  }
  __device__ bool empty() const { return r0 >= rows; }
  // Row r of the tile's (counted as r0 is) among all rows and heads.
  __device__ int64_t row_head(const KvAttention &a, int head, uint32_t r) const {
    return (row0 + r / group) * a.heads + head * group + r % group;
  }
  // The last key that a row at p may see: not past the table.
  __device__ int last_key(int p) const { return min(p, end - 1); }

  // A tile of all rows of a group of sequences over the tokens that they share.
  __device__ TileOf(Number group, const KvBatch &b, const KvGroups &g, int first, int past, int shared,
                    uint32_t tile, uint32_t width)
      : group(group) {
    row0 = b.first_row(first);
    const int64_t many = first < past ? b.first_row(past) - row0 : 0;
    all = (int)(many < 0 ? 0 : many);
    n = all < g.max_rows ? all : g.max_rows;
    len = end = shared;
    rows = (uint32_t)n * group;
    r0 = tile * width;
    p_lo = 0;
    p_hi = -1;
  }
  // The positions of its tokens, in two steps (KvBatch): lane l has that of token l from its
  // first one on, -1 past the last.
  template <int WIDTH>
  __device__ KvBatch::Guess guess(const KvBatch &b, int first, int past) const {
    return b.guess(row0 + min(token(), last_token<WIDTH>()), first, past, row0, all);
  }
  template <int WIDTH>
  __device__ int positions(const KvBatch &b, int first, int past, const KvBatch::Guess &g) {
    static_assert(WIDTH <= 64, "a lane for every token");
    const bool has = token() <= last_token<WIDTH>();
    const int at = has ? b.position(g, row0 + token(), first, past) : -1;
    p_hi = -lanes_min(-at);
    p_lo = lanes_min(has ? at : p_hi);
    return at;
  }
  __device__ int token() const { return (int)(r0 / group) + (int)(threadIdx.x & 63); }
  template <int WIDTH>
  __device__ int last_token() const { return (int)((min(r0 + WIDTH, rows) - 1) / group); }
};
using Tile = TileOf<uint32_t>;

// Where a workgroup works: the tile `index` of sequence (or group) `seq`, part `split` of
// its keys.
struct Range {
  int begin, end;  // of the list of steps
  bool one, none;  // the only part of the list; one past its last part
};

template <class S, int N>
struct Place {
  using Number = typename S::Number;
  const KvCache &c;
  const KvBatch &b;
  const KvAttention &a;
  const S &scope;
  int seq;
  uint32_t index, width;
  int split;
  Number max_splits;
  int split_steps;
  int first, past;  // sequences of the group
  KvBatch::Raw raw;
  int shared;
  int first_len;  // tokens of the group's first sequence
  const int32_t *table;

  __device__ Place(const KvCache &c, const KvBatch &b, const KvAttention &a, const S &scope,
                   int seq, uint32_t index, uint32_t width, int split, Number max_splits,
                   int split_steps)
      : c(c), b(b), a(a), scope(scope), seq(seq), index(index), width(width), split(split),
        max_splits(max_splits), split_steps(split_steps), first(seq), past(seq + 1), shared(0) {
    if constexpr (S::kPrefix) {
      first = scope.g.first_of(b, seq);
      past = scope.g.first_of(b, seq + 1);
      shared = scope.g.shared(b, seq);
    }
    if constexpr (!S::kPrefix) raw = b.raw(seq);
    if constexpr (S::kSuffix) shared = scope.g.shared_of(b, seq);
    // (a group without sequences has no rows: nothing of its table is read)
    const int64_t s = first < b.seqs ? first : 0;
    if constexpr (S::kPrefix) first_len = b.kv_len[s];
    table = b.table + s * b.table_stride;
  }
  // Shared tokens are read from the first sequence's pages, unless it has not got them all, as
  // one that was released or is behind the others: then `table` becomes another one's.  Asked
  // once that first pages' ids are on their way, so that the common case waits for nothing.
  __device__ bool elsewhere(const int32_t *&table) const {
    if constexpr (!S::kPrefix) return false;
    else {
      if (first_len >= shared) return false;
      const int s = scope.g.source(b, first, past, shared);
      table = b.table + (int64_t)s * b.table_stride;
      return s != first;
    }
  }
  using Tile = TileOf<typename S::Number>;
  __device__ Tile tile() const {
    if constexpr (S::kPrefix) return Tile(scope.group(c, a), b, scope.g, first, past, shared, index, width);
    else return Tile(scope.group(c, a), b, raw, index, width);
  }
  // Without a window what a prefix's rows see does not wait for their positions.
  __device__ bool ahead() const { return S::kPrefix && a.window == 0; }
  __device__ Steps<N> steps(const Tile &tl, int p_hi) const {
    if constexpr (S::kPrefix)
      return Steps<N>(0, tl.p_lo, ahead() ? shared - 1 : min(p_hi, shared - 1), a.window, a.sinks);
    return Steps<N>(shared / N, tl.p_lo, tl.last_key(p_hi), a.window, a.sinks);
  }
  // The steps that the host has planned for a part, or more where it has made room for
  // fewer parts; a prefix has all of its parts, some of them with nothing to do.
  __device__ Range range(const Steps<N> &s) const {
    const int per = S::kPrefix ? in_parts(s.count, max_splits)
                    : S::kSuffix ? suffix_steps(s.count, split_steps, max_splits) : split_steps;
    return Range{split * per, min(s.count, (split + 1) * per), !S::kPrefix && s.count <= per,
                 !S::kPrefix && split > 0 && split * per >= s.count};
  }
  // Whether a range holds all keys that the rows see.
  __device__ bool whole(const Range &r) const { return r.one && shared == 0; }
  __device__ int slot() const {
    if constexpr (S::kSuffix) return scope.prefix_slots + split;
    return split;
  }
  __device__ static int in_parts(int count, Number parts) {
    return (int)(((uint32_t)count + parts - 1) / parts);
  }
  __device__ static int suffix_steps(int count, int split_steps, Number max_splits) {
    return max(split_steps, in_parts(count, max_splits));
  }
};

// Workspace of a call whose keys are split: for every (item, split), an item
// being a tile of `width` rows, the rows' sums [width][D] and their (m, l).
__host__ __device__ inline int64_t part_floats(int width, int dim) {
  return (int64_t)width * (dim + 2);
}

__device__ inline uint32_t bf16_pair(float a, float b) {
  bf16x2 v;
  v[0] = (__bf16)a;
  v[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}

// Adds sums (m, l, x) of other keys to (mm, ll, xx).
__device__ inline void join(float &mm, float &ll, f32x4 &xx, float m, float l, f32x4 x) {
  if (m == -INFINITY) return;  // no key of these was seen
  const float top = fmaxf(mm, m);
  const float f = exp2_fast(mm - top), g = exp2_fast(m - top);
  ll = ll * f + l * g;
  xx = xx * f + x * g;
  mm = top;
}

// The log of a row's sum of weights: -inf if it saw no key, NaN if it has no sum.
__device__ inline float log_sum(float m, float l) {
  if (m == -INFINITY) return m;
  return l == 0.0f ? NAN : (m + __log2f(l)) * kLn2;
}

// The result of a row and head, values d .. d + 3, from its sums.
__device__ inline void store_sums(const KvCache &c, const KvAttention &a, int64_t at, int d, f32x4 x,
                                  float m, float l) {
  const bool none = m == -INFINITY;  // no key was seen
  const float inv = 1.0f / l;
  uint2 y;
  y.x = none ? 0u : bf16_pair(x[0] * inv, x[1] * inv);
  y.y = none ? 0u : bf16_pair(x[2] * inv, x[3] * inv);
  *reinterpret_cast<uint2 *>(a.out + at * c.head_dim + d) = y;
  if (a.lse && d == 0) a.lse[at] = log_sum(m, l);
}
// The same of row `cc` of a tile.
template <class T>
__device__ inline void store_row(const KvCache &c, const KvAttention &a, const T &tl, int head,
                                 int cc, int d, f32x4 x, float m, float l) {
  store_sums(c, a, tl.row_head(a, head, tl.r0 + cc), d, x, m, l);
}

// NaN codes in places that some row does not see would reach it as 0 * NaN, so
// steps that some row does not see whole take them as 0 (without_nan), and a
// product of their places with the visible ones (bits of `see`, keys as in the
// weights) makes the sums NaN where that is due.
template <int DT, class Sums>
__device__ inline void spread_nan(const uint32_t (&va)[DT], const uint32_t (&vc)[DT], uint32_t see,
                                  Sums (&o)[DT]) {
  constexpr int N = sizeof(Sums) / sizeof(float);
  uint32_t nan = 0;
#pragma unroll
  for (int t = 0; t < DT; ++t) nan |= nan_bytes(va[t]) | nan_bytes(vc[t]);
  if (!__any(nan != 0)) return;
  union {
    bf16x8 v;
    __bf16 e[8];
  } ones;
#pragma unroll
  for (int e = 0; e < 8; ++e) ones.e[e] = (__bf16)(see >> e & 1 ? 1.0f : 0.0f);
#pragma unroll
  for (int t = 0; t < DT; ++t) {
    const Sums hit = mfma(widen(nan_ones(va[t]), nan_ones(vc[t])), ones.v, Sums{});
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (hit[e] > 0.0f) o[t][e] = NAN;
    __builtin_amdgcn_sched_barrier(0);  // one at a time: registers
  }
}

// ---------------------------------------------------------------------------
// Few rows: one workgroup of W waves per (16 rows of a kv head, part of the
// keys), each wave every W-th step of 32 keys straight from memory to its
// registers, a step ahead.  Lane l owns query row l % 16; with g = l / 16 it
// holds keys 4g .. 4g + 3 of both blocks of a step.
//
// Memory bound: a step reads 8 KB (D = 128) for some 400 cycles of vector work.
// 64 sequences of up to 16384 tokens (1.11 GB): 217 us = 5.1 TB/s, the rate of
// a large copy; a bare read of the same pieces takes 185 us.  Six waves
// took 252 us, eight 247, loads marked as not to be kept some 20 more.  Small
// calls are bound by dependent trips to memory (lengths, page ids, keys, the
// waves' meeting): one sequence of 113 tokens 6.3 us, of which 1.6 an empty
// launch.
//
// The waves meet in LDS; the parts of split keys in the workspace, where each
// leaves its sums for the second launch.

template <int D>
struct Step {
  uint4 k[2][D / 64], v[2][D / 64];
};

template <int D, int W>
struct DecodeLds {
  static constexpr int kPitch = D + 4;  // of a row of sums, in floats
  float sums[W * 16 * kPitch];
  float ml[2][W][16];
};

template <int D, int W, class S>
__device__ inline void decode_part(const KvCache &c, int64_t layer, const KvBatch &b,
                                   const KvAttention &a, typename S::Number tiles,
                                   typename S::Number max_splits, int split_steps, const S &scope,
                                   uint32_t w, DecodeLds<D, W> &lds) {
  using Tile = TileOf<typename S::Number>;
  constexpr int KS = D / 32;   // k-steps of the first product
  constexpr int DT = D / 16;   // tiles of 16 values of the second
  constexpr int PITCH = DecodeLds<D, W>::kPitch;
  auto &sums = lds.sums;
  auto &ml = lds.ml;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  // neighbouring workgroups take the heads of one page, so that what is read
  // at a time lies side by side (64 sequences of up to 16384 tokens: 256 us
  // with the parts of a head side by side instead, 217 us this way)
  const int head = w % scope.heads(c);
  w = w / scope.heads(c);
  const int split = w % max_splits;
  w = w / max_splits;
  const uint32_t item = w * (uint32_t)c.kv_heads + head;
  const Place<S, 32> place(c, b, a, scope, w / tiles, w % tiles, 16, split, max_splits, split_steps);
  const int32_t *table = place.table;
  // without a window, where the first page ids stand does not depend on the
  // lengths: they are read beside them (as far as the longest one may reach)
  int page_ahead = -1;
  if (!S::kPrefix && !S::kSuffix && a.window == 0) {
    const int64_t t0 = (int64_t)(split * split_steps + wave + (lane >> 1) * W) * 32 + 16 * (lane & 1);
    page_ahead = table[min(t0, (int64_t)max(b.max_len - 1, 0)) >> c.page_shift];
  }
  if (S::kPrefix && place.shared == 0) return;
  Tile tl = place.tile();
  if (tl.empty()) return;
  int at = -1;  // a prefix's: positions of the tile's tokens
  if (S::kPrefix && !place.ahead())
    at = tl.template positions<16>(b, place.first, place.past, tl.template guess<16>(b, place.first, place.past));
  const Steps<32> steps = place.steps(tl, tl.p_hi);
  const Range range = place.range(steps);
  if (range.none) return;
  const int end = range.end;

  const bool mine = tl.r0 + col < tl.rows;
  const uint32_t r = mine ? tl.r0 + col : tl.rows - 1;
  const int tok = (int)(r / tl.group), qh = head * tl.group + (int)(r % tl.group);

  const int64_t layer_pages = layer * c.pages;
  const int page_blocks = 1 << (c.page_shift - 4);
  // What the wave's next 32 steps need to know of their blocks, lane 2s + h
  // for block h of step s: page (-1: none), c times the keys' scale, and for
  // the values' scale 2^e e and 2^-e.  Read ahead of the steps as vectors: a
  // scalar read per step would cost the step its whole latency, since scalar
  // reads return out of order and any use waits for all of them.
  const int first = range.begin + wave;
  int page_l = -1;
  float kc_l = 0.0f, ve_l = 0.0f, vi_l = 1.0f;
  uint64_t high_l = 0;  // bit 2s + h: that block's values need kLift
  auto block_of = [&](int page, int t0) {
    return ((layer_pages + page) * c.kv_heads + head) * page_blocks +
           ((t0 & (c.page_tokens() - 1)) >> 4);
  };
  auto look = [&](int i0) {
    const int i = i0 + (lane >> 1) * W;
    const int t0 = steps.key(i) + 16 * (lane & 1);
    page_l = -1;
    if (i < end && t0 < tl.end)
      page_l = !S::kPrefix && !S::kSuffix && a.window == 0 && i0 == first ? page_ahead
                                                                          : table[t0 >> c.page_shift];
    if (page_l >= c.pages) page_l = -1;
    const int64_t block = block_of(page_l < 0 ? 0 : page_l, t0);
    kc_l = c.ks[block];
    ve_l = c.vs[block];
  };
  auto looked = [&] {
    kc_l *= a.scale * kLog2e;
    // (held to what a cache can have: a block that was never written may lie
    // past the last token, and 0 weight times its 2^-e has to be 0)
    const int ve = kv_scale_exponent(ve_l);
    high_l = __ballot(ve > kLiftExp && page_l >= 0);
    ve_l = (float)ve;
    vi_l = __uint_as_float((uint32_t)(127 - ve) << 23);
  };
  auto load = [&](Step<D> &st, int i, int s) {
    const int key0 = steps.key(i);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int page = __builtin_amdgcn_readlane(page_l, 2 * s + h);
      const int64_t block = block_of(page < 0 ? 0 : page, key0 + 16 * h);
      const uint8_t *kp = c.k + block * (16 * D) + (col * D + g * 16);
      const uint8_t *vp = c.v + block * (16 * D) + (g * D + col * 4) * 4;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        st.k[h][j] = *reinterpret_cast<const uint4 *>(kp + 64 * j);
        st.v[h][j] = *reinterpret_cast<const uint4 *>(vp + 256 * j);
      }
    }
  };

  look(first);
  if (place.elsewhere(table)) look(first);
  KvBatch::Guess guess = {};
  if constexpr (S::kPrefix)
    if (place.ahead()) guess = tl.template guess<16>(b, place.first, place.past);

  bf16x8 q[KS];
  const uint16_t *qp = a.q + (tl.row0 + tok) * a.q_stride + (int64_t)qh * D + g * 16;
#pragma unroll
  for (int j = 0; j < KS; ++j)
    q[j] = *reinterpret_cast<const bf16x8 *>(qp + 64 * (j / 2) + 8 * (j % 2));
  if (S::kPrefix && place.ahead()) at = tl.template positions<16>(b, place.first, place.past, guess);
  const int row_pos = S::kPrefix ? __shfl(at, tok - (int)(tl.r0 / tl.group)) : tl.len - tl.n + tok;
  const int pos = mine ? row_pos : -1;

  const Visible<S> visible{a.window, a.sinks, place.shared};
  float m = -INFINITY, l = 0.0f;
  f32x4 o[DT] = {};

  auto compute = [&](const Step<D> &st, int i, int sl) {
    const int key0 = steps.key(i);
    uint32_t kw[2][D / 16], vw[2][D / 16];
    __builtin_memcpy(kw, st.k, sizeof(kw));
    __builtin_memcpy(vw, st.v, sizeof(vw));
    f32x4 s[2];
    bool hole[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[h] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < KS; ++j) s[h] = mfma(widen(kw[h][2 * j], kw[h][2 * j + 1]), q[j], s[h]);
      const float kc = lane_float(kc_l, 2 * sl + h);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[h][e] *= kc;
      hole[h] = __builtin_amdgcn_readlane(page_l, 2 * sl + h) < 0;
    }
    uint32_t see = 0xFF;  // bit 4h + e
    const bool masked = hole[0] || hole[1] || !visible.all(key0, 32, tl.p_lo, tl.p_hi);
    if (masked) {
      see = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool v = !hole[h] && visible(key0 + 16 * h + 4 * g + e, pos);
          see |= (uint32_t)v << (4 * h + e);
          if (!v) s[h][e] = -INFINITY;
        }
    }
    float mx = see != 0 ? kLeast : -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[h][e]);
    const float lift = (high_l >> (2 * sl) & 3) != 0 ? kLift : 0.0f;
    if (__any(mx > m + (kSlack - lift))) {
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float m_new = fmaxf(m, mx + lift);
      const float alpha = m_new == -INFINITY ? 1.0f : exp2_fast(m - m_new);
      m = m_new;
      l *= alpha;
#pragma unroll
      for (int t = 0; t < DT; ++t) o[t] *= alpha;
    }
    // two bf16 terms: memory bound, this kernel has the time (rel-L2 of the
    // result 0.0023 with one, 0.0017 with two, which is its own rounding)
    union {
      bf16x8 v;
      __bf16 e[8];
    } p, rest;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float sum = 0.0f;
      const float mv = m - lane_float(ve_l, 2 * sl + h);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = exp2_fast(s[h][e] - mv);
        if (!(see >> (4 * h + e) & 1)) x = 0.0f;  // also where m is still -inf
        sum += x;
        p.e[4 * h + e] = (__bf16)x;
        rest.e[4 * h + e] = (__bf16)(x - (float)p.e[4 * h + e]);
      }
      l += sum * lane_float(vi_l, 2 * sl + h);
    }
    if (masked) {  // the same for every lane
      spread_nan<DT>(vw[0], vw[1], see, o);
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        vw[0][t] = without_nan(vw[0][t]);
        vw[1][t] = without_nan(vw[1][t]);
      }
    }
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      const bf16x8 v = widen(vw[0][t], vw[1][t]);
      o[t] = mfma(v, p.v, o[t]);
      o[t] = mfma(v, rest.v, o[t]);
    }
  };

  // the loads of a step go out before the work on the step before it
  Step<D> st[2];
  for (int i = first; i < end; i += 32 * W) {
    if (i != first) look(i);
    const int n = min(32, (end - i + W - 1) / W);
    load(st[0], i, 0);
    looked();
    // every load is issued whether it is needed or not (the last step's
    // again), so that the number in flight is known at each wait
    for (int s = 0; s < n; s += 2) {
      const int s1 = min(s + 1, n - 1), s2 = min(s + 2, n - 1);
      load(st[1], i + s1 * W, s1);
      compute(st[0], i + s * W, s);
      load(st[0], i + s2 * W, s2);
      if (s + 1 < n) compute(st[1], i + s1 * W, s1);
    }
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);

  // the waves' sums, each scaled to the largest m
  if (g == 0) {
    ml[0][wave][col] = m;
    ml[1][wave][col] = l;
  }
  __syncthreads();
  float top = ml[0][0][col], f;
#pragma unroll
  for (int v = 1; v < W; ++v) top = fmaxf(top, ml[0][v][col]);
  f = m == -INFINITY ? 0.0f : exp2_fast(m - top);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    // element e of tile 4j + t is value 64j + 16g + 4e + t
    float *to = sums + (wave * 16 + col) * PITCH + g * 16 + e * 4;
#pragma unroll
    for (int t = 0; t < DT; t += 4)
      *reinterpret_cast<f32x4 *>(to + 16 * t) =
          f32x4{o[t][e] * f, o[t + 1][e] * f, o[t + 2][e] * f, o[t + 3][e] * f};
  }
  __syncthreads();

  // a thread's four neighbouring values of a row, over the waves
  constexpr int QUADS = D / 4;
  const int cols = (int)min(16u, tl.rows - tl.r0);
  float *part = static_cast<float *>(a.ws) +
                ((int64_t)item * max_splits + split) * part_floats(16, D);
  for (int u = threadIdx.x; u < cols * QUADS; u += 64 * W) {
    const int cc = u / QUADS, d = (u % QUADS) * 4;
    float mm = ml[0][0][cc], ll = 0.0f;
#pragma unroll
    for (int v = 1; v < W; ++v) mm = fmaxf(mm, ml[0][v][cc]);
    f32x4 x = {0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < W; ++v) {
      const float mv = ml[0][v][cc];
      ll += mv == -INFINITY ? 0.0f : ml[1][v][cc] * exp2_fast(mv - mm);
      x += *reinterpret_cast<const f32x4 *>(sums + (v * 16 + cc) * PITCH + d);
    }
    if (place.whole(range)) {
      store_row(c, a, tl, head, cc, d, x, mm, ll);
    } else if constexpr (S::kPrefix || S::kSuffix) {
      const uint32_t at = (uint32_t)tl.row_head(a, head, tl.r0 + cc);
      *scope.sums(a.ws, place.slot(), at, D, d) = x;
      if (d == 0) *scope.ml(a.ws, place.slot(), at, D) = make_float2(mm, ll);
    } else {
      *reinterpret_cast<f32x4 *>(part + cc * D + d) = x;
      if (d == 0) *reinterpret_cast<float2 *>(part + 16 * D + 2 * cc) = make_float2(mm, ll);
    }
  }
}

template <int D, int W>
__global__ __launch_bounds__(64 * W) void decode_kernel(KvCache c, int64_t layer, KvBatch b,
                                                        KvAttention a, uint32_t tiles,
                                                        int max_splits, int split_steps) {
  __shared__ DecodeLds<D, W> lds;
  decode_part(c, layer, b, a, tiles, max_splits, split_steps, Whole{}, blockIdx.x, lds);
}

// ---------------------------------------------------------------------------
// Many rows: one workgroup of 4 waves per (128 rows of a kv head, part of the
// keys), 32 rows a wave.  64 keys and values at a time are copied to LDS as
// they lie in memory, two steps ahead, each wave one block of 16; every wave
// widens what it reads.  Lane l owns row l % 32; with h = l / 32 it holds keys
// 8a + 4h + e of each 32 (a, e = 0 .. 3), element 4a + e of a product.
//
// Bound by the vector unit: per 32 rows and 64 keys (D = 128) the products
// take 32 matrix instructions of 32 cycles, and widening the codes 128 vector
// instructions, the softmax some 130 and 32 exponentials, 4 and 8 cycles each.
// 14449 rows of 28 heads over 4: 1385 to 1430 us = 1045 to 1080 TFLOP/s, the
// vector unit busy 0.73 of the time and the matrix cores 0.50; a product of
// large bf16 matrices reaches 1222 TFLOP/s.  Keys and values widened once per
// workgroup, bf16 in LDS, took 1538 us (LDS is then full), the scores of the
// next 32 keys beside the weights of these 1486 us.
constexpr int kTileKeys = 64;
constexpr int kTileWaves = 4;
constexpr int kTileRows = 32 * kTileWaves;
constexpr int kStages = 3;

template <int D>
struct TileLds {
  static constexpr int kV = kTileKeys * D;              // values, after the keys
  static constexpr int kS = 2 * kTileKeys * D;          // scales: 4 of keys, 4 of values
  static constexpr int kStage = kS + 64;
  static constexpr int kClean = kStages * kStage;       // values of a step without their NaN
  static constexpr int kBytes = kClean + kTileKeys * D;
  static constexpr int kCopies = 2 * (D / 64) + 2;      // per wave and stage
};

// The end of a tile of 64 rows (tile_part with H = 2), through LDS that nobody copies into
// any more: the two waves that share rows add their sums, each wave half of
// them, and the rows go through LDS once more, so that whole ones are stored side by
// side (a lane's own values are 16 bytes of every one of its pieces: 1.7 us to store
// them as they lie).
template <int D, class S, int DT>
__device__ inline void store_halves(const KvCache &c, const KvAttention &a, const S &scope, bool whole,
                                    int slot, const TileOf<typename S::Number> &tl, int head, int sub, int half,
                                    f32x16 (&o)[DT], float m, float sum, uint8_t *lds) {
  constexpr int PITCH = D + 4, QUADS = D / 4, AT_ONCE = 256 / QUADS;
  static_assert(64 * (PITCH * 4 + 8) <= TileLds<D>::kBytes && 4 * 64 * (32 * DT + 8) <= TileLds<D>::kBytes,
                "both have room in the stages");
  const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
  // what a wave gives to the other one, [wave][..][lane]
  f32x4 *given = reinterpret_cast<f32x4 *>(lds) + lane;
  float2 *given_ml = reinterpret_cast<float2 *>(lds + 4 * 2 * DT * 64 * 16) + lane;
  float *rows = reinterpret_cast<float *>(lds);
  float2 *rows_ml = reinterpret_cast<float2 *>(rows + 64 * PITCH);
  const int mine = 2 * half + sub, its = 2 * (1 - half) + sub;
  __syncthreads();
  // elements 8 half .. 8 half + 7 of every tile are the wave's own
  auto give = [&](auto from) {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        constexpr int E = decltype(from)::value;
        given[((mine * DT + t) * 2 + i) * 64] =
            f32x4{o[t][E + 4 * i], o[t][E + 4 * i + 1], o[t][E + 4 * i + 2], o[t][E + 4 * i + 3]};
      }
  };
  if (half) give(std::integral_constant<int, 0>());
  else give(std::integral_constant<int, 8>());
  given_ml[mine * 64] = make_float2(m, sum);
  __syncthreads();
  const float2 other = given_ml[its * 64];
  const float top = fmaxf(m, other.x);
  const float f0 = m == -INFINITY ? 0.0f : exp2_fast(m - top);
  const float f1 = other.x == -INFINITY ? 0.0f : exp2_fast(other.x - top);
  sum = sum * f0 + other.y * f1;
  float y[DT][8];
  auto add = [&](auto from) {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f32x4 x = given[((its * DT + t) * 2 + i) * 64];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          y[t][4 * i + e] = o[t][decltype(from)::value + 4 * i + e] * f0 + x[e] * f1;
      }
  };
  if (half) add(std::integral_constant<int, 8>());
  else add(std::integral_constant<int, 0>());
  __syncthreads();
  // element 4a + e of tile t is value DT (8a + 4h + e) + t
  float *to = rows + (32 * sub + col) * PITCH + (16 * half + 4 * h) * DT;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int x = 0; x < DT; ++x) {
      f32x4 z;
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = y[(4 * x + e) % DT][4 * i + (4 * x + e) / DT];
      *reinterpret_cast<f32x4 *>(to + i * 8 * DT + 4 * x) = z;
    }
  if (half == 0 && h == 0) rows_ml[32 * sub + col] = make_float2(top, sum);
  __syncthreads();
  const int count = (int)min(64u, tl.rows - tl.r0), d = threadIdx.x % QUADS * 4;
  // row r0 + cc among all rows and heads: its token, counted from the tile's first one, by a
  // product that is exact for r under 2^21
  const uint32_t from = tl.r0 % tl.group;
  const uint32_t first = (uint32_t)((tl.row0 + tl.r0 / tl.group) * a.heads) + head * tl.group;
  const float inverse = 1.0f / (float)tl.group;
  auto place_of = [&](int cc) {
    const uint32_t r = from + cc, tok = (uint32_t)(((float)r + 0.5f) * inverse);
    return first + tok * ((uint32_t)a.heads - tl.group) + r;
  };
  if (whole) {
    for (int cc = threadIdx.x / QUADS; cc < count; cc += AT_ONCE) {
      const float2 ml = rows_ml[cc];
      store_sums(c, a, place_of(cc), d, *reinterpret_cast<const f32x4 *>(rows + cc * PITCH + d), ml.x, ml.y);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 64 / AT_ONCE; ++i) {
    const int cc = i * AT_ONCE + threadIdx.x / QUADS;
    const f32x4 x = *reinterpret_cast<const f32x4 *>(rows + cc * PITCH + d);
    const float2 ml = rows_ml[cc];
    const uint32_t at = place_of(cc);
    if (cc < count) {
      *scope.sums(a.ws, slot, at, D, d) = x;
      if (d == 0) *scope.ml(a.ws, slot, at, D) = ml;
    }
  }
}

// H = 2: tiles of 64 rows, two waves for each 32 of them, which take the first and the
// last 32 keys of every step and meet in LDS at the end.
template <int D, int G, int H, class S>
__device__ inline void tile_part(const KvCache &c, int64_t layer, const KvBatch &b,
                                 const KvAttention &a, typename S::Number seqs, uint32_t tiles,
                                 typename S::Number max_splits, int split_steps, const S &scope,
                                 uint32_t w, uint8_t *all_lds) {
  using Tile = TileOf<typename S::Number>;
  using L = TileLds<D>;
  constexpr int DT = D / 32;   // tiles of 32 values
  constexpr int CH = D / 16;   // 16-byte pieces of a key
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & (kTileWaves - 1);
  // the team of four waves: team g takes steps g, g + G, .. with its own LDS
  const int team = __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * kTileWaves));
  uint8_t *const lds = all_lds + team * L::kBytes;
  static_assert(G == 1 || H == 1, "one way to share a tile");
  const int half = H == 2 ? wave >> 1 : 0;
  const int col = lane & 31, h = lane >> 5;
  // heads first: a kv head's workgroups run on the same dies and find its keys
  // in their cache; the last rows, which see most, start first
  const int head = w % scope.heads(c);
  w = w / scope.heads(c);
  const int split = w % max_splits;
  w = w / max_splits;
  const uint32_t seq = w % seqs;
  const uint32_t tile = tiles - 1 - w / seqs;
  const Place<S, kTileKeys> place(c, b, a, scope, seq, tile, kTileRows / H, split, max_splits, split_steps);
  if (S::kPrefix && place.shared == 0) return;
  Tile tl = place.tile();
  if (tl.empty()) return;
  int at = -1;  // a prefix's: positions of the tile's tokens
  if constexpr (S::kPrefix)
    if (!place.ahead())
      at = tl.template positions<kTileRows / H>(b, place.first, place.past,
                                                tl.template guess<kTileRows / H>(b, place.first, place.past));
  // the wave's rows: with two teams, waves w and w + 4 share a SIMD and hold
  // different halves of the tile
  const int sub = H == 2 ? wave & 1 : team == 0 ? wave : wave ^ 2;
  uint32_t r0 = tl.r0 + 32 * sub;
  int p_hi = tl.p_hi;
  if (!S::kPrefix && !S::kSuffix && G > 1 && a.window == 0 && max_splits == 1) {
    // the halves are the sequence's 64 rows number `tile` from its end (sub 0
    // and 1) and from its start, so that every tile has as much to do
    const uint32_t high = (2 * ((tl.rows + kTileRows - 1) / kTileRows) - 1 - tile) * 64;
    r0 = (sub < 2 ? high : 64 * tile) + 32 * (sub & 1);
    const uint32_t end = high < tl.rows ? high + 64 : 64 * tile + 64;
    p_hi = tl.len - tl.n + (int)((min(end, tl.rows) - 1) / tl.group);
  }
  const Steps<kTileKeys> steps = place.steps(tl, p_hi);
  const Range range = place.range(steps);
  if (range.none) return;
  const int begin = range.begin + team, mine_steps = range.end - range.begin;
  const int turns = (mine_steps + G - 1) / G;
  const int n = (mine_steps - team + G - 1) / G;

  const bool mine = r0 + col < tl.rows, idle = r0 >= tl.rows;
  const uint32_t r = mine ? r0 + col : tl.rows - 1;
  const int tok = (int)(r / tl.group), qh = head * tl.group + (int)(r % tl.group);
  int pos = mine ? tl.len - tl.n + tok : -1;
  int w_lo = idle ? 0 : tl.len - tl.n + (int)(r0 / tl.group);
  int w_hi = idle ? -1 : tl.len - tl.n + (int)(min(r0 + 31, tl.rows - 1) / tl.group);

  // copies of one step: the wave's block of 16 keys and values, and its scales
  const int32_t *table = place.table;
  uint32_t koff[D / 64];  // where in the block the lane's 16 bytes of each copy lie
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    // piece p of key row lies in LDS at piece p ^ (row / 2 % CH): 16 lanes of
    // a read then hit every bank once
    const int at = i * 64 + lane, row = at / CH, piece = (at % CH) ^ ((row >> 1) & (CH - 1));
    koff[i] = row * D + piece * 16;
  }
  // lane 4s + i: page of block i of step s of a group of 16, -1 for none
  auto pages_of = [&](int s0) {
    const int s = begin + (s0 + (lane >> 2)) * G;
    const int t0 = steps.key(s) + 16 * (lane & 3);
    int page = -1;
    if (s0 + (lane >> 2) < n && t0 < tl.end) page = table[t0 >> c.page_shift];
    return page;
  };
  int page_l = -1, page_next = pages_of(0);
  if (place.elsewhere(table)) page_next = pages_of(0);
  uint64_t hole_mask = 0;
  uint32_t holes = 0;  // four bits each for the steps that are in LDS or on their way
  const uint32_t page_bytes = (uint32_t)c.page_bytes();  // at most 2^25
  const int64_t first = (layer * c.pages * c.kv_heads + head) * ((int64_t)D << c.page_shift);
  const uint8_t *const k0 = c.k + first, *const v0 = c.v + first;
  const uint8_t *const ks0 = reinterpret_cast<const uint8_t *>(c.ks) + first / (4 * D);
  const uint8_t *const vs0 = reinterpret_cast<const uint8_t *>(c.vs) + first / (4 * D);
  const uint8_t *kb = k0, *vb = v0;
  uint64_t sb = 0;
  const uint32_t lds0 = lds_addr(lds);
  uint32_t to = lds0;  // the stage of the step that is issued
  auto issue = [&](int s) {
    if (s < n) {
      if ((s & 15) == 0) {
        page_l = page_next >= c.pages ? -1 : page_next;
        hole_mask = __ballot(page_l < 0);
        if (s + 16 < n) page_next = pages_of(s + 16);
      }
      const int at = 4 * (s & 15);
      holes |= ((uint32_t)(hole_mask >> at) & 15u) << (4 * (kStages - 1));
      const int page = __builtin_amdgcn_readlane(page_l, at + wave);
      const int t0 = steps.key(begin + s * G) + 16 * wave;
      const uint64_t off = (uint64_t)(uint32_t)(page < 0 ? 0 : page) * page_bytes +
                           (uint32_t)((t0 & (c.page_tokens() - 1)) * D);
      kb = k0 + off;
      vb = v0 + off;
      sb = off / (4 * D);
    }
    // past the last step: the last again, so that every step has as many
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      copy16_to_lds(to + wave * 16 * D + i * 1024, kb, koff[i]);
      copy16_to_lds(to + L::kV + wave * 16 * D + i * 1024, vb + i * 1024, lane * 16);
    }
    if (lane == 0) {
      copy4_to_lds(to + L::kS + wave * 4, ks0 + sb, 0);
      copy4_to_lds(to + L::kS + 16 + wave * 4, vs0 + sb, 0);
    }
    to = to == lds0 + (kStages - 1) * L::kStage ? lds0 : to + L::kStage;
  };

  KvBatch::Guess guess = {};
  if constexpr (S::kPrefix)
    if (place.ahead()) guess = tl.template guess<kTileRows / H>(b, place.first, place.past);

  // the element of key piece 2m + h that step 2m + e of the first product takes
  // is value 32m + 16h + 8e
  bf16x8 q[D / 16];
  const uint16_t *qp = a.q + (tl.row0 + tok) * a.q_stride + (int64_t)qh * D + h * 16;
#pragma unroll
  for (int j = 0; j < D / 16; ++j)
    q[j] = *reinterpret_cast<const bf16x8 *>(qp + 32 * (j / 2) + 8 * (j % 2));
  const Visible<S> visible{a.window, a.sinks, place.shared};
  const float cscale = a.scale * kLog2e;
  float m = -INFINITY, l[2] = {0.0f, 0.0f};
  f32x16 o[DT] = {};

  // values 8a + 4h .. of block k: quads h and 2 + h
  auto values = [&](const uint8_t *vt, int k, uint32_t (&va)[DT], uint32_t (&vc)[DT]) {
    const uint8_t *vr = vt + k * 16 * D + h * 4 * D + col * (D / 8);
    __builtin_memcpy(va, __builtin_assume_aligned(vr, D / 8), D / 8);
    __builtin_memcpy(vc, __builtin_assume_aligned(vr + 8 * D, D / 8), D / 8);
  };
  auto compute = [&](const uint8_t *st, int key0, uint32_t hole) {
    // scales: lane 4k + i holds block i's of keys (k = 0) or values (k = 1),
    // held to what a cache can have: a masked block's may never have been
    // written, and the -inf of its scores times 0, NaN or less would not stay -inf
    const int ve_l = kv_scale_exponent(reinterpret_cast<const float *>(st + L::kS)[lane & 7]);
    const float kc_l = __uint_as_float((uint32_t)(127 + ve_l) << 23) * cscale;
    const float vi_l = __uint_as_float((uint32_t)(127 - ve_l) << 23);
    f32x16 s[2 / H];  // of the wave's keys, 32 at a time
#pragma unroll
    for (int u = 0; u < 2 / H; ++u) {
      s[u] = f32x16{};
      const uint8_t *kr = st + (32 * (u + half) + col) * D;
#pragma unroll
      for (int j = 0; j < CH / 2; ++j) {
        const uint4 k = *reinterpret_cast<const uint4 *>(
            kr + (((2 * j + h) ^ ((col >> 1) & (CH - 1))) * 16));
        s[u] = mfma(widen(k.x, k.y), q[2 * j], s[u]);
        s[u] = mfma(widen(k.z, k.w), q[2 * j + 1], s[u]);
      }
    }
    const uint8_t *vt = st + L::kV;
    float mx = kLeast;
    // blocks whose values need kLift (lanes 4 to 7 hold the values' exponents)
    uint32_t high = (uint32_t)__ballot(ve_l > kLiftExp) & 0xF0u;
    if (hole != 0 || !visible.all(key0 + 32 * half, kTileKeys / H, w_lo, w_hi)) {
      uint64_t bits = visible.bits(key0, pos);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (hole >> k & 1) bits &= ~(0xFFFFull << (16 * k));
      if (H == 2) bits = bits >> (32 * half) & 0xFFFFFFFFu;
      mx = bits != 0 ? kLeast : -INFINITY;
      high &= ~(hole << 4);  // a hole's exponent is another block's
      bits >>= 4 * h;
      // bit 8a + e for element 4a + e of s[u]
      const uint32_t see[2] = {(uint32_t)bits, (uint32_t)(bits >> 32)};
#pragma unroll
      for (int u = 0; u < 2 / H; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t on = (uint32_t)__builtin_amdgcn_sbfe((int)see[u], 8 * (i >> 2) + (i & 3), 1);
          s[u][i] = __uint_as_float((on & __float_as_uint(s[u][i])) | (~on & 0xFF800000u));  // or -inf
        }
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < kTileKeys * D; i += 1024) {
        const uint4 v = *reinterpret_cast<const uint4 *>(vt + i + lane * 16);
        any |= nan_bytes(v.x) | nan_bytes(v.y) | nan_bytes(v.z) | nan_bytes(v.w);
      }
      if (__any(any != 0)) {
        // waves that come here in one step write the same bytes; the next
        // step's barrier is between their last read and the next write
        uint8_t *clean = lds + L::kClean;
#pragma unroll 1
        for (int i = 0; i < kTileKeys * D; i += 1024) {
          const uint4 v = *reinterpret_cast<const uint4 *>(vt + i + lane * 16);
          *reinterpret_cast<uint4 *>(clean + i + lane * 16) =
              make_uint4(without_nan(v.x), without_nan(v.y), without_nan(v.z), without_nan(v.w));
        }
#pragma unroll 1
        for (int k = 0; k < 4 / H; ++k) {
          uint32_t va[DT], vc[DT];
          values(vt, k + 2 * half, va, vc);
          const uint32_t w = (k >> 1 ? see[1] : see[0]) >> (16 * (k & 1));
          spread_nan<DT>(va, vc, (w & 15u) | (w >> 4 & 0xF0u), o);
        }
        vt = clean;
      }
    }
    float kc[4 / H];
#pragma unroll
    for (int k = 0; k < 4 / H; ++k) {
      kc[k] = lane_float(kc_l, k + 2 * half);
      const auto at = [&](int i) { return s[k >> 1][8 * (k & 1) + i]; };
      float t = max3(at(0), at(1), at(2));
      t = max3(t, at(3), at(4));
      t = max3(t, at(5), at(6));
      t = max3(t, at(7), at(7));
      mx = fmaxf(mx, t * kc[k]);  // kc is positive and finite
    }
    const float lift = high != 0 ? kLift : 0.0f;
    if (__any(mx > m + (kSlack - lift))) {
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float m_new = fmaxf(m, mx + lift);
      const float alpha = m_new == -INFINITY ? 1.0f : exp2_fast(m - m_new);
      m = m_new;
      l[0] *= alpha;
      l[1] *= alpha;
#pragma unroll
      for (int t = 0; t < DT; ++t) o[t] *= alpha;
    }
    // (a row that has seen nothing yet has only -inf here, which stays 0)
    const float base = m == -INFINITY ? 0.0f : m;
    union {
      bf16x8 v[4 / H];
      bf16x2 e[16 / H];
    } p, rest;  // rest: the second term, in tiles of 64 rows
#pragma unroll
    for (int k = 0; k < 4 / H; ++k) {
      const float mk = (float)__builtin_amdgcn_readlane(ve_l, 4 + k + 2 * half) - base;
      const float inv = lane_float(vi_l, 4 + k + 2 * half);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float x = exp2_fast(fmaf(s[k >> 1][8 * (k & 1) + i], kc[k], mk));
        const float y = exp2_fast(fmaf(s[k >> 1][8 * (k & 1) + i + 1], kc[k], mk));
        p.e[4 * k + i / 2][0] = (__bf16)x;
        p.e[4 * k + i / 2][1] = (__bf16)y;
        if (H == 2) {
          rest.e[4 * k + i / 2][0] = (__bf16)(x - (float)p.e[4 * k + i / 2][0]);
          rest.e[4 * k + i / 2][1] = (__bf16)(y - (float)p.e[4 * k + i / 2][1]);
        }
        l[0] = fmaf(x, inv, l[0]);
        l[1] = fmaf(y, inv, l[1]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4 / H; ++k) {
      uint32_t va[DT], vc[DT];
      values(vt, k + 2 * half, va, vc);
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        const bf16x8 v = widen(va[t], vc[t]);
        o[t] = mfma(v, p.v[k], o[t]);
        if (H == 2) o[t] = mfma(v, rest.v[k], o[t]);
      }
    }
  };

  for (int s = 0; s < kStages - 1; ++s) {
    issue(s);
    holes >>= 4;  // the steps issued now have the low places
  }
  if constexpr (S::kPrefix) {
    // (all of these loads are in flight together)
    if (place.ahead()) at = tl.template positions<kTileRows / H>(b, place.first, place.past, guess);
    const int row_pos = __shfl(at, tok - (int)(tl.r0 / tl.group));
    pos = mine ? row_pos : -1;
    w_lo = lanes_min(mine ? pos : 0x7FFFFFFF);
    w_hi = -lanes_min(-pos);
  }
  // q is waited for here: a wait inside the loop would be for the copies too
#pragma unroll
  for (int j = 0; j < D / 16; ++j) asm volatile("" : "+v"(q[j]));
  const uint8_t *st = lds;
  for (int s = 0; s < turns; ++s) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((kStages - 2) * L::kCopies) : "memory");
    issue(s + kStages - 1);
    const int key0 = steps.key(begin + s * G);
    // rows of this wave that see nothing here leave it out
    const int k_lo = key0 + 32 * half, k_hi = k_lo + kTileKeys / H - 1;
    const bool none = s >= n || k_lo > w_hi || (a.window > 0 && k_hi <= w_lo - a.window && k_lo >= a.sinks);
    if (!none) compute(st, key0, holes & 15u);
    st = st == lds + (kStages - 1) * L::kStage ? lds : st + L::kStage;
    holes >>= 4;
  }
  // copies into LDS land before the workgroup ends
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  float sum = l[0] + l[1];
  sum += __shfl_xor(sum, 32);
  if constexpr (H == 2) {
    store_halves<D>(c, a, scope, place.whole(range), place.slot(), tl, head, sub, half, o, m, sum, all_lds);
    return;
  }
  if (G > 1) {  // the teams' sums, through LDS that nobody copies into any more
    __syncthreads();
    float *of = reinterpret_cast<float *>(all_lds) + sub * (64 * (16 * DT + 2)) + lane;
    if (team == 1) {
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) of[64 * (16 * t + e)] = o[t][e];
      of[64 * 16 * DT] = m;
      of[64 * (16 * DT + 1)] = sum;
    }
    __syncthreads();
    if (team == 1) return;
    const float m1 = of[64 * 16 * DT], sum1 = of[64 * (16 * DT + 1)];
    const float top = fmaxf(m, m1);
    const float f0 = m == -INFINITY ? 0.0f : exp2_fast(m - top);
    const float f1 = m1 == -INFINITY ? 0.0f : exp2_fast(m1 - top);
    m = top;
    sum = sum * f0 + sum1 * f1;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[t][e] = o[t][e] * f0 + of[64 * (16 * t + e)] * f1;
  }
  // worked out again rather than kept in registers through the loop
  const int lane2 = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  const int my_col = lane2 & 31, my_h = lane2 >> 5;
  if (r0 + my_col >= tl.rows) return;
  // element 4a + e of tile t is value DT (8a + 4h + e) + t
  if (place.whole(range)) {
    const float inv = 1.0f / sum;
    const uint32_t keep = m == -INFINITY ? 0u : ~0u;  // no key was seen
    const uint32_t row = r0 + my_col;
    const int64_t at = tl.row_head(a, head, row);
    uint16_t *to = a.out + at * D + my_h * (4 * DT);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t y[2 * DT];
#pragma unroll
      for (int x = 0; x < 4 * DT; x += 2) {
        const float u = o[x % DT][4 * i + x / DT] * inv, v = o[(x + 1) % DT][4 * i + (x + 1) / DT] * inv;
        y[x / 2] = bf16_pair(u, v) & keep;
      }
#pragma unroll
      for (int x = 0; x < DT / 2; ++x)
        *reinterpret_cast<uint4 *>(to + i * 8 * DT + 8 * x) =
            make_uint4(y[4 * x], y[4 * x + 1], y[4 * x + 2], y[4 * x + 3]);
    }
    if (a.lse && my_h == 0) a.lse[at] = log_sum(m, sum);
    return;
  }
  const int64_t item = ((int64_t)seq * tiles + tile) * c.kv_heads + head;
  float *part = static_cast<float *>(a.ws) + (item * max_splits + split) * part_floats(kTileRows, D);
  const int row = 32 * sub + my_col;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int x = 0; x < DT; ++x) {
      f32x4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = o[(4 * x + e) % DT][4 * i + (4 * x + e) / DT];
      *reinterpret_cast<f32x4 *>(part + row * D + i * 8 * DT + my_h * 4 * DT + 4 * x) = y;
    }
  if (my_h == 0) *reinterpret_cast<float2 *>(part + kTileRows * D + 2 * row) = make_float2(m, sum);
}

template <int D, int G>
__global__ __launch_bounds__(64 * kTileWaves * G, 2) void tile_kernel(KvCache c, int64_t layer,
                                                                      KvBatch b, KvAttention a,
                                                                      uint32_t tiles,
                                                                      int max_splits,
                                                                      int split_steps) {
  __shared__ __align__(16) uint8_t lds[G * TileLds<D>::kBytes];
  tile_part<D, G, 1, Whole>(c, layer, b, a, (uint32_t)b.seqs, tiles, max_splits, split_steps, Whole{}, blockIdx.x, lds);
}

// Shared first tokens: the first workgroups take the prefixes of all groups, the others
// the suffixes of all sequences, in one launch: the former are bound by the vector
// unit, the latter by memory.  A group's rows of a kv head (sequences x rows x query heads
// to each) are the columns of one product, in tiles of 64 rows or 16, so that shared keys
// are read and widened once for all of them; a row's parts of the prefix and its
// sequence's suffix, each (m, l, sum), meet in join_shared_kernel by
//   m = max m_i,  l = sum l_i 2^(m_i - m),  out = sum x_i 2^(m_i - m) / l.
// Weights go into the products as two bf16 terms, as those of single tokens do in
// nf4_kv_attention, in whose place a call may stand: one term, which halves the second
// product of tiles of 64, took 17.5 us of 18.2 (eight beams over 14449 tokens, 28 heads over 4),
// 40.2 of 41.8 (64 sequences over 4096), 22.4 of 24.2 (24 of five rows over up to 3501), with the
// results' error up from 0.0017 to 0.0022.
//
// 64 sequences of up to 2000 tokens past 4096 shared ones, 32 heads over 8 of 128 (145 MB):
// 39.8 us in a trace, 3.6 TB/s; 512 of its 608 workgroups run at a time (211 registers, and
// 57.5 KB of LDS, of which a compute unit has 160), the rest
// start where short suffixes end, after some 15 us.  Short calls are bound by chains that
// nothing hides: 8 sequences past 14449, 28 heads over 4 (16 MB, 14.1 us in a trace), a
// prefix's workgroup takes, by clocks read while weights had one term, 9.6 us, 3.6 of them to
// its first step (arguments, groups, page ids and positions, trips to memory one after the
// other), 1.1 for its first keys, 1 for each of four steps, which is 3.9 TB/s by all of them, and
// 1.9 for the halves' meeting and the store.
struct SharedPlan {
  uint32_t prefix_grid;
  Divisor groups, prefix_tiles, prefix_splits;
  Divisor seqs, tiles, splits;
  int steps;  // of a suffix's part
};

// A workgroup's tile of ROWS rows: 16 or 64.
template <int D, int ROWS, class S>
__device__ inline void shared_part(const KvCache &c, int64_t layer, const KvBatch &b,
                                   const KvAttention &a, const Divisor &seqs, const Divisor &tiles,
                                   const Divisor &splits, int steps, const S &scope, uint32_t w,
                                   uint8_t *lds) {
  if constexpr (ROWS == 16)
    decode_part(c, layer, b, a, tiles, splits, steps, scope, w,
                *reinterpret_cast<DecodeLds<D, 4> *>(lds));
  else
    tile_part<D, 1, 2, S>(c, layer, b, a, seqs, tiles, splits, steps, scope, w, lds);
}

// What the kernel is called with.  It reads them where it takes its way, not at its
// start, as it would by itself: both ways' arguments together pass the scalar registers.
struct SharedArgs {
  KvCache c;
  int64_t layer;
  KvBatch b;
  KvAttention a;
  Shared scope;
  SharedPlan p;
};

template <int D, int PREFIX_ROWS, int ROWS>
__global__ __launch_bounds__(256, 2) void shared_kernel(SharedArgs) {
  constexpr int kTile = TileLds<D>::kBytes, kDecode = sizeof(DecodeLds<D, 4>);
  static_assert(kTile >= kDecode, "the larger of the two");
  __shared__ __align__(16) uint8_t lds[PREFIX_ROWS == 16 && ROWS == 16 ? kDecode : kTile];
  const SharedArgs *args = (const SharedArgs *)__builtin_amdgcn_kernarg_segment_ptr();
  const uint32_t prefix_grid = args->p.prefix_grid;
  if (blockIdx.x < prefix_grid) {
    asm volatile("; a prefix");
    const SharedArgs x = *args;
    shared_part<D, PREFIX_ROWS>(x.c, x.layer, x.b, x.a, x.p.groups, x.p.prefix_tiles,
                                x.p.prefix_splits, 0,
                                Prefix{x.scope}, blockIdx.x, lds);
  } else {
    asm volatile("; a suffix");
    const SharedArgs x = *args;
    shared_part<D, ROWS>(x.c, x.layer, x.b, x.a, x.p.seqs, x.p.tiles, x.p.splits, x.p.steps,
                         Suffix{x.scope}, blockIdx.x - prefix_grid, lds);
  }
}

// Joins the parts of rows: 256 threads take four neighbouring values each of
// 256 / (D / 4) / turns rows, and turns over the parts, in a fixed order.
// A second launch rather than the last workgroup to arrive: between eight
// dies, the stores, the count and the loads of that are each a trip to memory
// one after the other (two sequences of 14449 tokens, 28 heads over 4: 16.3 us
// that way, 13.6 us with the launch, 9.4 us without either).
template <int D, int N>
__global__ __launch_bounds__(256) void join_kernel(KvCache c, KvBatch b, KvAttention a,
                                                   uint32_t tiles, int width, int groups, int turns,
                                                   int max_splits, int split_steps) {
  constexpr int QUADS = D / 4;
  __shared__ f32x4 xs[256];
  __shared__ float2 mls[256];
  const int d = (threadIdx.x % QUADS) * 4, t = threadIdx.x / QUADS, turn = t % turns;
  const int rows = 256 / QUADS / turns;
  uint32_t w = blockIdx.x;
  const int cc = (w % (uint32_t)groups) * rows + t / turns;
  w /= (uint32_t)groups;
  const uint32_t item = w;
  const int head = w % (uint32_t)c.kv_heads;
  w /= (uint32_t)c.kv_heads;
  const float *part = static_cast<const float *>(a.ws) +
                      (int64_t)item * max_splits * part_floats(width, D);
  // the first parts are on their way before the lengths say how many there are
  float2 ml[8];
  f32x4 y[8];
  auto load = [&](int s0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float *from = part + min(s0 + j * turns, max_splits - 1) * part_floats(width, D);
      ml[j] = *reinterpret_cast<const float2 *>(from + width * D + 2 * min(cc, width - 1));
      y[j] = *reinterpret_cast<const f32x4 *>(from + min(cc, width - 1) * D + d);
    }
  };
  load(turn);
  const Tile tl(Whole::group(c, a), b, b.raw(w / tiles), w % tiles, width);
  if (tl.empty()) return;
  const Steps<N> steps(0, tl.p_lo, tl.last_key(tl.p_hi), a.window, a.sinks);
  if (steps.count <= split_steps) return;  // written already
  const int splits = (steps.count + split_steps - 1) / split_steps;
  const bool on = cc < width && tl.r0 + cc < tl.rows;
  float mm = -INFINITY, ll = 0.0f;
  f32x4 x = {0, 0, 0, 0};
  for (int s0 = turn; s0 < splits; s0 += 8 * turns) {
    if (s0 != turn) load(s0);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (s0 + j * turns < splits) join(mm, ll, x, ml[j].x, ml[j].y, y[j]);
  }
  if (turns > 1) {
    xs[threadIdx.x] = x;
    mls[threadIdx.x] = make_float2(mm, ll);
    __syncthreads();
    if (turn == 0)
      for (int j = 1; j < turns; ++j) {
        const float2 other = mls[threadIdx.x + j * QUADS];
        join(mm, ll, x, other.x, other.y, xs[threadIdx.x + j * QUADS]);
      }
  }
  if (on && turn == 0) store_row(c, a, tl, head, cc, d, x, mm, ll);
}

// The same for rows whose keys are those of a shared prefix and of the sequence's own
// suffix: a workgroup takes `256 / (D / 4) / turns` rows and heads of a sequence, which lie
// side by side in every slot.  Bound by its chain: arguments and groups 1 us, the parts, which
// other dies have written, 2, the turns' meeting 1; 4.0 to 5.1 us in traces.  The first
// parts read beside the groups, from where the rows most likely are, took longer
// (beams over 14449 tokens 17.1 us against 16.8 as a whole), by the instructions it added.
struct SharedJoin {
  Divisor splits;     // the suffix's plan
  int steps;
  int turns;          // a power of two
  Divisor per_seq;    // workgroups of a sequence
  Divisor heads;
};

template <int D, int N>
__global__ __launch_bounds__(256) void join_shared_kernel(KvCache c, KvBatch b, KvAttention a,
                                                          Shared scope, SharedJoin j) {
  constexpr int QUADS = D / 4;
  __shared__ f32x4 xs[256];
  __shared__ float2 mls[256];
  const int d = (threadIdx.x % QUADS) * 4, t = threadIdx.x / QUADS, turn = t & (j.turns - 1);
  const int turn_bits = __builtin_ctz(j.turns), row = t >> turn_bits;
  const int64_t seq = blockIdx.x / j.per_seq;
  const uint32_t first_row_head = (blockIdx.x % j.per_seq) * (256 / QUADS >> turn_bits);
  const KvBatch::Raw raw = b.raw(seq);
  int first = 0;
  const int shared = scope.g.shared_of(b, seq, &first);
  int64_t row0;
  int n, len, end;
  b.sequence(raw, row0, n, len, end);
  const int rows = n < b.max_rows ? n : b.max_rows;
  if (first_row_head >= (uint32_t)rows * a.heads) return;
  const uint32_t i = first_row_head + row;
  const bool on = i < (uint32_t)rows * a.heads;
  const int tok = on && b.max_rows > 1 ? (int)(i / j.heads) : 0;
  int splits = 1;
  if (j.splits > 1) {
    // the steps of the tile that the row is in
    constexpr int WIDTH = N == 32 ? 16 : 64;
    const Divisor &group_heads = scope.heads_each;
    const uint32_t r = tok * group_heads + (i % j.heads) % group_heads, r0 = r / WIDTH * WIDTH;
    const uint32_t r1 = min(r0 + WIDTH, (uint32_t)rows * group_heads) - 1;
    const int begin = len - n, p_lo = begin + (int)(r0 / group_heads), p_hi = begin + (int)(r1 / group_heads);
    const Steps<N> steps(shared / N, p_lo, min(p_hi, end - 1), a.window, a.sinks);
    const int per = Place<Suffix, N>::suffix_steps(steps.count, j.steps, j.splits);
    if (steps.count > per) splits = (steps.count + per - 1) / per;
  }
  const bool written = shared == 0 && splits == 1;
  int shared_parts = shared > 0 ? scope.prefix_slots : 0;
  if (scope.g.max_rows < b.rows && shared > 0) {
    const int64_t at = row0 + tok - b.first_row(first);  // the row among its group's
    if (at < 0 || at >= scope.g.max_rows) shared_parts = 0;
  }
  const uint32_t row_head = (uint32_t)row0 * a.heads + (on ? i : 0);
  const int parts = on && !written ? shared_parts + splits : 0;
  float mm = -INFINITY, ll = 0.0f;
  f32x4 x = {0, 0, 0, 0};
  for (int s0 = turn; s0 < parts; s0 += 8 * j.turns) {
    float2 ml[8];
    f32x4 y[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      int s = min(s0 + u * j.turns, parts - 1);
      if (s >= shared_parts) s += scope.prefix_slots - shared_parts;
      ml[u] = *scope.ml(a.ws, s, row_head, D);
      y[u] = *scope.sums(a.ws, s, row_head, D, d);
    }
    // all eight to the largest m of theirs and of those before
    float top = mm;
#pragma unroll
    for (int u = 0; u < 8; ++u) top = fmaxf(top, ml[u].x);  // (past the last part: the last one)
    const float f = mm == -INFINITY ? 0.0f : exp2_fast(mm - top);
    ll *= f;
    x *= f;
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (s0 + u * j.turns < parts && ml[u].x != -INFINITY) {
        const float g = exp2_fast(ml[u].x - top);
        ll += ml[u].y * g;
        x += y[u] * g;
      }
    mm = top;
  }
  if (j.turns > 1) {
    // every turn scales its own sums to the largest m, then they are added
    mls[threadIdx.x] = make_float2(mm, ll);
    __syncthreads();
    const int first_turn = threadIdx.x - turn * QUADS;
    float top = mm;
    for (int u = 0; u < j.turns; ++u) top = fmaxf(top, mls[first_turn + u * QUADS].x);
    const float f = mm == -INFINITY ? 0.0f : exp2_fast(mm - top);
    x = mm == -INFINITY ? f32x4{0, 0, 0, 0} : x * f;
    xs[threadIdx.x] = x;
    __syncthreads();
    if (turn == 0) {
      ll = ll * f;
      for (int u = 1; u < j.turns; ++u) {
        const float2 other = mls[threadIdx.x + u * QUADS];
        if (other.x == -INFINITY) continue;
        ll += other.y * exp2_fast(other.x - top);
        x += xs[threadIdx.x + u * QUADS];
      }
      mm = top;
    }
  }
  if (parts > 0 && turn == 0) store_sums(c, a, row_head, d, x, mm, ll);
}

// How a call is launched: in tiles of `width` rows, a workgroup taking
// split_steps steps of `keys` keys.
struct Plan {
  bool few;
  int width, keys, teams;
  int64_t tiles, items, splits;
  int split_steps;
};

// Few rows: a workgroup takes 64 steps (2048 keys), so that sequences of very
// different lengths fill the card evenly (64 sequences of up to 16384 tokens:
// 217 us, one workgroup each 238 us), and fewer, down to 16, where that leaves
// compute units without one (two sequences of 14449 tokens: 13.9 us with 16,
// 15.2 with 8).  Splitting costs the second launch, so a call whose rows all
// see at most that many steps is not split (48 sequences with a window of
// 1500: 20.4 us, split in two 25.5 us).
// Up to 32 rows: 16 sequences of up to 8000 tokens, 32 heads over 4: 32 rows 30.4
// us, as a tile of many rows 31.9; 40 rows 46.9 as three tiles of few, 32.9 as
// one of many, and 64 sequences of up to 500 19.5 and 12.4.  (One sequence alone
// favours tiles of few: 35 rows over 14449 tokens 15.5 us, 17.1 as one of many.)
// At most 256 parts: one sequence of 10^6 tokens, one kv head, takes 48.9 us,
// 99.7 in at most 64 parts, 52.9 in at most 1024.
constexpr int kWaves = 4;
constexpr int64_t kMinSteps = 16, kMostSteps = 64, kMaxSplits = 256;
constexpr int64_t kFewRows = 32;

// Many rows: no more tiles than compute units leave a unit one workgroup, and a
// SIMD one wave, which waits for its own products half of the time: then two
// teams of waves share a tile (1024 rows of 28 heads over 4, 224 tiles: 27.0 us
// against 29.3; and 23.7, by now 22.2, with a late and an early half in every
// tile, so that none has more keys to go through), and the keys are split as far as one
// workgroup per unit goes, in parts of 8 steps at least (113 rows over 14449
// tokens, 28 tiles: 9 parts of two teams 49 us, 18 parts of one 55 us, 10
// parts, past one workgroup per unit, 75 us).  Parts of 4 steps at least instead:
// 26.9 us against 25.1 for 300 rows over 3000 tokens, 8 heads over 2, 13.1
// against 15.1 for 40 rows over 2000, 8 heads; of 16: 29.3 and 20.1.
constexpr int64_t kMinTileSteps = 8;

// `seqs` sequences (or groups) of up to `max_rows` rows; most(keys, span): the most steps of
// that many keys for a tile whose rows stand at `span` positions.
template <class Most>
Plan plan_for(const KvCache &c, int64_t seqs, int64_t max_rows, int heads, Most most) {
  Plan p;
  const int64_t group = heads / c.kv_heads, rows = max_rows * group, cus = device_cu_count();
  p.teams = 1;
  p.few = rows <= kFewRows;
  p.width = p.few ? 16 : kTileRows;
  p.keys = p.few ? 32 : kTileKeys;
  p.tiles = (rows + p.width - 1) / p.width;
  p.items = seqs * p.tiles * c.kv_heads;
  const int64_t span = (p.width - 1 + group) / group + 1;  // positions of a tile's rows
  const int64_t steps = most(p.keys, (int)span);
  const int64_t even = (p.items * steps + cus - 1) / cus;
  int64_t per;
  if (p.few) {
    per = even < kMinSteps ? kMinSteps : even > kMostSteps ? kMostSteps : even;
    per = (per + kWaves - 1) / kWaves * kWaves;
    // sixteen tiles for every compute unit fill the card evenly by themselves
    // (512 sequences of up to 4000 tokens, 8 kv heads of 64: 198 us, split 224;
    // two tiles for each do not: 64 sequences above.  Eight, which are split,
    // would do better without: 256 sequences of up to 4000, 32 heads over 8, 127
    // us, unsplit 110)
    if (p.items >= 16 * cus) per = steps;
  } else {
    per = steps;
    p.teams = p.items <= cus ? 2 : 1;
    if (p.teams == 2) {
      const int64_t parts = cus / p.items;
      per = std::max(kMinTileSteps, (steps + parts - 1) / parts);
    }
  }
  if (per > steps) per = steps;
  if (per * kMaxSplits < steps) per = (steps + kMaxSplits - 1) / kMaxSplits;
  p.split_steps = (int)per;
  p.splits = (steps + per - 1) / per;
  return p;
}

Plan make_plan(const KvCache &c, const KvBatch &b, int heads, int window, int sinks) {
  return plan_for(c, b.seqs, b.max_rows, heads, [&](int keys, int span) {
    return most_steps(keys, b, span, window, sinks);
  });
}

// The suffixes are as long as the bounds say if the longest sequence has the longest
// prefix.  That is a guess: where it is not so, a part has more steps.
Plan suffix_plan(const KvCache &c, const KvBatch &b, const KvGroups &g, int heads, int window,
                 int sinks) {
  KvBatch guess = b;
  if (g.max_shared < b.max_len) guess.max_len = b.max_len - g.max_shared;
  Plan p = make_plan(c, guess, heads, window, sinks);
  p.teams = 1;
  if (p.few) return p;
  const int64_t group = heads / c.kv_heads, rows = b.max_rows * group;
  p.width = 64;
  p.tiles = (rows + p.width - 1) / p.width;
  p.items = b.seqs * p.tiles * c.kv_heads;
  const int64_t steps =
      most_steps(p.keys, guess, (int)((p.width - 1 + group) / group + 1), window, sinks);
  int64_t per = std::min<int64_t>(std::max<int64_t>(p.items * steps / (device_cu_count() / 2), 4), 32);
  per = std::max<int64_t>(per, (steps + kMaxSplits - 1) / kMaxSplits);
  p.splits = (steps + per - 1) / per;
  p.split_steps = (int)((steps + p.splits - 1) / p.splits);
  return p;
}

// The prefixes' part of a shared launch, beside suffixes by the plan `own`.  Tiles of 64
// rows, or 16 where a group has no more than kFewRows; how many steps a workgroup takes
// goes by the steps of all tiles: some 200 workgroups, of 2 to 12 steps (microseconds of
// the whole call: 9 sequences of two rows over 4888 tokens, 32 heads over 8 of 128, in parts
// of 6 steps 18.8, of 12 20.9; 62 over 4561, three groups, of 12 23.0, of 8 24.6; 8 over
// 14449, of 4 18.7, of 7 19.7), and more, up to 24, where that is more workgroups than
// run at a time, the suffixes' among them (23 sequences of three rows over 10477, two
// groups, of 16 34.9, of 12 41.5; 64 of up to 2000 tokens past 4096, which are as many as
// run at a time by themselves, of 24 46.0, of 16 48.2, of 12 53.9, of 32 46.7 against 44.3).
// Suffixes end early where they are short, and count by their length (19 sequences of five
// rows, 28 heads over 4, whose suffixes are tiles of 64 rows, over 12000 and up to 100 tokens
// 41.0, counted whole 44.7; over 6498 and up to 1331 41.9, counted whole 35.5).  Beside
// those, prefixes of 128 values take up to 32 steps (48 of five rows over 12000, three
// groups, 28 heads over 4, 69.4, with 24 73.2), of 64 values 24 (32 heads over 4, 50.0,
// with 32 55.0).  All of these with weights of one bf16 term in tiles of 64 rows; two take 2 to
// 8 % longer.  Every group counts as large as the largest: where they differ, some of the
// workgroups have nothing to do, and the others' parts are that much longer.
// Tiles of 16 rows: some 200 workgroups, of 16 to 40 steps of 32 keys (8 sequences over 20000,
// 16 heads over 8, in parts of 24 17.7, of 16 19.7, of 40 18.9; 8 over 32000, 8 heads, of 40
// 20.3, of 16 23.0, of 64 22.9; 16 over 3000, 16 heads over 8, of 16 13.9, of 24 15.4), and
// more where that is three for every compute unit (32 over 9000, 8 groups, 32 heads over 8, of
// 40 37.1, of 24 41.7).  A window's rows may stand anywhere: as many steps as it is long
// are counted.
Plan prefix_plan(const KvCache &c, const KvBatch &b, const KvGroups &g, int heads, int window,
                 const Plan &own) {
  const int64_t longest = std::min<int64_t>(g.max_shared, b.max_len), group = heads / c.kv_heads;
  const int64_t rows = g.max_rows * group, cus = device_cu_count();
  Plan p;
  p.teams = 1;
  p.few = rows <= kFewRows && own.few;
  p.width = p.few ? 16 : 64;
  p.keys = p.few ? 32 : kTileKeys;
  p.tiles = (rows + p.width - 1) / p.width;
  p.items = g.groups * p.tiles * c.kv_heads;
  int64_t steps = std::max<int64_t>((longest + p.keys - 1) / p.keys, 1);
  if (window > 0) steps = std::min<int64_t>(steps, window / p.keys + 2);
  int64_t per;
  if (p.few) {
    per = std::min<int64_t>(std::max<int64_t>(p.items * steps * 5 / (4 * cus), kMinSteps), 40);
    per = std::max<int64_t>(per, p.items * steps / (3 * cus));
  } else {
    per = std::min<int64_t>(std::max<int64_t>(p.items * steps * 5 / (4 * cus), 2), 12);
    const int64_t slots = (c.head_dim == 128 ? 2 : 3) * cus;
    const int64_t whole = own.few ? 1024 : 512;  // keys of a suffix that stays as long as prefixes
    const int64_t taken = own.items * own.splits * std::min<int64_t>(own.split_steps * own.keys, whole) / whole;
    const int64_t room = std::max<int64_t>((slots - taken) / p.items, 1);
    per = std::max<int64_t>(per, std::min<int64_t>((steps + room - 1) / room, !own.few && c.head_dim == 128 ? 32 : 24));
  }
  per = std::max<int64_t>(per, (steps + kMaxSplits - 1) / kMaxSplits);
  p.splits = (steps + per - 1) / per;
  p.split_steps = 0;  // as many as that leaves for each
  return p;
}

// Whether a call takes the shared keys apart.  Without that, every tile of 16 rows reads
// its own sequence's keys, which for shared ones mostly means from the caches, at some
// 9.5 TB/s, and a short call is one launch of 6.5 us where taking them apart costs two, 12
// us.  So it has to save reading kSavedBytes (a guess from the bounds): 53 sequences
// over up to 397 shared tokens, 8 heads of 64 (22 MB): 8.2 us as one, 14.3 apart; 28 over
// 776 (22 MB) 16.9 and 17.7; 8 over 14449, 4 heads of 128 (104 MB) 21.3 and 20.1; 32 over
// a window of 2048, 8 heads of 128 (130 MB) 30.2 and 24.2.  A sequence whose own rows fill
// a tile of 128 reads its keys once for them as it is.
constexpr int64_t kSavedBytes = int64_t(64) << 20;
// Nor where the parts would take more room than this: 400000 rows times heads of 128 in
// ten parts, whose queries alone are 100 MB.
constexpr int64_t kMostPartBytes = int64_t(2) << 30;

// Up to 2^31 threads a launch.
bool fits(const Plan &p) { return p.items * p.splits <= 0x7FFFFFFF / (256 * p.teams); }

// Rows of a tile side by side in a workgroup of the join, and turns over the parts: as
// many turns as there are four parts for each, the rest of the threads on other rows.
int join_turns(int head_dim, int64_t parts) {
  int turns = 256 / (head_dim / 4);
  while (turns > 1 && parts <= 2 * turns) turns /= 2;
  return turns;
}

struct SharedPlans {
  bool apart;
  Plan prefix, own;
  int turns;        // of the join, and its workgroups of a sequence
  int64_t per_seq;
  int64_t bytes;    // of the workspace
};

SharedPlans shared_plans(const KvCache &c, const KvBatch &b, const KvGroups &g, int heads,
                         int window, int sinks) {
  SharedPlans p{};
  const int64_t group = heads / c.kv_heads, rows = b.max_rows * group;
  int64_t keys = std::min(g.max_shared, b.max_len);
  if (window > 0) keys = std::min<int64_t>(keys, window);
  const int64_t tiles = b.seqs * ((rows + 15) / 16) - g.groups * ((g.max_rows * group + 63) / 64);
  if (rows > kTileRows || tiles <= 0 || keys <= kSavedBytes / (tiles * c.kv_heads * 2 * c.head_dim))
    return p;
  p.own = suffix_plan(c, b, g, heads, window, sinks);
  p.prefix = prefix_plan(c, b, g, heads, window, p.own);
  p.bytes = (p.prefix.splits + p.own.splits) * b.rows * heads * (c.head_dim + 2) * (int64_t)sizeof(float);
  p.turns = join_turns(c.head_dim, p.prefix.splits + p.own.splits);
  const int64_t at_once = 256 / (c.head_dim / 4) / p.turns;
  p.per_seq = (b.max_rows * (int64_t)heads + at_once - 1) / at_once;
  Plan both = p.own;  // one launch
  both.items = p.prefix.items * p.prefix.splits + p.own.items * p.own.splits;
  both.splits = 1;
  p.apart = p.bytes <= kMostPartBytes && fits(both) && b.seqs * p.per_seq <= 0x7FFFFFFF / 256;
  return p;
}

int64_t plan_floats(const Plan &p, int head_dim) {
  return p.items * p.splits * part_floats(p.width, head_dim);
}

}  // namespace

size_t kv_attention_workspace_bytes(const KvCache &c, const KvBatch &b, int heads, int window,
                                    int sinks) {
  const Plan p = make_plan(c, b, heads, window, sinks);
  if (p.splits == 1) return 0;
  return (size_t)plan_floats(p, c.head_dim) * sizeof(float);
}

size_t kv_attention_shared_workspace_bytes(const KvCache &c, const KvBatch &b, const KvGroups &g,
                                           int heads, int window, int sinks) {
  const SharedPlans p = shared_plans(c, b, g, heads, window, sinks);
  return p.apart ? (size_t)p.bytes : kv_attention_workspace_bytes(c, b, heads, window, sinks);
}

hipError_t launch_kv_attention(const KvCache &c, int64_t layer, const KvBatch &b,
                               const KvAttention &a, hipStream_t s) {
  const Plan p = make_plan(c, b, a.heads, a.window, a.sinks);
  const int64_t cols = std::min<int64_t>(p.width, (int64_t)b.max_rows * (a.heads / c.kv_heads));
  const int turns = join_turns(c.head_dim, p.splits);
  const int at_once = 256 / (c.head_dim / 4) / turns;
  const int64_t groups = (cols + at_once - 1) / at_once;
  if (!fits(p)) return hipErrorInvalidConfiguration;
  if (p.splits > 1 && p.items * groups > 0x7FFFFFFF / 256) return hipErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(p.items * p.splits)), dim3(256 * p.teams), 0, s, c,
                       layer, b, a, (uint32_t)p.tiles, (int)p.splits, p.split_steps);
  };
  if (p.few) {
    if (c.head_dim == 128) go(decode_kernel<128, kWaves>);
    else go(decode_kernel<64, kWaves>);
  } else {
    if (p.teams == 1) {
      if (c.head_dim == 128) go(tile_kernel<128, 1>);
      else go(tile_kernel<64, 1>);
    } else {
      if (c.head_dim == 128) go(tile_kernel<128, 2>);
      else go(tile_kernel<64, 2>);
    }
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  auto join = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(p.items * groups)), dim3(256), 0, s, c, b, a,
                       (uint32_t)p.tiles, p.width, (int)groups, turns, (int)p.splits,
                       p.split_steps);
  };
  if (p.few) {
    if (c.head_dim == 128) join(join_kernel<128, 32>);
    else join(join_kernel<64, 32>);
  } else {
    if (c.head_dim == 128) join(join_kernel<128, kTileKeys>);
    else join(join_kernel<64, kTileKeys>);
  }
  return hipGetLastError();
}

hipError_t launch_kv_attention_shared(const KvCache &c, int64_t layer, const KvBatch &b,
                                      const KvGroups &g, const KvAttention &a, hipStream_t s) {
  const SharedPlans plans = shared_plans(c, b, g, a.heads, a.window, a.sinks);
  if (!plans.apart) return launch_kv_attention(c, layer, b, a, s);
  const Plan &p = plans.prefix, &own = plans.own;
  const Shared scope{g, (uint32_t)(b.rows * a.heads), (int)p.splits, (int)(p.splits + own.splits),
                     Divisor::of(c.kv_heads), Divisor::of(a.heads / c.kv_heads)};
  const SharedPlan plan{(uint32_t)(p.items * p.splits), Divisor::of(g.groups), Divisor::of(p.tiles),
                        Divisor::of(p.splits), Divisor::of(b.seqs), Divisor::of(own.tiles),
                        Divisor::of(own.splits), own.split_steps};
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(p.items * p.splits + own.items * own.splits)), dim3(256),
                       0, s, SharedArgs{c, layer, b, a, scope, plan});
  };
  auto pick = [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    if (!own.few) go(shared_kernel<D, 64, 64>);
    else if (p.few) go(shared_kernel<D, 16, 16>);
    else go(shared_kernel<D, 64, 16>);
  };
  if (c.head_dim == 128) pick(std::integral_constant<int, 128>());
  else pick(std::integral_constant<int, 64>());
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const SharedJoin j{Divisor::of(own.splits), own.split_steps, plans.turns, Divisor::of(plans.per_seq),
                     Divisor::of(a.heads)};
  auto join = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(b.seqs * plans.per_seq)), dim3(256), 0, s, c, b, a, scope, j);
  };
  if (own.few) {
    if (c.head_dim == 128) join(join_shared_kernel<128, 32>);
    else join(join_shared_kernel<64, 32>);
  } else {
    if (c.head_dim == 128) join(join_shared_kernel<128, kTileKeys>);
    else join(join_shared_kernel<64, kTileKeys>);
  }
  return hipGetLastError();
}

}  // namespace nf4
