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

// The keys of one row: up to its position, inside the window or among the
// first tokens.
struct Visible {
  int window, sinks;
  __device__ bool operator()(int key, int pos) const {
    return (key <= pos) & ((window == 0) | (key > pos - window) | (key < sinks));
  }
  // Bit x: whether the row sees key + x, x = 0 .. 63.
  __device__ uint64_t bits(int key, int pos) const {
    auto upto = [](int t) {  // bits 0 .. t
      return t < 0 ? 0ull : t >= 63 ? ~0ull : ~0ull >> (63 - t);
    };
    uint64_t b = upto(pos - key);
    if (window > 0) b &= ~upto(pos - window - key) | upto(sinks - 1 - key);
    return b;
  }
  // Whether every row at p_lo .. p_hi sees all of key .. key + n - 1.
  __device__ bool all(int key, int n, int p_lo, int p_hi) const {
    return key + n - 1 <= p_lo && (window == 0 || key > p_hi - window || key + n <= sinks);
  }
};

// The steps of N keys that rows from p_lo on can see, as a list: those with
// first tokens, then from the start of the lowest row's window to the key `last`.
template <int N>
struct Steps {
  int sink_steps, from, count;
  __device__ Steps(int p_lo, int last, int window, int sinks) {
    sink_steps = from = 0;
    const int steps = last < 0 ? 0 : last / N + 1;
    if (window > 0 && p_lo - window + 1 > 0) {
      from = (p_lo - window + 1) / N;
      sink_steps = min((int)(((int64_t)sinks + N - 1) / N), steps);
      if (sink_steps >= from) from = sink_steps = 0;
    }
    count = sink_steps + max(steps - from, 0);
  }
  __device__ int key(int i) const { return (i < sink_steps ? i : i - sink_steps + from) * N; }
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
struct Tile {
  int64_t row0;
  uint32_t rows, r0, group;  // rows of a kv head of one sequence stay under 2^31
  int n, len, end, p_lo, p_hi;
  __device__ Tile(const KvCache &c, const KvBatch &b, const KvAttention &a, int64_t seq,
                  uint32_t tile, uint32_t width) {
    group = (uint32_t)a.heads / (uint32_t)c.kv_heads;
    b.sequence(seq, row0, n, len, end);
    rows = (uint32_t)(n < b.max_rows ? n : b.max_rows) * group;
    r0 = tile * width;
    const uint32_t last = r0 + width < rows ? r0 + width - 1 : rows - 1;
    p_lo = len - n + (int)(r0 / group);
    p_hi = len - n + (int)(last / group);
  }
  __device__ bool empty() const { return r0 >= rows; }
  // The last key that a row at p may see: not past the table.
  __device__ int last_key(int p) const { return min(p, end - 1); }
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

// The result of row `cc` of a tile, values d .. d + 3, from its sums.
__device__ inline void store_row(const KvCache &c, const KvAttention &a, const Tile &tl, int head,
                                 int cc, int d, f32x4 x, float m, float l) {
  const uint32_t r = tl.r0 + cc;
  const int64_t at = (tl.row0 + r / tl.group) * a.heads + head * tl.group + r % tl.group;
  const bool none = m == -INFINITY;  // no key was seen
  const float inv = 1.0f / l;
  uint2 y;
  y.x = none ? 0u : bf16_pair(x[0] * inv, x[1] * inv);
  y.y = none ? 0u : bf16_pair(x[2] * inv, x[3] * inv);
  *reinterpret_cast<uint2 *>(a.out + at * c.head_dim + d) = y;
  if (a.lse && d == 0) a.lse[at] = log_sum(m, l);
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
__global__ __launch_bounds__(64 * W) void decode_kernel(KvCache c, int64_t layer, KvBatch b,
                                                        KvAttention a, uint32_t tiles,
                                                        int max_splits,
                                                        int split_steps) {
  constexpr int KS = D / 32;   // k-steps of the first product
  constexpr int DT = D / 16;   // tiles of 16 values of the second
  constexpr int PITCH = D + 4; // of a row of sums in LDS, in floats
  __shared__ float sums[W * 16 * PITCH];
  __shared__ float ml[2][W][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  // neighbouring workgroups take the heads of one page, so that what is read
  // at a time lies side by side (64 sequences of up to 16384 tokens: 256 us
  // with the parts of a head side by side instead, 217 us this way)
  uint32_t w = blockIdx.x;
  const int head = w % (uint32_t)c.kv_heads;
  w /= (uint32_t)c.kv_heads;
  const int split = w % (uint32_t)max_splits;
  w /= (uint32_t)max_splits;
  const int64_t seq = w / tiles;
  const uint32_t item = w * (uint32_t)c.kv_heads + head;
  const int32_t *table = b.table + seq * b.table_stride;
  // without a window, where the first page ids stand does not depend on the
  // lengths: they are read beside them (as far as the longest one may reach)
  int page_ahead = -1;
  if (a.window == 0) {
    const int64_t t0 = (int64_t)(split * split_steps + wave + (lane >> 1) * W) * 32 + 16 * (lane & 1);
    page_ahead = table[min(t0, (int64_t)max(b.max_len - 1, 0)) >> c.page_shift];
  }
  const Tile tl(c, b, a, seq, w % tiles, 16);
  if (tl.empty()) return;
  const Steps<32> steps(tl.p_lo, tl.last_key(tl.p_hi), a.window, a.sinks);
  const int splits = steps.count <= split_steps ? 1 : (steps.count + split_steps - 1) / split_steps;
  if (split >= splits) return;
  const int end = min(steps.count, (split + 1) * split_steps);

  const bool mine = tl.r0 + col < tl.rows;
  const uint32_t r = mine ? tl.r0 + col : tl.rows - 1;
  const int tok = (int)(r / tl.group), qh = head * tl.group + (int)(r % tl.group);
  const int pos = mine ? tl.len - tl.n + tok : -1;

  const int64_t layer_pages = layer * c.pages;
  const int page_blocks = 1 << (c.page_shift - 4);
  // What the wave's next 32 steps need to know of their blocks, lane 2s + h
  // for block h of step s: page (-1: none), c times the keys' scale, and for
  // the values' scale 2^e e and 2^-e.  Read ahead of the steps as vectors: a
  // scalar read per step would cost the step its whole latency, since scalar
  // reads return out of order and any use waits for all of them.
  const int first = split * split_steps + wave;
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
      page_l = a.window == 0 && i0 == first ? page_ahead : table[t0 >> c.page_shift];
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

  bf16x8 q[KS];
  const uint16_t *qp = a.q + (tl.row0 + tok) * a.q_stride + (int64_t)qh * D + g * 16;
#pragma unroll
  for (int j = 0; j < KS; ++j)
    q[j] = *reinterpret_cast<const bf16x8 *>(qp + 64 * (j / 2) + 8 * (j % 2));

  const Visible visible{a.window, a.sinks};
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
    if (splits == 1) {
      store_row(c, a, tl, head, cc, d, x, mm, ll);
    } else {
      *reinterpret_cast<f32x4 *>(part + cc * D + d) = x;
      if (d == 0) *reinterpret_cast<float2 *>(part + 16 * D + 2 * cc) = make_float2(mm, ll);
    }
  }
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

template <int D, int G>
__global__ __launch_bounds__(64 * kTileWaves * G, 2) void tile_kernel(KvCache c, int64_t layer,
                                                                      KvBatch b, KvAttention a,
                                                                      uint32_t tiles,
                                                                      int max_splits,
                                                                      int split_steps) {
  using L = TileLds<D>;
  constexpr int DT = D / 32;   // tiles of 32 values
  constexpr int CH = D / 16;   // 16-byte pieces of a key
  __shared__ __align__(16) uint8_t all_lds[G * L::kBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & (kTileWaves - 1);
  // the team of four waves: team g takes steps g, g + G, .. with its own LDS
  const int team = __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * kTileWaves));
  uint8_t *const lds = all_lds + team * L::kBytes;
  const int col = lane & 31, h = lane >> 5;
  // heads first: a kv head's workgroups run on the same dies and find its keys
  // in their cache; the last rows, which see most, start first
  uint32_t w = blockIdx.x;
  const int head = w % (uint32_t)c.kv_heads;
  w /= (uint32_t)c.kv_heads;
  const int split = w % (uint32_t)max_splits;
  w /= (uint32_t)max_splits;
  const uint32_t seq = w % (uint32_t)b.seqs;
  const uint32_t tile = tiles - 1 - w / (uint32_t)b.seqs;
  const Tile tl(c, b, a, seq, tile, kTileRows);
  if (tl.empty()) return;
  // the wave's rows: with two teams, waves w and w + 4 share a SIMD and hold
  // different halves of the tile
  const int sub = team == 0 ? wave : wave ^ 2;
  uint32_t r0 = tl.r0 + 32 * sub;
  int p_hi = tl.p_hi;
  if (G > 1 && a.window == 0 && max_splits == 1) {
    // the halves are the sequence's 64 rows number `tile` from its end (sub 0
    // and 1) and from its start, so that every tile has as much to do
    const uint32_t high = (2 * ((tl.rows + kTileRows - 1) / kTileRows) - 1 - tile) * 64;
    r0 = (sub < 2 ? high : 64 * tile) + 32 * (sub & 1);
    const uint32_t end = high < tl.rows ? high + 64 : 64 * tile + 64;
    p_hi = tl.len - tl.n + (int)((min(end, tl.rows) - 1) / tl.group);
  }
  const Steps<kTileKeys> steps(tl.p_lo, tl.last_key(p_hi), a.window, a.sinks);
  const int splits = steps.count <= split_steps ? 1 : (steps.count + split_steps - 1) / split_steps;
  if (split >= splits) return;
  const int begin = split * split_steps + team;
  const int turns = (min(steps.count - split * split_steps, split_steps) + G - 1) / G;
  const int n = (min(steps.count - split * split_steps, split_steps) - team + G - 1) / G;

  const bool mine = r0 + col < tl.rows, idle = r0 >= tl.rows;
  const uint32_t r = mine ? r0 + col : tl.rows - 1;
  const int tok = (int)(r / tl.group), qh = head * tl.group + (int)(r % tl.group);
  const int pos = mine ? tl.len - tl.n + tok : -1;
  const int w_lo = idle ? 0 : tl.len - tl.n + (int)(r0 / tl.group);
  const int w_hi = idle ? -1 : tl.len - tl.n + (int)(min(r0 + 31, tl.rows - 1) / tl.group);

  // copies of one step: the wave's block of 16 keys and values, and its scales
  const int32_t *table = b.table + (int64_t)seq * b.table_stride;
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
      holes |= ((uint32_t)(hole_mask >> at) & 15u) << 8;
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

  // the element of key piece 2m + h that step 2m + e of the first product takes
  // is value 32m + 16h + 8e
  bf16x8 q[D / 16];
  const uint16_t *qp = a.q + (tl.row0 + tok) * a.q_stride + (int64_t)qh * D + h * 16;
#pragma unroll
  for (int j = 0; j < D / 16; ++j)
    q[j] = *reinterpret_cast<const bf16x8 *>(qp + 32 * (j / 2) + 8 * (j % 2));
  const Visible visible{a.window, a.sinks};
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
    f32x16 s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u] = f32x16{};
      const uint8_t *kr = st + (32 * u + col) * D;
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
    if (hole != 0 || !visible.all(key0, kTileKeys, w_lo, w_hi)) {
      uint64_t bits = visible.bits(key0, pos);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (hole >> k & 1) bits &= ~(0xFFFFull << (16 * k));
      mx = bits != 0 ? kLeast : -INFINITY;
      high &= ~(hole << 4);  // a hole's exponent is another block's
      bits >>= 4 * h;
      // bit 8a + e for element 4a + e of s[u]
      const uint32_t see[2] = {(uint32_t)bits, (uint32_t)(bits >> 32)};
#pragma unroll
      for (int u = 0; u < 2; ++u)
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
        for (int k = 0; k < 4; ++k) {
          uint32_t va[DT], vc[DT];
          values(vt, k, va, vc);
          const uint32_t w = (k >> 1 ? see[1] : see[0]) >> (16 * (k & 1));
          spread_nan<DT>(va, vc, (w & 15u) | (w >> 4 & 0xF0u), o);
        }
        vt = clean;
      }
    }
    float kc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      kc[k] = lane_float(kc_l, k);
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
      bf16x8 v[4];
      bf16x2 e[16];
    } p;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float mk = (float)__builtin_amdgcn_readlane(ve_l, 4 + k) - base;
      const float inv = lane_float(vi_l, 4 + k);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float x = exp2_fast(fmaf(s[k >> 1][8 * (k & 1) + i], kc[k], mk));
        const float y = exp2_fast(fmaf(s[k >> 1][8 * (k & 1) + i + 1], kc[k], mk));
        p.e[4 * k + i / 2][0] = (__bf16)x;
        p.e[4 * k + i / 2][1] = (__bf16)y;
        l[0] = fmaf(x, inv, l[0]);
        l[1] = fmaf(y, inv, l[1]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t va[DT], vc[DT];
      values(vt, k, va, vc);
#pragma unroll
      for (int t = 0; t < DT; ++t) o[t] = mfma(widen(va[t], vc[t]), p.v[k], o[t]);
    }
  };

  issue(0);
  holes >>= 4;
  issue(1);
  holes >>= 4;  // steps 0 and 1 now have the two low places
  // q is waited for here: a wait inside the loop would be for the copies too
#pragma unroll
  for (int j = 0; j < D / 16; ++j) asm volatile("" : "+v"(q[j]));
  const uint8_t *st = lds;
  for (int s = 0; s < turns; ++s) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(L::kCopies) : "memory");
    issue(s + 2);
    const int key0 = steps.key(begin + s * G);
    // rows of this wave that see nothing here leave it out
    const bool none = s >= n || key0 > w_hi || (a.window > 0 && key0 + kTileKeys - 1 <= w_lo - a.window &&
                                      key0 >= a.sinks);
    if (!none) compute(st, key0, holes & 15u);
    st = st == lds + (kStages - 1) * L::kStage ? lds : st + L::kStage;
    holes >>= 4;
  }
  // copies into LDS land before the workgroup ends
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  float sum = l[0] + l[1];
  sum += __shfl_xor(sum, 32);
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
  if (splits == 1) {
    const float inv = 1.0f / sum;
    const uint32_t keep = m == -INFINITY ? 0u : ~0u;  // no key was seen
    const uint32_t row = r0 + my_col;
    const int64_t at = (tl.row0 + row / tl.group) * a.heads + head * tl.group + row % tl.group;
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
  const Tile tl(c, b, a, w / tiles, w % tiles, width);
  if (tl.empty()) return;
  const Steps<N> steps(tl.p_lo, tl.last_key(tl.p_hi), a.window, a.sinks);
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

Plan make_plan(const KvCache &c, const KvBatch &b, int heads, int window, int sinks) {
  Plan p;
  const int64_t group = heads / c.kv_heads, rows = b.max_rows * group, cus = device_cu_count();
  p.teams = 1;
  p.few = rows <= kFewRows;
  p.width = p.few ? 16 : kTileRows;
  p.keys = p.few ? 32 : kTileKeys;
  p.tiles = (rows + p.width - 1) / p.width;
  p.items = b.seqs * p.tiles * c.kv_heads;
  const int64_t span = (p.width - 1 + group) / group + 1;  // positions of a tile's rows
  const int64_t steps = most_steps(p.keys, b, (int)span, window, sinks);
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

}  // namespace

size_t kv_attention_workspace_bytes(const KvCache &c, const KvBatch &b, int heads, int window,
                                    int sinks) {
  const Plan p = make_plan(c, b, heads, window, sinks);
  if (p.splits == 1) return 0;
  return (size_t)(p.items * p.splits * part_floats(p.width, c.head_dim)) * sizeof(float);
}

hipError_t launch_kv_attention(const KvCache &c, int64_t layer, const KvBatch &b,
                               const KvAttention &a, hipStream_t s) {
  const Plan p = make_plan(c, b, a.heads, a.window, a.sinks);
  const int64_t grid = p.items * p.splits;
  // the join: as many turns as there are four parts for each, the rest of the
  // threads on other rows
  const int64_t cols = std::min<int64_t>(p.width, (int64_t)b.max_rows * (a.heads / c.kv_heads));
  int turns = 256 / (c.head_dim / 4);
  while (turns > 1 && p.splits <= 2 * turns) turns /= 2;
  const int at_once = 256 / (c.head_dim / 4) / turns;
  const int64_t groups = (cols + at_once - 1) / at_once;
  // up to 2^31 threads a launch
  if (grid > 0x7FFFFFFF / (256 * p.teams)) return hipErrorInvalidConfiguration;
  if (p.splits > 1 && p.items * groups > 0x7FFFFFFF / 256) return hipErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(256 * p.teams), 0, s, c, layer, b, a,
                       (uint32_t)p.tiles, (int)p.splits, p.split_steps);
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
  hipError_t e = hipGetLastError();
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

}  // namespace nf4
