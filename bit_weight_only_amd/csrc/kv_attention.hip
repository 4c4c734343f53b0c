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

namespace nf4 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

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

__device__ inline f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Exponent of a block's scale, held to what a cache can have.
__device__ inline int kv_scale_exponent(float s) {
  const int e = (int)((__float_as_uint(s) >> 23) & 255u) - 127;
  return e < kKvExpMin ? kKvExpMin : e > kKvExpMax ? kKvExpMax : e;
}

// The keys of one row: up to its position, inside the window or among the
// first tokens.
struct Visible {
  int window, sinks;
  __device__ bool operator()(int key, int pos) const {
    return (key <= pos) & ((window == 0) | (key > pos - window) | (key < sinks));
  }
  // Whether every row at p_lo .. p_hi sees all of key .. key + n - 1.
  __device__ bool all(int key, int n, int p_lo, int p_hi) const {
    return key + n - 1 <= p_lo && (window == 0 || key > p_hi - window || key + n <= sinks);
  }
};

// The steps of N keys that rows p_lo .. p_hi can see, as a list: those with
// first tokens, then from the start of the lowest row's window on.
template <int N>
struct Steps {
  int sink_steps, from, count;
  __device__ Steps(int p_lo, int p_hi, int window, int sinks) {
    sink_steps = from = 0;
    if (window > 0 && p_lo - window + 1 > 0) {
      from = (p_lo - window + 1) / N;
      sink_steps = (int)(((int64_t)sinks + N - 1) / N);
      if (sink_steps >= from) from = sink_steps = 0;
    }
    count = p_hi < 0 ? 0 : sink_steps + p_hi / N + 1 - from;
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
  int n, len, p_lo, p_hi;
  __device__ Tile(const KvCache &c, const KvBatch &b, const KvAttention &a, int64_t seq,
                  uint32_t tile, uint32_t width) {
    group = (uint32_t)a.heads / (uint32_t)c.kv_heads;
    b.sequence(seq, c.page_shift, row0, n, len);
    rows = (uint32_t)(n < b.max_rows ? n : b.max_rows) * group;
    r0 = tile * width;
    const uint32_t last = r0 + width < rows ? r0 + width - 1 : rows - 1;
    p_lo = len - n + (int)(r0 / group);
    p_hi = len - n + (int)(last / group);
  }
  __device__ bool empty() const { return r0 >= rows; }
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

// The result of row `cc` of a tile, values d .. d + 3, from its sums.
__device__ inline void store_row(const KvCache &c, const KvAttention &a, const Tile &tl, int head,
                                 int cc, int d, f32x4 x, float m, float l) {
  const uint32_t r = tl.r0 + cc;
  const int64_t at = (tl.row0 + r / tl.group) * a.heads + head * tl.group + r % tl.group;
  const bool none = l == 0.0f;  // no key was seen
  const float inv = none ? 0.0f : 1.0f / l;
  uint2 y;
  y.x = none ? 0u : bf16_pair(x[0] * inv, x[1] * inv);
  y.y = none ? 0u : bf16_pair(x[2] * inv, x[3] * inv);
  *reinterpret_cast<uint2 *>(a.out + at * c.head_dim + d) = y;
  if (a.lse && d == 0) a.lse[at] = none ? -INFINITY : (m + __log2f(l)) * kLn2;
}

// NaN codes in places that some row does not see would reach it as 0 * NaN.
// They become 0 here, and a product of their places with the visible ones
// makes the sums NaN where that is due.
template <int DT>
__device__ inline void hide_nan(uint32_t (&vw)[2][DT], uint32_t see, f32x4 (&o)[DT]) {
  uint32_t nan = 0;
#pragma unroll
  for (int t = 0; t < DT; ++t) nan |= nan_bytes(vw[0][t]) | nan_bytes(vw[1][t]);
  if (!__any(nan != 0)) return;
  union {
    bf16x8 v;
    __bf16 e[8];
  } ones;
#pragma unroll
  for (int e = 0; e < 8; ++e) ones.e[e] = (__bf16)(see >> e & 1 ? 1.0f : 0.0f);
#pragma unroll
  for (int t = 0; t < DT; ++t) {
    const f32x4 hit =
        mfma16(widen(nan_ones(vw[0][t]), nan_ones(vw[1][t])), ones.v, f32x4{0, 0, 0, 0});
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (hit[e] > 0.0f) o[t][e] = NAN;
    vw[0][t] = without_nan(vw[0][t]);
    vw[1][t] = without_nan(vw[1][t]);
  }
}

// ---------------------------------------------------------------------------
// Few rows: one workgroup of W waves per (16 rows of a kv head, part of the
// keys), each wave every W-th step of 32 keys straight from memory to its
// registers, a step ahead.  Lane l owns query row l % 16; with g = l / 16 it
// holds keys 4g .. 4g + 3 of both blocks of a step.  Memory bound: a step
// reads 8 KB (D = 128) for some 400 cycles of vector work.
//
// The waves meet in LDS, the parts in the workspace: each writes its sums and
// counts its arrival, the last one adds them in order.

template <int D>
struct Step {
  uint4 k[2][D / 64], v[2][D / 64];
};

__device__ inline float lane_float(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

template <int D, int W>
__global__ __launch_bounds__(64 * W) void decode_kernel(KvCache c, int64_t layer, KvBatch b,
                                                        KvAttention a, int tiles, int max_splits,
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
  // with the parts of a head side by side instead, 221 us this way)
  uint32_t w = blockIdx.x;
  const int head = w % (uint32_t)c.kv_heads;
  w /= (uint32_t)c.kv_heads;
  const int split = w % (uint32_t)max_splits;
  w /= (uint32_t)max_splits;
  const int64_t seq = w / (uint32_t)tiles;
  const uint32_t item = w * (uint32_t)c.kv_heads + head;
  const Tile tl(c, b, a, seq, w % (uint32_t)tiles, 16);
  if (tl.empty()) return;
  const Steps<32> steps(tl.p_lo, tl.p_hi, a.window, a.sinks);
  const int splits = steps.count <= split_steps ? 1 : (steps.count + split_steps - 1) / split_steps;
  if (split >= splits) return;
  const int end = min(steps.count, (split + 1) * split_steps);

  const bool mine = tl.r0 + col < tl.rows;
  const uint32_t r = mine ? tl.r0 + col : tl.rows - 1;
  const int tok = (int)(r / tl.group), qh = head * tl.group + (int)(r % tl.group);
  const int pos = mine ? tl.len - tl.n + tok : -1;

  const int32_t *table = b.table + seq * b.table_stride;
  const int64_t layer_pages = layer * c.pages;
  const int page_blocks = 1 << (c.page_shift - 4);
  // What the wave's next 32 steps need to know of their blocks, lane 2s + h
  // for block h of step s: page (-1: none), c times the keys' scale, and for
  // the values' scale 2^e e and 2^-e.  Read ahead of the steps as vectors: a
  // scalar read per step would cost the step its whole latency, since scalar
  // reads return out of order and any use waits for all of them.
  int page_l = -1;
  float kc_l = 0.0f, ve_l = 0.0f, vi_l = 1.0f;
  auto block_of = [&](int page, int t0) {
    return ((layer_pages + page) * c.kv_heads + head) * page_blocks +
           ((t0 & (c.page_tokens() - 1)) >> 4);
  };
  auto look = [&](int i0) {
    const int i = i0 + (lane >> 1) * W;
    const int t0 = steps.key(i) + 16 * (lane & 1);
    page_l = i < end && t0 < tl.len ? table[t0 >> c.page_shift] : -1;
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

  const int first = split * split_steps + wave;
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
      for (int j = 0; j < KS; ++j) s[h] = mfma16(widen(kw[h][2 * j], kw[h][2 * j + 1]), q[j], s[h]);
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
    float mx = s[0][0];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[h][e]);
    // m only has to be near the maximum: it is raised, and the sums rescaled,
    // when a weight would pass 2^8 (as the first key's would)
    if (__any(mx > m + 8.0f)) {
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float m_new = fmaxf(m, mx);
      const float alpha = m_new == -INFINITY ? 1.0f : exp2_fast(m - m_new);
      m = m_new;
      l *= alpha;
#pragma unroll
      for (int t = 0; t < DT; ++t) o[t] *= alpha;
    }
    union {
      bf16x8 v;
      __bf16 e[8];
    } p;
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
      }
      l += sum * lane_float(vi_l, 2 * sl + h);
    }
    if (masked) hide_nan<DT>(vw, see, o);  // the same for every lane
#pragma unroll
    for (int t = 0; t < DT; ++t) o[t] = mfma16(widen(vw[0][t], vw[1][t]), p.v, o[t]);
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

// Joins the parts of a row, one workgroup per (item, row): 256 threads take
// four neighbouring values each and turns over the parts, in a fixed order.
// A second launch rather than the last workgroup to arrive: between eight
// dies, the stores, the count and the loads of that are each a trip to memory
// one after the other (two sequences of 14449 tokens, 28 heads over 4: 16.3 us
// that way, 13.6 us with the launch, 9.4 us without either).
template <int D, int N>
__global__ __launch_bounds__(256) void join_kernel(KvCache c, KvBatch b, KvAttention a,
                                                   uint32_t tiles, int width, int cols,
                                                   int max_splits, int split_steps) {
  constexpr int QUADS = D / 4, TURNS = 256 / QUADS;
  __shared__ f32x4 xs[256];
  __shared__ float ms[TURNS], ls[TURNS];
  const int d = (threadIdx.x % QUADS) * 4, turn = threadIdx.x / QUADS;
  uint32_t w = blockIdx.x;
  const int cc = w % (uint32_t)cols;
  w /= (uint32_t)cols;
  const uint32_t item = w;
  const int head = w % (uint32_t)c.kv_heads;
  w /= (uint32_t)c.kv_heads;
  const Tile tl(c, b, a, w / tiles, w % tiles, width);
  if (tl.r0 + cc >= tl.rows) return;
  const Steps<N> steps(tl.p_lo, tl.p_hi, a.window, a.sinks);
  if (steps.count <= split_steps) return;  // written already
  const int splits = (steps.count + split_steps - 1) / split_steps;
  const float *part = static_cast<const float *>(a.ws) +
                      (int64_t)item * max_splits * part_floats(width, D);
  float mm = -INFINITY, ll = 0.0f;
  f32x4 x = {0, 0, 0, 0};
  for (int s0 = turn; s0 < splits; s0 += 8 * TURNS) {
    float2 ml[8];
    f32x4 y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float *from = part + min(s0 + j * TURNS, splits - 1) * part_floats(width, D);
      ml[j] = *reinterpret_cast<const float2 *>(from + width * D + 2 * cc);
      y[j] = *reinterpret_cast<const f32x4 *>(from + cc * D + d);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (s0 + j * TURNS < splits) join(mm, ll, x, ml[j].x, ml[j].y, y[j]);
  }
  xs[threadIdx.x] = x;
  if (d == 0) ms[turn] = mm, ls[turn] = ll;
  __syncthreads();
  if (turn != 0) return;
  for (int t = 1; t < TURNS; ++t) join(mm, ll, x, ms[t], ls[t], xs[threadIdx.x + t * QUADS]);
  store_row(c, a, tl, head, cc, d, x, mm, ll);
}

// How the keys of a call are split: a workgroup takes split_steps steps.
struct Plan {
  int64_t tiles, items, splits;
  int split_steps;
};

// A workgroup takes 64 steps (2048 keys), so that sequences of very different
// lengths fill the card evenly (64 sequences of up to 16384 tokens: 221 us,
// one workgroup each 238 us), and fewer, down to 16, where that leaves
// compute units without one (two sequences of 14449 tokens: 13.7 us with 16,
// 15.2 with 8).  Splitting costs the second launch, so a call whose rows all
// see at most that many steps is not split (48 sequences with a window of
// 1500: 19.0 us, split in two 25.5 us).
constexpr int kWaves = 4;
constexpr int64_t kMinSteps = 16, kMostSteps = 64, kMaxSplits = 256;

Plan decode_plan(const KvCache &c, const KvBatch &b, int heads, int window, int sinks) {
  Plan p;
  const int group = heads / c.kv_heads;
  p.tiles = ((int64_t)b.max_rows * group + 15) / 16;
  p.items = b.seqs * p.tiles * c.kv_heads;
  const int64_t steps = most_steps(32, b, (15 + group) / group + 1, window, sinks);
  const int64_t even = (p.items * steps + device_cu_count() - 1) / device_cu_count();
  int64_t per = even < kMinSteps ? kMinSteps : even > kMostSteps ? kMostSteps : even;
  // sixteen tiles for every compute unit fill the card evenly by themselves
  if (p.items >= 16 * device_cu_count()) per = steps;
  if (per * kMaxSplits < steps) per = (steps + kMaxSplits - 1) / kMaxSplits;
  per = (per + kWaves - 1) / kWaves * kWaves;
  p.split_steps = (int)per;
  p.splits = (steps + per - 1) / per;
  return p;
}

size_t plan_bytes(const KvCache &c, const Plan &p) {
  if (p.splits == 1) return 0;
  return (size_t)(p.items * p.splits * part_floats(16, c.head_dim)) * sizeof(float);
}

}  // namespace

size_t kv_attention_workspace_bytes(const KvCache &c, const KvBatch &b, int heads, int window,
                                    int sinks) {
  return plan_bytes(c, decode_plan(c, b, heads, window, sinks));
}

hipError_t launch_kv_attention(const KvCache &c, int64_t layer, const KvBatch &b,
                               const KvAttention &a, hipStream_t s) {
  const Plan p = decode_plan(c, b, a.heads, a.window, a.sinks);
  const int64_t grid = p.items * p.splits;
  if (grid > 0x7FFFFFFF / (64 * kWaves)) return hipErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(64 * kWaves), 0, s, c, layer, b, a,
                       (int)p.tiles, (int)p.splits, p.split_steps);
  };
  if (c.head_dim == 128) go(decode_kernel<128, kWaves>);
  else go(decode_kernel<64, kWaves>);
  if (p.splits > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    auto join = [&](auto kernel) {
      const int cols = (int)std::min<int64_t>(16, (int64_t)b.max_rows * (a.heads / c.kv_heads));
      hipLaunchKernelGGL(kernel, dim3((unsigned)(p.items * cols)), dim3(256), 0, s, c, b, a,
                         (uint32_t)p.tiles, 16, cols, (int)p.splits, p.split_steps);
    };
    if (c.head_dim == 128) join(join_kernel<128, 32>);
    else join(join_kernel<64, 32>);
  }
  return hipGetLastError();
}

}  // namespace nf4
