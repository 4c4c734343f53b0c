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

struct Visible {
  int len, window, sinks;
  __device__ bool operator()(int key, int pos) const {
    return key <= pos && (window == 0 || key > pos - window || key < sinks);
  }
};

// One wave: 16 query rows of a kv head (a row is a token and a head of the
// group) against the keys, 32 at a time.  Lane l owns query row l % 16; with
// g = l / 16 it holds keys 4g .. 4g + 3 of both blocks of a step.
template <int D>
__global__ __launch_bounds__(64) void attention16_kernel(KvCache c, int64_t layer, KvBatch b,
                                                         KvAttention a, int64_t tiles) {
  constexpr int KS = D / 32;  // k-steps of the first product
  constexpr int DT = D / 16;  // tiles of 16 values of the second
  const int lane = threadIdx.x, col = lane & 15, g = lane >> 4;
  int64_t w = blockIdx.x;
  const int head = (int)(w % c.kv_heads);
  w /= c.kv_heads;
  const int64_t tile = w % tiles, seq = w / tiles;
  const int group = a.heads / c.kv_heads;
  int64_t row0;
  int n, len;
  b.sequence(seq, c.page_shift, row0, n, len);
  const int64_t rows = (int64_t)(n < b.max_rows ? n : b.max_rows) * group;
  if (tile * 16 >= rows) return;
  const int64_t r = tile * 16 + col;
  const bool mine = r < rows;
  const int64_t tok = mine ? r / group : (rows - 1) / group;
  const int qh = head * group + (int)(mine ? r % group : 0);
  const int pos = mine ? len - n + (int)tok : -1;
  const int p_lo = len - n + (int)(tile * 16 / group);
  const int64_t last_row = tile * 16 + 15 < rows ? tile * 16 + 15 : rows - 1;
  const int p_hi = len - n + (int)(last_row / group);

  bf16x8 q[KS];
  const uint16_t *qp = a.q + (row0 + tok) * a.q_stride + (int64_t)qh * D + g * (D / 4);
#pragma unroll
  for (int j = 0; j < KS; ++j) q[j] = *reinterpret_cast<const bf16x8 *>(qp + 8 * j);

  const float cscale = a.scale * kLog2e;
  const Visible visible{len, a.window, a.sinks};
  float m = -INFINITY, l = 0.0f;
  f32x4 o[DT] = {};

  // steps of 32 keys: those that hold visible first tokens, then from the
  // window of the lowest row on
  int from = 0, sink_steps = 0;
  if (a.window > 0 && p_lo - a.window + 1 > 0) {
    from = (p_lo - a.window + 1) / 32;
    sink_steps = (a.sinks + 31) / 32;
    if (sink_steps >= from) from = sink_steps = 0;
  }
  const int steps = p_hi < 0 ? 0 : sink_steps + p_hi / 32 + 1 - from;
  for (int st = 0; st < steps; ++st) {
    const int key0 = (st < sink_steps ? st : st - sink_steps + from) * 32;
    f32x4 s[2];
    uint32_t vw[2][DT];
    float vlog[2], vinv[2];
    bool hole[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t0 = key0 + 16 * h;
      int page = -1;
      if (t0 < len) page = b.table[seq * b.table_stride + (t0 >> c.page_shift)];
      hole[h] = page < 0 || page >= c.pages;
      const int64_t block = ((layer * c.pages + (hole[h] ? 0 : page)) * c.kv_heads + head) *
                                (int64_t)(1 << (c.page_shift - 4)) +
                            ((t0 & (c.page_tokens() - 1)) >> 4);
      const uint8_t *kp = c.k + block * (16 * D) + col * D + g * (D / 4);
      const uint8_t *vp = c.v + block * (16 * D) + (g * D + col * DT) * 4;
      uint32_t kw[D / 16];
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        *reinterpret_cast<uint4 *>(kw + 4 * i) = *reinterpret_cast<const uint4 *>(kp + 16 * i);
        *reinterpret_cast<uint4 *>(vw[h] + 4 * i) = *reinterpret_cast<const uint4 *>(vp + 16 * i);
      }
      s[h] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < KS; ++j) s[h] = mfma16(widen(kw[2 * j], kw[2 * j + 1]), q[j], s[h]);
      const float kc = cscale * c.ks[block];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[h][i] *= kc;
      // (held to what a cache can have: a block that was never written may
      // lie past the last token, and 0 weight times its 2^-e has to be 0)
      int ve = (int)((__float_as_uint(c.vs[block]) >> 23) & 255u) - 127;
      ve = ve < kKvExpMin ? kKvExpMin : ve > kKvExpMax ? kKvExpMax : ve;
      vlog[h] = (float)ve;
      vinv[h] = __uint_as_float((uint32_t)(127 - ve) << 23);
    }
    bool see[2][4];
    float mx = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        see[h][i] = !hole[h] && visible(key0 + 16 * h + 4 * g + i, pos);
        if (see[h][i]) mx = fmaxf(mx, s[h][i]);
      }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float m_new = fmaxf(m, mx);
    const float alpha = m_new == -INFINITY ? 1.0f : exp2_fast(m - m_new);
    m = m_new;
    l *= alpha;
#pragma unroll
    for (int t = 0; t < DT; ++t) o[t] *= alpha;
    union {
      bf16x8 v;
      __bf16 e[8];
    } p, ones;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = see[h][i] ? exp2_fast(s[h][i] - m + vlog[h]) : 0.0f;
        sum += x;
        p.e[4 * h + i] = (__bf16)x;
        ones.e[4 * h + i] = (__bf16)(see[h][i] ? 1.0f : 0.0f);
      }
      l += sum * vinv[h];
    }
    // NaN codes in places that some row does not see would reach it as 0 * NaN:
    // they count as 0, and 1 per visible NaN makes the sum NaN where it is due
    uint32_t nan = 0;
#pragma unroll
    for (int t = 0; t < DT; ++t) nan |= nan_bytes(vw[0][t]) | nan_bytes(vw[1][t]);
    if (__any(nan != 0)) {
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        const f32x4 hit = mfma16(widen(nan_ones(vw[0][t]), nan_ones(vw[1][t])), ones.v,
                                 f32x4{0, 0, 0, 0});
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (hit[i] > 0.0f) o[t][i] = NAN;
        vw[0][t] = without_nan(vw[0][t]);
        vw[1][t] = without_nan(vw[1][t]);
      }
    }
#pragma unroll
    for (int t = 0; t < DT; ++t) o[t] = mfma16(widen(vw[0][t], vw[1][t]), p.v, o[t]);
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (!mine) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  // element i of tile t is value (4g + i) DT + t
  uint16_t *op = a.out + (row0 + tok) * a.heads * D + (int64_t)qh * D + g * (D / 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    union {
      uint4 v[DT / 4 > 1 ? DT / 8 + (DT % 8 != 0) : 1];
      __bf16 e[DT];
    } y;
#pragma unroll
    for (int t = 0; t < DT; ++t) y.e[t] = (__bf16)(l == 0.0f ? 0.0f : o[t][i] * inv);
    if (DT == 8) *reinterpret_cast<uint4 *>(op + i * DT) = y.v[0];
    else *reinterpret_cast<uint2 *>(op + i * DT) = *reinterpret_cast<uint2 *>(&y.v[0]);
  }
  if (a.lse && g == 0)
    a.lse[(row0 + tok) * a.heads + qh] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2;
}

}  // namespace

size_t kv_attention_workspace_bytes(const KvCache &, const KvBatch &, int, int, int) { return 0; }

hipError_t launch_kv_attention(const KvCache &c, int64_t layer, const KvBatch &b,
                               const KvAttention &a, hipStream_t s) {
  const int64_t tiles = ((int64_t)b.max_rows * (a.heads / c.kv_heads) + 15) / 16;
  const int64_t grid = b.seqs * tiles * c.kv_heads;
  if (grid > 0x7FFFFFFF / 64) return hipErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(64), 0, s, c, layer, b, a, tiles);
  };
  if (c.head_dim == 128) go(attention16_kernel<128>);
  else go(attention16_kernel<64>);
  return hipGetLastError();
}

}  // namespace nf4
