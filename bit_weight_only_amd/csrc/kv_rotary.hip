// kv_rotary.hip -- rotary positions: heads turned by their positions, normed
// first where the model does, and the same for the queries and keys of new tokens
// in the pass that quantizes keys and values into their pages.
//
// A pair (a, b) of a head at position p is turned by the angle p f,
//
//   (a cos - b sin, a sin + b cos) gain,
//
// the norm before it is x (mean x^2 + eps)^-1/2 w over the whole head.  Frequencies
// come as turns a token in 64-bit fixed point, so that p f modulo a full turn is a
// 64-bit product, exact to 2^-35 of a turn at the longest position; its sine and
// cosine are summed in 64 bits and rounded once.
//
// vibevoice.c README: the decoder's positions are rotary; the block format and its
// rules are include/nf4.h's.
#include "kv_internal.h"
#include "kv_quant.h"

namespace nf4 {
namespace {

constexpr int kThreads = 256;

// Cosine and sine of u 2^-32 turns, times gain.  With the nearest quarter turn taken
// off, |x| <= pi / 4, and what the Taylor sums leave out is under x^11 / 11! = 2e-9.
__device__ inline float2 turned(uint32_t u, double gain) {
  const uint32_t quarter = (u + 0x20000000u) >> 30;
  const double x = (double)(int)(u - (quarter << 30)) * (6.283185307179586 / 4294967296.0);
  const double y = x * x;
  double s = fma(y, 1.0 / 362880, -1.0 / 5040);
  s = fma(y, s, 1.0 / 120);
  s = fma(y, s, -1.0 / 6);
  s = fma(y * x, s, x) * gain;
  double c = fma(y, -1.0 / 3628800, 1.0 / 40320);
  c = fma(y, c, -1.0 / 720);
  c = fma(y, c, 1.0 / 24);
  c = fma(y, c, -0.5);
  c = fma(y, c, 1.0) * gain;
  const float sf = (float)s, cf = (float)c;
  const float co = quarter & 1 ? sf : cf, si = quarter & 1 ? cf : sf;
  // quarters 1 and 2 have a negative cosine, 2 and 3 a negative sine
  return make_float2((quarter + 1) & 2 ? -co : co, quarter & 2 ? -si : si);
}

// What the workgroup's waves share: cosines and sines of 16 tokens, and for each
// wave a few rows of a head, where lanes find the other values of their pairs.
// (Rows are padded by 16 bytes, so that neighbouring ones start at other banks.)
template <int D>
struct alignas(16) TurnLds {
  float2 cs[kKvBlock][D / 2 + 2];
  float rows[kThreads / 64][512 / D][D + 4];  // 64 lanes of up to 8 values
};

// The table for tokens t0 + r, r = 0 .. 15, of which those in [lo, hi) count.
template <int D, class Position>
__device__ inline void fill_table(TurnLds<D> &lds, const KvRotary &rot, int lo, int hi,
                                  Position position) {
  constexpr int PAIRS = D / 2;
  for (int i = threadIdx.x; i < kKvBlock * PAIRS; i += kThreads) {
    const int r = i / PAIRS, p = i % PAIRS;
    if (r < lo || r >= hi || 2 * p >= rot.dims) continue;
    const uint64_t at = (uint64_t)position(r) * rot.turns[p];
    lds.cs[r][p] = turned((uint32_t)(at >> 32), rot.gain);
  }
}

// Norms (w not null) and turns one token's values of one row: `v` are the lane's, from
// value VEC * piece on; `r` the token's row of the table; `row` the wave's row in
// LDS for this lane's token.  All lanes of the wave come here together.
template <int D, int VEC>
__device__ inline void turn_row(const TurnLds<D> &lds, float *row, const KvRotary &rot,
                                const float (&w)[VEC], bool norm, double eps, int r, int piece,
                                float (&v)[VEC]) {
  constexpr int CHUNKS = D / VEC;
  if (norm) {
    // in 64 bits: squares of fp32 values keep their range
    double sum = 0.0;
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum = fma((double)v[e], (double)v[e], sum);
#pragma unroll
    for (int o = 1; o < CHUNKS; o <<= 1) sum += __shfl_xor(sum, o);
    const double mean = fma(sum, 1.0 / D, eps);
    const bool big = mean > 0x1p100;  // its root then leaves too little of 1 / root's range
    const float t = (float)(mean * (big ? 0x1p-128 : 1.0)), pre = big ? 0x1p-64f : 1.0f;
    float inv = __builtin_amdgcn_rsqf(t);
    // one step towards the root, for the last bit (not from 1 / infinity)
    if (inv > 0.0f) inv = fmaf(0.5f * inv, fmaf(-t * inv, inv, 1.0f), inv);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = v[e] * pre * inv * w[e];
  }
  const int e0 = piece * VEC;
  if (rot.dims == 0) return;
  if (rot.pairs) {
    float cs[VEC];
    __builtin_memcpy(cs, __builtin_assume_aligned(&lds.cs[r][piece * (VEC / 2)], 16), sizeof(cs));
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      const float a = v[j], b = v[j + 1];
      const bool on = e0 + j < rot.dims;
      v[j] = on ? fmaf(a, cs[j], -(b * cs[j + 1])) : a;
      v[j + 1] = on ? fmaf(b, cs[j], a * cs[j + 1]) : b;
    }
    return;
  }
  const int half = rot.dims / 2;
#pragma unroll
  for (int e = 0; e < VEC; e += 4)
    *reinterpret_cast<float4 *>(row + e0 + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (half % VEC == 0) {  // the other values of a lane's pairs are one piece
    const bool low = e0 < half, on = e0 < rot.dims;
    const int other = on ? (low ? e0 + half : e0 - half) : e0, p0 = on ? (low ? e0 : e0 - half) : 0;
    float x[VEC], cs[2 * VEC];
    __builtin_memcpy(x, __builtin_assume_aligned(row + other, 16), sizeof(x));
    __builtin_memcpy(cs, __builtin_assume_aligned(&lds.cs[r][p0], 16), sizeof(cs));
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float y = fmaf(v[e], cs[2 * e], x[e] * (low ? -cs[2 * e + 1] : cs[2 * e + 1]));
      v[e] = on ? y : v[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int at = e0 + e;
      const bool low = at < half, on = at < rot.dims;
      const float2 cs = lds.cs[r][on ? (low ? at : at - half) : 0];
      const float y = fmaf(v[e], cs.x, row[on ? (low ? at + half : at - half) : at] * (low ? -cs.y : cs.y));
      v[e] = on ? y : v[e];
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ inline uint32_t bf16_bits(float x) {
  return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// VEC values to a row of fp32 or bf16, `at` values from its start.
template <int VEC>
__device__ inline void store_values(void *row, int64_t at, bool f32, const float (&v)[VEC]) {
  if (f32) {
    float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(row) + at);
#pragma unroll
    for (int h = 0; h < VEC / 4; ++h)
      to[h] = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
    return;
  }
  uint32_t y[VEC / 2];
#pragma unroll
  for (int h = 0; h < VEC / 2; ++h) y[h] = bf16_bits(v[2 * h]) | bf16_bits(v[2 * h + 1]) << 16;
  uint16_t *to = static_cast<uint16_t *>(row) + at;
  if (VEC == 8) {
    *reinterpret_cast<uint4 *>(to) = make_uint4(y[0], y[1], y[VEC / 2 - 2], y[VEC / 2 - 1]);
  } else {
    *reinterpret_cast<uint2 *>(to) = make_uint2(y[0], y[1]);
  }
}

// One head of a block of 16 rows, of which [lo, hi) count, as a wave takes it
// (Block): row r's values of head `head` lie at src + r * stride bytes.
template <bool F32, int D>
__device__ inline void load_head(const uint8_t *src, int64_t stride, int head, int lo, int hi,
                                 float (&val)[Block<F32, D>::PER][4][Block<F32, D>::VEC]) {
  using B = Block<F32, D>;
  const int lane = threadIdx.x & 63;
  uint4 raw[B::PER][4];
#pragma unroll
  for (int i = 0; i < B::PER; ++i) {
    const int task = lane + i * kWave, quad = task / B::CHUNKS, piece = task % B::CHUNKS;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int r = 4 * quad + t;
      raw[i][t] = make_uint4(0, 0, 0, 0);
      if (task < B::TASKS && r >= lo && r < hi)
        raw[i][t] = *reinterpret_cast<const uint4 *>(
            src + r * stride + ((int64_t)head * D + piece * B::VEC) * (F32 ? 4 : 2));
    }
  }
#pragma unroll
  for (int i = 0; i < B::PER; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t rw[4] = {raw[i][t].x, raw[i][t].y, raw[i][t].z, raw[i][t].w};
#pragma unroll
      for (int e = 0; e < B::VEC; ++e)
        val[i][t][e] = __uint_as_float(F32 ? rw[e]
                                           : (e & 1) ? rw[e >> 1] & 0xFFFF0000u : rw[e >> 1] << 16);
    }
}

// Norms and turns the values of load_head.
template <bool F32, int D>
__device__ inline void turn_head(TurnLds<D> &lds, const KvRotary &rot, const float *weight,
                                 double eps,
                                 float (&val)[Block<F32, D>::PER][4][Block<F32, D>::VEC]) {
  using B = Block<F32, D>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float w[B::VEC] = {};
  const int piece = lane % B::CHUNKS;  // the same for every i: CHUNKS divides 64
  float *row = lds.rows[wave][lane / B::CHUNKS];
  if (weight) {
#pragma unroll
    for (int e = 0; e < B::VEC; ++e) w[e] = weight[piece * B::VEC + e];
  }
#pragma unroll
  for (int i = 0; i < B::PER; ++i) {
    // (where a head has few pieces, the lanes past its 16 tokens go along on any row of
    // the table: theirs are not stored)
    const int quad = ((lane + i * kWave) / B::CHUNKS) % 4;
#pragma unroll
    for (int t = 0; t < 4; ++t)
      turn_row<D, B::VEC>(lds, row, rot, w, weight != nullptr, eps, 4 * quad + t,
                          piece, val[i][t]);
  }
}

struct RotateArgs {
  const uint8_t *x;
  int64_t x_stride;  // bytes
  const int32_t *positions;
  int64_t rows;
  int heads, per;  // heads of a workgroup
  const float *weight;
  double eps;
  uint8_t *y;
  int64_t y_stride;  // bytes
};

// A workgroup takes `per` heads of 16 rows, a wave one head at a time.
template <bool F32, int D>
__global__ __launch_bounds__(kThreads) void rotate_kernel(KvRotary rot, RotateArgs a, bool y32,
                                                          uint32_t slices) {
  using B = Block<F32, D>;
  __shared__ TurnLds<D> lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slice = blockIdx.x % slices;
  const int64_t row0 = (int64_t)(blockIdx.x / slices) * kKvBlock;
  const int n = (int)(a.rows - row0 < kKvBlock ? a.rows - row0 : kKvBlock);
  const int end = min(a.heads, (slice + 1) * a.per);
  fill_table<D>(lds, rot, 0, n, [&](int r) { return (int64_t)a.positions[row0 + r]; });
  __syncthreads();
  for (int head = slice * a.per + wave; head < end; head += kThreads / 64) {
    float val[B::PER][4][B::VEC];
    load_head<F32, D>(a.x + row0 * a.x_stride, a.x_stride, head, 0, n, val);
    turn_head<F32, D>(lds, rot, a.weight, a.eps, val);
#pragma unroll
    for (int i = 0; i < B::PER; ++i) {
      const int task = lane + i * kWave, quad = task / B::CHUNKS, piece = task % B::CHUNKS;
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (task < B::TASKS && 4 * quad + t < n)
          store_values(a.y + (row0 + 4 * quad + t) * a.y_stride,
                       (int64_t)head * D + piece * B::VEC, y32, val[i][t]);
    }
  }
}

// New tokens: a workgroup takes `per` heads (queries, then keys, then values) of one
// block of 16 positions of a sequence, a wave one head at a time.
template <bool F32, int D>
__global__ __launch_bounds__(kThreads) void append_rotated_kernel(KvCache c, int64_t layer, KvBatch b,
                                                                  KvRotary rot, KvTurned a,
                                                                  uint32_t blocks_per_seq,
                                                                  uint32_t slices, int per) {
  using B = Block<F32, D>;
  __shared__ TurnLds<D> lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t w = blockIdx.x;
  const int slice = w % slices;
  w /= slices;
  const int64_t seq = w / blocks_per_seq;
  int64_t row0;
  int n, len, end;
  b.sequence(seq, row0, n, len, end);
  const int begin = len - n;                // position of row 0, may be negative
  const int first = begin < 0 ? 0 : begin;  // first new token
  const int past = begin + (n < b.max_rows ? n : b.max_rows);  // past the last row's position
  const int last = past < end ? past : end;                    // past the last token with a place
  const int blk = first / kKvBlock + (int)(w % blocks_per_seq);
  const int t0 = blk * kKvBlock;
  const int from = slice * per, to = min(a.heads + 2 * c.kv_heads, from + per);
  if (begin < 0 && w % blocks_per_seq == 0) {
    // rows that are no tokens: zeros
    const int none = min(-begin, min(n, b.max_rows));
    const int heads = min(to, a.heads) - from;
    for (int64_t i = threadIdx.x; heads > 0 && i < (int64_t)none * heads * (D / 8); i += kThreads) {
      const int64_t row = i / (heads * (D / 8)), at = i % (heads * (D / 8));
      reinterpret_cast<uint4 *>(a.q_out + ((row0 + row) * a.heads + from) * D)[at] =
          make_uint4(0, 0, 0, 0);
    }
  }
  if (first >= past || t0 >= past) return;
  int page = -1;
  if (to > a.heads && t0 < last) page = b.table[seq * b.table_stride + (t0 >> c.page_shift)];
  if (page >= c.pages) page = -1;
  const int lo = first > t0 ? first - t0 : 0, hi = past - t0 < kKvBlock ? past - t0 : kKvBlock;
  if (from < a.heads + c.kv_heads) {
    fill_table<D>(lds, rot, lo, hi, [&](int r) { return (int64_t)(t0 + r); });
    __syncthreads();
  }
  const int64_t row = row0 + (t0 - begin);  // of token t0, which may be an earlier sequence's
  for (int task = from + wave; task < to; task += kThreads / 64) {
    const int part = task < a.heads ? 0 : task < a.heads + c.kv_heads ? 1 : 2;
    const int head = part == 0 ? task : part == 1 ? task - a.heads : task - a.heads - c.kv_heads;
    if (part > 0 && (page < 0 || t0 + lo >= last)) break;
    const uint8_t *src = part == 0 ? a.q : part == 1 ? a.k : a.v;
    const int64_t stride = part == 0 ? a.q_stride : part == 1 ? a.k_stride : a.v_stride;
    const int rows = part == 0 ? hi : min(hi, last - t0);
    float val[B::PER][4][B::VEC];
    load_head<F32, D>(src + row * stride, stride, head, lo, rows, val);
    if (part < 2) turn_head<F32, D>(lds, rot, part == 0 ? a.q_weight : a.k_weight, a.eps, val);
    if (part == 0) {
#pragma unroll
      for (int i = 0; i < B::PER; ++i) {
        const int u = lane + i * kWave, quad = u / B::CHUNKS, piece = u % B::CHUNKS;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int r = 4 * quad + t;
          if (u < B::TASKS && r >= lo && r < rows)
            store_values(a.q_out + (row + r) * a.heads * D, (int64_t)head * D + piece * B::VEC, false,
                         val[i][t]);
        }
      }
      continue;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < B::PER; ++i) {
      const int u = lane + i * kWave, quad = u / B::CHUNKS;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int r = 4 * quad + t;
        const bool on = u < B::TASKS && r >= lo && r < rows;
#pragma unroll
        for (int e = 0; e < B::VEC; ++e) {
          const uint32_t mag = __float_as_uint(val[i][t][e]) & 0x7FFFFFFFu;
          if (on && mag < 0x7F800000u && mag > top) top = mag;
        }
      }
    }
    store_block<F32, D>(c, layer, page, head, part - 1, t0, t0 + lo, t0 + rows, val, top);
  }
}

// Heads of a workgroup: one for each wave, as long as that makes no more workgroups
// than the card takes at a time, else three, which share a table.
int heads_each(int64_t blocks, int64_t heads) {
  const int64_t waves = kThreads / 64;
  const int64_t per = blocks * ((heads + waves - 1) / waves) <= 4 * (int64_t)device_cu_count() ? waves : 3 * waves;
  return (int)(per < heads ? per : heads);
}

}  // namespace

hipError_t launch_rotate(const KvRotary &rot, const KvRows &x, const int32_t *positions,
                         int64_t rows, int heads, int head_dim, const float *weight, double eps,
                         const KvRows &y, hipStream_t s) {
  const int64_t blocks = (rows + kKvBlock - 1) / kKvBlock;
  const int per = heads_each(blocks, heads);
  const int64_t slices = (heads + per - 1) / per;
  if (blocks * slices > 0x7FFFFFFF / kThreads) return hipErrorInvalidConfiguration;
  const RotateArgs a{static_cast<const uint8_t *>(x.at), x.stride * (x.f32 ? 4 : 2), positions, rows,
                     heads, per, weight, eps, static_cast<uint8_t *>(y.at),
                     y.stride * (y.f32 ? 4 : 2)};
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks * slices)), dim3(kThreads), 0, s, rot, a, y.f32,
                       (uint32_t)slices);
  };
  if (x.f32) {
    if (head_dim == 128) go(rotate_kernel<true, 128>);
    else go(rotate_kernel<true, 64>);
  } else {
    if (head_dim == 128) go(rotate_kernel<false, 128>);
    else go(rotate_kernel<false, 64>);
  }
  return hipGetLastError();
}

hipError_t launch_kv_append_rotated(const KvCache &c, int64_t layer, const KvBatch &b,
                                    const KvRotary &rot, const KvTurned &a, bool f32,
                                    hipStream_t s) {
  // n consecutive tokens touch at most (n + 30) / 16 blocks
  const int64_t blocks = ((int64_t)b.max_rows + 2 * kKvBlock - 2) / kKvBlock;
  const int heads = a.heads + 2 * c.kv_heads, per = heads_each(b.seqs * blocks, heads);
  const int64_t slices = (heads + per - 1) / per, grid = b.seqs * blocks * slices;
  if (grid > 0x7FFFFFFF / kThreads) return hipErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, c, layer, b, rot, a,
                       (uint32_t)blocks, (uint32_t)slices, per);
  };
  if (f32) {
    if (c.head_dim == 128) go(append_rotated_kernel<true, 128>);
    else go(append_rotated_kernel<true, 64>);
  } else {
    if (c.head_dim == 128) go(append_rotated_kernel<false, 128>);
    else go(append_rotated_kernel<false, 64>);
  }
  return hipGetLastError();
}

}  // namespace nf4
