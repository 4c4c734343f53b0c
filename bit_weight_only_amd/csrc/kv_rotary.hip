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
// 64-bit product, off by the position times what rounding the turns left; its sine and
// cosine are summed in 64 bits, to 2^-37.
//
// What leaves as bf16 is worked out in fp32.  Keys, which go on to be quantized, and
// fp32 results are worked out in 64 bits and rounded once: a code then differs from
// that of the exact key only where an fp32 rounding crosses between two codes (a
// multiply-add in 64 bits costs no more here than one in 32).
//
// vibevoice.c README: the decoder's positions are rotary; the block format and its
// rules are include/nf4.h's.
#include <type_traits>

#include "kv_internal.h"
#include "kv_quant.h"

namespace nf4 {
namespace {

constexpr int kThreads = 256;

// Cosine and sine of u 2^-64 turns, times gain.  With the nearest quarter turn taken
// off, |x| <= pi / 4, and what the Taylor sums leave out is under x^13 / 13! = 7e-12.
// All 64 bits go in: the upper 32 alone are up to 1.5e-9 rad off, which is more than an fp32
// rounding of a result under a fortieth of its pair.
struct Turn {
  double c, s;
};
__device__ inline Turn turned(uint64_t u, double gain) {
  const uint32_t quarter = ((uint32_t)(u >> 32) + 0x20000000u) >> 30;
  const double x = (double)(int64_t)(u - ((uint64_t)quarter << 62)) * (6.283185307179586 * 0x1p-64);
  const double y = x * x;
  double s = fma(y, -1.0 / 39916800, 1.0 / 362880);
  s = fma(y, s, -1.0 / 5040);
  s = fma(y, s, 1.0 / 120);
  s = fma(y, s, -1.0 / 6);
  s = fma(y * x, s, x) * gain;
  double c = fma(y, 1.0 / 479001600, -1.0 / 3628800);
  c = fma(y, c, 1.0 / 40320);
  c = fma(y, c, -1.0 / 720);
  c = fma(y, c, 1.0 / 24);
  c = fma(y, c, -0.5);
  c = fma(y, c, 1.0) * gain;
  const double co = quarter & 1 ? s : c, si = quarter & 1 ? c : s;
  // quarters 1 and 2 have a negative cosine, 2 and 3 a negative sine
  return Turn{(quarter + 1) & 2 ? -co : co, quarter & 2 ? -si : si};
}

// What the workgroup's waves share: what turns the values of 16 tokens, in fp32 and, where
// something is worked out in 64 bits (T double), what that leaves of it, and for each
// wave some rows of heads, where lanes find the other values of their pairs.  In pairs entry
// i holds (cos, sin) of pair i; in halves every value has its own, (cos, -sin) for the
// first one of a pair and (cos, sin) for the second.  Rows are padded by 16 bytes,
// so that neighbouring ones start at other banks.
template <class T, int D>
struct alignas(16) TurnLds {
  static constexpr bool LOW = sizeof(T) == 8;
  float2 cs[kKvBlock][D + 2];
  float2 low[LOW ? kKvBlock : 1][D + 2];
  T rows[kThreads / 64][512 / D][D + D / 8 + 4];  // 64 lanes of up to 8 values
};

// The table for tokens r of 16, lo <= r < hi, at the positions `position(r)`.  A thread
// has one pair in all of its turns.
template <class T, int D, class Lds, class Position>
__device__ inline void fill_table(Lds &lds, const KvRotary &rot, uint64_t turns, int lo, int hi,
                                  Position position) {
  constexpr int PAIRS = D / 2;
  const int p = threadIdx.x % PAIRS;
  if (2 * p >= rot.dims) return;
  for (int r = threadIdx.x / PAIRS; r < hi; r += kThreads / PAIRS) {
    if (r < lo) continue;
    const Turn t = turned((uint64_t)position(r) * turns, rot.gain);
    const float2 cs = make_float2((float)t.c, (float)t.s);
    const float2 low = make_float2((float)(t.c - cs.x), (float)(t.s - cs.y));
    auto set = [&](int at, float sign) {
      lds.cs[r][at] = make_float2(cs.x, sign * cs.y);
      if constexpr (sizeof(T) == 8) lds.low[r][at] = make_float2(low.x, sign * low.y);
    };
    set(p, rot.pairs ? 1.0f : -1.0f);
    if (!rot.pairs) set(p + rot.dims / 2, 1.0f);
  }
}

// Sum over the 8, 16 or 32 neighbouring lanes that hold a row.
template <int CTRL>
__device__ inline float moved(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ inline double moved(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int LANES, class T>
__device__ inline T row_sum(T v) {
  v += moved<0xB1>(v);   // lane ^ 1
  v += moved<0x4E>(v);   // lane ^ 2
  v += moved<0x141>(v);  // 7 - lane of 8
  if (LANES >= 16) v += moved<0x140>(v);  // 15 - lane of 16
  if (LANES == 32) v += __shfl_xor(v, 16);
  return v;
}

// 1 / sqrt(t) for a normal t, infinity (0) and NaN.
__device__ inline float inverse_root(float t) {
  const float y = __builtin_amdgcn_rsqf(t);
  // one step towards the root, for the last bit (not from 1 / infinity)
  return y > 0.0f ? fmaf(0.5f * y, fmaf(-t * y, y, 1.0f), y) : y;
}
__device__ inline double inverse_root(double t) {
  double y = __builtin_amdgcn_rsq(t);  // half of the bits
  if (!(y > 0.0)) return y;
#pragma unroll
  for (int i = 0; i < 2; ++i) y = fma(0.5 * y, fma(-t * y, y, 1.0), y);
  return y;
}

// The norm of a row's values.
template <int D, int VEC>
__device__ inline void norm_row(const float (&w)[VEC], double eps, double (&v)[VEC]) {
  double sum = 0.0;
#pragma unroll
  for (int e = 0; e < VEC; ++e) sum = fma(v[e], v[e], sum);
  const double inv = inverse_root(fma(row_sum<D / VEC>(sum), 1.0 / D, eps));
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] *= inv * w[e];
}
template <int D, int VEC>
__device__ inline void norm_row(const float (&w)[VEC], double eps, float (&v)[VEC]) {
  float sum = 0.0f;
#pragma unroll
  for (int e = 0; e < VEC; ++e) sum = fmaf(v[e], v[e], sum);
  const float mean = fmaf(row_sum<D / VEC>(sum), 1.0f / D, (float)eps);
  const float inv = inverse_root(mean);
  const bool large = !(mean < 0x1p100f);
  if (__any(large)) {  // squares that pass fp32 have to be summed in 64 bits
    double x[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = v[e];
    norm_row<D, VEC>(w, eps, x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = large ? (float)x[e] : v[e] * inv * w[e];
    return;
  }
  // (the value first: inv w passes fp32 for rows of zeros under large weights)
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = v[e] * inv * w[e];
}

// What one lane's value is to the lane that holds the other half of its row, CHUNKS / 2 lanes
// away from it.
template <int CHUNKS>
__device__ inline uint32_t across(uint32_t v) {
  if constexpr (CHUNKS == 8) {  // lane ^ 4: 7 - lane of 8, then 3 - lane of 4
    const int m = __builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true);
    return (uint32_t)__builtin_amdgcn_update_dpp(0, m, 0x1B, 0xF, 0xF, true);
  } else if constexpr (CHUNKS == 16) {  // rotated by 8 in 16
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, true);
  } else {
    // rows of 16 lanes: [0] has the even ones twice, [1] the odd ones
    const auto x = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return threadIdx.x & 16 ? x[0] : x[1];
  }
}
template <int CHUNKS>
__device__ inline float across(float v) {
  return __uint_as_float(across<CHUNKS>(__float_as_uint(v)));
}
template <int CHUNKS>
__device__ inline double across(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)across<CHUNKS>((uint32_t)(u >> 32)) << 32 |
                                        across<CHUNKS>((uint32_t)u));
}

// A value turned, by what the table holds for it and the other value of its pair.
__device__ inline float turn(float x, float other, float2 cs, float2) {
  return fmaf(x, cs.x, other * cs.y);
}
__device__ inline double turn(double x, double other, float2 cs, float2 low) {
  return fma(x, (double)cs.x + low.x, other * ((double)cs.y + low.y));
}

// N values at p, which is aligned to `ALIGN` bytes.
template <int ALIGN, class T, int N>
__device__ inline void load_n(T (&x)[N], const T *p) {
  __builtin_memcpy(x, __builtin_assume_aligned(p, ALIGN), sizeof(x));
}

// What a wave's lanes have written to LDS before this, any of them reads after it.
__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Where in a wave's row of LDS a lane finds the other values of its pairs, where these start
// anywhere (an odd number of pairs, or one that pieces end inside of): a place is left
// free after every eight values, so that lanes find theirs in different banks.  For eight values
// (bf16) the places are byte offsets, two in a register: worked out for every row they are a
// fifth of its instructions (the append of 5 times 701 rows, 32 heads over 8 of 64: 16.7 us,
// kept 14.9).  For four (fp32) they are worked out there, since the kernel has no registers left
// to keep them (14449 rows of 28 heads over 4 78.3 us, kept 90.5).
template <class T, int VEC>
struct Others {
  static constexpr bool KEPT = VEC == 8;
  uint32_t at[KEPT ? VEC / 2 : 1];
  __device__ static int place(int value) { return value + value / 8; }
  __device__ static int other(const KvRotary &rot, int v) {
    const int half = rot.dims / 2;
    return place(v >= rot.dims ? v : v < half ? v + half : v - half);
  }
  // Whether a lane's values have theirs at places of their own.
  __device__ static bool apart(const KvRotary &rot) { return rot.dims / 2 % VEC != 0; }
  __device__ Others(const KvRotary &rot, int piece) {
    if (!KEPT || rot.pairs || !apart(rot)) return;
#pragma unroll
    for (int e = 0; e < VEC; e += 2)
      at[KEPT ? e / 2 : 0] = (uint32_t)(other(rot, piece * VEC + e) * sizeof(T)) |
                             (uint32_t)(other(rot, piece * VEC + e + 1) * sizeof(T)) << 16;
  }
  // Through the row: x the lane's values, from value `first` on, y the others.
  __device__ void exchange(const KvRotary &rot, T *row, int first, const T (&x)[VEC], T (&y)[VEC]) const {
    // (the compiler is not to keep places from row to row: registers)
    if (!KEPT) asm volatile("" : "+v"(first));
#pragma unroll
    for (int e = 0; e < VEC; ++e) row[place(first) + e] = x[e];
    wave_sync();
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      if constexpr (KEPT) {
        uint32_t both = at[e / 2];
        asm volatile("" : "+v"(both));
        const uint8_t *bytes = reinterpret_cast<const uint8_t *>(row);
        y[e] = *reinterpret_cast<const T *>(bytes + (both & 0xFFFFu));
        y[e + 1] = *reinterpret_cast<const T *>(bytes + (both >> 16));
      } else {
        y[e] = row[other(rot, first + e)];
        y[e + 1] = row[other(rot, first + e + 1)];
      }
    }
  }
};

// Norms (weight w) and turns one token's values of one row: `v` are the lane's, from
// value VEC * piece on; `r` the token's row of the table; `row` the row in LDS for this
// lane's token.  All lanes of the wave come here together.
template <class T, int D, int VEC, class Lds>
__device__ inline void turn_row(const Lds &lds, T *row, const KvRotary &rot,
                                const Others<T, VEC> &others, const float (&w)[VEC], bool norm,
                                double eps, int r, int piece, float (&v)[VEC]) {
  constexpr bool LOW = sizeof(T) == 8;
  T x[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) x[e] = v[e];
  if (norm) norm_row<D, VEC>(w, eps, x);
  const int e0 = piece * VEC;
  if (rot.dims > 0 && rot.pairs) {
    float2 cs[VEC / 2], low[VEC / 2] = {};
    load_n<16>(cs, &lds.cs[r][piece * (VEC / 2)]);
    if (LOW) load_n<16>(low, &lds.low[LOW ? r : 0][piece * (VEC / 2)]);
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      const T a = x[2 * j], b = x[2 * j + 1];
      const bool on = e0 + 2 * j < rot.dims;
      x[2 * j] = on ? turn(a, b, make_float2(cs[j].x, -cs[j].y), make_float2(low[j].x, -low[j].y)) : a;
      x[2 * j + 1] = on ? turn(b, a, cs[j], low[j]) : b;
    }
  } else if (rot.dims > 0) {
    const int half = rot.dims / 2;
    T other[VEC];
    if (rot.dims == D) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) other[e] = across<D / VEC>(x[e]);
    } else {
      if (!others.apart(rot)) {  // the other values of a lane's pairs are one piece
        __builtin_memcpy(__builtin_assume_aligned(row + e0, 16), x, sizeof(x));
        wave_sync();
        load_n<16>(other, row + (e0 >= rot.dims ? e0 : e0 < half ? e0 + half : e0 - half));
      } else {
        others.exchange(rot, row, e0, x, other);  // one at a time
      }
      wave_sync();
    }
#pragma unroll
    for (int c = 0; c < VEC; c += 4) {
      float2 cs[4], low[4] = {};
      load_n<16>(cs, &lds.cs[r][e0 + c]);
      if (LOW) load_n<16>(low, &lds.low[LOW ? r : 0][e0 + c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const T y = turn(x[c + e], other[c + e], cs[e], low[e]);
        x[c + e] = e0 + c + e < rot.dims ? y : x[c + e];
      }
      if (LOW) __builtin_amdgcn_sched_barrier(0);  // registers
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = (float)x[e];
}

__device__ inline uint32_t bf16_bits(float x) {
  return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// VEC values to `to`, as fp32 or bf16.
template <bool F32, int VEC>
__device__ inline void store_values(uint8_t *to, const float (&v)[VEC]) {
  if (F32) {
#pragma unroll
    for (int h = 0; h < VEC / 4; ++h)
      reinterpret_cast<float4 *>(to)[h] = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
    return;
  }
  uint32_t y[VEC / 2];
#pragma unroll
  for (int h = 0; h < VEC / 2; ++h) y[h] = bf16_bits(v[2 * h]) | bf16_bits(v[2 * h + 1]) << 16;
  if (VEC == 8) *reinterpret_cast<uint4 *>(to) = make_uint4(y[0], y[1], y[VEC / 2 - 2], y[VEC / 2 - 1]);
  else *reinterpret_cast<uint2 *>(to) = make_uint2(y[0], y[1]);
}

// How a wave takes 16 rows of its heads: as Block, and where one head leaves lanes over
// (64 values of bf16), as many more heads as they have room for.  Sixteen rows are less
// than 2^31 bytes apart (kKvWidestRows).
template <bool F32, int D>
struct Heads : Block<F32, D> {
  using B = Block<F32, D>;
  static constexpr int SUB = B::TASKS < 64 ? 64 / B::TASKS : 1;
  static constexpr int LANES = 64 / SUB;  // of a head
  uint4 raw[B::PER][4];

  __device__ static int sub() { return (threadIdx.x & 63) / LANES; }
  __device__ static int quad(int i) { return ((threadIdx.x & (LANES - 1)) + i * kWave) / B::CHUNKS; }
  __device__ static int piece() { return threadIdx.x % B::CHUNKS; }

  // Loads rows lo .. hi - 1 of head `head` (< 0: none): row r's heads lie at src + r * stride bytes.
  __device__ void load(const uint8_t *src, uint32_t stride, int head, int lo, int hi) {
    const uint32_t at = ((uint32_t)head * D + piece() * B::VEC) * (F32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < B::PER; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int r = 4 * quad(i) + t;
        raw[i][t] = make_uint4(0, 0, 0, 0);
        if (head >= 0 && r >= lo && r < hi)
          raw[i][t] = *reinterpret_cast<const uint4 *>(src + (uint32_t)(r * stride + at));
      }
  }
  // One row's values of the lane.
  __device__ void values(int i, int t, float (&val)[B::VEC]) const {
    const uint32_t rw[4] = {raw[i][t].x, raw[i][t].y, raw[i][t].z, raw[i][t].w};
#pragma unroll
    for (int e = 0; e < B::VEC; ++e)
      val[e] = __uint_as_float(F32 ? rw[e] : (e & 1) ? rw[e >> 1] & 0xFFFF0000u : rw[e >> 1] << 16);
  }
  // A lane's part of the norms' weights.
  __device__ static void weights(const float *weight, float (&w)[B::VEC]) {
#pragma unroll
    for (int e = 0; e < B::VEC; ++e) w[e] = 0.0f;
    if (weight) load_n<16>(w, weight + piece() * B::VEC);
  }
  template <class T, class Lds>
  __device__ static void turn(Lds &lds, const KvRotary &rot, const Others<T, B::VEC> &others,
                              const float (&w)[B::VEC], bool norm, double eps, int i, int t,
                              float (&val)[B::VEC]) {
    T *row = lds.rows[threadIdx.x >> 6][(threadIdx.x & 63) / B::CHUNKS];
    turn_row<T, D, B::VEC>(lds, row, rot, others, w, norm, eps, 4 * quad(i) + t, piece(), val);
    __builtin_amdgcn_sched_barrier(0);  // one at a time: registers
  }
  // All rows turned and stored, T what they are worked out in: row r's lie at dst + r *
  // stride bytes.
  template <class T, bool Y32, class Lds>
  __device__ void turn_and_store(Lds &lds, const KvRotary &rot, const Others<T, B::VEC> &others,
                                 const float (&w)[B::VEC], bool norm, double eps, uint8_t *dst,
                                 uint32_t stride, int head, int lo, int hi) const {
    const uint32_t at = ((uint32_t)head * D + piece() * B::VEC) * (Y32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < B::PER; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int r = 4 * quad(i) + t;
        const bool mine = head >= 0 && r >= lo && r < hi;
        if (!__any(mine)) continue;
        float val[B::VEC];
        values(i, t, val);
        turn<T>(lds, rot, others, w, norm, eps, i, t, val);
        if (mine) store_values<Y32>(dst + (uint32_t)(r * stride + at), val);
      }
  }
};

struct RotateArgs {
  const uint8_t *x;
  const int32_t *positions;
  int64_t rows, x_stride, y_stride;  // bytes
  int heads, per;                    // heads, and those of a workgroup
  const float *weight;
  double eps;
  uint8_t *y;
};

// A workgroup takes `per` heads of 16 rows, a wave SUB heads at a time, the next ones'
// values on their way while these are worked on.  The 16 rows' sines and cosines are
// worked out once for all of the workgroup's heads, some 40 instructions of 64 bits each: by
// every head for itself they would take longer than the rows' way through memory.
// Memory bound, other rows in every call: 14449 rows of 32 heads of 128, normed, bf16 to bf16
// (237 MB) 45.4 us = 5.2 TB/s, the rate of a large copy; bf16 to fp32 and back (355 MB)
// 76 us = 4.7; fp32 to fp32 (473 MB) 103 us = 4.6, 0.9 of that rate: where fp32 leaves, 52 KB of
// LDS keep it to three workgroups per compute unit.  One row of 28 heads: 3.7 us in a trace, 1.6
// of them an empty launch.
template <bool F32, bool Y32, int D>
__global__ __launch_bounds__(kThreads) void rotate_kernel(KvRotary rot, RotateArgs a,
                                                          uint32_t slices) {
  using H = Heads<F32, D>;
  using T = std::conditional_t<Y32, double, float>;
  __shared__ TurnLds<T, D> lds;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t turns = rot.turns[threadIdx.x % (D / 2)];
  const int slice = blockIdx.x % slices;
  const int64_t row0 = (int64_t)(blockIdx.x / slices) * kKvBlock;
  const int n = (int)(a.rows - row0 < kKvBlock ? a.rows - row0 : kKvBlock);
  const int end = min(a.heads, (slice + 1) * a.per);
  const uint8_t *src = a.x + row0 * a.x_stride;
  uint8_t *dst = a.y + row0 * a.y_stride;
  constexpr int STEP = kThreads / 64 * H::SUB;
  int first = slice * a.per + wave * H::SUB;
  auto head = [&](int first) { return first + H::sub() < end ? first + H::sub() : -1; };
  float w[H::VEC];
  H::weights(a.weight, w);
  const Others<T, H::VEC> others(rot, H::piece());
  H now, next;
  now.load(src, (uint32_t)a.x_stride, head(first), 0, n);
  fill_table<T, D>(lds, rot, turns, 0, n, [&](int r) { return (int64_t)a.positions[row0 + r]; });
  __syncthreads();
  for (; first < end; first += STEP) {
    next.load(src, (uint32_t)a.x_stride, head(first + STEP), 0, n);
    now.template turn_and_store<T, Y32>(lds, rot, others, w, a.weight != nullptr, a.eps, dst,
                                        (uint32_t)a.y_stride, head(first), 0, n);
    now = next;
  }
}

// What append_rotated_kernel is called with.  Its two ways read them where they begin, not
// at the kernel's start, as it would by itself: all together pass the scalar registers.
struct AppendArgs {
  uint32_t blocks_per_seq;
  int q_slices, q_per, kv_slices, kv_per;  // workgroups of a block, units of each
  KvBatch b;
  KvTurned a;
  KvCache c;
  int64_t layer;
  KvRotary rot;
};

// The rows of a workgroup: those of a sequence at the 16 positions of a block.
struct NewRows {
  int64_t row;      // of the block's first position, which may be an earlier sequence's
  int t0, lo, hi;   // the block's first position; rows lo .. hi - 1 of the block are new
  int kv_hi;        // those up to here have a place in the table
  int none;         // rows that are no tokens, from row0 on, where the block is the first
  int64_t row0;
  __device__ NewRows(const KvBatch &b, int64_t seq, uint32_t block) {
    int n, len, end;
    b.sequence(seq, row0, n, len, end);
    const int begin = len - n;                // position of row 0, may be negative
    const int first = begin < 0 ? 0 : begin;  // first new token
    const int rows = n < b.max_rows ? n : b.max_rows;
    const int past = begin + rows;            // past the last row's position
    t0 = (first / kKvBlock + (int)block) * kKvBlock;
    row = row0 + (t0 - begin);
    lo = first > t0 ? first - t0 : 0;
    hi = past - t0 < kKvBlock ? past - t0 : kKvBlock;
    kv_hi = min(hi, min(past, end) - t0);
    none = begin < 0 && block == 0 ? min(-begin, rows) : 0;
  }
};

// Queries: a workgroup takes `q_per` units of one block, a wave one at a time, the next one's
// values on their way.  A unit is SUB heads.
template <bool F32, int D>
__device__ inline void append_queries(const AppendArgs &x, int64_t seq, uint32_t block, int slice,
                                      TurnLds<float, D> &lds) {
  using H = Heads<F32, D>;
  constexpr int WAVES = kThreads / 64;
  const KvTurned a = x.a;  // all at once
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), heads = a.heads;
  const uint64_t turns = x.rot.turns[threadIdx.x % (D / 2)];
  const NewRows r(x.b, seq, block);
  int first = (slice * x.q_per + wave) * H::SUB;
  const int end = min(heads, (slice + 1) * x.q_per * H::SUB);
  if (r.none > 0) {  // zeros
    const int h0 = slice * x.q_per * H::SUB, pieces = (end - h0) * (D / 8);
    for (int64_t i = threadIdx.x; pieces > 0 && i < (int64_t)r.none * pieces; i += kThreads)
      reinterpret_cast<uint4 *>(a.q_out + ((r.row0 + i / pieces) * heads + h0) * D)[i % pieces] =
          make_uint4(0, 0, 0, 0);
  }
  if (r.lo >= r.hi) return;
  const uint8_t *src = a.q + r.row * a.q_stride;
  uint8_t *dst = reinterpret_cast<uint8_t *>(a.q_out + r.row * heads * D);
  auto head = [&](int first) { return first + H::sub() < end ? first + H::sub() : -1; };
  float w[H::VEC];
  H::weights(a.q_weight, w);
  const Others<float, H::VEC> others(x.rot, H::piece());
  H now, next;
  now.load(src, (uint32_t)a.q_stride, head(first), r.lo, r.hi);
  fill_table<float, D>(lds, x.rot, turns, r.lo, r.hi, [&](int i) { return (int64_t)(r.t0 + i); });
  __syncthreads();
  for (; first < end; first += WAVES * H::SUB) {
    next.load(src, (uint32_t)a.q_stride, head(first + WAVES * H::SUB), r.lo, r.hi);
    now.template turn_and_store<float, false>(lds, x.rot, others, w, a.q_weight != nullptr, a.eps, dst,
                                              (uint32_t)(heads * D * 2), head(first), r.lo, r.hi);
    now = next;
  }
}

// Keys, then values: units as above.  What a block that is new in part held before is read
// beside the new values.
template <bool F32, int D>
__device__ inline void append_block(const AppendArgs &x, int64_t seq, uint32_t block, int slice,
                                    TurnLds<double, D> &lds) {
  using H = Heads<F32, D>;
  constexpr int SUB = H::SUB, WAVES = kThreads / 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const KvTurned a = x.a;  // all at once
  const KvCache c = x.c;
  const uint64_t turns = x.rot.turns[threadIdx.x % (D / 2)];
  const NewRows r(x.b, seq, block);
  if (r.lo >= r.kv_hi) return;  // no place
  const int page = x.b.table[seq * x.b.table_stride + (r.t0 >> c.page_shift)];
  const int units = (c.kv_heads + SUB - 1) / SUB, end = min(2 * units, (slice + 1) * x.kv_per);
  int unit = slice * x.kv_per + wave;
  const bool turned = slice * x.kv_per < units;
  const Others<double, H::VEC> others(x.rot, H::piece());
  H now;
  auto load = [&] {
    const int value = unit >= units, h = (unit - (value ? units : 0)) * SUB + H::sub();
    const int64_t stride = value ? a.v_stride : a.k_stride;
    now.load((value ? a.v : a.k) + r.row * stride, (uint32_t)stride,
             unit < end && h < c.kv_heads ? h : -1, r.lo, r.kv_hi);
  };
  load();
  if (turned) {
    fill_table<double, D>(lds, x.rot, turns, r.lo, r.kv_hi, [&](int i) { return (int64_t)(r.t0 + i); });
    __syncthreads();
  }
  if (page < 0 || page >= c.pages) return;
  for (; unit < end; unit += WAVES) {
    const int value = unit >= units, at = (unit - (value ? units : 0)) * SUB + H::sub();
    const int h = at < c.kv_heads ? at : -1;
    const OldBlock<F32, D, SUB> was(c, x.layer, page, h, value, r.t0, r.t0 + r.lo, r.t0 + r.kv_hi);
    float w[H::VEC], val[H::PER][4][H::VEC];
    const bool norm = a.k_weight != nullptr;
    H::weights(value ? nullptr : a.k_weight, w);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < H::PER; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = 4 * H::quad(i) + t;
        const bool mine = row >= r.lo && row < r.kv_hi;
        now.values(i, t, val[i][t]);
        if (!__any(mine)) continue;
        if (!value) H::template turn<double>(lds, x.rot, others, w, norm, a.eps, i, t, val[i][t]);
#pragma unroll
        for (int e = 0; e < H::VEC; ++e) {
          const uint32_t mag = __float_as_uint(val[i][t][e]) & 0x7FFFFFFFu;
          if (mine && mag < 0x7F800000u && mag > top) top = mag;
        }
      }
    store_block<F32, D>(was, h, value, r.t0, r.t0 + r.lo, r.t0 + r.kv_hi, val, top);
    if (unit + WAVES < end) {
      unit += WAVES;
      load();
      unit -= WAVES;
    }
  }
}

// New rows of queries, keys and values: each block of 16 positions of a sequence by
// q_slices workgroups that turn queries and kv_slices that turn keys and write keys and
// values into their page.  One launch, so that a decoded token waits for one chain of trips
// to memory (place and length, then rows beside the page id, then the old scale beside
// the old codes): 5.8 us in a trace for one token of 28 heads over 4, 7.1 for 64 of 32 over
// 8, an empty launch 1.6.  Long prompts are memory bound: 14449 fp32 rows of 28 heads over 4 of
// 128 (385 MB) 78.3 us back to back = 4.9 TB/s (83.4 alone in a trace).  In between the vector
// unit takes part, and LDS, where lanes read the sines' table 64 bytes apart in halves of
// bf16 (32 in pairs): 5 chunks of up to 701 rows, 32 heads over 8 of 64, normed, 50 values
// turned (40 MB) 14.8 us back to back, of which some 4 go if nothing turns; conflicts of
// LDS banks are 6500 cycles of a compute unit, up to 2.7 us.
// Every sequence has as many workgroups as the longest chunk: 63 single tokens beside a chunk
// of 1024 rows, 28 fp32 heads over 4, 33.6 us in a graph, beside one of 113 14.7.
template <bool F32, int D>
__global__ __launch_bounds__(kThreads) void append_rotated_kernel(AppendArgs) {
  __shared__ union {
    TurnLds<float, D> queries;
    TurnLds<double, D> keys;
  } lds;
  const AppendArgs *args = (const AppendArgs *)__builtin_amdgcn_kernarg_segment_ptr();
  const uint32_t slices = args->q_slices + args->kv_slices, blocks = args->blocks_per_seq;
  const int slice = blockIdx.x % slices;
  const uint32_t w = blockIdx.x / slices;
  if (slice < args->q_slices) {
    asm volatile("; queries");
    append_queries<F32, D>(*args, w / blocks, w % blocks, slice, lds.queries);
  } else {
    asm volatile("; keys and values");
    append_block<F32, D>(*args, w / blocks, w % blocks, slice - args->q_slices, lds.keys);
  }
}

// Units of a workgroup: one for each wave, as long as that makes no more workgroups
// than the card takes at a time, else two, which share a table.  In replayed graphs of one
// call: 14449 rows of 32 heads one 56.9 us, two 50.2, three 51.8; 300 rows one 17.5, two
// 17.6, three 19.2; an append of 5 times 701 rows, 32 heads over 8, one 27.2, two 22.3, three
// 22.1.
int units_each(int64_t blocks, int64_t units) {
  const int64_t waves = kThreads / 64;
  const int64_t per = blocks * ((units + waves - 1) / waves) <= 4 * (int64_t)device_cu_count() ? waves : 2 * waves;
  return (int)(per < units ? per : units);
}

template <bool F32>
int sub_of(int head_dim) {
  return head_dim == 128 ? Heads<F32, 128>::SUB : Heads<F32, 64>::SUB;
}

}  // namespace

hipError_t launch_rotate(const KvRotary &rot, const KvRows &x, const int32_t *positions,
                         int64_t rows, int heads, int head_dim, const float *weight, double eps,
                         const KvRows &y, hipStream_t s) {
  const int64_t blocks = (rows + kKvBlock - 1) / kKvBlock;
  const int sub = x.f32 ? sub_of<true>(head_dim) : sub_of<false>(head_dim);
  const int per = units_each(blocks, (heads + sub - 1) / sub) * sub;
  const int64_t slices = (heads + per - 1) / per;
  if (blocks * slices > 0x7FFFFFFF / kThreads) return hipErrorInvalidConfiguration;
  const RotateArgs a{static_cast<const uint8_t *>(x.at), positions, rows, x.stride * (x.f32 ? 4 : 2),
                     y.stride * (y.f32 ? 4 : 2), heads, per, weight, eps, static_cast<uint8_t *>(y.at)};
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks * slices)), dim3(kThreads), 0, s, rot, a,
                       (uint32_t)slices);
  };
  auto pick = [&](auto f32, auto y32) {
    constexpr bool F32 = decltype(f32)::value, Y32 = decltype(y32)::value;
    if (head_dim == 128) go(rotate_kernel<F32, Y32, 128>);
    else go(rotate_kernel<F32, Y32, 64>);
  };
  if (x.f32 && y.f32) pick(std::true_type(), std::true_type());
  else if (x.f32) pick(std::true_type(), std::false_type());
  else if (y.f32) pick(std::false_type(), std::true_type());
  else pick(std::false_type(), std::false_type());
  return hipGetLastError();
}

hipError_t launch_kv_append_rotated(const KvCache &c, int64_t layer, const KvBatch &b,
                                    const KvRotary &rot, const KvTurned &a, bool f32,
                                    hipStream_t s) {
  // n consecutive tokens touch at most (n + 30) / 16 blocks
  const int64_t blocks = ((int64_t)b.max_rows + 2 * kKvBlock - 2) / kKvBlock;
  const int sub = f32 ? sub_of<true>(c.head_dim) : sub_of<false>(c.head_dim);
  const int q_units = (a.heads + sub - 1) / sub, kv_units = 2 * ((c.kv_heads + sub - 1) / sub);
  const int per = units_each(b.seqs * blocks, q_units + kv_units);
  const int q_slices = (q_units + per - 1) / per, kv_slices = (kv_units + per - 1) / per;
  const int q_per = (q_units + q_slices - 1) / q_slices, kv_per = (kv_units + kv_slices - 1) / kv_slices;
  const int64_t grid = b.seqs * blocks * (q_slices + kv_slices);
  if (grid > 0x7FFFFFFF / kThreads) return hipErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(kThreads), 0, s,
                       AppendArgs{(uint32_t)blocks, q_slices, q_per, kv_slices, kv_per, b, a, c, layer, rot});
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
