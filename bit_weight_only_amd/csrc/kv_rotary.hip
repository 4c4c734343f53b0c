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
// cosine are summed in 64 bits.
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

// Cosine and sine of u 2^-32 turns, times gain.  With the nearest quarter turn taken
// off, |x| <= pi / 4, and what the Taylor sums leave out is under x^13 / 13! = 7e-12.
struct Turn {
  double c, s;
};
__device__ inline Turn turned(uint32_t u, double gain) {
  const uint32_t quarter = (u + 0x20000000u) >> 30;
  const double x = (double)(int)(u - (quarter << 30)) * (6.283185307179586 / 4294967296.0);
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

// What the workgroup's waves share: cosines and sines of 16 tokens, (cos, sin) in fp32
// and, where something is worked out in 64 bits (T double), what that leaves of them, and
// for each wave some rows of heads, where lanes find the other values of their pairs.
// Rows are padded by 16 bytes, so that neighbouring ones start at other banks.
template <class T, int D>
struct alignas(16) TurnLds {
  static constexpr bool LOW = sizeof(T) == 8;
  float2 cs[kKvBlock][D / 2 + 2];
  float2 low[LOW ? kKvBlock : 1][D / 2 + 2];
  // 64 lanes of up to 8 values, and what a read of a last row may pass it by
  T rows[kThreads / 64][512 / D * (D + 16 / sizeof(T)) + 8];
};
// Values of a row in LDS.
template <class T, int D>
constexpr int kRow = D + 16 / (int)sizeof(T);

// The table for tokens r of 16, lo <= r < hi, at the positions `position(r)`.  A thread
// has one pair in all of its turns.
template <class T, int D, class Position>
__device__ inline void fill_table(TurnLds<T, D> &lds, const KvRotary &rot, uint64_t turns, int lo,
                                  int hi, Position position) {
  constexpr int PAIRS = D / 2;
  const int p = threadIdx.x % PAIRS;
  if (2 * p >= rot.dims) return;
  for (int r = threadIdx.x / PAIRS; r < hi; r += kThreads / PAIRS) {
    if (r < lo) continue;
    const Turn t = turned((uint32_t)(((uint64_t)position(r) * turns) >> 32), rot.gain);
    const float2 cs = make_float2((float)t.c, (float)t.s);
    lds.cs[r][p] = cs;
    if constexpr (TurnLds<T, D>::LOW)
      lds.low[r][p] = make_float2((float)(t.c - cs.x), (float)(t.s - cs.y));
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
  if (__any(!(mean < 0x1p100f))) {  // squares that pass fp32 have to be summed in 64 bits
    double x[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = v[e];
    norm_row<D, VEC>(w, eps, x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = (float)x[e];
    return;
  }
  const float inv = inverse_root(mean);
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] *= inv * w[e];
}

__device__ inline float turn_a(float a, float b, float2 cs, float2) { return fmaf(a, cs.x, -(b * cs.y)); }
__device__ inline float turn_b(float a, float b, float2 cs, float2) { return fmaf(b, cs.x, a * cs.y); }
__device__ inline double turn_a(double a, double b, float2 cs, float2 low) {
  return fma(a, (double)cs.x + low.x, -(b * ((double)cs.y + low.y)));
}
__device__ inline double turn_b(double a, double b, float2 cs, float2 low) {
  return fma(b, (double)cs.x + low.x, a * ((double)cs.y + low.y));
}

// N values at p, which is aligned to `ALIGN` bytes.
template <int ALIGN, class T, int N>
__device__ inline void load_n(T (&x)[N], const T *p) {
  __builtin_memcpy(x, __builtin_assume_aligned(p, ALIGN), sizeof(x));
}

// Norms (weight w) and turns one token's values of one row: `v` are the lane's, from
// value VEC * piece on; `r` the token's row of the table; `row` the row in LDS for this
// lane's token.  All lanes of the wave come here together.
template <class T, int D, int VEC, class Lds>
__device__ inline void turn_row(const Lds &lds, T *row, const KvRotary &rot,
                                const float (&w)[VEC], bool norm, double eps, int r, int piece,
                                float (&v)[VEC]) {
  constexpr bool LOW = sizeof(T) == 8;
  T x[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) x[e] = v[e];
  if (norm) norm_row<D, VEC>(w, eps, x);
  const int e0 = piece * VEC;
  if (rot.dims > 0 && rot.pairs) {
    float2 cs[VEC / 2], low[VEC / 2] = {};
    load_n<VEC * 4 < 16 ? 8 : 16>(cs, &lds.cs[r][piece * (VEC / 2)]);
    if (LOW) load_n<VEC * 4 < 16 ? 8 : 16>(low, &lds.low[LOW ? r : 0][piece * (VEC / 2)]);
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      const T a = x[2 * j], b = x[2 * j + 1];
      const bool on = e0 + 2 * j < rot.dims;
      x[2 * j] = on ? turn_a(a, b, cs[j], low[j]) : a;
      x[2 * j + 1] = on ? turn_b(a, b, cs[j], low[j]) : b;
    }
  } else if (rot.dims > 0) {
    const int half = rot.dims / 2;
    __builtin_memcpy(__builtin_assume_aligned(row + e0, 16), x, sizeof(x));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    T other[VEC];
    float2 cs[VEC], low[VEC] = {};
    if (half % VEC == 0) {  // the other values of a lane's pairs are one piece
      const bool on = e0 < rot.dims, first = e0 < half;
      const int p = first || !on ? e0 % (D / 2) : e0 - half;
      load_n<16>(other, row + (!on ? e0 : first ? e0 + half : e0 - half));
      load_n<16>(cs, &lds.cs[r][p]);
      if (LOW) load_n<16>(low, &lds.low[LOW ? r : 0][p]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const T y = first ? turn_a(x[e], other[e], cs[e], low[e]) : turn_b(other[e], x[e], cs[e], low[e]);
        x[e] = on ? y : x[e];
      }
    } else {
      // they start anywhere, and a lane may have first and second values of pairs: it reads
      // the others of both kinds (of a kind that it has none of, anything of the row)
      const int up = min(e0 + half, D - 1), down = e0 + VEC > half ? e0 - half : 0;
      T below[VEC];
      load_n<sizeof(T)>(other, row + up);
      load_n<sizeof(T)>(below, row + down);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int at = e0 + e;
        const bool on = at < rot.dims, first = at < half;
        const int p = !on ? 0 : first ? at : at - half;
        const float2 t = lds.cs[r][p], l = LOW ? lds.low[LOW ? r : 0][p] : float2{};
        const T y = first ? turn_a(x[e], other[e], t, l) : turn_b(below[e], x[e], t, l);
        x[e] = on ? y : x[e];
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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
  __device__ static void turn(Lds &lds, const KvRotary &rot, const float (&w)[B::VEC], bool norm,
                              double eps, int i, int t, float (&val)[B::VEC]) {
    T *row = reinterpret_cast<T *>(lds.rows[threadIdx.x >> 6]) + (threadIdx.x & 63) / B::CHUNKS * kRow<T, D>;
    turn_row<T, D, B::VEC>(lds, row, rot, w, norm, eps, 4 * quad(i) + t, piece(), val);
    __builtin_amdgcn_sched_barrier(0);  // one at a time: registers
  }
  // All rows turned and stored, T what they are worked out in: row r's lie at dst + r *
  // stride bytes.
  template <class T, bool Y32, class Lds>
  __device__ void turn_and_store(Lds &lds, const KvRotary &rot, const float (&w)[B::VEC], bool norm,
                                 double eps, uint8_t *dst, uint32_t stride, int head, int lo,
                                 int hi) const {
    const uint32_t at = ((uint32_t)head * D + piece() * B::VEC) * (Y32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < B::PER; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int r = 4 * quad(i) + t;
        float val[B::VEC];
        values(i, t, val);
        turn<T>(lds, rot, w, norm, eps, i, t, val);
        if (head >= 0 && r >= lo && r < hi) store_values<Y32>(dst + (uint32_t)(r * stride + at), val);
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
// values on their way while these are worked on.
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
  H now, next;
  now.load(src, (uint32_t)a.x_stride, head(first), 0, n);
  fill_table<T, D>(lds, rot, turns, 0, n, [&](int r) { return (int64_t)a.positions[row0 + r]; });
  __syncthreads();
  for (; first < end; first += STEP) {
    next.load(src, (uint32_t)a.x_stride, head(first + STEP), 0, n);
    now.template turn_and_store<T, Y32>(lds, rot, w, a.weight != nullptr, a.eps, dst,
                                        (uint32_t)a.y_stride, head(first), 0, n);
    now = next;
  }
}

// What append_rotated_kernel is called with.  It reads them where it wants them, not at its
// start, as it would by itself: all together pass the scalar registers.
struct AppendArgs {
  KvCache c;
  int64_t layer;
  KvBatch b;
  KvRotary rot;
  KvTurned a;
  uint32_t blocks_per_seq, slices;
  int per;
};

// New tokens: a workgroup takes `per` units of one block of 16 positions of a sequence, a
// wave one at a time.  A unit is SUB heads of queries, keys or values, in this order.
template <bool F32, int D>
__global__ __launch_bounds__(kThreads) void append_rotated_kernel(AppendArgs) {
  using H = Heads<F32, D>;
  constexpr int SUB = H::SUB, WAVES = kThreads / 64;
  __shared__ TurnLds<double, D> lds;
  const AppendArgs *args = (const AppendArgs *)__builtin_amdgcn_kernarg_segment_ptr();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t turns = args->rot.turns[threadIdx.x % (D / 2)];
  const uint32_t slices = args->slices, blocks_per_seq = args->blocks_per_seq;
  uint32_t w = blockIdx.x;
  const int slice = w % slices;
  w /= slices;
  const int64_t seq = w / blocks_per_seq;
  int64_t row0;
  int n, len, end;
  const int max_rows = args->b.max_rows, heads = args->a.heads, kv_heads = args->c.kv_heads;
  args->b.sequence(seq, row0, n, len, end);
  const int begin = len - n;                // position of row 0, may be negative
  const int first = begin < 0 ? 0 : begin;  // first new token
  const int past = begin + (n < max_rows ? n : max_rows);  // past the last row's position
  const int last = past < end ? past : end;                // past the last token with a place
  const int blk = first / kKvBlock + (int)(w % blocks_per_seq);
  const int t0 = blk * kKvBlock;
  const int q_units = (heads + SUB - 1) / SUB, kv_units = (kv_heads + SUB - 1) / SUB;
  const int from = slice * args->per, to = min(q_units + 2 * kv_units, from + args->per);
  const int q_to = min(to, q_units);
  if (begin < 0 && w % blocks_per_seq == 0) {
    // rows that are no tokens: zeros
    const int none = min(-begin, min(n, max_rows));
    const int h0 = from * SUB, pieces = (min(to * SUB, heads) - h0) * (D / 8);
    for (int64_t i = threadIdx.x; pieces > 0 && i < (int64_t)none * pieces; i += kThreads)
      reinterpret_cast<uint4 *>(args->a.q_out + ((row0 + i / pieces) * heads + h0) * D)[i % pieces] =
          make_uint4(0, 0, 0, 0);
  }
  if (first >= past || t0 >= past) return;
  int page = -1;
  if (to > q_units && t0 < last)
    page = args->b.table[seq * args->b.table_stride + (t0 >> args->c.page_shift)];
  const int lo = first > t0 ? first - t0 : 0, hi = past - t0 < kKvBlock ? past - t0 : kKvBlock;
  const int64_t row = row0 + (t0 - begin);  // of token t0, which may be an earlier sequence's
  KvRotary rot;
  rot.dims = args->rot.dims;
  rot.pairs = args->rot.pairs;
  rot.gain = args->rot.gain;
  const double eps = args->a.eps;

  const uint8_t *src = args->a.q + row * args->a.q_stride;
  const uint32_t stride = (uint32_t)args->a.q_stride;
  auto head = [&](int unit, int end, int heads) {
    const int h = unit * SUB + H::sub();
    return unit < end && h < heads ? h : -1;
  };
  H now, next;
  if (from < q_units) now.load(src, stride, head(from + wave, q_to, heads), lo, hi);
  if (from < q_units + kv_units) {
    fill_table<double, D>(lds, rot, turns, lo, hi, [&](int r) { return (int64_t)(t0 + r); });
    __syncthreads();
  }
  if (from < q_units) {
    const float *weight = args->a.q_weight;
    float qw[H::VEC];
    H::weights(weight, qw);
    uint8_t *dst = reinterpret_cast<uint8_t *>(args->a.q_out + row * heads * D);
    for (int unit = from + wave; unit < q_to; unit += WAVES) {
      next.load(src, stride, head(unit + WAVES, q_to, heads), lo, hi);
      now.template turn_and_store<float, false>(lds, rot, qw, weight != nullptr, eps, dst,
                                                (uint32_t)(heads * D * 2), head(unit, q_to, heads), lo, hi);
      now = next;
    }
  }
  const int kv_hi = min(hi, last - t0);
  if (to <= q_units || lo >= kv_hi || page < 0) return;  // no place for keys and values
  KvCache c = args->c;
  if (page >= c.pages) return;
  const float *weight = args->a.k_weight;
  // the wave's first unit past the queries
  int unit = from + wave;
  if (unit < q_units) unit += (q_units - unit + WAVES - 1) / WAVES * WAVES;
  for (; unit < to; unit += WAVES) {
    const bool value = unit >= q_units + kv_units;
    const int h = head(unit - q_units - (value ? kv_units : 0), kv_units, kv_heads);
    const int64_t stride = value ? args->a.v_stride : args->a.k_stride;
    now.load((value ? args->a.v : args->a.k) + row * stride, (uint32_t)stride, h, lo, kv_hi);
    float kw[H::VEC], val[H::PER][4][H::VEC];
    H::weights(value ? nullptr : weight, kw);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < H::PER; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        now.values(i, t, val[i][t]);
        if (!value) H::template turn<double>(lds, rot, kw, weight != nullptr, eps, i, t, val[i][t]);
        const int r = 4 * H::quad(i) + t;
#pragma unroll
        for (int e = 0; e < H::VEC; ++e) {
          const uint32_t mag = __float_as_uint(val[i][t][e]) & 0x7FFFFFFFu;
          if (r >= lo && r < kv_hi && mag < 0x7F800000u && mag > top) top = mag;
        }
      }
    store_block<F32, D, SUB>(c, args->layer, page, h, value, t0, t0 + lo, t0 + kv_hi, val, top);
  }
}

// Heads of a workgroup: one unit for each wave, as long as that makes no more workgroups
// than the card takes at a time, else three, which share a table.
int units_each(int64_t blocks, int64_t units) {
  const int64_t waves = kThreads / 64;
  const int64_t per = blocks * ((units + waves - 1) / waves) <= 4 * (int64_t)device_cu_count() ? waves : 3 * waves;
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
  const int units = (a.heads + sub - 1) / sub + 2 * ((c.kv_heads + sub - 1) / sub);
  const int per = units_each(b.seqs * blocks, units);
  const int64_t slices = (units + per - 1) / per, grid = b.seqs * blocks * slices;
  if (grid > 0x7FFFFFFF / kThreads) return hipErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(kThreads), 0, s,
                       AppendArgs{c, layer, b, rot, a, (uint32_t)blocks, (uint32_t)slices, per});
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
