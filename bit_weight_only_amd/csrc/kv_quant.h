// kv_quant.h -- the 8-bit format on the device: exponents, codes, and a block of
// new tokens written into its page.  Shared by the kernels that write the cache
// or read it back.  Not installed.
#pragma once

#include "kv_internal.h"

namespace nf4 {

constexpr int kWave = 64;

// The largest of 64 (or each 32) neighbouring lanes' values.
template <int LANES = 64>
__device__ inline uint32_t wave_max(uint32_t v) {
  auto max_with = [&](uint32_t w) { v = w > v ? w : v; };
  max_with(__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));   // lane ^ 1
  max_with(__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));   // lane ^ 2
  max_with(__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));  // 7 - lane of 8
  max_with(__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));  // 15 - lane of 16
  uint32_t row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) row[i] = (uint32_t)__builtin_amdgcn_readlane((int)v, 16 * i);
  const uint32_t low = row[0] > row[1] ? row[0] : row[1], high = row[2] > row[3] ? row[2] : row[3];
  if (LANES == 32) return threadIdx.x & 32 ? high : low;
  return low > high ? low : high;
}

// Exponent of the block scale for the bits of a magnitude a = m 2^E, 1 <= m <
// 2: the least e with a <= 448 2^e = 1.75 2^(8 + e), clamped.  Zero and
// subnormals have E = -127 here, which the clamp takes to kKvExpMin either way.
__device__ inline int block_exponent(uint32_t bits) {
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < kKvExpMin ? kKvExpMin : e > kKvExpMax ? kKvExpMax : e;
}

__device__ inline float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Exponent of a scale that the cache holds; whatever else lies there is
// taken into the range (it can only be a block that was never written).
__device__ inline int scale_exponent(float s) {
  const int e = (int)((__float_as_uint(s) >> 23) & 255u) - 127;
  return e < kKvExpMin ? kKvExpMin : e > kKvExpMax ? kKvExpMax : e;
}

// e4m3 codes of four values (byte i = value i): to nearest even, past +-448
// as +-448, NaN as NaN.
__device__ inline uint32_t codes4(float a, float b, float c, float d) {
  auto hold = [](float x) { return x != x ? x : fminf(fmaxf(x, -448.0f), 448.0f); };
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(hold(a), hold(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(hold(c), hold(d), w, true);
}

// The codes of a dword at a scale 2^shift times as large.
__device__ inline uint32_t rescale4(uint32_t w, float factor) {
  auto v = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  auto u = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return codes4(v[0] * factor, v[1] * factor, u[0] * factor, u[1] * factor);
}

// How a wave takes a block of 16 tokens of one head, rows of D values in fp32 or
// bf16: a lane 16 bytes (VEC values, piece `task % CHUNKS` of a row) of the four
// consecutive tokens of quad `task / CHUNKS`, which are pieces of four key rows
// and whole dwords of a quad of values; task = lane + 64 i, i < PER.
template <bool F32, int D>
struct Block {
  static constexpr int VEC = F32 ? 4 : 8;
  static constexpr int CHUNKS = D / VEC;
  static constexpr int TASKS = 4 * CHUNKS;
  static constexpr int PER = (TASKS + kWave - 1) / kWave;
};

// What a block that is new in part held before, read ahead of the new values' way
// through the kernel: its scale, and the values' quads that have old or no tokens in them.
template <bool F32, int D, int SUB = 1>
struct OldBlock {
  using B = Block<F32, D>;
  uint8_t *codes;
  float *scale;
  float old_scale;
  uint32_t had[B::PER][B::VEC];

  // The block that starts at t0 of keys (kv 0) or values (1), of which the tokens first ..
  // last - 1 are new.  SUB: as many heads are taken by as many parts of the wave.
  __device__ OldBlock(const KvCache &c, int64_t layer, int64_t page, int head, int kv, int t0,
                      int first, int last) {
    const int lane = threadIdx.x & (64 / SUB - 1);
    const int64_t block = ((layer * c.pages + page) * c.kv_heads + head) *
                              (int64_t)(1 << (c.page_shift - 4)) +
                          ((t0 & (c.page_tokens() - 1)) >> 4);
    codes = (kv ? c.v : c.k) + block * (kKvBlock * D);
    scale = (kv ? c.vs : c.ks) + block;
    old_scale = 0.0f;
    if (head < 0) return;
    if (first > t0) old_scale = *scale;
#pragma unroll
    for (int i = 0; i < B::PER; ++i) {
      const int task = lane + i * kWave, quad = task / B::CHUNKS, piece = task % B::CHUNKS;
      const int q0 = t0 + 4 * quad;
      if (kv && task < B::TASKS && q0 < last && (q0 < first || q0 + 4 > last))
        __builtin_memcpy(had[i], __builtin_assume_aligned(codes + (quad * D + piece * B::VEC) * 4, 16),
                         sizeof(had[i]));
    }
  }
};

// Writes the tokens first .. last - 1 of the block that starts at t0 (kv 0: keys,
// 1: values) into its page: val holds them as above, top is the lane's largest
// finite magnitude of them, as bits.  Tokens before `first` are the sequence's
// own earlier ones; what lies past `last` is left as it is.  head < 0: a part of the wave
// that has none.
template <bool F32, int D, int SUB = 1, int VEC, int PER>
__device__ inline void store_block(const OldBlock<F32, D, SUB> &was, int head, int kv, int t0,
                                   int first, int last, const float (&val)[PER][4][VEC],
                                   uint32_t top) {
  constexpr int CHUNKS = Block<F32, D>::CHUNKS, TASKS = Block<F32, D>::TASKS;
  constexpr int LANES = 64 / SUB;
  const int lane = threadIdx.x & (LANES - 1);
  const uint32_t top_of_all = wave_max<LANES>(top);
  if (SUB > 1 && head < 0) return;
  uint8_t *const codes = was.codes;
  int e = block_exponent(top_of_all);
  const bool has_old = first > t0;
  int e_old = e;
  if (has_old) {
    e_old = scale_exponent(was.old_scale);
    e = e_old > e ? e_old : e;
  }
  const float inv = pow2(-e), factor = pow2(e_old - e < -126 ? -126 : e_old - e);
  const bool grew = has_old && e != e_old;

#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int task = lane + i * kWave, quad = task / CHUNKS, piece = task % CHUNKS;
    if (task >= TASKS) continue;
    const int q0 = t0 + 4 * quad;
    if (kv == 0) {
      // keys: VEC bytes of each of the four rows
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int tok = q0 + t;
        uint32_t *p = reinterpret_cast<uint32_t *>(codes + (4 * quad + t) * D + piece * VEC);
        if (tok >= first && tok < last) {
#pragma unroll
          for (int h = 0; h < VEC / 4; ++h)
            p[h] = codes4(val[i][t][4 * h] * inv, val[i][t][4 * h + 1] * inv,
                          val[i][t][4 * h + 2] * inv, val[i][t][4 * h + 3] * inv);
        } else if (tok < first && grew) {
#pragma unroll
          for (int h = 0; h < VEC / 4; ++h) p[h] = rescale4(p[h], factor);
        }
      }
    } else if (q0 < last && (q0 + 3 >= first || grew)) {
      // values: VEC dwords of a quad, each byte a token
      uint32_t *p = reinterpret_cast<uint32_t *>(codes + (quad * D + piece * VEC) * 4);
      uint32_t keep = 0, old = 0;  // bytes of the quad that are not new
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (q0 + t < first || q0 + t >= last) keep |= 0xFFu << (8 * t);
        if (q0 + t < first) old |= 0xFFu << (8 * t);
      }
      uint32_t out[VEC];
#pragma unroll
      for (int d = 0; d < VEC; ++d) {
        uint32_t y = codes4(val[i][0][d] * inv, val[i][1][d] * inv, val[i][2][d] * inv,
                            val[i][3][d] * inv);
        if (keep) {
          const uint32_t had = was.had[i][d];
          const uint32_t kept = grew ? (rescale4(had, factor) & old) | (had & ~old) : had;
          y = (y & ~keep) | (kept & keep);
        }
        out[d] = y;
      }
      __builtin_memcpy(__builtin_assume_aligned(p, 16), out, sizeof(out));
    }
  }
  if (lane == 0) *was.scale = pow2(e);
}

}  // namespace nf4
