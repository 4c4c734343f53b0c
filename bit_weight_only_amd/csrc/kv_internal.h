// kv_internal.h -- geometry of the key-value cache, kernel argument blocks and
// the launchers shared by the entry points in kv_abi.hip.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nf4 {

constexpr int kKvBlock = 16;    // tokens under one scale
constexpr int kKvExpMin = -40;  // exponents that a block's scale may have: the
constexpr int kKvExpMax = 100;  // attention folds them into exponents of its weights
                                // (kLift there keeps the sums in range)

// Positions are held to this, and windows: the most tokens of a table that the
// library reads and as many rows past them, so that a row there is past every
// key, and positions less windows stay in 32 bits.
constexpr int kKvLongest = (1 << 30) + (1 << 23);

// Values that the rows of queries, keys and the like may lie apart: offsets inside a block
// of 16 rows stay in 31 bits.
constexpr int64_t kKvWidestRows = int64_t(1) << 24;

// The cache as a kernel sees it.  A page of one layer is kv_heads runs of
// page_tokens * D bytes (k and v alike) and kv_heads * page_tokens / 16 scales.
struct KvCache {
  uint8_t *k, *v;
  float *ks, *vs;
  int64_t layers, pages;
  int kv_heads;
  int page_shift;  // log2 of the tokens of a page
  int head_dim;
  __host__ __device__ int page_tokens() const { return 1 << page_shift; }
  __host__ __device__ int64_t page_blocks() const {
    return (int64_t)kv_heads << (page_shift - 4);
  }
  __host__ __device__ int64_t page_bytes() const {
    return page_blocks() * kKvBlock * head_dim;
  }
};

struct KvBatch {
  int64_t seqs, rows;
  int max_rows;
  int max_len;   // no more than the table's entries have room for
  int held_len;  // what the host holds lengths to, kKvLongest where only the table does
  const int32_t *row_start, *kv_len, *table;
  int64_t table_stride;

  // Rows of sequence s: the first one's index and their number; the tokens of
  // the sequence, and how many of them have a place in the table.  Only the
  // rows' positions come from the former: a sequence that has outgrown its
  // table must not find its new tokens on the places of older ones.
  __device__ void sequence(int64_t s, int64_t &row0, int &n, int &len, int &end) const {
    sequence(raw(s), row0, n, len, end);
  }
  // The same in two steps, so that other loads can go out beside these.
  struct Raw {
    int64_t r0, r1;
    int len;
  };
  __device__ Raw raw(int64_t s) const {
    Raw x{s, s + 1, 0};
    if (row_start) {
      x.r0 = row_start[s];
      x.r1 = row_start[s + 1];
    }
    x.len = kv_len[s];
    return x;
  }
  __device__ void sequence(const Raw &x, int64_t &row0, int &n, int &len, int &end) const {
    const int64_t r0 = x.r0 < 0 ? 0 : x.r0 > rows ? rows : x.r0;
    const int64_t r1 = x.r1 < r0 ? r0 : x.r1 > rows ? rows : x.r1;
    row0 = r0;
    n = (int)(r1 - r0);
    len = x.len < 0 ? 0 : x.len > held_len ? held_len : x.len;
    end = len > max_len ? max_len : len;
  }
  // The first row of sequence s, s = seqs: past the last one's.
  __device__ int64_t first_row(int64_t s) const {
    const int64_t r = row_start ? row_start[s] : s;
    return r < 0 ? 0 : r > rows ? rows : r;
  }
  // The position of a row of one of the sequences first .. past - 1, in two steps, so that
  // the loads of the first one are in flight beside others.  It takes the sequence
  // that the row is in if all have as many rows; the second one searches if that is not it.
  struct Guess {
    int seq, from, to, len;
  };
  __device__ Guess guess(int64_t row, int first, int past, int64_t row0, int rows_of_all) const {
    Guess g;
    const int n = past - first, each = rows_of_all > n ? rows_of_all / n : 1;
    g.seq = first + (int)(row - row0) / each;
    g.seq = g.seq < past ? g.seq : past - 1;
    g.from = row_start ? row_start[g.seq] : g.seq;
    g.to = row_start ? row_start[g.seq + 1] : g.seq + 1;
    g.len = kv_len[g.seq];
    return g;
  }
  __device__ int position(const Guess &g, int64_t row, int first, int past) const {
    if (g.from <= row && row < g.to && g.from >= 0 && g.to <= rows)
      return (g.len < 0 ? 0 : g.len > held_len ? held_len : g.len) - (g.to - g.from) + (int)(row - g.from);
    int s = first, hi = past;
    while (row_start && hi - s > 1) {
      const int mid = s + (hi - s) / 2;
      (row_start[mid] <= row ? s : hi) = mid;
    }
    int64_t row0;
    int n, len, end;
    sequence(s, row0, n, len, end);
    return len - n + (int)(row - row0);
  }
};

// Sequences first[g] .. first[g + 1] - 1 begin with the same shared_len[g] tokens.
struct KvGroups {
  int groups, max_rows, max_shared;
  const int32_t *first, *shared_len;  // first null: one group of all

  __device__ int first_of(const KvBatch &b, int g) const {
    const int n = (int)b.seqs, s = first ? first[g] : g == 0 ? 0 : n;
    return s < 0 ? 0 : s > n ? n : s;
  }
  // Tokens that group g shares and the table has a place for.
  __device__ int shared(const KvBatch &b, int g) const { return held(b, shared_len[g]); }
  __device__ int held(const KvBatch &b, int n) const {
    const int most = max_shared < b.max_len ? max_shared : b.max_len;
    return n < 0 ? 0 : n > most ? most : n;
  }
  // The sequence of first .. past - 1 whose pages the group's `shared` tokens are read from: the
  // first one that has them all, or has the most of them.  The whole wave looks.
  __device__ int source(const KvBatch &b, int first, int past, int shared) const {
    int most = -1, at = first;
    for (int s0 = first; s0 < past; s0 += 64) {
      const int s = s0 + (int)(threadIdx.x & 63), len = s < past ? b.kv_len[s] : -1;
      const uint64_t all = __ballot(len >= shared);
      if (all) return s0 + __builtin_ctzll(all);
      if (len > most) {
        most = len;
        at = s;
      }
    }
    for (int o = 1; o < 64; o *= 2) {
      const int len = __shfl_xor(most, o), s = __shfl_xor(at, o);
      if (len > most || (len == most && s < at)) {
        most = len;
        at = s;
      }
    }
    return __builtin_amdgcn_readfirstlane(at);
  }
  // The same of the group that sequence s is in (0: in none), and that group's first
  // sequence.  The whole wave looks, a lane at every 64th place, so that up to 64 groups
  // take one trip to memory.
  __device__ int shared_of(const KvBatch &b, int s, int *first_seq = nullptr) const {
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = groups;
    for (;;) {
      const int step = (hi - lo + 63) / 64, at = lo + lane * step;
      const int here = at < hi ? at : hi - 1;
      const int from = first_of(b, here), to = first_of(b, here + 1), len = shared_len[here];
      const int in = __popcll(__ballot(at < hi && from <= s));  // ascending: the first ones
      if (in == 0) return 0;
      const int l = in - 1;
      if (step == 1) {
        if (first_seq) *first_seq = __builtin_amdgcn_readlane(from, l);
        return s < __builtin_amdgcn_readlane(to, l) ? held(b, __builtin_amdgcn_readlane(len, l)) : 0;
      }
      lo += l * step;
      hi = lo + step < hi ? lo + step : hi;
    }
  }
};

struct KvPool {
  int32_t *refs, *table;
  int64_t rows, stride;
  int32_t *len, *missing;
};

// Compute units of the current device (queried once per device).
int device_cu_count();

hipError_t launch_kv_append(const KvCache &c, int64_t layer, const KvBatch &b, const void *k,
                            int64_t k_stride, const void *v, int64_t v_stride, bool f32,
                            hipStream_t s);

// How heads turn: the first `dims` values, pair i by turns[i] / 2^64 of a full turn a
// token; `pairs`: neighbouring values, else value i and i + dims / 2.
struct KvRotary {
  int dims;
  bool pairs;
  double gain;
  uint64_t turns[64];
};

// Rows of values, `stride` of them apart.
struct KvRows {
  void *at;
  int64_t stride;
  bool f32;
};
hipError_t launch_rotate(const KvRotary &rot, const KvRows &x, const int32_t *positions,
                         int64_t rows, int heads, int head_dim, const float *weight, double eps,
                         const KvRows &y, hipStream_t s);

// The new rows of an append that turns queries and keys, strides in bytes.
struct KvTurned {
  const uint8_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  int heads;
  const float *q_weight, *k_weight;  // of the norms, or null
  double eps;
  uint16_t *q_out;
};
hipError_t launch_kv_append_rotated(const KvCache &c, int64_t layer, const KvBatch &b,
                                    const KvRotary &rot, const KvTurned &a, bool f32,
                                    hipStream_t s);

hipError_t launch_kv_read(const KvCache &c, int64_t layer, const KvBatch &b, const KvRows &k,
                          const KvRows &v, hipStream_t s);

struct KvAttention {
  const uint16_t *q;
  int64_t q_stride;
  int heads;
  float scale;
  int window, sinks;  // window 0: none
  uint16_t *out;
  float *lse;
  void *ws;
};
size_t kv_attention_workspace_bytes(const KvCache &c, const KvBatch &b, int heads, int window,
                                    int sinks);
hipError_t launch_kv_attention(const KvCache &c, int64_t layer, const KvBatch &b,
                               const KvAttention &a, hipStream_t s);

size_t kv_attention_shared_workspace_bytes(const KvCache &c, const KvBatch &b, const KvGroups &g,
                                           int heads, int window, int sinks);
hipError_t launch_kv_attention_shared(const KvCache &c, int64_t layer, const KvBatch &b,
                                      const KvGroups &g, const KvAttention &a, hipStream_t s);

hipError_t launch_kv_copy_pages(const KvCache &c, const int32_t *src, const int32_t *dst,
                                int64_t n, hipStream_t s);
hipError_t launch_kv_reserve(const KvCache &c, const KvPool &p, const int32_t *add, hipStream_t s);
hipError_t launch_kv_fork(const KvCache &c, const KvPool &p, const int32_t *src,
                          const int32_t *dst, int64_t n, hipStream_t s);
hipError_t launch_kv_release(const KvCache &c, const KvPool &p, const int32_t *rows, int64_t n,
                             hipStream_t s);
size_t kv_compact_workspace_bytes(const KvCache &c);
hipError_t launch_kv_compact(const KvCache &c, const KvPool &p, int32_t *refs_out,
                             int32_t *table_out, void *ws, hipStream_t s);

}  // namespace nf4
