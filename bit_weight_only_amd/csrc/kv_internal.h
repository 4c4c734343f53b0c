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
    int64_t r0 = s, r1 = s + 1;
    if (row_start) {
      r0 = row_start[s];
      r1 = row_start[s + 1];
    }
    r0 = r0 < 0 ? 0 : r0 > rows ? rows : r0;
    r1 = r1 < r0 ? r0 : r1 > rows ? rows : r1;
    row0 = r0;
    n = (int)(r1 - r0);
    const int l = kv_len[s];
    len = l < 0 ? 0 : l > held_len ? held_len : l;
    end = len > max_len ? max_len : len;
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
