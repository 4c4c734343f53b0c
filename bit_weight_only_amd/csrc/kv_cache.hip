// kv_cache.hip -- writing the 8-bit key-value cache (quantization of new
// tokens into their pages) and the pool its pages come from (reserving,
// forking, copying, releasing and compacting them).
//
// vibevoice.c README: the KV cache may be kept in FP8, and in pages that the
// slots of a server share.  The block format, its scales and every rule of the pool are this
// library's own (include/nf4.h states them).
#include "kv_internal.h"
#include "kv_quant.h"

namespace nf4 {
namespace {

struct Rows {
  const void *k, *v;
  int64_t k_stride, v_stride;
};

// One wave per (sequence, block that its new tokens touch, head, keys or
// values).  A lane takes 16 bytes of four consecutive tokens, which are whole
// dwords of a quad of values and pieces of four key rows.  Memory bound: the
// new rows are read once and their codes written once; a block that was full
// in part also has its old codes read, once more written where the scale grew.
// 14449 fp32 tokens of 8 heads of 128 (148 MB): 26 us in a trace = 5.7 TB/s.  A
// single token, of which 1.6 us are an empty launch, is bound by trips to memory
// one after the other: its place among the rows and the length, the page id beside
// the rows, and the old scale beside the quad of values that it is a byte of
// (OldBlock), which are then merged and stored.
template <bool F32, int D>
__global__ __launch_bounds__(256) void append_kernel(KvCache c, int64_t layer, KvBatch b, Rows x,
                                                     int64_t blocks_per_seq) {
  using B = Block<F32, D>;
  constexpr int VEC = B::VEC, CHUNKS = B::CHUNKS, TASKS = B::TASKS, PER = B::PER;
  const int lane = threadIdx.x & 63;
  int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int kv = (int)(w & 1);
  w >>= 1;
  const int head = (int)(w % c.kv_heads);
  w /= c.kv_heads;
  const int64_t seq = w / blocks_per_seq;
  if (seq >= b.seqs) return;
  int64_t row0;
  int n, len, end;
  b.sequence(seq, row0, n, len, end);
  const int begin = len - n;                    // position of row 0, may be negative
  const int first = begin < 0 ? 0 : begin;      // first new token
  int last = begin + (n < b.max_rows ? n : b.max_rows);  // past the last one
  last = last < end ? last : end;
  const int64_t blk = first / kKvBlock + w % blocks_per_seq;
  const int t0 = (int)(blk * kKvBlock);
  if (blk * kKvBlock >= last) return;
  const int page = b.table[seq * b.table_stride + (t0 >> c.page_shift)];
  const uint8_t *src = static_cast<const uint8_t *>(kv ? x.v : x.k);
  const int64_t stride = (kv ? x.v_stride : x.k_stride) * (F32 ? 4 : 2);

  float val[PER][4][VEC];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int task = lane + i * kWave, quad = task / CHUNKS, piece = task % CHUNKS;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int tok = t0 + 4 * quad + t;
      uint4 r = make_uint4(0, 0, 0, 0);
      if (task < TASKS && tok >= first && tok < last)
        r = *reinterpret_cast<const uint4 *>(src + (row0 + (tok - begin)) * stride +
                                             ((int64_t)head * D + piece * VEC) * (F32 ? 4 : 2));
      const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const uint32_t bits =
            F32 ? rw[e] : (e & 1) ? rw[e >> 1] & 0xFFFF0000u : rw[e >> 1] << 16;
        val[i][t][e] = __uint_as_float(bits);
        const uint32_t mag = bits & 0x7FFFFFFFu;
        if (mag < 0x7F800000u && mag > top) top = mag;
      }
    }
  }
  // the rows are on their way before the page is known
  if (page < 0 || page >= c.pages) return;
  const OldBlock<F32, D> was(c, layer, page, head, kv, t0, first, last);
  store_block<F32, D>(was, head, kv, t0, first, last, val, top);
}

struct ReadRows {
  uint8_t *k, *v;
  int64_t k_stride, v_stride;  // bytes
};

// The reverse of append_kernel, by the same division of the work: a wave per
// (sequence, block that its rows touch, head, keys or values).  Rows that have no
// place get zeros.  Memory bound: 6 sequences of up to 14449 tokens, 8 heads of 128, to bf16
// (291 MB), other ones in every call: 62.6 us = 4.6 TB/s; a chunk of 113 tokens, 4 heads, to
// fp32 3.8 us in a trace, of which 1.6 an empty launch and the rest three trips to memory one
// after the other (place and length, page id, codes).
template <bool F32, int D>
__global__ __launch_bounds__(256) void read_kernel(KvCache c, int64_t layer, KvBatch b, ReadRows y,
                                                   int64_t blocks_per_seq) {
  using B = Block<F32, D>;
  constexpr int VEC = B::VEC, CHUNKS = B::CHUNKS, TASKS = B::TASKS, PER = B::PER;
  const int lane = threadIdx.x & 63;
  int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int kv = (int)(w & 1);
  w >>= 1;
  const int head = (int)(w % c.kv_heads);
  w /= c.kv_heads;
  const int64_t seq = w / blocks_per_seq;
  if (seq >= b.seqs) return;
  int64_t row0;
  int n, len, end;
  b.sequence(seq, row0, n, len, end);
  const int begin = len - n;                // position of row 0, may be negative
  const int first = begin < 0 ? 0 : begin;  // first token
  const int past = begin + (n < b.max_rows ? n : b.max_rows);  // past the last row's position
  uint8_t *to = kv ? y.v : y.k;
  const int64_t stride = kv ? y.v_stride : y.k_stride;
  if (begin < 0 && w % blocks_per_seq == 0) {
    const int none = min(-begin, min(n, b.max_rows));  // rows that are no tokens
    for (int64_t i = lane; i < (int64_t)none * CHUNKS; i += kWave)
      *reinterpret_cast<uint4 *>(to + (row0 + i / CHUNKS) * stride +
                                 ((int64_t)head * CHUNKS + i % CHUNKS) * 16) =
          make_uint4(0, 0, 0, 0);
  }
  const int blk = first / kKvBlock + (int)(w % blocks_per_seq), t0 = blk * kKvBlock;
  if (first >= past || t0 >= past) return;
  int page = -1;
  if (t0 < end) page = b.table[seq * b.table_stride + (t0 >> c.page_shift)];
  const bool there = page >= 0 && page < c.pages;
  const int64_t block = ((layer * c.pages + (there ? page : 0)) * c.kv_heads + head) *
                            (int64_t)(1 << (c.page_shift - 4)) +
                        ((t0 & (c.page_tokens() - 1)) >> 4);
  const uint8_t *codes = (kv ? c.v : c.k) + block * (kKvBlock * D);
  const float scale = pow2(scale_exponent((kv ? c.vs : c.ks)[block]));
  const int last = min(past, end);  // past the last token with a place
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int task = lane + i * kWave, quad = task / CHUNKS, piece = task % CHUNKS;
    if (task >= TASKS) continue;
    // four tokens' codes of VEC values: dword h of token t
    uint32_t code[4][VEC / 4];
    if (kv == 0) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        __builtin_memcpy(code[t], __builtin_assume_aligned(codes + (4 * quad + t) * D + piece * VEC, VEC),
                         VEC);
    } else {
      uint32_t q[VEC];  // a value's four tokens each
      __builtin_memcpy(q, __builtin_assume_aligned(codes + (quad * D + piece * VEC) * 4, 16), 4 * VEC);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int h = 0; h < VEC / 4; ++h) {
          code[t][h] = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) code[t][h] |= (q[4 * h + e] >> (8 * t) & 255u) << (8 * e);
        }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int tok = t0 + 4 * quad + t;
      if (tok < first || tok >= past) continue;
      float v[VEC];
#pragma unroll
      for (int h = 0; h < VEC / 4; ++h) {
        const auto x = __builtin_amdgcn_cvt_pk_f32_fp8((int)code[t][h], false);
        const auto z = __builtin_amdgcn_cvt_pk_f32_fp8((int)code[t][h], true);
        v[4 * h] = x[0] * scale;
        v[4 * h + 1] = x[1] * scale;
        v[4 * h + 2] = z[0] * scale;
        v[4 * h + 3] = z[1] * scale;
      }
      uint4 out = make_uint4(0, 0, 0, 0);
      if (there && tok < last) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)  // few bits each: as bf16, a value is its upper half
          u[e] = F32 ? __float_as_uint(v[e])
                     : __float_as_uint(v[(2 * e) % VEC]) >> 16 |
                           (__float_as_uint(v[(2 * e + 1) % VEC]) & 0xFFFF0000u);
        out = make_uint4(u[0], u[1], u[2], u[3]);
      }
      *reinterpret_cast<uint4 *>(to + (row0 + (tok - begin)) * stride +
                                 ((int64_t)head * CHUNKS + piece) * 16) = out;
    }
  }
}

// ------------------------------------------------------------------ the pool

constexpr int kPlanThreads = 256;

// Exclusive prefix sum of v (0 .. 2^28) over the workgroup's threads in thread
// order; `total` gets the sum.  Both stop at kManyPages, more than a pool has:
// 256 requests may pass 32 bits.  `part`: one int per wave in LDS.
constexpr int kManyPages = 1 << 28;

__device__ inline int block_prefix(int v, int *part, int &total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o);
    if (lane >= o) x = min(x + y, kManyPages);
  }
  __syncthreads();  // the previous call's reads of part are over
  if (lane == 63) part[wave] = x;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    const int p = part[w];
    before += w < wave ? p : 0;
    sum += p;
  }
  total = min(sum, kManyPages);
  const int below = __shfl_up(x, 1);
  return min(before + (lane > 0 ? below : 0), kManyPages);
}

// Requests for pages, in an order that fixes which free page answers which:
// Fork asks for one page per pair whose source's last page is full in part,
// Reserve for the pages between a row's old and new length.
struct ForkRequests {
  const int32_t *src, *dst;
  int64_t n;
  __device__ int64_t count() const { return n; }
  // Pages that item i asks for, the table row and the first entry they go to.
  __device__ int ask(const KvCache &c, const KvPool &p, int64_t i, int64_t &row, int64_t &entry,
                     int &lost) const {
    const int64_t a = src[i], d = dst[i];
    lost = 0;
    if (a < 0 || a >= p.rows || d < 0 || d >= p.rows) return 0;
    const int len = p.len[a];
    row = d;
    entry = len >> c.page_shift;
    if (len <= 0 || (len & (c.page_tokens() - 1)) == 0 || entry >= p.stride) return 0;
    const int page = p.table[a * p.stride + entry];
    return page >= 0 && page < c.pages ? 1 : 0;
  }
  __device__ void done(const KvPool &p, int64_t i) const {
    const int64_t a = src[i], d = dst[i];
    if (a >= 0 && a < p.rows && d >= 0 && d < p.rows) p.len[d] = p.len[a];
  }
};

struct ReserveRequests {
  const int32_t *add;
  __device__ int64_t count() const { return -1; }
  __device__ int ask(const KvCache &c, const KvPool &p, int64_t i, int64_t &row, int64_t &entry,
                     int &lost) const {
    lost = 0;
    row = i;
    const int64_t more = add[i], len = p.len[i] < 0 ? 0 : p.len[i];
    const int64_t pt = c.page_tokens();
    entry = (len + pt - 1) >> c.page_shift;
    if (more <= 0) return 0;
    int64_t end = (len + more + pt - 1) >> c.page_shift;
    if (end > p.stride) {
      lost = (int)(end - (entry > p.stride ? entry : p.stride));
      end = p.stride;
    }
    return end > entry ? (int)(end - entry) : 0;
  }
  __device__ void done(const KvPool &p, int64_t i) const {
    if (add[i] <= 0) return;
    const int64_t len = (int64_t)(p.len[i] < 0 ? 0 : p.len[i]) + add[i];
    p.len[i] = (int)(len > 0x7FFFFFFF ? 0x7FFFFFFF : len);
  }
};

// The counts of 2048 pages: a wave takes 512 consecutive ones, 64 at a time, a
// page per lane, so that pages are numbered by counting bits of ballots.
constexpr int kRunGroups = 8;
constexpr int kRunPages = kPlanThreads * kRunGroups;

__device__ inline int64_t run_page(int64_t page0, int g) {
  return page0 + ((threadIdx.x >> 6) * kRunGroups + g) * 64 + (threadIdx.x & 63);
}
__device__ inline void read_run(const KvCache &c, const int32_t *refs, int64_t page0,
                                int32_t (&r)[kRunGroups]) {
#pragma unroll
  for (int g = 0; g < kRunGroups; ++g) {
    const int64_t page = run_page(page0, g);
    r[g] = page < c.pages ? refs[page] : -1;
  }
}
// Number of ones below the lane.
__device__ inline int ones_below(uint64_t bits) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(bits >> 32),
                                   __builtin_amdgcn_mbcnt_lo((uint32_t)bits, 0u));
}
// `before`: ones of the waves before this one, out of each wave's own number;
// `total`: of all waves.  `part`: one int per wave in LDS.
__device__ inline void wave_prefix(int mine, int *part, int &before, int &total) {
  const int wave = threadIdx.x >> 6;
  __syncthreads();  // the previous call's reads of part are over
  if ((threadIdx.x & 63) == 0) part[wave] = mine;
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    const int p = part[w];
    before += w < wave ? p : 0;
    total += p;
  }
}

// One workgroup: items 256 at a time, their requests numbered by a prefix
// sum, then the free pages numbered the same way from page 0 on until every
// request has its page.  Latency bound, a few dependent reads and barriers (32
// requests, 512 pages: 4.2 us); one workgroup, so that the order needs no second
// launch.
template <class Requests>
__global__ __launch_bounds__(kPlanThreads) void assign_pages_kernel(KvCache c, KvPool p,
                                                                    Requests rq) {
  __shared__ int part[kPlanThreads / 64];
  __shared__ int first[kPlanThreads];        // number of an item's first request
  __shared__ int64_t where[kPlanThreads];    // table place of its first page
  __shared__ unsigned long long missing;     // pages that requests did not get
  const int tid = threadIdx.x;
  int32_t refs[kRunGroups];
  read_run(c, p.refs, 0, refs);  // the first pages, beside the requests
  if (tid == 0) missing = 0;
  const int64_t items = rq.count() < 0 ? p.rows : rq.count();
  for (int64_t i0 = 0; i0 < items; i0 += kPlanThreads) {
    const int64_t i = i0 + tid;
    int64_t row = 0, entry = 0;
    int lost = 0, want = 0, total;
    if (i < items) want = rq.ask(c, p, i, row, entry, lost);
    const int mine = block_prefix(want, part, total);
    first[tid] = mine;
    where[tid] = row * p.stride + entry;
    int found = 0;
    for (int64_t page0 = 0; page0 < c.pages && found < total; page0 += kRunPages) {
      if (i0 + page0 > 0) read_run(c, p.refs, page0, refs);
      uint64_t free[kRunGroups];
      int count = 0, before, here;
#pragma unroll
      for (int g = 0; g < kRunGroups; ++g) {
        free[g] = __ballot(refs[g] == 0);
        count += __popcll(free[g]);
      }
      wave_prefix(count, part, before, here);  // its barriers are first's and where's too
      int rank0 = found + before;
#pragma unroll
      for (int g = 0; g < kRunGroups; ++g) {
        const int rank = rank0 + ones_below(free[g]);
        rank0 += __popcll(free[g]);
        if (refs[g] != 0 || rank >= total) continue;
        const int64_t page = run_page(page0, g);
        int lo = 0, hi = kPlanThreads;  // the last item whose first request is <= rank
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          (first[mid] <= rank ? lo : hi) = mid;
        }
        p.table[where[lo] + (rank - first[lo])] = (int32_t)page;
        p.refs[page] = 1;
      }
      found += here;
    }
    found = found < total ? found : total;
    const int got = min(max(found - mine, 0), want);
    for (int r = got; r < want; ++r) p.table[where[tid] + r] = -1;
    if (lost + (want - got) > 0) atomicAdd(&missing, (unsigned long long)lost + (want - got));
    if (i < items) rq.done(p, i);
    __syncthreads();
  }
  if (tid == 0 && p.missing)
    *p.missing = (int32_t)(missing > 0x7FFFFFFF ? 0x7FFFFFFF : missing);
}

// Page copies are cut into pieces of 16 KB of codes per workgroup, four 16-byte
// loads for each of 256 lanes.  The compiler holds what is loaded in LDS (16 KB a
// workgroup) and waits for each load before the next, so that a lane has one in
// flight, and the many workgroups are what keeps the memory busy (pieces twice
// as large, which halve them: a third slower).  Memory bound: 32 forks of a page
// of 1.8 MB each (28 layers) 25 us = 4.7 TB/s, the 465 MB of a compaction 107 us
// = 4.3 TB/s; a large copy reaches 5.1.
constexpr int kPieceLoads = 4;
constexpr int kPieceBytes = kPieceLoads * 256 * 16;

__host__ __device__ inline int64_t page_pieces(const KvCache &c) {
  return (c.page_bytes() + kPieceBytes - 1) / kPieceBytes;
}

// Piece `piece` of the 2 * page_pieces(c) of one page (keys, then values;
// the first piece of each also takes the scales).
__device__ inline void copy_piece(const KvCache &c, int64_t layer, int64_t from, int64_t to,
                                  int64_t piece) {
  const int64_t per = page_pieces(c);
  const bool kv = piece >= per;
  const int64_t at = (kv ? piece - per : piece) * kPieceBytes;
  const int64_t bytes = c.page_bytes(), blocks = c.page_blocks();
  uint8_t *base = kv ? c.v : c.k;
  const uint4 *s = reinterpret_cast<const uint4 *>(base + (layer * c.pages + from) * bytes + at);
  uint4 *d = reinterpret_cast<uint4 *>(base + (layer * c.pages + to) * bytes + at);
  const int left = (int)((bytes - at < kPieceBytes ? bytes - at : kPieceBytes) / 16);
  uint4 r[kPieceLoads];
#pragma unroll
  for (int i = 0; i < kPieceLoads; ++i)
    if ((int)threadIdx.x + i * 256 < left) r[i] = s[threadIdx.x + i * 256];
#pragma unroll
  for (int i = 0; i < kPieceLoads; ++i)
    if ((int)threadIdx.x + i * 256 < left) d[threadIdx.x + i * 256] = r[i];
  if (at == 0) {
    float *sc = kv ? c.vs : c.ks;
    for (int64_t i = threadIdx.x; i < blocks; i += 256)
      sc[(layer * c.pages + to) * blocks + i] = sc[(layer * c.pages + from) * blocks + i];
  }
}

__global__ __launch_bounds__(256) void copy_pages_kernel(KvCache c, const int32_t *src,
                                                         const int32_t *dst) {
  const int64_t per = 2 * page_pieces(c);
  int64_t w = blockIdx.x;
  const int64_t piece = w % per;
  w /= per;
  const int64_t layer = w % c.layers, i = w / c.layers;
  const int64_t from = src[i], to = dst[i];
  if (from < 0 || from >= c.pages || to < 0 || to >= c.pages) return;
  copy_piece(c, layer, from, to, piece);
}

// After assign_pages_kernel: the first `copies` workgroups copy the pages
// that are full in part, the others share the whole ones.
__global__ __launch_bounds__(256) void fork_kernel(KvCache c, KvPool p, const int32_t *src,
                                                   const int32_t *dst, int64_t copies,
                                                   int64_t entry_groups) {
  int64_t w = blockIdx.x;
  const bool copy = w < copies;
  const int64_t per = 2 * page_pieces(c);
  int64_t piece = 0, layer = 0, group = 0, i;
  if (copy) {
    piece = w % per;
    w /= per;
    layer = w % c.layers;
    i = w / c.layers;
  } else {
    w -= copies;
    group = w % entry_groups;
    i = w / entry_groups;
  }
  const int64_t a = src[i], d = dst[i];
  if (a < 0 || a >= p.rows || d < 0 || d >= p.rows) return;
  const int len = p.len[a];
  const int64_t full = len <= 0 ? 0 : len >> c.page_shift;
  const bool part = len > 0 && (len & (c.page_tokens() - 1)) != 0 && full < p.stride;
  if (copy) {
    if (!part) return;
    const int64_t from = p.table[a * p.stride + full], to = p.table[d * p.stride + full];
    if (from < 0 || from >= c.pages || to < 0 || to >= c.pages) return;
    copy_piece(c, layer, from, to, piece);
    return;
  }
  const int64_t entry = group * 256 + threadIdx.x;
  if (entry >= p.stride) return;
  const int64_t page = p.table[a * p.stride + entry];
  const bool valid = page >= 0 && page < c.pages;
  if (entry < full) {
    p.table[d * p.stride + entry] = valid ? (int32_t)page : -1;
    if (valid) atomicAdd(&p.refs[page], 1);
  } else if (entry > full || !part || !valid) {
    p.table[d * p.stride + entry] = -1;
  }
}

__global__ __launch_bounds__(256) void release_kernel(KvCache c, KvPool p, const int32_t *rows,
                                                      int64_t entry_groups) {
  const int64_t i = blockIdx.x / entry_groups;
  const int64_t entry = (blockIdx.x % entry_groups) * 256 + threadIdx.x;
  const int64_t row = rows[i];
  if (row < 0 || row >= p.rows || entry >= p.stride) return;
  // the exchange lets a row that is named twice give its pages up once
  const int page = atomicExch(&p.table[row * p.stride + entry], -1);
  if (page >= 0 && page < c.pages) atomicSub(&p.refs[page], 1);
  if (entry == 0) p.len[row] = 0;
}

// Workspace of a compaction, int32 each: [0] the number of moves, then from
// kMoveWords on the sources, the destinations and the new id of every page.
constexpr int kMoveWords = 64;

// One workgroup: counts the live pages n, then numbers the free pages before
// n and the live ones at or past it; equal numbers pair up.  Latency bound
// (2000 pages: 6.1 us).
__global__ __launch_bounds__(kPlanThreads) void compact_plan_kernel(KvCache c, KvPool p,
                                                                    int32_t *refs_out,
                                                                    int32_t *ws) {
  __shared__ int part[kPlanThreads / 64];
  int32_t *src = ws + kMoveWords, *dst = src + c.pages, *to = dst + c.pages;
  const int tid = threadIdx.x;
  int32_t refs[kRunGroups];
  int count = 0, before, live;
  for (int64_t page0 = 0; page0 < c.pages; page0 += kRunPages) {
    read_run(c, p.refs, page0, refs);
#pragma unroll
    for (int g = 0; g < kRunGroups; ++g) count += __popcll(__ballot(refs[g] > 0));
  }
  wave_prefix(count, part, before, live);
  int moves = 0, holes = 0;
  for (int64_t page0 = 0; page0 < c.pages; page0 += kRunPages) {
    if (c.pages > kRunPages) read_run(c, p.refs, page0, refs);  // else they are there
    uint64_t high[kRunGroups], hole[kRunGroups];
    int highs = 0, free = 0, h0, f0, all_high, all_free;
#pragma unroll
    for (int g = 0; g < kRunGroups; ++g) {
      const int64_t page = run_page(page0, g);
      high[g] = __ballot(page >= live && refs[g] > 0);
      hole[g] = __ballot(page < live && refs[g] <= 0);
      highs += __popcll(high[g]);
      free += __popcll(hole[g]);
    }
    wave_prefix(highs, part, h0, all_high);
    wave_prefix(free, part, f0, all_free);
    h0 += moves;
    f0 += holes;
#pragma unroll
    for (int g = 0; g < kRunGroups; ++g) {
      const int64_t page = run_page(page0, g);
      if (page < c.pages) {
        const bool used = refs[g] > 0;
        if (used && page >= live) src[h0 + ones_below(high[g])] = (int32_t)page;
        if (!used && page < live) dst[f0 + ones_below(hole[g])] = (int32_t)page;
        to[page] = used ? (int32_t)page : -1;
        refs_out[page] = used ? refs[g] : 0;
      }
      h0 += __popcll(high[g]);
      f0 += __popcll(hole[g]);
    }
    moves += all_high;
    holes += all_free;
  }
  __syncthreads();
  // refs_out holds the old counts of the moved pages (it may be refs itself)
  for (int j = tid; j < moves; j += kPlanThreads) {
    const int32_t a = src[j], b = dst[j];
    to[a] = b;
    refs_out[b] = refs_out[a];
  }
  __syncthreads();
  for (int j = tid; j < moves; j += kPlanThreads) refs_out[src[j]] = 0;
  if (tid == 0) ws[0] = moves;
}

// The first `map` workgroups renumber the table, the others move pages.
__global__ __launch_bounds__(256) void compact_move_kernel(KvCache c, KvPool p,
                                                           int32_t *table_out, const int32_t *ws,
                                                           int64_t map) {
  const int32_t *src = ws + kMoveWords, *dst = src + c.pages, *to = dst + c.pages;
  if (blockIdx.x < map) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < p.rows * p.stride) {
      const int page = p.table[i];
      table_out[i] = page >= 0 && page < c.pages ? to[page] : -1;
    }
    return;
  }
  const int64_t per = 2 * page_pieces(c), units = ws[0] * c.layers * per;
  for (int64_t u = blockIdx.x - map; u < units; u += gridDim.x - map) {
    const int64_t piece = u % per, w = u / per;
    copy_piece(c, w % c.layers, src[w / c.layers], dst[w / c.layers], piece);
  }
}

int64_t entry_groups(const KvPool &p) { return (p.stride + 255) / 256; }

}  // namespace

hipError_t launch_kv_append(const KvCache &c, int64_t layer, const KvBatch &b, const void *k,
                            int64_t k_stride, const void *v, int64_t v_stride, bool f32,
                            hipStream_t s) {
  // n consecutive tokens touch at most (n + 30) / 16 blocks
  const int64_t blocks = ((int64_t)b.max_rows + 2 * kKvBlock - 2) / kKvBlock;
  const int64_t waves = b.seqs * blocks * c.kv_heads * 2;
  const int64_t grid = (waves + 3) / 4;
  if (grid > 0x7FFFFFFF / 256) return hipErrorInvalidConfiguration;
  const Rows x{k, v, k_stride, v_stride};
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(256), 0, s, c, layer, b, x, blocks);
  };
  if (f32) {
    if (c.head_dim == 128) go(append_kernel<true, 128>);
    else go(append_kernel<true, 64>);
  } else {
    if (c.head_dim == 128) go(append_kernel<false, 128>);
    else go(append_kernel<false, 64>);
  }
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache &c, int64_t layer, const KvBatch &b, const KvRows &k,
                          const KvRows &v, hipStream_t s) {
  const int64_t blocks = ((int64_t)b.max_rows + 2 * kKvBlock - 2) / kKvBlock;  // as in an append
  const int64_t waves = b.seqs * blocks * c.kv_heads * 2;
  const int64_t grid = (waves + 3) / 4;
  if (grid > 0x7FFFFFFF / 256) return hipErrorInvalidConfiguration;
  const int64_t size = k.f32 ? 4 : 2;
  const ReadRows y{static_cast<uint8_t *>(k.at), static_cast<uint8_t *>(v.at), k.stride * size,
                   v.stride * size};
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(256), 0, s, c, layer, b, y, blocks);
  };
  if (k.f32) {
    if (c.head_dim == 128) go(read_kernel<true, 128>);
    else go(read_kernel<true, 64>);
  } else {
    if (c.head_dim == 128) go(read_kernel<false, 128>);
    else go(read_kernel<false, 64>);
  }
  return hipGetLastError();
}

hipError_t launch_kv_copy_pages(const KvCache &c, const int32_t *src, const int32_t *dst,
                                int64_t n, hipStream_t s) {
  const int64_t grid = n * c.layers * 2 * page_pieces(c);
  if (grid > 0x7FFFFFFF / 256) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(copy_pages_kernel, dim3((unsigned)grid), dim3(256), 0, s, c, src, dst);
  return hipGetLastError();
}

hipError_t launch_kv_reserve(const KvCache &c, const KvPool &p, const int32_t *add,
                             hipStream_t s) {
  hipLaunchKernelGGL(assign_pages_kernel<ReserveRequests>, dim3(1), dim3(kPlanThreads), 0, s, c, p,
                     ReserveRequests{add});
  return hipGetLastError();
}

hipError_t launch_kv_fork(const KvCache &c, const KvPool &p, const int32_t *src,
                          const int32_t *dst, int64_t n, hipStream_t s) {
  const int64_t copies = n * c.layers * 2 * page_pieces(c), groups = entry_groups(p);
  const int64_t grid = copies + n * groups;
  if (grid > 0x7FFFFFFF / 256) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(assign_pages_kernel<ForkRequests>, dim3(1), dim3(kPlanThreads), 0, s, c, p,
                     ForkRequests{src, dst, n});
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fork_kernel, dim3((unsigned)grid), dim3(256), 0, s, c, p, src, dst, copies,
                     groups);
  return hipGetLastError();
}

hipError_t launch_kv_release(const KvCache &c, const KvPool &p, const int32_t *rows, int64_t n,
                             hipStream_t s) {
  const int64_t groups = entry_groups(p), grid = n * groups;
  if (grid > 0x7FFFFFFF / 256) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(release_kernel, dim3((unsigned)grid), dim3(256), 0, s, c, p, rows, groups);
  return hipGetLastError();
}

size_t kv_compact_workspace_bytes(const KvCache &c) {
  return (kMoveWords + 3 * (size_t)c.pages) * sizeof(int32_t);
}

hipError_t launch_kv_compact(const KvCache &c, const KvPool &p, int32_t *refs_out,
                             int32_t *table_out, void *ws, hipStream_t s) {
  int32_t *w = static_cast<int32_t *>(ws);
  const int64_t map = (p.rows * p.stride + 255) / 256;
  // the number of moves is known on the device only: enough workgroups to
  // fill it, each taking pieces in turn
  const int64_t most = c.pages / 2 * c.layers * 2 * page_pieces(c);
  const int64_t movers = most < 1 ? 1 : most > 4096 ? 4096 : most;
  if (map + movers > 0x7FFFFFFF / 256) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, c, p, refs_out, w);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(compact_move_kernel, dim3((unsigned)(map + movers)), dim3(256), 0, s, c, p,
                     table_out, w, map);
  return hipGetLastError();
}

}  // namespace nf4
