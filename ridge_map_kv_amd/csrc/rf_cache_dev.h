// Device helpers shared by the kernels that read the paged cache.
#pragma once

#include "rf_cache.h"
#include "rf_common.h"

namespace rf {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Division of 0 .. 2^31 - 1 by a divisor known on the host: (mulhi(x, m) + x) >> s.
struct Divide {
  unsigned m, s, d;
};
inline Divide divide_by(unsigned d) {
  Divide v{0u, 0u, d};
  while ((1ull << v.s) < d) ++v.s;
  v.m = (unsigned)((((1ull << v.s) - d) << 32) / d + 1);
  return v;
}
__device__ __forceinline__ unsigned quotient(unsigned x, Divide v) {
  return (__umulhi(x, v.m) + x) >> v.s;
}

// Sequence `seq`: its length, first query and number of queries; false if it is to be skipped
// (with *bad set where that is an error).
__device__ __forceinline__ bool sequence_of(const Batch& b, const Queries& q, int seq, int* len,
                                            int* first, int* n, bool* bad) {
  *len = b.lengths[seq];
  *first = q.start[seq];
  const int end = q.start[seq + 1];
  *n = (int)((unsigned)end - (unsigned)*first);
  *bad = *len < 0 || *len > b.max_len || *first < 0 || end < *first || *n > q.max_q || *n > *len ||
         end > q.n_q;
  return !*bad && *n > 0;
}

// What a query sees of its sequence's drafts, a bit each: its word of the mask, or a chain.
__device__ __forceinline__ uint64_t draft_word(const Queries& q, int query, int i) {
  return q.mask ? q.mask[query] : i < 63 ? (2ull << i) - 1 : ~0ull;
}

// Which of the 32 cache rows from `base` on a query sees; d = base less the row of the first
// draft, > -32.
__device__ __forceinline__ uint32_t seen_rows(uint64_t word, int d) {
  if (d >= 0) return d < 64 ? (uint32_t)(word >> d) : 0u;
  return (uint32_t)(word << -d) | ((1u << -d) - 1u);
}

// What a query sees of the 64 cache rows from `base` on, d = base less the first draft's row.
__device__ __forceinline__ uint64_t seen64(uint64_t word, int d) {
  if (d >= 0) return d < 64 ? word >> d : 0ull;
  return d <= -64 ? ~0ull : word << -d | ((1ull << -d) - 1ull);
}

// The status word from one workgroup: every sequence and every page that it uses, eight lookups
// of a thread at a time.
__device__ inline void scan_status(const Batch& b, const Queries& q, unsigned* status) {
  const int each = (b.max_len - 1) / b.page_size + 1, total = b.batch * each;
  int bits = 0;
  for (int i0 = threadIdx.x; i0 < total; i0 += 8 * blockDim.x) {
    bool wrong[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * (int)blockDim.x < total ? i0 + j * (int)blockDim.x : i0;
      const int s = i / each, p = i - s * each;
      int len, first, n;
      bool bad;
      const bool go = sequence_of(b, q, s, &len, &first, &n, &bad);
      const int page = b.tables[(int64_t)s * b.table_stride + p];
      wrong[j] = bad || (go && (int64_t)p * b.page_size < len && (page < 0 || page >= b.num_pages));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) bits |= wrong[j];
  }
  bits = __syncthreads_or(bits);
  if (threadIdx.x == 0) *status = bits ? kStatusRowsBit : 0u;
}

// Of a call of one launch, the status word is written by a workgroup that scans the tables beside
// the others where that takes no longer than they do (4,096 entries: two rounds of lookups); else it
// is cleared first and the workgroups report what they meet.
inline bool scans(const Batch& b) {
  return (int64_t)b.batch * ((b.max_len - 1) / b.page_size + 1) <= 4096;
}

// A call of two launches clears the status in the first, and workgroups of the second add to it, part
// `part` of `parts` of a sequence's pages each: a workgroup that scans in the first would keep one
// that needs a whole compute unit waiting (weights of 32,768 rows: 37.4 instead of 35.4 us; trees on 4
// sequences with a clearing launch instead: 168 instead of 164 us, caches cold).
__device__ inline void scan_sequence(const Batch& b, const Queries& q, int seq, int part, int parts,
                                     unsigned* status) {
  int len, first, n;
  bool bad;
  const bool go = sequence_of(b, q, seq, &len, &first, &n, &bad);
  const int pages = go ? (len - 1) / b.page_size + 1 : 0, step = blockDim.x;
  const int32_t* table = b.tables + (int64_t)seq * b.table_stride;
  int bits = bad;
  for (int64_t i0 = (int64_t)part * 8 * step + threadIdx.x; i0 < pages; i0 += (int64_t)parts * 8 * step) {
    int page[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) page[j] = table[i0 + j * step < pages ? i0 + j * step : i0];
#pragma unroll
    for (int j = 0; j < 8; ++j) bits |= page[j] < 0 || page[j] >= b.num_pages;
  }
  bits = __syncthreads_or(bits);
  if (bits && threadIdx.x == 0) atomicOr(status, kStatusRowsBit);
}

// How many workgroups scan a sequence: one for 4,096 pages (two rounds of lookups), sixteen at most.
inline int scan_parts(const Batch& b) {
  const int pages = (b.max_len - 1) / b.page_size + 1;
  return pages > 16 * 4096 ? 16 : (pages + 4095) / 4096;
}

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

}  // namespace rf
