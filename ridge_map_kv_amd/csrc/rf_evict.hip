// Eviction from the paged cache by accumulated weight, on gfx950.
//
// Two launches.  The first, one workgroup per sequence, picks the kept rows and lists the
// moves; the second copies them in every pool.  Rows are kept by a 32-bit key (the weight's
// bits in unsigned order, all ones for a protected row, 0 for a NaN), the n_keep-th largest
// found by a radix select of 8 bits a pass; of the rows at that key the lowest are kept.  The
// keys stay in LDS (up to 32,768 rows; in registers they, and the votes that the compiler kept
// with them, spilled), and there are sixteen histograms side by side: weights share most of
// their leading bits, so in one all lanes would count in the same few words, one after another.
//
// A kept row below n_keep stays where it is and a kept row above moves into a free row below:
// the sources (>= n_keep) and the destinations (< n_keep) are disjoint, so rows move in place
// and in parallel, and only k (1 - k/n) of the k kept rows move (of n, evenly spread), 64 of
// 4096 where 64 new rows have been appended, while closing the gaps in order would move nearly
// all of them.
// What the first launch is bound by is one compute unit's instructions, so it leaves the second,
// which has the whole chip, the looking up of pages and the moved rows' weights and positions.
// 8 sequences of 4,160 rows cut to 4,096, 4 layers: 14 + 6 us (with the lookups in the first
// launch 19 + 6); one of 32,768 cut to 16,384: 32 + 61 us (57 + 65), the moving of 8,192 rows at
// 4.4 TB/s.  Of the 32 us 6 go to reading weights and positions, 10 to the radix select.  65,536 cut to
// 32,768, keys formed anew in each pass: 98 + 115 us.
#include "rf_cache_dev.h"

namespace rf {

namespace {

constexpr int kSel = 1024;      // threads of the selecting workgroup
constexpr int kWaves = kSel / 64;

struct __attribute__((aligned(16))) MoveRow {
  int from, to;
  float weight;
  int pos;
};
struct EvictHead {              // of a sequence
  int moves, err, old_len;      // old_len: 0 where nothing is cut
};

// Workspace: status; per sequence its head; per sequence the moving rows.
struct EvictWs {
  size_t head, rows, total;
  int64_t most;                 // moves of one sequence at most
};
EvictWs evict_ws(const Batch& b, int n_keep) {
  EvictWs w;
  const int64_t over = b.max_len > n_keep ? b.max_len - n_keep : 0;
  w.most = over < n_keep ? over : n_keep;
  w.head = kStatusBytes;
  w.rows = w.head + align256((size_t)b.batch * sizeof(EvictHead));
  w.total = w.rows + align256((size_t)b.batch * w.most * sizeof(MoveRow));
  return w;
}

__device__ __forceinline__ uint32_t weight_order(float s) {
  uint32_t u = __float_as_uint(s);
  if (s != s) return 0u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kCopies = 16;     // histograms, one to two banks
constexpr int kRun = 33;        // most rows in a row that a thread takes where their order counts
constexpr int kMostPer = 512;   // moves of a copying workgroup: 1,024 pieces of rows of two or more
constexpr int kHeldRows = (kRun - 1) * kSel;    // rows that LDS holds at a time

// Inclusive prefix sum over the wave, by row shifts and broadcasts in registers.
__device__ __forceinline__ int wave_scan(int v) {
#define RF_ADD(ctrl, rows) v += __builtin_amdgcn_update_dpp(0, v, ctrl, rows, 0xf, false)
  RF_ADD(0x111, 0xf);            // one, two, four, eight lanes to the right in rows of 16
  RF_ADD(0x112, 0xf);
  RF_ADD(0x114, 0xf);
  RF_ADD(0x118, 0xf);
  RF_ADD(0x142, 0xa);            // a row's last lane to the next row, then the first half's to the second
  RF_ADD(0x143, 0xc);
#undef RF_ADD
  return v;
}

// Sum of v over the threads before this one; the sum over all in *all.  part: [kWaves] in LDS.
__device__ __forceinline__ int block_before(int v, int* part, int* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int upto = wave_scan(v);
  if (lane == 63) part[wave] = upto;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += part[w];
    sum += part[w];
  }
  __syncthreads();
  *all = sum;
  return before + upto - v;
}

// kHold: the keys of all rows lie in LDS (max_len <= kHeldRows); else they are formed anew in each
// pass, and LDS holds those of 32,768 rows at a time where their order counts.
template <bool kHold>
__global__ __launch_bounds__(kSel) void evict_select_kernel(Batch b, EvictCall c, EvictHead* head,
                                                            MoveRow* rows, int64_t most,
                                                            unsigned* status) {
  extern __shared__ uint32_t held[];            // keys, then the lists of free and of moving rows
  __shared__ unsigned hist[256 * kCopies], digits[256];
  __shared__ int red[kWaves];
  __shared__ unsigned sh_digit, sh_need, sh_all;
  const int seq = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int len = b.lengths[seq];
  if (seq == 0 && tid == 0) *status = 0u;       // the second launch adds the errors
  if (len < 0 || len > b.max_len) {
    if (tid == 0) head[seq] = {0, (int)kStatusRowsBit, 0};
    return;
  }
  const float* acc = c.acc + seq * c.stride;
  const int32_t* pos = c.pos + seq * c.stride;
  float* acc_out = c.acc_out + seq * c.stride;
  int32_t* pos_out = c.pos_out + seq * c.stride;
  const int keep = c.n_keep;
  int err = 0;

  // Thread tid looks after rows tid, tid + 1024, ..: chunk i's is 1024 i + tid.  Values are fetched
  // eight chunks at a time, or each chunk would wait for its own (sixteen: longer code, which is fetched
  // once for each launch: 15.4 instead of 14.4 us for 4,160 rows, no gain for 32,768).
  const int chunks = (len + kSel - 1) / kSel;
  constexpr int kFetch = 8;
  const auto batches = [&](int to, auto fetch, auto body) {             // body(i, fetch(i))
    for (int i0 = 0; i0 < to; i0 += kFetch) {
      decltype(fetch(0)) v[kFetch];
#pragma unroll
      for (int j = 0; j < kFetch; ++j)
        if (i0 + (j & ~3) < to) v[j] = fetch(i0 + j);
#pragma unroll
      for (int j = 0; j < kFetch; ++j)
        if (i0 + j < to) body(i0 + j, v[j]);
    }
  };
  struct Row {
    float w;
    int p;
  };
  const auto at = [&](int i) { return i * kSel + tid < len ? i * kSel + tid : len - 1; };   // len > 0
  const auto row_at = [&](int i) -> Row { return {acc[at(i)], pos[at(i)]}; };
  const auto copy_rows = [&](int n) {           // rows that stay, unless they are there already
    if (acc_out == acc && pos_out == pos) return;
    batches((n + kSel - 1) / kSel, row_at, [&](int i, const Row& r) {
      if (i * kSel + tid >= n) return;
      acc_out[i * kSel + tid] = r.w;
      pos_out[i * kSel + tid] = r.p;
    });
  };
  int top = INT32_MIN, bottom = INT32_MAX;
  batches(chunks, row_at, [&](int i, const Row& r) {
    top = max(top, r.p);
    bottom = min(bottom, r.p);
    if (r.w != r.w) err = 1;
    if constexpr (kHold) held[i * kSel + tid] = i * kSel + tid < len ? weight_order(r.w) : 0u;
  });
  // whole eights of chunks: keys of 0, the lowest, after the last row change nothing below
  if constexpr (kHold)
    for (int i = chunks; i & 7; ++i) held[i * kSel + tid] = 0u;
  for (int x = tid; x < 256 * kCopies; x += kSel) hist[x] = 0u;
#pragma unroll
  for (int d = 32; d; d >>= 1) top = max(top, __shfl_xor(top, d));
#pragma unroll
  for (int d = 32; d; d >>= 1) bottom = min(bottom, __shfl_xor(bottom, d));
  const int wave_top = top;
  if (lane == 0) red[wave] = top;
  err = __syncthreads_or(err) ? (int)kStatusScoreBit : 0;
  for (int w = 0; w < kWaves; ++w) top = max(top, red[w]);

  if (len <= keep) {                                // nothing to cut
    copy_rows(len);
    if (tid == 0) {
      c.len_out[seq] = len;
      head[seq] = {0, err, 0};
    }
    return;
  }

  const int64_t newest = (int64_t)top - c.n_recent;   // protected above this position
  const auto safe = [&](int p) { return p < c.n_sink || p > newest; };
  if constexpr (kHold)
    if (safe(bottom) || safe(wave_top))             // few waves have a protected row
      batches(chunks, [&](int i) { return pos[at(i)]; },
              [&](int i, int p) {
                if (i * kSel + tid < len && safe(p)) held[i * kSel + tid] = 0xffffffffu;
              });
  const auto key_of = [&](const Row& r) { return safe(r.p) ? 0xffffffffu : weight_order(r.w); };
  // the keep-th largest key, digit by digit; `need` of the rows at it are kept.  Where all rows of a
  // digit are needed the digits after it are not (after three of them that is nearly always so).
  uint32_t prefix = 0u, mask = 0u;
  unsigned need = (unsigned)keep;
  for (int shift = 24; keep > 0 && shift >= 0; shift -= 8) {
    const auto count = [&](uint32_t k) {
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift & 0xffu) * kCopies + lane % kCopies], 1u);
    };
    if constexpr (kHold) {                          // a thread reads its own entries
      for (int i0 = 0; i0 < chunks; i0 += 8) {
        uint32_t k[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) k[j] = held[(i0 + j) * kSel + tid];
#pragma unroll
        for (int j = 0; j < 8; ++j) count(k[j]);
      }
    } else {
      batches(chunks, row_at, [&](int i, const Row& r) {
        if (i * kSel + tid < len) count(key_of(r));
      });
    }
    __syncthreads();
    // four lanes a digit add up its copies, each starting at another bank, and clear them
    unsigned part = 0u;
#pragma unroll
    for (int x = 0; x < kCopies / 4; ++x) {
      unsigned* h = hist + (tid >> 2) * kCopies + (tid & 3) * (kCopies / 4) + ((x + (tid >> 3)) & (kCopies / 4 - 1));
      part += *h;
      *h = 0u;
    }
    part += __shfl_xor(part, 1);
    part += __shfl_xor(part, 2);
    if ((tid & 3) == 0) digits[tid >> 2] = part;
    __syncthreads();
    if (wave == 0) {                                // lane l: digits 255-4l down to 252-4l
      unsigned v[4], s = 0u;
      for (int i = 0; i < 4; ++i) s += v[i] = digits[255 - 4 * lane - i];
      const unsigned run = (unsigned)wave_scan((int)s);
      unsigned above = run - s;                     // keys with a larger digit
      for (int i = 0; i < 4; ++i) {
        if (above < need && need <= above + v[i]) {
          sh_digit = 255u - 4u * lane - i;
          sh_need = need - above;
          sh_all = need - above == v[i];
        }
        above += v[i];
      }
    }
    __syncthreads();
    prefix |= sh_digit << shift;
    mask |= 0xffu << shift;
    need = sh_need;
    if (sh_all) {                                   // all from `prefix` on: those above prefix - 1, which
      --prefix;                                     // is not below 0, or all rows would be kept
      need = 0u;
      break;
    }
  }

  // In order: which rows are kept, the free rows below keep, the kept rows from keep on.  A thread
  // takes up to 33 rows in a row (an odd number: no two of 64 runs begin at one bank), a bit each, so
  // that counts of bits and scans over the threads rank them; the free rows replace the keys from
  // the first on, the moving ones from the last on back, and go from there to the list side by side.
  MoveRow* list = rows + seq * most;
  int ties = 0, holes = 0, movers = 0;                // of the rows before these
  for (int t0 = 0; t0 < len; t0 += kHeldRows) {
    const int here = len - t0 < kHeldRows ? len - t0 : kHeldRows, deal = (here + kSel - 1) / kSel;
    const int size = deal | 1;
    if constexpr (!kHold)
      for (int i0 = 0; i0 < deal; i0 += 8) {
        Row r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = row_at(t0 / kSel + i0 + j);
#pragma unroll
        for (int j = 0; j < 8; ++j) held[(i0 + j) * kSel + tid] = key_of(r[j]);
      }
    __syncthreads();
    const int run0 = tid * size, n = here - run0 < 0 ? 0 : here - run0 < size ? here - run0 : size;
    const uint32_t* run = held + (n ? run0 : 0);
    const uint64_t valid = (1ull << n) - 1;
    uint64_t larger = 0, equal = 0;
    if (keep > 0 && n)
      for (int j0 = 0; j0 < size; j0 += 8) {          // past the run: other rows' words, not used
        uint32_t gt = 0u, eq = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t k = run[j0 + j];
          gt |= k > prefix ? 1u << j : 0u;
          eq |= k == prefix ? 1u << j : 0u;
        }
        larger |= (uint64_t)gt << j0;
        equal |= (uint64_t)eq << j0;
      }
    equal &= valid;
    int all;
    const int rank = ties + block_before(__popcll(equal), red, &all);
    ties += all;
    // of the rows at the key itself the lowest: those past `need` are dropped from the end
    for (int drop = __popcll(equal) - ((int)need - rank < 0 ? 0 : (int)need - rank); drop > 0 && equal; --drop)
      equal &= ~(1ull << (63 - __clzll((long long)equal)));
    const uint64_t kept = (larger & valid) | equal;
    const int under = keep - (t0 + run0);             // of the run, the rows below keep
    const uint64_t low = under >= n ? valid : under <= 0 ? 0ull : (1ull << under) - 1;
    uint64_t open = low & ~kept, moving = kept & ~low;
    int new_holes, new_movers;
    uint32_t* hole = held + block_before(__popcll(open), red, &new_holes);
    uint32_t* mover = held + here - 1 - block_before(__popcll(moving), red, &new_movers);
    for (; open; open &= open - 1) *hole++ = (uint32_t)(t0 + run0 + __ffsll((unsigned long long)open) - 1);
    for (; moving; moving &= moving - 1) *mover-- = (uint32_t)(t0 + run0 + __ffsll((unsigned long long)moving) - 1);
    __syncthreads();
    if constexpr (!kHold)                             // else as many as rows that move: with those
      for (int x = tid; x < new_holes; x += kSel) list[holes + x].to = (int)held[x];
    for (int x0 = tid; x0 < new_movers; x0 += 8 * kSel) {   // eight at a time
      MoveRow r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int x = x0 + j * kSel < new_movers ? x0 + j * kSel : x0;
        r[j].from = (int)held[here - 1 - x];
        if constexpr (kHold) r[j].to = (int)held[x];
        r[j].weight = acc[r[j].from];
        r[j].pos = pos[r[j].from];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (x0 + j * kSel < new_movers) {
          MoveRow* m = list + movers + x0 + j * kSel;
          if constexpr (kHold) {
            *m = r[j];
          } else {
            m->from = r[j].from;
            m->weight = r[j].weight;
            m->pos = r[j].pos;
          }
        }
    }
    holes += new_holes;
    movers += new_movers;
    __syncthreads();                                  // LDS is written again
  }
  copy_rows(keep);
  if (tid == 0) {
    c.len_out[seq] = keep;
    head[seq] = {movers, err, len};
  }
}

// blockIdx.x: `per` of a sequence's moves, y: pool, z: sequence.  A row is n_kv * hd bf16
// values in one piece, row16 pieces of 16 bytes; a thread has up to four of them under way.
// With `status` the first y is none of the pools but the rows' weights and positions (weights of
// 0 from keep on) and, of its first workgroup, the errors.
__global__ __launch_bounds__(256) void evict_move_kernel(EvictPools pools, Batch b, EvictCall c,
                                                         const EvictHead* head, const MoveRow* rows,
                                                         int64_t most, int per, int row16,
                                                         Divide by_row, Divide by_page,
                                                         unsigned* status) {
  __shared__ int2 sh_move[kMostPer];
  const int seq = blockIdx.z;
  const MoveRow* list = rows + seq * most;
  const auto slot_of = [&](int t) -> int {
    const int pi = (int)quotient((unsigned)t, by_page), page = b.tables[(int64_t)seq * b.table_stride + pi];
    return page < 0 || page >= b.num_pages ? -1 : page * b.page_size + (t - pi * b.page_size);
  };
  const EvictHead h = head[seq];
  if (status && blockIdx.y == 0) {
    float* acc_out = c.acc_out + seq * c.stride;
    int32_t* pos_out = c.pos_out + seq * c.stride;
    const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    bool bad = false;
    for (int64_t i = first; i < h.moves; i += step) {
      const MoveRow r = list[i];
      if (slot_of(r.from) < 0 || slot_of(r.to) < 0) {     // no pool moves it: the place keeps its own
        bad = true;
        continue;
      }
      acc_out[r.to] = r.weight;
      pos_out[r.to] = r.pos;
    }
    for (int64_t t = c.n_keep + first; t < h.old_len; t += step) acc_out[t] = 0.f;
    const unsigned bits = (blockIdx.x == 0 ? (unsigned)h.err : 0u) | (__any(bad) ? kStatusRowsBit : 0u);
    if (bits && (threadIdx.x & 63) == 0) atomicOr(status, bits);
    return;
  }
  const int64_t first = (int64_t)blockIdx.x * per, left = h.moves - first;
  if (left <= 0) return;
  const int n = (int)(left < per ? left : per), total = n * row16;
  for (int i = threadIdx.x; i < n; i += 256) {
    const MoveRow r = list[first + i];
    const int2 m = make_int2(slot_of(r.from), slot_of(r.to));
    sh_move[i] = m.x < 0 || m.y < 0 ? make_int2(-1, -1) : m;
  }
  __syncthreads();
  u32x4* p = reinterpret_cast<u32x4*>(pools.p[blockIdx.y - (status ? 1 : 0)]);
  for (int i0 = threadIdx.x; i0 < total; i0 += 1024) {
    u32x4 v[4];
    int64_t to[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 256 * j;
      to[j] = -1;
      if (i < total) {
        const int m = (int)quotient((unsigned)i, by_row), e = i - m * row16;
        const int2 w = sh_move[m];
        if (w.x >= 0) {
          v[j] = p[(int64_t)w.x * row16 + e];
          to[j] = (int64_t)w.y * row16 + e;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (to[j] >= 0) p[to[j]] = v[j];
  }
}

}  // namespace

size_t evict_workspace(const Batch& b, int n_keep) { return evict_ws(b, n_keep).total; }

hipError_t launch_evict(const Batch& b, const EvictCall& c, uint16_t* const* pools, int n_pools,
                        void* ws, hipStream_t stream) {
  const EvictWs w = evict_ws(b, c.n_keep);
  unsigned char* p = static_cast<unsigned char*>(ws);
  unsigned* status = reinterpret_cast<unsigned*>(p);
  EvictHead* head = reinterpret_cast<EvictHead*>(p + w.head);
  MoveRow* rows = reinterpret_cast<MoveRow*>(p + w.rows);
  const bool hold = b.max_len <= kHeldRows;
  const int deal = hold ? (b.max_len + 8 * kSel - 1) / (8 * kSel) * 8 : kHeldRows / kSel;
  const size_t lds = ((size_t)deal * kSel + kRun + 7) * 4;   // runs are read eight words at a time
  if (lds > 32768) {                                  // beyond what a launch gets unasked
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void*>(hold ? evict_select_kernel<true> : evict_select_kernel<false>),
        hipFuncAttributeMaxDynamicSharedMemorySize, (kHeldRows + kRun + 7) * 4);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(hold ? evict_select_kernel<true> : evict_select_kernel<false>, dim3(b.batch), dim3(kSel),
                     lds, stream, b, c, head, rows, w.most, status);
  const int row16 = b.n_kv * b.hd / 8;
  int per = row16 < 1024 ? 1024 / row16 : 1;
  if (w.most / per > 1 << 22) per = (int)(w.most >> 22) + 1;    // within a grid's threads
  const unsigned blocks = w.most > 0 ? (unsigned)((w.most + per - 1) / per) : 1u;
  for (int first = 0; first == 0 || first < n_pools; first += kEvictPools) {
    EvictPools e = {};
    const int n = n_pools - first < kEvictPools ? n_pools - first : kEvictPools;
    for (int i = 0; i < n; ++i) e.p[i] = pools[first + i];
    hipLaunchKernelGGL(evict_move_kernel, dim3(blocks, n + (first == 0 ? 1 : 0), b.batch), dim3(256), 0, stream,
                       e, b, c, head, rows, w.most, per, row16, divide_by((unsigned)row16),
                       divide_by((unsigned)b.page_size), first == 0 ? status : nullptr);
  }
  return hipGetLastError();
}

}  // namespace rf
