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
#include "rf_cache_dev.h"

namespace rf {

namespace {

constexpr int kSel = 1024;      // threads of the selecting workgroup
constexpr int kWaves = kSel / 64;

// Workspace: status; per sequence {moves, error bits}; per sequence the list of moves as pool
// slots {from, to} and, before that, the moving rows' {from, to, weight, position}.
struct EvictWs {
  size_t head, moves, rows, total;
  int64_t most;                 // moves of one sequence at most
};
EvictWs evict_ws(const Batch& b, int n_keep) {
  EvictWs w;
  const int64_t over = b.max_len > n_keep ? b.max_len - n_keep : 0;
  w.most = over < n_keep ? over : n_keep;
  w.head = kStatusBytes;
  w.moves = w.head + align256((size_t)b.batch * 8);
  w.rows = w.moves + align256((size_t)b.batch * w.most * 8);
  w.total = w.rows + align256((size_t)b.batch * w.most * 16);
  return w;
}

__device__ __forceinline__ uint32_t weight_order(float s) {
  uint32_t u = __float_as_uint(s);
  if (s != s) return 0u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct MoveRow {
  int from, to;
  float weight;
  int pos;
};

constexpr int kCopies = 16;     // histograms, one to two banks
constexpr int kRun = 33;        // most rows in a row that a thread takes where their order counts
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
__global__ __launch_bounds__(kSel) void evict_select_kernel(Batch b, EvictCall c, int2* head,
                                                            int2* moves, MoveRow* mrows,
                                                            int64_t most, Divide by_page) {
  extern __shared__ uint32_t held[];            // keys, then what becomes of the rows: [whole runs]
  __shared__ unsigned hist[256 * kCopies];
  __shared__ int red[kWaves];
  __shared__ unsigned sh_digit, sh_need;
  const int seq = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int len = b.lengths[seq];
  if (len < 0 || len > b.max_len) {
    if (tid == 0) head[seq] = make_int2(0, (int)kStatusRowsBit);
    return;
  }
  const float* acc = c.acc + seq * c.stride;
  const int32_t* pos = c.pos + seq * c.stride;
  float* acc_out = c.acc_out + seq * c.stride;
  int32_t* pos_out = c.pos_out + seq * c.stride;
  const int keep = c.n_keep;
  int err = 0;

  // Thread tid looks after rows tid, tid + 1024, ..: chunk i's is 1024 i + tid.  Values are fetched
  // eight chunks at a time, or each chunk would wait for its own.
  const int chunks = (len + kSel - 1) / kSel;
  const auto batches = [&](int from, int to, auto fetch, auto body) {   // body(i, fetch(i))
    for (int i0 = from; i0 < to; i0 += 8) {
      decltype(fetch(0)) v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = fetch(i0 + j);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + j < to) body(i0 + j, v[j]);
    }
  };
  struct Row {
    float w;
    int p;
  };
  const auto row_at = [&](int i) -> Row {             // past the end: the last row (len > 0)
    const int t = i * kSel + tid < len ? i * kSel + tid : len - 1;
    return {acc[t], pos[t]};
  };
  int top = INT32_MIN;
  batches(0, chunks, row_at, [&](int i, const Row& r) {
    top = max(top, r.p);
    if (r.w != r.w) err = 1;
    if constexpr (kHold) held[i * kSel + tid] = i * kSel + tid < len ? weight_order(r.w) : 0u;
  });
#pragma unroll
  for (int d = 32; d; d >>= 1) top = max(top, __shfl_xor(top, d));
  if (lane == 0) red[wave] = top;
  err = __syncthreads_or(err) ? (int)kStatusScoreBit : 0;
  for (int w = 0; w < kWaves; ++w) top = max(top, red[w]);

  if (len <= keep) {                                // nothing to cut
    batches(0, chunks, row_at, [&](int i, const Row& r) {
      const int t = i * kSel + tid;
      if (t < len) {
        acc_out[t] = r.w;
        pos_out[t] = r.p;
      }
    });
    if (tid == 0) {
      c.len_out[seq] = len;
      head[seq] = make_int2(0, err);
    }
    return;
  }

  const int64_t newest = (int64_t)top - c.n_recent;   // protected above this position
  const auto safe = [&](int p) { return p < c.n_sink || p > newest; };
  if constexpr (kHold)
    batches(0, chunks, [&](int i) { return pos[i * kSel + tid < len ? i * kSel + tid : len - 1]; },
            [&](int i, int p) {
              if (i * kSel + tid < len && safe(p)) held[i * kSel + tid] = 0xffffffffu;
            });
  const auto key_at = [&](int i) -> uint32_t {        // a thread reads its own entries only
    if constexpr (kHold) return held[(i < chunks ? i : chunks - 1) * kSel + tid];
    const Row r = row_at(i);
    return safe(r.p) ? 0xffffffffu : weight_order(r.w);
  };
  // the keep-th largest key, digit by digit; `need` of the rows at it are kept
  uint32_t prefix = 0u, mask = 0u;
  unsigned need = (unsigned)keep;
  for (int shift = 24; keep > 0 && shift >= 0; shift -= 8) {
    for (int x = tid; x < 256 * kCopies; x += kSel) hist[x] = 0u;
    __syncthreads();
    batches(0, chunks, key_at, [&](int i, uint32_t k) {
      if (i * kSel + tid < len && (k & mask) == prefix)
        atomicAdd(&hist[(k >> shift & 0xffu) * kCopies + lane % kCopies], 1u);
    });
    __syncthreads();
    // four lanes a digit add up its copies, each starting at another bank
    unsigned part = 0u;
#pragma unroll
    for (int x = 0; x < kCopies / 4; ++x)
      part += hist[(tid >> 2) * kCopies + (tid & 3) * (kCopies / 4) + ((x + (tid >> 3)) & (kCopies / 4 - 1))];
    part += __shfl_xor(part, 1);
    part += __shfl_xor(part, 2);
    __syncthreads();
    if ((tid & 3) == 0) hist[tid >> 2] = part;
    __syncthreads();
    if (wave == 0) {                                // lane l: digits 255-4l down to 252-4l
      unsigned v[4], s = 0u;
      for (int i = 0; i < 4; ++i) s += v[i] = hist[255 - 4 * lane - i];
      const unsigned run = (unsigned)wave_scan((int)s);
      unsigned above = run - s;                     // keys with a larger digit
      for (int i = 0; i < 4; ++i) {
        if (above < need && need <= above + v[i]) {
          sh_digit = 255u - 4u * lane - i;
          sh_need = need - above;
        }
        above += v[i];
      }
    }
    __syncthreads();
    prefix |= sh_digit << shift;
    mask |= 0xffu << shift;
    need = sh_need;
  }

  // In order: which rows are kept, the free rows below keep, the kept rows from keep on.  A thread
  // takes up to 33 rows in a row (an odd number: no two of 64 runs begin at one bank), a bit each, so
  // that counts of bits and scans over the threads rank them; what becomes of a row replaces its
  // key, and is done with the rows dealt out as before.
  constexpr uint32_t kStays = 0u, kFree = 1u, kMoves = 2u, kCut = 3u;   // in the top two bits; the rank below
  MoveRow* list = mrows + seq * most;
  int ties = 0, holes = 0, movers = 0;                // of the rows before these
  for (int t0 = 0; t0 < len; t0 += kHeldRows) {
    const int here = len - t0 < kHeldRows ? len - t0 : kHeldRows, deal = (here + kSel - 1) / kSel;
    const int c0 = t0 / kSel, size = deal | 1;
    if constexpr (!kHold)
      batches(c0, c0 + deal, key_at, [&](int i, uint32_t k) { held[(i - c0) * kSel + tid] = k; });
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
    int hole = holes + block_before(__popcll(low & ~kept), red, &all);
    holes += all;
    int mover = movers + block_before(__popcll(kept & ~low), red, &all);
    movers += all;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const bool is = kept >> j & 1, lo = low >> j & 1;
      held[run0 + j] = is ? lo ? kStays << 30 : kMoves << 30 | (uint32_t)mover : lo ? kFree << 30 | (uint32_t)hole : kCut << 30;
      hole += lo && !is;
      mover += !lo && is;
    }
    __syncthreads();
    batches(c0, c0 + deal, row_at, [&](int i, const Row& r) {
      const int t = i * kSel + tid;
      if (t >= len) return;
      const uint32_t x = held[t - t0], what = x >> 30, at = x & 0x3fffffffu;
      if (what == kFree) list[at].to = t;
      if (what == kMoves) {
        list[at].from = t;
        list[at].weight = r.w;
        list[at].pos = r.p;
      }
      if (what == kStays) {
        acc_out[t] = r.w;
        pos_out[t] = r.p;
      }
      if (t >= keep) acc_out[t] = 0.f;
    });
    __syncthreads();                                  // LDS is written again; the list is whole
  }
  const auto slot_of = [&](int t) -> int {
    const int pi = (int)quotient((unsigned)t, by_page), page = b.tables[(int64_t)seq * b.table_stride + pi];
    return page < 0 || page >= b.num_pages ? -1 : page * b.page_size + (t - pi * b.page_size);
  };
  int bad = 0;
#pragma unroll 1
  for (int i0 = tid; i0 < movers; i0 += 8 * kSel) {   // eight at a time
    MoveRow r[8];
    int2 m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = list[i0 + j * kSel < movers ? i0 + j * kSel : i0];
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = make_int2(slot_of(r[j].from), slot_of(r[j].to));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * kSel;
      if (i >= movers) continue;
      acc_out[r[j].to] = r[j].weight;
      pos_out[r[j].to] = r[j].pos;
      if (m[j].x < 0 || m[j].y < 0) {
        bad = 1;
        m[j] = make_int2(-1, -1);
      }
      moves[seq * most + i] = m[j];
    }
  }
  bad = __syncthreads_or(bad);
  if (tid == 0) {
    c.len_out[seq] = keep;
    head[seq] = make_int2(movers, err | (bad ? (int)kStatusRowsBit : 0));
  }
}

// blockIdx.x: `per` of a sequence's moves, y: pool, z: sequence.  A row is n_kv * hd bf16
// values in one piece, row16 pieces of 16 bytes; a thread has up to four of them under way.
__global__ __launch_bounds__(256) void evict_move_kernel(EvictPools pools, const int2* head,
                                                         const int2* moves, int64_t most, int per,
                                                         int row16, Divide by_row, int batch,
                                                         unsigned* status) {
  if (status && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
    int bits = 0;
    for (int s = threadIdx.x; s < batch; s += 256) bits |= head[s].y;
    const int rows = __syncthreads_or(bits & (int)kStatusRowsBit);
    const int nan = __syncthreads_or(bits & (int)kStatusScoreBit);
    if (threadIdx.x == 0) *status = (rows ? kStatusRowsBit : 0u) | (nan ? kStatusScoreBit : 0u);
  }
  const int64_t first = (int64_t)blockIdx.x * per;
  const int64_t left = head[blockIdx.z].x - first;
  if (left <= 0) return;
  const int total = (int)(left < per ? left : per) * row16;
  const int2* mv = moves + blockIdx.z * most + first;
  u32x4* p = reinterpret_cast<u32x4*>(pools.p[blockIdx.y]);
  for (int i0 = threadIdx.x; i0 < total; i0 += 1024) {
    u32x4 v[4];
    int64_t to[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 256 * j;
      to[j] = -1;
      if (i < total) {
        const int m = (int)quotient((unsigned)i, by_row), e = i - m * row16;
        const int2 w = mv[m];
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
  int2* head = reinterpret_cast<int2*>(p + w.head);
  int2* moves = reinterpret_cast<int2*>(p + w.moves);
  const bool hold = b.max_len <= kHeldRows;
  const int deal = hold ? (b.max_len + kSel - 1) / kSel : kRun - 1;
  const size_t lds = ((size_t)deal * kSel + kRun + 7) * 4;   // runs are read eight words at a time
  if (lds > 32768) {                                  // beyond what a launch gets unasked
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void*>(hold ? evict_select_kernel<true> : evict_select_kernel<false>),
        hipFuncAttributeMaxDynamicSharedMemorySize, (kHeldRows + kRun + 7) * 4);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(hold ? evict_select_kernel<true> : evict_select_kernel<false>, dim3(b.batch), dim3(kSel),
                     lds, stream, b, c, head, moves, reinterpret_cast<MoveRow*>(p + w.rows), w.most,
                     divide_by((unsigned)b.page_size));
  const int row16 = b.n_kv * b.hd / 8;
  int per = row16 < 1024 ? 1024 / row16 : 1;
  if (w.most / per > 1 << 22) per = (int)(w.most >> 22) + 1;    // within a grid's threads
  const unsigned blocks = w.most > 0 ? (unsigned)((w.most + per - 1) / per) : 1u;
  for (int first = 0; first == 0 || first < n_pools; first += kEvictPools) {
    EvictPools e = {};
    const int n = n_pools - first < kEvictPools ? n_pools - first : kEvictPools;
    for (int i = 0; i < n; ++i) e.p[i] = pools[first + i];
    hipLaunchKernelGGL(evict_move_kernel, n ? dim3(blocks, n, b.batch) : dim3(1), dim3(256), 0, stream, e,
                       head, moves, w.most, per, n ? row16 : 0, divide_by((unsigned)row16), b.batch,
                       first == 0 ? status : nullptr);
  }
  return hipGetLastError();
}

}  // namespace rf
