// Eviction from the paged cache by accumulated weight, on gfx950.
//
// Two launches.  The first, one workgroup per sequence, picks the kept rows and lists the
// moves; the second copies them in every pool.  Rows are kept by a 32-bit key (the weight's
// bits in unsigned order, all ones for a protected row, 0 for a NaN), the n_keep-th largest
// found by a radix select of 8 bits a pass; of the rows at that key the lowest are kept.
//
// A kept row below n_keep stays where it is and a kept row above moves into a free row below:
// the sources (>= n_keep) and the destinations (< n_keep) are disjoint, so rows move in place
// and in parallel, and only k (1 - k/n) of the k kept rows move (of n, evenly spread), 64 of
// 4096 where 64 new rows have been appended, while closing the gaps in order would move nearly
// all of them.
#include "rf_cache.h"
#include "rf_common.h"

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

__global__ __launch_bounds__(kSel) void evict_select_kernel(Batch b, EvictCall c, int2* head,
                                                            int2* moves, MoveRow* mrows,
                                                            int64_t most) {
  __shared__ unsigned hist[256];
  __shared__ int red[kWaves];
  __shared__ int counts[kWaves][3];
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

  int top = INT32_MIN;
  for (int t = tid; t < len; t += kSel) {
    top = max(top, pos[t]);
    if (acc[t] != acc[t]) err = (int)kStatusScoreBit;
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) top = max(top, __shfl_xor(top, d));
  if (lane == 0) red[wave] = top;
  err = __syncthreads_or(err);
  err = err ? (int)kStatusScoreBit : 0;
  for (int w = 0; w < kWaves; ++w) top = max(top, red[w]);

  if (len <= keep) {                                // nothing to cut
    for (int t = tid; t < len; t += kSel) {
      const float a = acc[t];
      const int p = pos[t];
      acc_out[t] = a;
      pos_out[t] = p;
    }
    if (tid == 0) {
      c.len_out[seq] = len;
      head[seq] = make_int2(0, err);
    }
    return;
  }

  const int64_t newest = (int64_t)top - c.n_recent;   // protected above this position
  auto key_of = [&](int t) -> uint32_t {
    const int p = pos[t];
    return (p < c.n_sink || p > newest) ? 0xffffffffu : weight_order(acc[t]);
  };
  // the keep-th largest key, digit by digit; `need` of the rows at it are kept
  uint32_t prefix = 0u, mask = 0u;
  unsigned need = (unsigned)keep;
  for (int shift = 24; keep > 0 && shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0u;
    __syncthreads();
    for (int t = tid; t < len; t += kSel) {
      const uint32_t k = key_of(t);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 0xffu], 1u);
    }
    __syncthreads();
    if (wave == 0) {                                // lane l: digits 255-4l down to 252-4l
      unsigned v[4], s = 0u;
      for (int i = 0; i < 4; ++i) s += v[i] = hist[255 - 4 * lane - i];
      unsigned run = s;
      for (int d = 1; d < 64; d <<= 1) {
        const unsigned o = __shfl_up(run, d);
        if (lane >= d) run += o;
      }
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

  // in order: which rows are kept, the free rows below keep, the kept rows from keep on
  MoveRow* list = mrows + seq * most;
  int ties = 0, holes = 0, movers = 0;              // so far, over all rows before this chunk
  for (int base = 0; base < len; base += kSel) {
    const int t = base + tid;
    const bool in = t < len;
    const uint32_t k = in && keep > 0 ? key_of(t) : 0u;
    const bool tie = in && keep > 0 && k == prefix;
    const float a = in ? acc[t] : 0.f;
    const int p = in ? pos[t] : 0;
    const uint64_t below = (1ull << lane) - 1;
    uint64_t vote = __ballot(tie);
    if (lane == 0) counts[wave][0] = __popcll(vote);
    __syncthreads();
    int rank = ties + __popcll(vote & below);
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) rank += counts[w][0];
      ties += counts[w][0];
    }
    const bool kept = in && keep > 0 && (k > prefix || (tie && rank < (int)need));
    const bool hole = in && t < keep && !kept, mover = t >= keep && kept;
    const uint64_t vh = __ballot(hole), vm = __ballot(mover);
    if (lane == 0) {
      counts[wave][1] = __popcll(vh);
      counts[wave][2] = __popcll(vm);
    }
    __syncthreads();
    int rh = holes + __popcll(vh & below), rm = movers + __popcll(vm & below);
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) {
        rh += counts[w][1];
        rm += counts[w][2];
      }
      holes += counts[w][1];
      movers += counts[w][2];
    }
    if (hole) list[rh].to = t;
    if (mover) {
      list[rm].from = t;
      list[rm].weight = a;
      list[rm].pos = p;
    }
    if (in && t >= keep) acc_out[t] = 0.f;
    if (kept && t < keep) {
      acc_out[t] = a;
      pos_out[t] = p;
    }
    __syncthreads();                                // counts are written again
  }
  // the list is complete for this workgroup's own eyes after the barrier above
  auto slot_of = [&](int t) -> int {
    const int page = b.tables[(int64_t)seq * b.table_stride + t / b.page_size];
    return page < 0 || page >= b.num_pages ? -1 : page * b.page_size + t % b.page_size;
  };
  int bad = 0;
  for (int i = tid; i < movers; i += kSel) {
    const MoveRow r = list[i];
    acc_out[r.to] = r.weight;
    pos_out[r.to] = r.pos;
    int2 m = make_int2(slot_of(r.from), slot_of(r.to));
    if (m.x < 0 || m.y < 0) {
      bad = 1;
      m = make_int2(-1, -1);
    }
    moves[seq * most + i] = m;
  }
  bad = __syncthreads_or(bad);
  if (tid == 0) {
    c.len_out[seq] = keep;
    head[seq] = make_int2(movers, err | (bad ? (int)kStatusRowsBit : 0));
  }
}

// blockIdx.x: chunk of a sequence's moves, y: pool, z: sequence.  A row is n_kv * hd bf16
// values in one piece; each lane copies 16 bytes of one.
__global__ __launch_bounds__(256) void evict_move_kernel(EvictPools pools, const int2* head,
                                                         const int2* moves, int64_t most,
                                                         int row16, int batch, unsigned* status) {
  if (status && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
    int bits = 0;
    for (int s = threadIdx.x; s < batch; s += 256) bits |= head[s].y;
    const int rows = __syncthreads_or(bits & (int)kStatusRowsBit);
    const int nan = __syncthreads_or(bits & (int)kStatusScoreBit);
    if (threadIdx.x == 0) *status = (rows ? kStatusRowsBit : 0u) | (nan ? kStatusScoreBit : 0u);
  }
  const int n = head[blockIdx.z].x;
  u32x4* p = reinterpret_cast<u32x4*>(pools.p[blockIdx.y]);
  const int64_t total = (int64_t)n * row16;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int m = (int)(i / row16), e = (int)(i % row16);
    const int2 mv = moves[blockIdx.z * most + m];
    if (mv.x >= 0) p[(int64_t)mv.y * row16 + e] = p[(int64_t)mv.x * row16 + e];
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
  hipLaunchKernelGGL(evict_select_kernel, dim3(b.batch), dim3(kSel), 0, stream, b, c, head, moves,
                     reinterpret_cast<MoveRow*>(p + w.rows), w.most);
  const int row16 = b.n_kv * b.hd / 8;
  int64_t blocks = (w.most * row16 + 1023) / 1024;   // four 16-byte pieces a thread
  blocks = blocks < 1 ? 1 : blocks > 4096 ? 4096 : blocks;
  for (int first = 0; first == 0 || first < n_pools; first += kEvictPools) {
    EvictPools e = {};
    const int n = n_pools - first < kEvictPools ? n_pools - first : kEvictPools;
    for (int i = 0; i < n; ++i) e.p[i] = pools[first + i];
    hipLaunchKernelGGL(evict_move_kernel, n ? dim3((unsigned)blocks, n, b.batch) : dim3(1), dim3(256),
                       0, stream, e, head, moves, n ? w.most : 0, n ? row16 : 0, b.batch,
                       first == 0 ? status : nullptr);
  }
  return hipGetLastError();
}

}  // namespace rf
