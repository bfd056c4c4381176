// The attention weight that the rows of the paged cache receive, on gfx950 (section "Which
// rows to compute exactly" of the English RidgeFill review: the attention that a prompt's last
// tokens pay to its rows ranks them).
//
// With the queries' log-sum-exp at hand one pass over K suffices: a row's weight is the sum of
// exp(scale q.k - lse) over the queries and heads.  As in the attention, the n queries of a
// sequence and the G query heads of one key head are M = n G rows of a matrix Q, and a wave
// computes S^T = K Q^T (16x16x32 MFMAs, A = 16 cache rows straight from memory, B = 16 query
// rows): lane (c, g) holds rows 4 g + r of query c, so the sum over queries is a lane's own
// over the query tiles, and one over the 16 lanes c at the end.  Sums run in a fixed order.
//
// M <= 64 (decoding, small trees): bound by the read of K.  A workgroup takes 64 or more cache
// rows and all key heads (its waves share them out), joins the heads in LDS and writes the
// accumulated weight: one launch.  16 sequences of up to 16,384 rows, one token, 8 key heads of
// 128 (380 MB): 73 us, 5.2 TB/s, as a large copy.
// M > 64: bound by the exponentials (16 cycles a wave of 64) and the matrix cores.  Q of one key
// head (256 rows a block) lies in LDS and a workgroup walks a long range of cache rows with it;
// the heads' sums meet in a second launch.  The last 64 tokens of 32,768 rows, 32 query heads: 33 + 5
// us, 35 in one call after another, 485 TFLOP/s; the exponentials alone are 12 us (24 cycles with
// their addition), staging Q 7 (whose writes meet in LDS banks: 40% of the kernel's LDS cycles).
#include "rf_cache_dev.h"
#include "rf_split.h"

namespace rf {

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 64;             // cache rows of one step of a wave
constexpr int kBlock = 256;           // query rows in LDS
constexpr int kHeadWaves = 8;         // waves that share them
constexpr int kHeadThreads = 64 * kHeadWaves;

struct WeightArgs {
  Batch b;
  Queries q;
  const uint16_t* kp;
  const float* lse;
  const float* acc;
  float* acc_out;
  unsigned* status;
  float* part;                  // [batch][n_kv mblocks][max_len]
  int64_t acc_stride;
  Divide page, by_group;
  float decay;
  int chunk, splits;            // cache rows of a workgroup, workgroups along them
  int mblocks, group;
  int scan;                     // 1: the first workgroup of the only launch looks all pages over
  int scan_parts;               // of a sequence, in the second launch
};

// Sum over the 16 lanes of a row of the wave, in every one of them.
__device__ __forceinline__ float sum16(float v) {
#define RF_ROR(n) \
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + n, 0xf, 0xf, false))
  RF_ROR(8);
  RF_ROR(4);
  RF_ROR(2);
  RF_ROR(1);
#undef RF_ROR
  return v;
}

template <int HD>
struct Keys {                   // 64 cache rows of one head
  u32x4 k[4][HD / 32];          // rows 16 t + c, features 32 s + 8 g ..
};

template <int HD>
__device__ __forceinline__ void load_keys(Keys<HD>& t, const uint16_t* kh, int64_t row, int slot,
                                          int c, int g) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint16_t* p = kh + (int64_t)__shfl(slot, 16 * h + c) * row + 8 * g;
#pragma unroll
    for (int s = 0; s < HD / 32; ++s) t.k[h][s] = *reinterpret_cast<const u32x4*>(p + 32 * s);
  }
}

// Adds the weights that 16 queries give to the 64 rows.  `some`: not all of them see all rows;
// then `seen` says which (0 for a lane without a query or whose query sees nothing).
template <int HD>
__device__ __forceinline__ void add_weights(const Keys<HD>& keys, const bf16x8 (&q)[HD / 32],
                                            float scale2, float lse2, bool some, uint64_t seen,
                                            int g, float (&w)[4][4]) {
  f32x4 s[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int st = 0; st < HD / 32; ++st)                // four independent sums side by side
#pragma unroll
    for (int t = 0; t < 4; ++t) s[t] = mfma16(__builtin_bit_cast(bf16x8, keys.k[t][st]), q[st], s[t]);
  if (!some) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) w[t][r] += __builtin_amdgcn_exp2f(fmaf(s[t][r], scale2, -lse2));
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t bits = (uint32_t)(seen >> (16 * t + 4 * g));
#pragma unroll
      for (int r = 0; r < 4; ++r)
        w[t][r] += bits >> r & 1 ? __builtin_amdgcn_exp2f(fmaf(s[t][r], scale2, -lse2)) : 0.f;
    }
  }
}

// Pool slot of cache row `row`; -1 past the last row and on a bad page (*err).
__device__ __forceinline__ int key_slot(const WeightArgs& a, const int32_t* table, int row, int len,
                                        bool* err) {
  if (row >= len) return -1;
  const int pi = (int)quotient((unsigned)row, a.page);
  const int page = table[pi];
  if (page < 0 || page >= a.b.num_pages) {
    *err = true;
    return -1;
  }
  return page * a.b.page_size + (row - pi * a.b.page_size);
}

// M <= 16 MT: workgroup = rows x all heads.  hw waves share the key heads, the others take
// further rows.
template <int HD, int MT>
__global__ __launch_bounds__(kThreads) void weight_rows_kernel(WeightArgs a) {
  constexpr int kSteps = HD / 32;
  __shared__ float sh[kWaves][kRows];
  if (a.scan && blockIdx.x == 0) return scan_status(a.b, a.q, a.status);
  const int id = blockIdx.x - a.scan, seq = id / a.splits, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int hw = a.b.n_kv >= 4 ? 4 : a.b.n_kv >= 2 ? 2 : 1;
  int len, first, n;
  bool bad;
  const bool go = sequence_of(a.b, a.q, seq, &len, &first, &n, &bad);
  if (bad && !a.scan && threadIdx.x == 0) atomicOr(a.status, kStatusRowsBit);
  const int base = (id % a.splits) * a.chunk + wave / hw * kRows;
  if (!go || (id % a.splits) * a.chunk >= len) return;
  const int ctx = len - n, m_rows = n * a.group;
  const int32_t* table = a.b.tables + (int64_t)seq * a.b.table_stride;
  bool err = false;
  const int slot = key_slot(a, table, base + lane, len, &err);
  const uint64_t there = __ballot(slot >= 0);
  if (!a.scan && __any(err) && lane == 0) atomicOr(a.status, kStatusRowsBit);
  const bool part_rows = ~there || base + kRows > ctx;

  float w[4][4];
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) w[t][r] = 0.f;
  const float scale2 = a.q.scale * kLog2e;
  if (there) {
    for (int kh = wave % hw; kh < a.b.n_kv; kh += hw) {
      Keys<HD> keys;
      load_keys<HD>(keys, a.kp + kh * HD, (int64_t)a.b.n_kv * HD, slot < 0 ? 0 : slot, c, g);
#pragma unroll
      for (int qt = 0; qt < MT; ++qt) {
        const int m = 16 * qt + c;
        if (16 * qt >= m_rows) break;
        const bool in = m < m_rows;
        const int i = in ? (int)quotient((unsigned)m, a.by_group) : 0, h = kh * a.group + (in ? m - i * a.group : 0);
        const uint16_t* p = a.q.q + (int64_t)(first + i) * a.q.q_stride + h * HD + 8 * g;
        bf16x8 q[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) q[s] = *reinterpret_cast<const bf16x8*>(p + 32 * s);
        const float l = in ? a.lse[(int64_t)(first + i) * a.q.n_heads + h] : -INFINITY;
        const bool live = l != -INFINITY;
        uint64_t seen = live ? there : 0ull;
        if (base + kRows > ctx) seen &= seen64(draft_word(a.q, first + i, i), base - ctx);
        add_weights<HD>(keys, q, scale2, l * kLog2e, part_rows || __any(!live), seen, g, w);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      w[t][r] = sum16(w[t][r]);
      if (c == 0) sh[wave][16 * t + 4 * g + r] = w[t][r];
    }
  __syncthreads();
  const int row = base + lane;
  if (wave % hw == 0 && row < len) {
    float v = 0.f;
    for (int i = 0; i < hw; ++i) v += sh[wave + i][lane];
    const int64_t at = seq * a.acc_stride + row;
    a.acc_out[at] = a.acc ? a.decay * a.acc[at] + v : v;
  }
}

// M > 64: workgroup = one key head, a block of its query rows, a range of cache rows.
template <int HD>
__global__ __launch_bounds__(kHeadThreads, 2) void weight_heads_kernel(WeightArgs a) {
  constexpr int kSteps = HD / 32;
  __shared__ u32x4 sh_q[kBlock / 16][kSteps][64];   // as the lanes read them
  __shared__ float sh_lse[kBlock];                  // in log2
  __shared__ uint64_t sh_word[kBlock];
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0u;      // the sum's launch adds what is wrong
  const int id = blockIdx.x, split = id % a.splits, unit = id / a.splits;
  const int mb = unit % a.mblocks, kh = unit / a.mblocks % a.b.n_kv, seq = unit / a.mblocks / a.b.n_kv;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  int len, first, n;
  bool bad;
  const bool go = sequence_of(a.b, a.q, seq, &len, &first, &n, &bad);
  const int begin = split * a.chunk, m0 = mb * kBlock;
  const int m_rows = n * a.group - m0 < kBlock ? n * a.group - m0 : kBlock;
  if (!go || begin >= len || m_rows <= 0) return;
  const int end = len < begin + a.chunk ? len : begin + a.chunk;
  const int ctx = len - n, tiles = (m_rows + 15) / 16;

  // the first rows on their way, then Q into LDS
  const int32_t* table = a.b.tables + (int64_t)seq * a.b.table_stride;
  const uint16_t* kbase = a.kp + kh * HD;
  const int64_t row_size = (int64_t)a.b.n_kv * HD;
  bool err = false;                                 // reported by the sum's launch
  int base = begin + wave * kRows;
  Keys<HD> keys;
  int slot = -1;
  if (base < end) {
    slot = key_slot(a, table, base + lane, len, &err);
    load_keys<HD>(keys, kbase, row_size, slot < 0 ? 0 : slot, c, g);
  }
  constexpr int kPieces = kBlock * (HD / 8) / kHeadThreads;
  u32x4 piece[kPieces];
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int x = tid + j * kHeadThreads, m = x / (HD / 8), ch = x % (HD / 8), mc = m < m_rows ? m : m_rows - 1;
    const int i = (int)quotient((unsigned)(m0 + mc), a.by_group), h = kh * a.group + (m0 + mc - i * a.group);
    piece[j] = *reinterpret_cast<const u32x4*>(a.q.q + (int64_t)(first + i) * a.q.q_stride + h * HD + 8 * ch);
  }
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int x = tid + j * kHeadThreads, m = x / (HD / 8), ch = x % (HD / 8);
    sh_q[m / 16][ch / 4][ch % 4 * 16 + m % 16] = m < m_rows ? piece[j] : u32x4{0u, 0u, 0u, 0u};
  }
  bool off = false;                                 // some query of the tiles gives nothing
  for (int m = tid; m < kBlock; m += kHeadThreads) {
    const bool in = m < m_rows;
    const int i = in ? (int)quotient((unsigned)(m0 + m), a.by_group) : 0, h = kh * a.group + (in ? m0 + m - i * a.group : 0);
    sh_lse[m] = in ? a.lse[(int64_t)(first + i) * a.q.n_heads + h] * kLog2e : -INFINITY;
    sh_word[m] = in ? draft_word(a.q, first + i, i) : 0ull;
    if (m < 16 * tiles && sh_lse[m] == -INFINITY) off = true;
  }
  const bool some_off = __syncthreads_or(off);

  float* part = a.part + ((int64_t)(seq * a.b.n_kv + kh) * a.mblocks + mb) * a.b.max_len;
  const float scale2 = a.q.scale * kLog2e;
  for (; base < end; base += kHeadWaves * kRows) {
    const int ahead = base + kHeadWaves * kRows;
    int slot_next = -1;
    Keys<HD> next;
    if (ahead < end) {
      slot_next = key_slot(a, table, ahead + lane, len, &err);
      load_keys<HD>(next, kbase, row_size, slot_next < 0 ? 0 : slot_next, c, g);
    }
    const uint64_t there = __ballot(slot >= 0);
    const bool part_rows = ~there || base + kRows > ctx;
    float w[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) w[t][r] = 0.f;
    // Two tiles of queries in turn, the fragments of one on their way while the other is used.
    const auto fetch = [&](int qt, bf16x8 (&q)[kSteps], float& l) {
      const int at = qt < tiles ? qt : tiles - 1;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) q[s] = __builtin_bit_cast(bf16x8, sh_q[at][s][lane]);
      l = sh_lse[16 * at + c];
    };
    const auto all_tiles = [&](auto add) {
      bf16x8 q0[kSteps], q1[kSteps];
      float l0, l1;
      fetch(0, q0, l0);
      for (int qt = 0; qt < tiles; qt += 2) {
        fetch(qt + 1, q1, l1);
        add(qt, q0, l0);
        if (qt + 1 >= tiles) break;
        fetch(qt + 2, q0, l0);
        add(qt + 1, q1, l1);
      }
    };
    if (!part_rows && !some_off)
      all_tiles([&](int, const bf16x8 (&q)[kSteps], float l) { add_weights<HD>(keys, q, scale2, l, false, 0ull, g, w); });
    else
      all_tiles([&](int qt, const bf16x8 (&q)[kSteps], float l) {
        uint64_t seen = l != -INFINITY ? there : 0ull;
        if (base + kRows > ctx) seen &= seen64(sh_word[16 * qt + c], base - ctx);
        add_weights<HD>(keys, q, scale2, l, true, seen, g, w);
      });
    f32x4 mine = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float v = sum16(w[t][r]);
        if (c == t) mine[r] = v;
      }
    if (c < 4) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = base + 16 * c + 4 * g + r;
        if (row < len) part[row] = mine[r];
      }
    }
    keys = next;
    slot = slot_next;
  }
}

// The heads' sums, in order; the last a.scan_parts of a sequence's workgroups look its pages over.
__global__ __launch_bounds__(kThreads) void weight_sum_kernel(WeightArgs a) {
  const int seq = blockIdx.y, row = blockIdx.x * kThreads + threadIdx.x;
  int len, first, n;
  bool bad;
  const int scan = (int)blockIdx.x - (int)(gridDim.x - a.scan_parts);
  if (scan >= 0) return scan_sequence(a.b, a.q, seq, scan, a.scan_parts, a.status);
  if (!sequence_of(a.b, a.q, seq, &len, &first, &n, &bad) || row >= len) return;
  const int live = (n * a.group + kBlock - 1) / kBlock;    // blocks of query rows
  const float* p = a.part + (int64_t)seq * a.b.n_kv * a.mblocks * a.b.max_len + row;
  float v = 0.f;
  for (int kh = 0; kh < a.b.n_kv; ++kh)
    for (int mb = 0; mb < live; ++mb) v += p[(int64_t)(kh * a.mblocks + mb) * a.b.max_len];
  const int64_t at = seq * a.acc_stride + row;
  a.acc_out[at] = a.acc ? a.decay * a.acc[at] + v : v;
}

struct WeightPlan {
  int group, mt, mblocks, chunk, splits;    // mt 0: with Q in LDS
  size_t part, total;
};
WeightPlan weight_plan(const Batch& b, int n_heads, int max_q) {
  WeightPlan p;
  p.group = n_heads / b.n_kv;
  const int rows = max_q * p.group;
  p.part = kStatusBytes;
  if (rows <= 64) {
    p.mt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    p.mblocks = 1;
    p.chunk = kRows * (b.n_kv >= 4 ? 1 : b.n_kv >= 2 ? 2 : 4);
    p.splits = (b.max_len + p.chunk - 1) / p.chunk;
    p.total = p.part;
    return p;
  }
  p.mt = 0;
  p.mblocks = (rows + kBlock - 1) / kBlock;
  // one workgroup to a compute unit, each of at least one step of its waves (rounded up whatever the
  // rounds, 64 queries of 3 sequences of 32,768 rows took 133 us in 264 workgroups, 97 in 240; 6: 219, 155)
  const int64_t units = (int64_t)b.batch * b.n_kv * p.mblocks;
  p.chunk = chunk_rows(units, b.max_len, kHeadWaves * kRows);
  p.splits = (b.max_len + p.chunk - 1) / p.chunk;
  p.total = p.part + align256((size_t)units * b.max_len * sizeof(float));
  return p;
}

template <int HD>
void launch_weight_head(const WeightArgs& a, const WeightPlan& p, hipStream_t stream) {
  const int64_t units = p.mt ? a.b.batch : (int64_t)a.b.batch * a.b.n_kv * p.mblocks;
  const dim3 grid((unsigned)(units * p.splits + a.scan)), block(kThreads);
  if (p.mt == 1) {
    hipLaunchKernelGGL((weight_rows_kernel<HD, 1>), grid, block, 0, stream, a);
  } else if (p.mt == 2) {
    hipLaunchKernelGGL((weight_rows_kernel<HD, 2>), grid, block, 0, stream, a);
  } else if (p.mt == 4) {
    hipLaunchKernelGGL((weight_rows_kernel<HD, 4>), grid, block, 0, stream, a);
  } else {
    hipLaunchKernelGGL((weight_heads_kernel<HD>), grid, dim3(kHeadThreads), 0, stream, a);
    hipLaunchKernelGGL(weight_sum_kernel, dim3((a.b.max_len + kThreads - 1) / kThreads + a.scan_parts, a.b.batch),
                       block, 0, stream, a);
  }
}

}  // namespace

size_t weight_workspace(const Batch& b, int n_heads, int max_q) {
  return weight_plan(b, n_heads, max_q).total;
}

hipError_t launch_weight(const Batch& b, const uint16_t* kp, const Queries& q, const float* lse,
                         float decay, const float* acc, float* acc_out, int64_t acc_stride,
                         void* ws, hipStream_t stream) {
  const WeightPlan p = weight_plan(b, q.n_heads, q.max_q);
  unsigned char* w = static_cast<unsigned char*>(ws);
  WeightArgs a = {};
  a.b = b;
  a.q = q;
  a.kp = kp;
  a.lse = lse;
  a.acc = acc;
  a.acc_out = acc_out;
  a.status = reinterpret_cast<unsigned*>(w);
  a.part = reinterpret_cast<float*>(w + p.part);
  a.acc_stride = acc_stride;
  a.page = divide_by((unsigned)b.page_size);
  a.by_group = divide_by((unsigned)p.group);
  a.decay = decay;
  a.chunk = p.chunk;
  a.splits = p.splits;
  a.mblocks = p.mblocks;
  a.group = p.group;
  a.scan = p.mt && scans(b) ? 1 : 0;
  a.scan_parts = scan_parts(b);
  if (p.mt && !a.scan) {
    const hipError_t e = launch_clear_status(a.status, stream);
    if (e != hipSuccess) return e;
  }
  if (b.hd == 128)
    launch_weight_head<128>(a, p, stream);
  else
    launch_weight_head<64>(a, p, stream);
  return hipGetLastError();
}

}  // namespace rf
