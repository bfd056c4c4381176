// Attention over the paged cache: how a call is laid out, and the join of its parts.  The kernels are
// in rf_attend_dev.h; those of plain bf16 caches are compiled here, those that know prefixes or codes in
// rf_attend_shared.hip, rf_attend_fp8.hip and rf_attend_int8.hip.
#include "rf_attend_dev.h"

namespace rf {

namespace {

// The plan of more than 64 groups.
__global__ __launch_bounds__(64) void plan_kernel(AttendArgs a) {
  GroupLine line = {0, 0};
  const Group first = look_up_groups(a, 0, &line);
  const int each = grains_of_prefix_part<true>(a, first, line);
  write_plan<true>(a, first, line, each);
  if (threadIdx.x == 0) *a.sh.each = each;
}

// What is wrong with a group or its prefix's pages, part `part` of them.
__device__ inline void scan_prefix(const AttendArgs& a, int g, int part) {
  const bool counts = a.sh.plan[g].w;
  const int len = a.sh.lengths[g], pages = counts && len > 0 ? (len - 1) / a.b.page_size + 1 : 0, step = blockDim.x;
  const int32_t* table = a.sh.tables + (int64_t)g * a.sh.table_stride;
  int bits = !counts;
  for (int64_t i = (int64_t)part * step + threadIdx.x; i < pages; i += (int64_t)a.sh.scan_parts * step) {
    const int page = table[i];
    bits |= page < 0 || page >= a.b.num_pages;
  }
  bits = __syncthreads_or(bits);
  if (bits && threadIdx.x == 0) atomicOr(a.status, kStatusRowsBit);
}

// Joins the parts of one output row by kPer waves: sixteen lanes hold the row, four parts to a
// wave at a time (and several of those in flight: one at a time, 128 parts took 80 us).  One token
// over 65,536 rows, 8 key heads: 64 us by four waves a row, 72 by one; one key head 26 and 40.
// Eight workgroups fit a compute unit (with more registers for the scan: five, 12.6 instead of 9.4
// us for the trees above).
// Sequences of more than 128 parts in the mean (of codes, whose workgroups of four key heads make four times as many, or
// of prefixes): sixteen waves a row.  One fp8 sequence of 65,536 rows, 8 key heads, 512 parts: 48.5 us by
// four, 42.7 by sixteen.
constexpr int kManyWaves = 16;
template <int HD, int kPer, bool kShared>
__global__ __launch_bounds__(kPer > kWaves ? 64 * kPer : kThreads, 8) void join_kernel(AttendArgs a) {
  constexpr int kE = HD / 16;
  __shared__ float sh_o[kPer][HD + 1];
  const int rows = a.q.max_q * a.group;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = threadIdx.x >> 6, g0 = 4 * (wave % kPer) + g;
  const int own_scans = a.b.batch * a.scan_parts, scans = own_scans + (kShared ? a.sh.groups * a.sh.scan_parts : 0);
  if ((int)blockIdx.x < own_scans)
    return scan_sequence(a.b, a.q, blockIdx.x / a.scan_parts, blockIdx.x % a.scan_parts, a.scan_parts, a.status);
  if constexpr (kShared) {
    const int i = blockIdx.x - own_scans;
    if ((int)blockIdx.x < scans) return scan_prefix(a, i / a.sh.scan_parts, i % a.sh.scan_parts);
  }
  const int64_t id = kPer > kWaves ? (int64_t)blockIdx.x - scans : (int64_t)(blockIdx.x - scans) * (kWaves / kPer) + wave / kPer;
  const int sh = (int)(id / rows), m = (int)(id % rows);
  if (sh >= a.b.batch * a.b.n_kv) return;
  const int kh = sh % a.b.n_kv, seq = sh / a.b.n_kv;
  const Seq mine = look_up(a, lane), self = look_up(a, seq);
  const int n = self.n, first = self.first;
  if (!self.grains || m >= n * a.group) return;
  // parts of its own rows, then of its prefix
  int own = 1, before = seq;
  if (!kShared || a.goal) {
    const int each = (int)*a.each;
    own = (self.grains + each - 1) / each;
    before = lane < seq ? (mine.grains + each - 1) / each : 0;
    for (int b = 64 + lane; b < seq; b += 64) before += (look_up(a, b).grains + each - 1) / each;
    before = wave_sum(before);
  }
  const int64_t at = ((int64_t)before * a.b.n_kv + kh) * rows + m, step = (int64_t)a.b.n_kv * rows;
  int64_t more_at = 0, more_step = 0;
  int parts = own;
  if constexpr (kShared) {
    int g = -1;
    for (int g0 = 0; g0 < a.sh.groups && g < 0; g0 += 64) {
      const int l = g0 + lane;
      const uint64_t has = __ballot(l < a.sh.groups && a.sh.starts[l] <= seq && seq < a.sh.starts[l + 1]);
      if (has) g = g0 + __ffsll((unsigned long long)has) - 1;
    }
    if (g >= 0) {
      const uint4 plan = a.sh.plan[g];
      const Group r = look_up_group(a, g);
      // a sequence whose prefix is not known has no answer, nor has one outside its group's queries
      if (!plan.w || first < r.first || (int64_t)first + n > (int64_t)r.first + r.n) return;
      if (plan.y) {
        const int x = (first - r.first) * a.group + m, block = x / a.sh.rows;
        parts += (int)plan.z;
        more_at = a.sh.first_row + ((int64_t)(plan.x + block) * a.b.n_kv + kh) * a.sh.rows + x % a.sh.rows;
        more_step = (int64_t)plan.y * a.b.n_kv * a.sh.rows;
      }
    }
  }
  if (!kShared && parts == 1) return;               // written by its workgroup
  const auto place = [&](int s) { return kShared && s >= own ? more_at + (s - own) * more_step : at + s * step; };
  float top = -INFINITY;
  for (int s = lane; s < parts; s += 64) top = fmaxf(top, a.part_ml[place(s)].x);
#pragma unroll
  for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  const float zero = top == -INFINITY ? 0.f : top;
  float sum = 0.f, o[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) o[e] = 0.f;
  if (a.out) {
    const float* po = a.part_o + c * kE;
#pragma unroll 4
    for (int s = g0; s < parts; s += 4 * kPer) {
      const int64_t i0 = place(s);
      const float2 v = a.part_ml[i0];
      const float w = __builtin_amdgcn_exp2f(v.x - zero);
      sum += v.y * w;
#pragma unroll
      for (int e = 0; e < kE; e += 4) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(po + i0 * HD + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[e + i] += x[i] * w;
      }
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      o[e] += __shfl_xor(o[e], 16);
      o[e] += __shfl_xor(o[e], 32);
    }
  } else {
    for (int s = g0; s < parts; s += 4 * kPer) {
      const float2 v = a.part_ml[place(s)];
      sum += v.y * __builtin_amdgcn_exp2f(v.x - zero);
    }
  }
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if constexpr (kPer > 1) {                         // one row to a workgroup: all its waves are here
    static_assert(kPer >= kWaves, "a row is one workgroup's");
    if (a.out && g == 0) {
#pragma unroll
      for (int e = 0; e < kE; ++e) sh_o[wave][c * kE + e] = o[e];
    }
    if (lane == 0) sh_o[wave][HD] = sum;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < kPer; ++w) {
      sum += sh_o[w][HD];
      if (a.out) {
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] += sh_o[w][c * kE + e];
      }
    }
  }
  const int h = kh * a.group + m % a.group;
  const int64_t row = first + m / a.group;
  const bool none = sum == 0.f;
  if (a.lse && lane == 0) a.lse[row * a.q.n_heads + h] = none ? -INFINITY : top * kLn2 + __logf(sum);
  if (a.out && g == 0) {
    uint16_t* p = a.out + row * a.out_stride + h * HD + c * kE;
    const float inv = none ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < kE; e += 4) {
      const u32x2 x = {pack_bf16x2(o[e] * inv, o[e + 1] * inv), pack_bf16x2(o[e + 2] * inv, o[e + 3] * inv)};
      *reinterpret_cast<u32x2*>(p + e) = none ? u32x2{0u, 0u} : x;
    }
  }
}

// How a call is laid out.
struct AttendPlan {
  int rows;                     // query rows of a workgroup
  int heads;                    // key heads of a workgroup
  int mblocks, group, parts, goal, least;
  size_t ml, o, total;
};
// Key heads of a workgroup: of codes up to four (where they share lines of scales), each for its own waves.
int heads_together(const Batch& b, int rows, bool codes) {
  return !codes || rows != 16 ? 1 : b.n_kv % 4 == 0 ? 4 : b.n_kv % 2 == 0 ? 2 : 1;
}
// `joined`: all parts are joined, also those of sequences that have one.
// `codes`: a cache of 8 bits.
AttendPlan attend_plan(const Batch& b, int n_heads, int max_q, bool joined = false, bool codes = false) {
  AttendPlan p;
  p.group = n_heads / b.n_kv;
  const int rows = max_q * p.group;
  p.rows = rows <= 16 ? 16 : rows <= 128 ? 128 : 256;
  p.mblocks = (rows + p.rows - 1) / p.rows;
  // Enough workgroups for the chip: up to four a compute unit with registers alone, one with LDS; of codes beside
  // prefixes half as many (48 sequences of up to 2,048 rows on four prefixes in fp8 137 instead of 145 us).
  p.heads = heads_together(b, p.rows, codes);
  const int per_part = b.n_kv / p.heads * p.mblocks, want = p.rows == 16 ? (joined && codes ? 512 : 1024) : 256;
  p.least = p.rows == 16 ? least_rows(b.batch, b.max_len, per_part, want, p.heads, joined) : 128;
  p.goal = parts_goal(want, per_part);
  if (p.goal <= b.batch || b.max_len <= p.least) p.goal = 0;
  const int64_t most = (int64_t)b.batch * ((b.max_len + p.least - 1) / p.least);
  p.parts = p.goal == 0 ? b.batch : most < p.goal ? (int)most : p.goal;
  const size_t held = p.goal || joined ? (size_t)p.parts * b.n_kv * rows : 0;
  p.ml = kStatusBytes;
  p.o = p.ml + align256(held * sizeof(float2));
  p.total = p.o + align256(held * b.hd * sizeof(float));
  return p;
}

// The prefixes of a call: their form, and the pairs of a part and a block of query rows.
struct PrefixPlan {
  int rows, heads, goal, least, parts, pairs;
};
PrefixPlan prefix_plan(const Batch& b, const PrefixCall& pre, int n_heads, int max_q, int64_t n_q, bool codes) {
  PrefixPlan p;
  const int group = n_heads / b.n_kv;
  const int64_t most = (int64_t)b.batch * max_q, n = n_q < most ? n_q : most;      // queries that can have sequences
  const int64_t groups = n < pre.groups ? n : pre.groups, all = n * group, mean = groups ? all / groups : 0;
  p.rows = prefix_block(mean, all);
  p.heads = heads_together(b, p.rows, codes);
  p.least = p.rows == 16 ? 256 / p.heads : 128;
  p.goal = parts_goal(p.rows == 16 ? 1024 : 256, b.n_kv / p.heads);
  p.parts = (pre.max_len + p.least - 1) / p.least;      // of one block, at most
  p.pairs = (int)most_pairs(most_blocks(all, groups, p.rows), p.parts, p.goal);
  return p;
}

struct CacheLayout {
  size_t plan, ml, o, total;
  int64_t own_rows;             // of partial results
};
CacheLayout cache_layout(const Batch& b, const PrefixCall& pre, const AttendPlan& p, const PrefixPlan& q, int rows) {
  CacheLayout l;
  l.own_rows = (int64_t)p.parts * b.n_kv * rows;
  const size_t held = (size_t)(l.own_rows + (int64_t)q.pairs * b.n_kv * q.rows);
  l.plan = kStatusBytes;
  l.ml = l.plan + align256((size_t)pre.groups * sizeof(uint4));
  l.o = l.ml + align256(held * sizeof(float2));
  l.total = l.o + align256(held * b.hd * sizeof(float));
  return l;
}

// `parts`: what sequences have in the mean; `many`: sixteen waves a row where they pay (not for plain bf16
// caches: their sums keep their order).
template <int HD, bool kShared>
void launch_join(const AttendArgs& a, int most_parts, int parts, bool many, hipStream_t stream) {
  const int64_t rows = (int64_t)a.b.batch * a.b.n_kv * a.q.max_q * a.group;
  const int64_t scans = (int64_t)a.b.batch * a.scan_parts + (kShared ? (int64_t)a.sh.groups * a.sh.scan_parts : 0);
  // More waves to a row where it has more parts than a wave has under way, and the chip has room for them: with
  // 33 parts 7,680 rows take 425 us of a call with one wave each and 437 with four, 6,144 rows of 11 parts 137
  // and 145; 2,048 rows of 33 parts 104 with either.
  const bool room = rows <= 2048;
  if (many && parts > 128 && room)
    hipLaunchKernelGGL((join_kernel<HD, kManyWaves, kShared>), dim3((unsigned)(rows + scans)), dim3(64 * kManyWaves), 0, stream, a);
  else if (kShared ? parts > 16 && room : most_parts > 32)
    hipLaunchKernelGGL((join_kernel<HD, kWaves, kShared>), dim3((unsigned)(rows + scans)), dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((join_kernel<HD, 1, kShared>), dim3((unsigned)((rows + kWaves - 1) / kWaves + scans)),
                       dim3(kThreads), 0, stream, a);
}

// What all calls set, with the workspace of one that has no prefixes.
AttendArgs attend_args(const Batch& b, const Queries& q, const AttendPlan& p, uint16_t* out, int64_t out_stride,
                       float* lse, unsigned char* ws) {
  AttendArgs a = {};
  a.b = b;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.status = reinterpret_cast<unsigned*>(ws);
  a.each = a.status + 1;
  a.part_ml = reinterpret_cast<float2*>(ws + p.ml);
  a.part_o = reinterpret_cast<float*>(ws + p.o);
  a.out_stride = out_stride;
  a.page = divide_by((unsigned)b.page_size);
  a.parts = p.parts;
  a.goal = p.goal;
  a.least = p.least;
  a.heads = p.heads;
  a.mblocks = p.mblocks;
  a.group = p.group;
  a.scan_parts = scan_parts(b);
  return a;
}

// A call without prefixes: one launch, and the join where sequences are split.
hipError_t launch_plain(AttendArgs& a, const AttendPlan& p, bool codes, void (*rows)(const AttendArgs&, int, unsigned, hipStream_t),
                        hipStream_t stream) {
  a.scan = !p.goal && scans(a.b) ? 1 : 0;
  a.report = !p.goal && !a.scan ? 1 : 0;
  if (a.report) {
    const hipError_t e = launch_clear_status(a.status, stream);
    if (e != hipSuccess) return e;
  }
  a.own = (int)((int64_t)p.parts * (a.b.n_kv / p.heads) * p.mblocks);
  rows(a, p.rows, (unsigned)a.own + a.scan, stream);
  const auto join = a.b.hd == 128 ? launch_join<128, false> : launch_join<64, false>;
  if (p.goal) join(a, p.goal, p.parts / a.b.batch, codes, stream);
  return hipGetLastError();
}

}  // namespace

size_t attend_workspace(const Batch& b, int n_heads, int max_q) {
  return attend_plan(b, n_heads, max_q).total;
}

hipError_t launch_attend(const Batch& b, const uint16_t* kp, const uint16_t* vp, const Queries& q,
                         uint16_t* out, int64_t out_stride, float* lse, void* ws,
                         hipStream_t stream) {
  const AttendPlan p = attend_plan(b, q.n_heads, q.max_q);
  AttendArgs a = attend_args(b, q, p, out, out_stride, lse, static_cast<unsigned char*>(ws));
  a.kp = kp;
  a.vp = vp;
  return launch_plain(a, p, false, launch_rows<RF_CACHE_BF16, false>, stream);
}

// What caches of either kind need.
size_t cache_attend_workspace(const Batch& b, const PrefixCall* prefix, int n_heads, int max_q, int64_t n_q) {
  size_t most = 0;
  for (const bool codes : {false, true}) {
    const AttendPlan p = attend_plan(b, n_heads, max_q, prefix != nullptr, codes);
    const size_t need = prefix ? cache_layout(b, *prefix, p, prefix_plan(b, *prefix, n_heads, max_q, n_q, codes), max_q * p.group).total
                               : p.total;
    most = most < need ? need : most;
  }
  return most;
}

hipError_t launch_cache_attend(const Batch& b, const PrefixCall* prefix, const Pools& pools, const Queries& q,
                               uint16_t* out, int64_t out_stride, float* lse, void* ws, hipStream_t stream) {
  const uint16_t* kp = static_cast<const uint16_t*>(pools.k);
  const uint16_t* vp = static_cast<const uint16_t*>(pools.v);
  if (!prefix && pools.type == RF_CACHE_BF16) return launch_attend(b, kp, vp, q, out, out_stride, lse, ws, stream);
  const auto rows = pools.type == RF_CACHE_BF16  ? launch_rows<RF_CACHE_BF16, true>
                    : pools.type == RF_CACHE_FP8 ? launch_rows<RF_CACHE_FP8, true>
                                                 : launch_rows<RF_CACHE_INT8, true>;
  const bool codes = pools.type != RF_CACHE_BF16;
  const AttendPlan p = attend_plan(b, q.n_heads, q.max_q, prefix != nullptr, codes);
  unsigned char* w = static_cast<unsigned char*>(ws);
  AttendArgs a = attend_args(b, q, p, out, out_stride, lse, w);
  a.kp = kp;
  a.vp = vp;
  a.ks = pools.ks;
  a.vs = pools.vs;
  if (!prefix) return launch_plain(a, p, codes, rows, stream);
  const PrefixPlan pp = prefix_plan(b, *prefix, q.n_heads, q.max_q, q.n_q, codes);
  const CacheLayout l = cache_layout(b, *prefix, p, pp, q.max_q * p.group);
  a.part_ml = reinterpret_cast<float2*>(w + l.ml);
  a.part_o = reinterpret_cast<float*>(w + l.o);
  Batch as = b;                                     // for the pages to look over
  as.max_len = prefix->max_len;
  a.sh = {prefix->tables, prefix->lengths, prefix->starts, prefix->table_stride, prefix->groups, prefix->max_len,
          pp.goal, pp.least, pp.rows, l.own_rows, scan_parts(as), reinterpret_cast<uint4*>(w + l.plan), a.status + 2};
  if (prefix->groups > 64) hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(64), 0, stream, a);
  // The sequences' own rows and the prefixes, in one launch where both take the same kernel.
  const int own = (int)((int64_t)p.parts * (b.n_kv / p.heads) * p.mblocks), more = pp.pairs * (b.n_kv / pp.heads);
  a.own = own;
  rows(a, p.rows, (unsigned)(p.rows == pp.rows ? own + more : own), stream);
  if (p.rows != pp.rows) {
    a.own = 0;
    a.heads = pp.heads;
    rows(a, pp.rows, (unsigned)more, stream);
  }
  const int most_parts = p.parts > pp.pairs ? p.parts : pp.pairs;
  // its own parts, and those of a prefix
  const int groups = prefix->groups < b.batch ? prefix->groups : b.batch, shared = pp.goal / groups;
  const int mean = p.parts / b.batch + (shared < pp.parts ? shared : pp.parts);
  (b.hd == 128 ? launch_join<128, true> : launch_join<64, true>)(a, most_parts, mean, true, stream);
  return hipGetLastError();
}

}  // namespace rf
