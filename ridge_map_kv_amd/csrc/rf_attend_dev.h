// Attention of drafted tokens over the paged cache, on gfx950 (section "Two numbers set the
// skip range" of the English RidgeFill review: rows that are not filled attend over the cache).
//
// For one key head, the n queries of a sequence and the G query heads that share it are M = n G
// rows of one matrix: S = Q K^T, softmax over the cache rows, O = P V.  K and V are read once
// for all of them, so with M of a few rows the call is bound by that read (2 hd bytes a row
// and head for each of K and V against 4 M hd operations), with M of some hundreds by the
// matrix cores and the exponentials.
//
// A wave computes the transposed products with 16x16x32 MFMAs and needs no LDS for them:
//   S^T (16 cache rows x 16 queries) = K Q^T: A = K, lane (c, g) = (lane % 16, lane / 16) holds
//     row c, features 8 g .. 8 g + 7 of each 32: one 16-byte load of the cache row;
//   the result has query c in lane (c, g) and cache rows 4 g + r: the softmax statistics of a
//     query are a running maximum and sum per lane, joined over g by two lane exchanges;
//   O^T (16 features x 16 queries) += V^T P^T over 32 cache rows: P^T as the B operand is what
//     the lane already holds, with the cache rows taken in the order k = 8 g + j <->
//     row 16 (j / 4) + 4 g + j % 4.  The A operand needs, for one feature, those eight rows'
//     values: the lane loads 16 bytes of each of the eight rows (hd 128; features 8 c ..
//     8 c + 7) and transposes the 8 x 8 block in its registers by byte permutes, so feature
//     tile m consists of the features 8 c + m.  O^T then has features 8 (4 g + r) + m in
//     lane (c, g): eight in a row for each r.
// The wave loads the next 32 rows while it computes; block-table entries are read two steps
// ahead.  A workgroup's four waves take the 32-row tiles of its row range in turn and are joined
// in LDS; long caches are split over workgroups, whose partial results (fp32) a second kernel joins.
#pragma once

#include "rf_cache_dev.h"
#include "rf_held_dev.h"
#include "rf_split.h"

namespace rf {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 32;             // cache rows of one step of a wave
// The running maximum follows a larger score only when that is more than 2^8 times as heavy: the
// weights relative to it then stay below 2^8, which costs neither fp32 sums nor bf16 weights any
// precision, and the outputs are rescaled a few times in all instead of in every other step.
constexpr float kSlack = 8.f;

// Prefixes that groups of sequences share (rf_prefix), and how their work is laid out.
struct Shared {
  const int32_t* tables;
  const int32_t* lengths;
  const int32_t* starts;        // first sequence of each group
  int64_t table_stride;
  int groups, max_len;
  int goal, least;              // pairs of a part and a block of query rows wanted, rows of a part
  int rows;                     // query rows of a block
  int64_t first_row;            // of the pairs' partial results
  int scan_parts;               // workgroups that look over a prefix's pages
  uint4* plan;                  // [groups]: first pair, blocks, parts, and whether the group counts
  unsigned* each;               // grains of a part, of more than 64 groups
};

struct AttendArgs {
  Batch b;
  Queries q;
  const uint16_t* kp;           // bf16 rows, or codes
  const uint16_t* vp;
  const uint8_t* ks;            // scales of codes
  const uint8_t* vs;
  Shared sh;
  uint16_t* out;
  float* lse;
  unsigned* status;
  unsigned* each;               // grains of a part, from the first launch to the join
  float* part_o;                // [parts][n_kv][max_q G][hd]
  float2* part_ml;              // [parts][n_kv][max_q G]: running maximum (log2), sum
  int64_t out_stride;
  Divide page;
  int parts, goal, least;       // parts of the grid; wanted of all sequences (0: one each), rows of one
  int own;                      // workgroups before those of the prefixes
  int heads;                    // key heads of a workgroup of the kernel over codes: 1, 2 or 4
  int mblocks;                  // blocks of query rows
  int group;                    // query heads of a key head
  int scan;                     // 1: the first workgroup looks all pages over for the status
  int report;                   // 1: the workgroups report bad pages and sequences
  int scan_parts;               // of a sequence, in the join
};

__device__ __forceinline__ uint32_t half_pair(uint32_t lo, uint32_t hi, int half) {
  return __builtin_amdgcn_perm(hi, lo, half ? 0x07060302u : 0x05040100u);
}

// Two weights, e^(s - max), as operands of the product with V: the leading eight bits of each, cut
// off, and what these leave, in bf16 too, so that the products add up to weights within 2^-15.  One
// bf16 a weight put the outputs as far off (0.0011 of them) as their own rounding does (0.0017), and
// more than the scores and sums in fp32 do.  The second products cost nothing where the read of the
// cache is the bound (16 sequences of up to 16,384 rows, one token: 200 us before and after, caches
// cold), 11 and 26% where the matrix cores are (162 -> 180 us for trees of 48 on 4 sequences of up to
// 32,768 rows, 143 -> 180 for one of 64 over 65,536).
// The rest is taken from the weight times 1 + 2^-23: it is above 0 wherever the weight is, so that an
// infinite value, which both products take, stays what it is (0 or a rest below 0 would make it NaN).
struct Weights {
  uint32_t lead, rest;
};
__device__ __forceinline__ Weights split_weights(float a, float b) {
  const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
  constexpr float kUp = 1.f + 0x1p-23f;
  return {half_pair(x, y, 1), pack_bf16x2(fmaf(a, kUp, -__uint_as_float(x & 0xffff0000u)),
                                          fmaf(b, kUp, -__uint_as_float(y & 0xffff0000u)))};
}

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// The same value, unknown to the compiler: what is formed from it in a loop is formed there
// and not before the loop, where it would stay in registers all along and push others out (a
// reload of those would wait for the rows in flight).
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Long caches are split into parts of about equal length over all sequences, `goal` of them at
// most: with one workgroup to a compute unit one part too many costs a second round (trees on 4
// sequences, 35 parts of 8 heads instead of 32: 239 instead of 149 us; one of 64 tokens over 32,768
// rows, 5 key heads, 52 parts instead of 51: 74 instead of 62).  The lengths are known only here, so
// each wave works the split out for itself, and the join takes it from the workspace (worked out for
// each row there too: 290 instead of 273 us for trees on 24 sequences).
constexpr int kGrain = 64;              // parts are multiples of this many rows

// One sequence of a batch as a lane looks it up; grains 0: it is skipped.
struct Seq {
  int len, first, n, grains;
};
__device__ __forceinline__ Seq look_up(const AttendArgs& a, int b) {
  Seq s = {};
  bool bad;
  if (b < a.b.batch && sequence_of(a.b, a.q, b, &s.len, &s.first, &s.n, &bad)) s.grains = (s.len + kGrain - 1) / kGrain;
  return s;
}

// Grains of one part; `mine`: sequence lane.
inline __device__ int grains_of_part(const AttendArgs& a, const Seq& mine) {
  const int lane = threadIdx.x & 63;
  int total = mine.grains;                  // batch * max_len <= 2^36: below 2^31
  for (int b = 64 + lane; b < a.b.batch; b += 64) total += look_up(a, b).grains;
  return part_grains(wave_sum(total), a.b.batch, a.goal, a.least / kGrain, [&](int each) {
    int parts = (mine.grains + each - 1) / each;
    for (int b = 64 + lane; b < a.b.batch; b += 64) parts += (look_up(a, b).grains + each - 1) / each;
    return wave_sum(parts);
  });
}

// What a workgroup computes: rows [begin, end) of a sequence, or of a prefix, for one key head.
struct Part {
  int kh, len, first, n, begin, end;
  int ctx;                              // rows that all its queries see
  const int32_t* table;
  int64_t at;                           // where its partial results go; -1: it is the sequence's only part
};
__device__ __forceinline__ void place_part(const AttendArgs& a, int seq, int id, bool whole, Part* p) {
  p->ctx = p->len - p->n;
  p->table = a.b.tables + (int64_t)seq * a.b.table_stride;
  p->at = whole ? -1 : ((int64_t)id * a.b.n_kv + p->kh) * (a.q.max_q * a.group);
}
// `heads`: key heads of a workgroup, of which this wave takes number `head`.
template <bool kShared>
__device__ bool find_part(const AttendArgs& a, int unit, Part* p, int heads = 1, int head = 0) {
  const int lane = threadIdx.x & 63;
  const int groups = a.b.n_kv / heads, id = unit / groups;
  p->kh = unit % groups * heads + head;
  if (!a.goal) {
    const bool shared = kShared && a.sh.groups;
    if (shared && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0u;    // the join adds what is wrong
    bool bad;
    const bool go = sequence_of(a.b, a.q, id, &p->len, &p->first, &p->n, &bad);
    if (bad && a.report && threadIdx.x == 0) atomicOr(a.status, kStatusRowsBit);
    p->begin = 0;
    p->end = p->len;
    place_part(a, id, id, !shared, p);
    return go;
  }
  Seq s = look_up(a, lane);
  const int each = grains_of_part(a, s);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *a.status = 0u;                     // the join adds what is wrong
    *a.each = each;
  }
  int before = 0;                       // parts of the sequences before these 64
  for (int b0 = 0; b0 < a.b.batch; b0 += 64) {
    if (b0) s = look_up(a, b0 + lane);
    const int mine = (s.grains + each - 1) / each;
    const int upto = wave_scan(mine);
    const uint64_t past = __ballot(before + upto > id);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
      const int parts = of(mine), split = id - before - (of(upto) - parts);
      p->len = of(s.len);
      p->first = of(s.first);
      p->n = of(s.n);
      p->begin = __builtin_amdgcn_readfirstlane((int)((int64_t)split * each * kGrain));
      p->end = p->len - p->begin < each * kGrain ? p->len : p->begin + each * kGrain;
      place_part(a, b0 + l, id, parts == 1 && !(kShared && a.sh.groups), p);
      return true;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// One group as a lane looks it up; blocks 0: nothing to do.
struct Group {
  int from, to, len, first, n, blocks, grains;
  bool ok;
};
__device__ __forceinline__ Group look_up_group(const AttendArgs& a, int g) {
  Group r = {};
  if (g >= a.sh.groups) return r;
  r.from = a.sh.starts[g];
  r.to = a.sh.starts[g + 1];
  r.len = a.sh.lengths[g];
  if (r.from < 0 || r.from > a.b.batch || r.to < 0 || r.to > a.b.batch) return r;  // not to be looked up
  r.first = a.q.start[r.from];
  const int end = a.q.start[r.to];
  r.n = (int)((unsigned)end - (unsigned)r.first);
  r.ok = is_group(r.from, r.to, r.len, r.first, end, a.b.batch, a.sh.max_len, a.q.max_q, a.q.n_q);
  if (!r.ok || r.n == 0 || r.len == 0) return r;
  r.blocks = query_blocks(r.n, a.group, a.sh.rows);
  r.grains = (r.len + kGrain - 1) / kGrain;
  return r;
}
// Groups g0 .. g0 + 63, one a lane; those that do not count (rf_split.h) are not ok.  *line: where the groups before
// them end, and then where these do.  All lanes take part.
__device__ __forceinline__ Group look_up_groups(const AttendArgs& a, int g0, GroupLine* line) {
  const int lane = threadIdx.x & 63;
  Group r = look_up_group(a, g0 + lane);
  const auto at = [](int v, int l) { return __builtin_amdgcn_readlane(v, l); };
  const int last = a.sh.groups - g0 < 64 ? a.sh.groups - g0 - 1 : 63;
  if (!__ballot(!r.ok && lane <= last) && begins_at(at(r.from, 0), at(r.first, 0), *line)) {
    // without a fault among them each ends where the next one begins
    *line = {at(r.to, last), at(r.first + r.n, last)};
    return r;
  }
  const int seq = wave_scan_max(r.ok ? r.to : 0), query = wave_scan_max(r.ok ? r.first + r.n : 0);
  const int seq_before = __shfl_up(seq, 1), query_before = __shfl_up(query, 1);
  const auto most = [](int x, int y) { return x > y ? x : y; };
  const GroupLine before = {most(line->seq, lane ? seq_before : 0), most(line->query, lane ? query_before : 0)};
  if (!begins_at(r.from, r.first, before)) {
    r.ok = false;
    r.blocks = r.grains = 0;
  }
  *line = {most(line->seq, at(seq, 63)), most(line->query, at(query, 63))};
  return r;
}

// How the groups' rows are cut into parts, and their query rows into blocks: the grains of a part, and one wave's plan
// of all groups, by which the join finds the pairs of a part and a block (it reads nothing that nobody wrote).
// `first`: groups 0 .. 63, `line`: where they end; kMany: there are more.
__device__ __forceinline__ int parts_of(const Group& r, int each) { return r.blocks * ((r.grains + each - 1) / each); }
template <bool kMany, typename Use>
__device__ __forceinline__ void past_first(const AttendArgs& a, GroupLine line, Use use) {
  if constexpr (kMany)
    for (int g0 = 64; g0 < a.sh.groups; g0 += 64) use(g0, look_up_groups(a, g0, &line));
}
template <bool kMany>
__device__ __forceinline__ int grains_of_prefix_part(const AttendArgs& a, const Group& first, GroupLine line) {
  long long total = (long long)first.blocks * first.grains;
  int blocks = first.blocks;
  past_first<kMany>(a, line, [&](int, const Group& r) {
    total += (long long)r.blocks * r.grains;
    blocks += r.blocks;
  });
  return group_grains(wave_sum(total), wave_sum(blocks), a.sh.goal, a.sh.least / kGrain, [&](int each) {
    int parts = parts_of(first, each);
    past_first<kMany>(a, line, [&](int, const Group& r) { parts += parts_of(r, each); });
    return wave_sum(parts);
  });
}
template <bool kMany>
__device__ __forceinline__ void write_plan(const AttendArgs& a, const Group& first, GroupLine line, int each) {
  int before = 0;
  const auto write = [&](int g0, const Group& r) {
    const int parts = (r.grains + each - 1) / each, mine = r.blocks * parts, upto = wave_scan(mine), g = g0 + (threadIdx.x & 63);
    if (g < a.sh.groups) a.sh.plan[g] = {(unsigned)(before + upto - mine), (unsigned)r.blocks, (unsigned)parts, r.ok};
    before += __builtin_amdgcn_readlane(upto, 63);
  };
  write(0, first);
  past_first<kMany>(a, line, write);
}

// What a workgroup computes of the prefixes: the pairs of a part and a block take turns with the key heads, blocks
// first, so that the workgroups that read the same rows run side by side.  *mb: the block.  Up to 64 groups every wave
// lays out for itself, and the first unit, which is always there, writes the plan; more are laid out by a launch
// before, and looked for in its plan (1,000 groups of two sequences, one token each: 725 us, with every wave looking all
// groups over 1,252; 65 groups 178 and 176).
inline __device__ bool find_prefix(const AttendArgs& a, int unit, Part* p, int* mb, int heads = 1, int head = 0) {
  const int lane = threadIdx.x & 63, per = a.b.n_kv / heads, id = unit / per;
  p->kh = unit % per * heads + head;
  int g, n_blocks, at, each;
  if (a.sh.groups <= 64) {
    GroupLine line = {0, 0};
    const Group r = look_up_groups(a, 0, &line);
    each = grains_of_prefix_part<false>(a, r, line);
    if (unit == 0 && threadIdx.x < 64) write_plan<false>(a, r, line, each);
    const int mine = parts_of(r, each), upto = wave_scan(mine);
    const uint64_t past = __ballot(upto > id);
    if (!past) return false;
    g = __ffsll((unsigned long long)past) - 1;
    const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, g); };
    n_blocks = of(r.blocks);
    at = id - (of(upto) - of(mine));
    p->len = of(r.len);
    p->first = of(r.first);
    p->n = of(r.n);
  } else {
    // the last group whose first pair is not past this one: those without pairs come before the next with some
    g = 0;
    for (int count = a.sh.groups; count > 1;) {
      const int step = (count + 63) / 64;
      const int upto = __popcll(__ballot(lane * step < count && (int)a.sh.plan[g + lane * step].x <= id)) - 1;
      g += upto * step;
      count = count - upto * step < step ? count - upto * step : step;
    }
    g = __builtin_amdgcn_readfirstlane(g);
    const uint4 plan = a.sh.plan[g];
    n_blocks = (int)plan.y;
    at = id - (int)plan.x;
    if (at >= n_blocks * (int)plan.z) return false;
    each = (int)*a.sh.each;
    const Group r = look_up_group(a, g);
    p->len = r.len;
    p->first = r.first;
    p->n = r.n;
  }
  const int split = at / n_blocks;
  *mb = at - split * n_blocks;
  p->ctx = p->len;
  p->begin = __builtin_amdgcn_readfirstlane((int)((int64_t)split * each * kGrain));
  p->end = p->len - p->begin < (int64_t)each * kGrain ? p->len : p->begin + each * kGrain;
  p->table = a.sh.tables + (int64_t)g * a.sh.table_stride;
  p->at = a.sh.first_row + ((int64_t)id * a.b.n_kv + p->kh) * a.sh.rows - (int64_t)*mb * a.sh.rows;
  return true;
}

// A workgroup's unit (part and key head) and block of query rows: the blocks of one unit go to
// one XCD (blockIdx % 8), side by side, where they share its cache.
__device__ __forceinline__ void place_block(const AttendArgs& a, int* unit, int* mb) {
  if (a.mblocks == 1) return;
  const int per = 8 * a.mblocks, full = (a.parts * a.b.n_kv) / 8 * per;
  const int id = *unit;
  if (id < full) {
    *mb = id % per / 8;
    *unit = id / per * 8 + id % 8;
  } else {
    *mb = (id - full) % a.mblocks;
    *unit = full / a.mblocks + (id - full) / a.mblocks;
  }
}

template <int HD>
struct Tile {                   // 32 cache rows of one head, as a wave holds them
  static constexpr int kSteps = HD / 32;
  u32x4 k[2][kSteps];           // rows 16 t + c, features 32 s + 8 g ..
  uint32_t v[8][HD / 32];       // rows 16 (j/4) + 4 g + j % 4, features (HD/16) c ..
};

template <int HD, bool kV>
__device__ __forceinline__ void load_tile(Tile<HD>& t, const AttendArgs& a, const uint16_t* kh,
                                          const uint16_t* vh, int slot, int c, int g) {
  const int64_t row = (int64_t)a.b.n_kv * HD;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint16_t* p = kh + (int64_t)__shfl(slot, 16 * h + c) * row + 8 * g;
#pragma unroll
    for (int s = 0; s < HD / 32; ++s) t.k[h][s] = *reinterpret_cast<const u32x4*>(p + 32 * s);
  }
  if constexpr (kV) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint16_t* p = vh + (int64_t)__shfl(slot, 16 * (j / 4) + 4 * g + j % 4) * row + (HD / 16) * c;
      if constexpr (HD == 128) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) t.v[j][i] = w[i];
      } else {
        const u32x2 w = *reinterpret_cast<const u32x2*>(p);
        t.v[j][0] = w[0];
        t.v[j][1] = w[1];
      }
    }
  }
}

// The end of the kernels of up to 16 query rows: the workgroup's waves' results joined and written, those of
// waves w and w + heads where the workgroup has several key heads.
template <int HD, bool kOut>
__device__ __forceinline__ void join_waves(const AttendArgs& a, const Part& pt, int heads, int m, bool in, int64_t row, int head, float m_run,
                                           float l_run, f32x4 (&o)[kOut ? HD / 16 : 1], float (*sh_o)[16][HD + 4],
                                           float2 (*sh_ml)[16]) {
  constexpr int kFeat = HD / 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  // sums over g, then the waves: 2 and 3 into 0 and 1, then 1 into 0
  l_run += __shfl_xor(l_run, 16);
  l_run += __shfl_xor(l_run, 32);
  for (int half = kWaves / 2; half >= heads; half /= 2) {
    if (wave >= half && wave < 2 * half) {
      const int w = wave - half;
      if (g == 0) sh_ml[w][c] = make_float2(m_run, l_run);
      if constexpr (kOut) {
#pragma unroll
        for (int f = 0; f < kFeat; ++f)
#pragma unroll
          for (int r = 0; r < 4; ++r) sh_o[w][c][kFeat * (4 * g + r) + f] = o[f][r];
      }
    }
    __syncthreads();
    if (wave < half) {
      const float2 ml = sh_ml[wave][c];
      const float m_new = fmaxf(m_run, ml.x), zero = m_new == -INFINITY ? 0.f : m_new;
      const float mine = __builtin_amdgcn_exp2f(m_run - zero), theirs = __builtin_amdgcn_exp2f(ml.x - zero);
      m_run = m_new;
      l_run = l_run * mine + ml.y * theirs;
      if constexpr (kOut) {
#pragma unroll
        for (int f = 0; f < kFeat; ++f)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[f][r] = o[f][r] * mine + sh_o[wave][c][kFeat * (4 * g + r) + f] * theirs;
      }
    }
    __syncthreads();
  }
  if (wave >= heads || !in) return;
  if (pt.at >= 0) {
    const int64_t part = pt.at + m;
    if (g == 0) a.part_ml[part] = make_float2(m_run, l_run);
    if constexpr (kOut) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float* p = a.part_o + part * HD + kFeat * (4 * g + r);
#pragma unroll
        for (int f = 0; f < kFeat; f += 4)
          *reinterpret_cast<f32x4*>(p + f) = f32x4{o[f][r], o[f + 1][r], o[f + 2][r], o[f + 3][r]};
      }
    }
    return;
  }
  const bool none = l_run == 0.f;
  if (a.lse && g == 0) a.lse[row * a.q.n_heads + head] = none ? -INFINITY : m_run * kLn2 + __logf(l_run);
  if constexpr (kOut) {
    const float inv = none ? 0.f : 1.f / l_run;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      uint16_t* p = a.out + row * a.out_stride + head * HD + kFeat * (4 * g + r);
#pragma unroll
      for (int f = 0; f < kFeat; f += 4) {
        u32x2 w;
        w[0] = pack_bf16x2(o[f][r] * inv, o[f + 1][r] * inv);
        w[1] = pack_bf16x2(o[f + 2][r] * inv, o[f + 3][r] * inv);
        *reinterpret_cast<u32x2*>(p + f) = none ? u32x2{0u, 0u} : w;
      }
    }
  }
}

// kOut: with the product with V (else only the statistics).
// At most 16 query rows: bound by the read of K and V.  16 sequences of up to 16,384 rows, one token,
// 8 key heads of 128 (760 MB): 148 us of the call's 153, 5.1 TB/s, as a large copy.  (The tile kernel
// below took 187 us there; this one, with four tiles of 16 queries, 120 us for 64 query rows over 65,536
// where that took 70; both with one operand a weight.)
template <int HD, bool kOut, bool kShared>
__global__ __launch_bounds__(kThreads, 2) void attend_kernel(AttendArgs a) {
  constexpr int kSteps = HD / 32, kFeat = HD / 16;
  __shared__ float sh_o[kWaves / 2][16][HD + 4];
  __shared__ float2 sh_ml[kWaves / 2][16];
  if (a.scan && blockIdx.x == 0) return scan_status(a.b, a.q, a.status);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  Part pt;
  int mb = 0;
  bool prefix = false;
  const int unit = blockIdx.x - a.scan;
  if constexpr (kShared) prefix = unit >= a.own;
  if (prefix ? !find_prefix(a, unit - a.own, &pt, &mb) : !find_part<kShared>(a, unit, &pt)) return;
  // the end as a value of each lane: counted in scalars the loop spills (and lost 5 us of 200 before)
  const int kh = pt.kh, len = pt.len, first = pt.first, begin = pt.begin, end = fresh(pt.end);
  const int m_rows = pt.n * a.group, ctx = pt.ctx, m = 16 * mb + c;

  // Q^T fragments: query row m, zero past the last
  const bool in = m < m_rows;
  const int qi = in ? m / a.group : 0, head = kh * a.group + (in ? m % a.group : 0);
  const uint64_t word = kShared && prefix ? 0ull : draft_word(a.q, first + qi, qi);
  bf16x8 qf[kSteps];
  {
    const uint16_t* p = a.q.q + (int64_t)(first + qi) * a.q.q_stride + head * HD + 8 * g;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      u32x4 w = {0u, 0u, 0u, 0u};
      if (in) w = *reinterpret_cast<const u32x4*>(p + 32 * s);
      qf[s] = __builtin_bit_cast(bf16x8, w);
    }
  }

  f32x4 o[kOut ? kFeat : 1];
  float m_run = -INFINITY, l_run = 0.f;
#pragma unroll
  for (int f = 0; f < (kOut ? kFeat : 1); ++f) o[f] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int32_t* table = pt.table;
  const uint16_t* kbase = a.kp + kh * HD;
  const uint16_t* vbase = kOut ? a.vp + kh * HD : nullptr;
  const float scale2 = a.q.scale * kLog2e;
  int page_err = 0;
  // page of row r (the last row for rows past it), then the pool slot: -1 on a bad page
  const auto page_of = [&](int base) -> int {
    const int r = base + (lane & 31);
    return table[quotient((unsigned)(r < len ? r : len - 1), a.page)];
  };
  const auto slot_of = [&](int base, int page) -> int {
    const int r0 = base + (lane & 31), r = r0 < len ? r0 : len - 1;
    if (page < 0 || page >= a.b.num_pages) return -1;
    return page * a.b.page_size + (r - (int)quotient((unsigned)r, a.page) * a.b.page_size);
  };

  int base = begin + wave * kRows;
  constexpr int kStride = kWaves * kRows;
  Tile<HD> cur;
  int page_next = 0, slot = -1;
  if (base < end) {
    slot = slot_of(base, page_of(base));
    load_tile<HD, kOut>(cur, a, kbase, vbase, slot < 0 ? 0 : slot, c, g);
    page_next = page_of(base + kStride);
  }
  for (; base < end; base += kStride) {
    // the next rows on their way (rows past the end repeat the last one, and are not used)
    const int slot_next = slot_of(base + kStride, page_next);
    Tile<HD> next;
    if (base + kStride < end) load_tile<HD, kOut>(next, a, kbase, vbase, slot_next < 0 ? 0 : slot_next, c, g);
    page_next = page_of(base + 2 * kStride);

    const uint64_t good64 = __ballot(slot >= 0);
    const uint32_t good = (uint32_t)good64;
    const bool masked = base + kRows > ctx || base + kRows > end || good != 0xffffffffu;
    if (good != 0xffffffffu) page_err = 1;
    uint32_t there = good;                            // rows of this step that exist
    if (end - base < 32) there &= (1u << (end - base)) - 1u;

    // V^T fragments
    bf16x8 vf[kOut ? kFeat : 1];
    bool wild = false;                                // a value that is not finite
    if constexpr (kOut) {
      if (masked) {
        bool w = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool in = there >> (16 * (j / 4) + 4 * g + j % 4) & 1;
#pragma unroll
          for (int i = 0; i < HD / 32; ++i) {
            if (!in) cur.v[j][i] = 0u;
            w |= (cur.v[j][i] & 0x7f80u) == 0x7f80u || (cur.v[j][i] & 0x7f800000u) == 0x7f800000u;
          }
        }
        wild = __any(w);
      }
#pragma unroll
      for (int f = 0; f < kFeat; ++f) {
        u32x4 w;
#pragma unroll
        for (int p = 0; p < 4; ++p) w[p] = half_pair(cur.v[2 * p][f / 2], cur.v[2 * p + 1][f / 2], f & 1);
        vf[f] = __builtin_bit_cast(bf16x8, w);
      }
    }

    f32x4 s[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
#pragma unroll
      for (int h = 0; h < 2; ++h) s[h] = mfma16(__builtin_bit_cast(bf16x8, cur.k[h][st]), qf[st], s[h]);
    uint32_t seen = 0xffffffffu;                    // rows that this lane's query sees
    if (masked) {
      seen = there;
      if (base + kRows > ctx) seen &= seen_rows(word, base - ctx);
    }
    float x[8], top = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = s[j / 4][j % 4] * scale2;
      if (masked && !(seen >> (16 * (j / 4) + 4 * g + j % 4) & 1)) x[j] = -INFINITY;
      top = fmaxf(top, x[j]);
    }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    if (__any(top > m_run + kSlack)) {
      const float m_new = fmaxf(m_run, top);
      const float shrink = __builtin_amdgcn_exp2f(m_run - (m_new == -INFINITY ? 0.f : m_new));
      l_run *= shrink;
      if constexpr (kOut) {
#pragma unroll
        for (int f = 0; f < kFeat; ++f) o[f] *= shrink;
      }
      m_run = m_new;
    }
    const float zero = m_run == -INFINITY ? 0.f : m_run;
    float p[8], sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = __builtin_amdgcn_exp2f(x[j] - zero);
      sum += p[j];
    }
    l_run += sum;
    if constexpr (kOut) {
      u32x4 pw[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Weights w = split_weights(p[2 * i], p[2 * i + 1]);
        pw[0][i] = w.lead;
        pw[1][i] = w.rest;
      }
      if (!wild) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int f = 0; f < kFeat; ++f) o[f] = mfma16(vf[f], __builtin_bit_cast(bf16x8, pw[k]), o[f]);
      } else {
        // Some value is infinite or NaN, and 0 times it is not 0: row by row, added only
        // for the queries that see the row.
        for (int r = 0; r < kRows; ++r) {
          const int rg = r % 16 / 4, j = r / 16 * 4 + r % 4;
          const bool vis = __shfl(seen, 16 * rg + c) >> r & 1;
          const uint32_t keep = j & 1 ? 0xffff0000u : 0x0000ffffu;
          u32x4 pr[2];
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) pr[k][i] = g == rg && i == j / 2 ? pw[k][i] & keep : 0u;
#pragma unroll
          for (int f = 0; f < kFeat; ++f) {
            const u32x4 vw = __builtin_bit_cast(u32x4, vf[f]);
            u32x4 vr;
#pragma unroll
            for (int i = 0; i < 4; ++i) vr[i] = g == rg && i == j / 2 ? vw[i] & keep : 0u;
            f32x4 add = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 2; ++k) add = mfma16(__builtin_bit_cast(bf16x8, vr), __builtin_bit_cast(bf16x8, pr[k]), add);
            if (vis) o[f] += add;
          }
        }
      }
    }
    cur = next;
    slot = slot_next;
  }
  if (page_err && a.report && lane == 0) atomicOr(a.status, kStatusRowsBit);
  join_waves<HD, kOut>(a, pt, 1, m, in, first + qi, head, m_run, l_run, o, sh_o, sh_ml);
}

// 16 bytes per lane from base + off (bytes) to the LDS address lds + 16 lane (lds: the same in the wave).  The
// compiler does not see the load: dma_wait before the barrier that hands the data on.
__device__ __forceinline__ void dma_row(const uint16_t* base, uint64_t off, uint32_t lds) {
  const unsigned char* p = reinterpret_cast<const unsigned char*>(base) + off;
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(p), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory", "m0");
}
template <int kLeft>                  // until at most kLeft loads are under way
__device__ __forceinline__ void dma_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(kLeft) : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

template <int kBytes>                 // 4 or 16 of each lane
__device__ __forceinline__ void dma_to(const uint8_t* p, uint32_t lds) {
  if constexpr (kBytes == 16)
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(p), "s"(__builtin_amdgcn_readfirstlane(lds))
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
                 :
                 : "v"(p), "s"(__builtin_amdgcn_readfirstlane(lds))
                 : "memory", "m0");
}
// The value of lane ^ 32.
__device__ __forceinline__ float other_half(float v) {
  const int x = __builtin_bit_cast(int, v);
  const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return __builtin_bit_cast(float, (threadIdx.x & 32) ? r[0] : r[1]);
}

// The value of lane ^ 16.
__device__ __forceinline__ float other_sixteen(float v) {
  const int x = __builtin_bit_cast(int, v);
  const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  return __builtin_bit_cast(float, (threadIdx.x & 16) ? r[0] : r[1]);
}

// What was read of LDS has arrived: it may be overwritten.
__device__ __forceinline__ void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }

// The same over codes.  A step's bytes are half as many, so twice as many waves have to be under way:
// each has its 32 rows in LDS of its own, where direct loads put them without holding registers, and
// sends for the next rows' keys as soon as the scores are formed, for their values as soon as the
// product is.  No wave waits for another.  Values exist two features at a time.
// A head's scales are 4 bytes of each line of 128, and what a compute unit can have under way is counted in
// lines (its first cache holds 256): four waves that take different rows of one head have 80 lines of a
// step where 64 hold its codes.  So they take the same rows of four heads, whose scales share the lines.
// Row r lies at place r ^ (r / 4 & kSwap), its pieces of 16 bytes turned by the place, so that few of the keys'
// reads (16 rows at a time) and the values' (rows 4 apart) meet in a bank: LDS moves data in 13% of the
// cycles, a quarter of those are conflicts.
// Bound by memory: one token of 16 fp8 sequences of up to 16,384 rows, 8 key heads of 128 (402 MB), 86 us of the
// call's 93, 4.6 TB/s; reading the rows and nothing else takes 78.  In registers, two waves a SIMD, 110.
constexpr int kCodeTiles = 8;         // steps of a wave whose slots are looked up at a time
template <int HD>
struct WaveRows {                     // a wave's rows in LDS
  static constexpr int kSwap = HD == 128 ? 1 : 3, kPieces = HD / 16;
  unsigned char k[kRows * HD], v[kRows * HD];
  unsigned scales[2][64];             // k's, then v's, by turns
  int slot[kCodeTiles * kRows];
  static constexpr unsigned turn_shift = HD == 128 ? 1 : 2;
  __host__ __device__ static constexpr unsigned place(unsigned row) { return row ^ (row >> 2 & kSwap); }
  __host__ __device__ static constexpr unsigned turn(unsigned place) { return place >> turn_shift & (kPieces - 1); }
  // Byte offsets in k or v; the parts that the lane and the loop's index give differ in their bits, so that
  // one kept address and a constant make each.
  // Features 32 s + 8 g .. of row c (and of 16 + c, 16 HD further).
  __device__ static unsigned key(unsigned c, unsigned g) { return place(c) * HD + (((g >> 1) ^ turn(place(c))) << 4) + 8 * (g & 1); }
  static constexpr unsigned key_step(int s) { return 32u * s; }
  // Features (HD/16) c .. of row 4 g + j, j < 4 (and of 16 + 4 g + j).
  __device__ static unsigned value(unsigned c, unsigned g) {
    return place(4 * g) * HD + (((c * (HD / 16) >> 4) ^ turn(place(4 * g))) << 4) + c * (HD / 16) % 16;
  }
  static constexpr unsigned value_step(int j) { return (unsigned)j * HD + (turn((unsigned)j) << 4); }
};
// Rows 4 g + j for j < 4 lie at place(4 g) ^ j and are turned by turn(place(4 g)) ^ turn(j); rows c and 16 + c
// are turned alike.
template <int HD>
constexpr bool places_split() {
  using R = WaveRows<HD>;
  for (unsigned r = 0; r < 32; ++r) {
    if (R::place(r) != (R::place(r & ~3u) ^ (r & 3))) return false;
    if (R::turn(R::place(r)) != (R::turn(R::place(r & ~3u)) ^ R::turn(r & 3))) return false;
    if (R::turn(R::place(r & 15)) != R::turn(R::place(r))) return false;
    if (R::place(R::place(r)) != r) return false;
  }
  return true;
}
static_assert(places_split<128>() && places_split<64>(), "how rows lie in LDS");

template <int HD, bool kOut, int kType>
__global__ __launch_bounds__(kThreads, 4) void attend_codes_kernel(AttendArgs a) {
  constexpr int kSteps = HD / 32, kFeat = HD / 16;
  using Rows = WaveRows<HD>;
  constexpr int kLoads = kRows * HD / 1024;             // direct loads of a step's keys, and values
  struct Join {
    float o[kWaves / 2][16][HD + 4];
    float2 ml[kWaves / 2][16];
  };
  __shared__ union __attribute__((aligned(256))) {
    Rows rows[kWaves];
    Join join;
  } sh;
  if (a.scan && blockIdx.x == 0) return scan_status(a.b, a.q, a.status);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  Part pt;
  int mb = 0;
  const int unit = blockIdx.x - a.scan;
  const bool prefix = unit >= a.own;
  const int heads = a.heads, rank = wave / heads, ranks = kWaves / heads;   // which of a head's waves this is
  if (prefix ? !find_prefix(a, unit - a.own, &pt, &mb, heads, wave % heads) : !find_part<true>(a, unit, &pt, heads, wave % heads)) return;
  const auto same = [](int v) { return __builtin_amdgcn_readfirstlane(v); };   // in all lanes: scalar
  const int kh = same(pt.kh), len = same(pt.len), first = same(pt.first), begin = same(pt.begin), end = same(pt.end);
  const int m_rows = same(pt.n * a.group), ctx = same(pt.ctx);
  const auto same_pointer = [&](const void* p) {
    typedef const __attribute__((address_space(1))) uint8_t* global;
    const uint64_t bits = reinterpret_cast<uint64_t>(p);
    return (global)((uint64_t)(uint32_t)same((int)(bits >> 32)) << 32 | (uint32_t)same((int)bits));
  };
  const auto table = (const __attribute__((address_space(1))) int32_t*)same_pointer(pt.table);
  // query row of this lane, its query and head; formed where they are used
  struct Row {
    int m, qi, head;
    bool in;
  };
  const auto row_of_query = [&]() -> Row {
    const int m = 16 * mb + (fresh(lane) & 15);
    const bool in = m < m_rows;
    return {m, in ? m / a.group : 0, kh * a.group + (in ? m % a.group : 0), in};
  };
  bf16x8 qf[kSteps];
  // a load of it in the loop would be waited for with the rows under way
  uint64_t word = 0ull;
  {
    const Row q = row_of_query();
    if (!prefix) word = draft_word(a.q, first + q.qi, q.qi);
    const uint16_t* p = a.q.q + (int64_t)(first + q.qi) * a.q.q_stride + q.head * HD + 8 * g;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      u32x4 w = {0u, 0u, 0u, 0u};
      if (q.in) w = *reinterpret_cast<const u32x4*>(p + 32 * s);
      qf[s] = __builtin_bit_cast(bf16x8, w);
    }
  }
  f32x4 o[kOut ? kFeat : 1];
  float m_run = -INFINITY, l_run = 0.f;
#pragma unroll
  for (int f = 0; f < (kOut ? kFeat : 1); ++f) o[f] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float scale2 = a.q.scale * kLog2e;
  int page_err = 0;
  Rows& rows = sh.rows[wave];
  constexpr int kPages = kCodeTiles * kRows / 64;
  const int stride = ranks * kRows, base0 = begin + rank * kRows;
  const int tiles = base0 < end ? (end - base0 + stride - 1) / stride : 0;
  // the wave's row of one of its steps; rows past the last repeat it
  const auto row_of = [&](int i) {
    const int r = base0 + i / kRows * stride + i % kRows;
    return r < len ? r : len - 1;
  };
  const auto look_up_pages = [&](int tile, int (&page)[kPages]) {
    const int ln = fresh(lane);
#pragma unroll
    for (int i = 0; i < kPages; ++i) page[i] = table[quotient((unsigned)row_of(tile * kRows + 64 * i + ln), a.page)];
  };
  const auto set_slots = [&](int tile, const int (&page)[kPages]) {
    const int ln = fresh(lane);
#pragma unroll
    for (int i = 0; i < kPages; ++i) {
      const int r = row_of(tile * kRows + 64 * i + ln);
      rows.slot[64 * i + ln] = page[i] < 0 || page[i] >= a.b.num_pages
                                     ? -1 : page[i] * a.b.page_size + (r - (int)quotient((unsigned)r, a.page) * a.b.page_size);
    }
  };
  // Where a row lies in the pools: slot n_kv + kh, in rows of one head.  Of a direct load's 64 / kPieces rows this
  // lane loads one piece; the rows of the next load are 64 / kPieces on in either order.
  const unsigned row_bytes = a.b.n_kv * HD;
  const uint8_t* kbase = reinterpret_cast<const uint8_t*>(a.kp) + (int64_t)kh * HD;
  const uint8_t* vbase = reinterpret_cast<const uint8_t*>(a.vp) + (int64_t)kh * HD;
  constexpr int kEach = 64 / Rows::kPieces;
  static_assert(Rows::turn(kEach) == 0 || Rows::turn(kEach) == Rows::kPieces / 2, "every other load is turned the other way");
  const unsigned mine = lane / Rows::kPieces, my_row = Rows::place(mine), my_piece = 16 * ((lane % Rows::kPieces) ^ Rows::turn(mine));
  const auto slots_of = [&](int tile) { return rows.slot + tile % kCodeTiles * kRows; };
  const auto load_rows = [&](const uint8_t* base, unsigned char* to, int tile) {
    const unsigned row0 = fresh(my_row), piece0 = fresh(my_piece);   // what is formed from them is not kept
    int slot[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) slot[i] = slots_of(tile)[row0 + kEach * i];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint64_t off = (uint64_t)(unsigned)(slot[i] < 0 ? 0 : slot[i]) * row_bytes;
      dma_to<16>(base + off + (piece0 ^ Rows::turn(kEach * i) << 4), lds_address(to) + 1024 * i);
    }
  };
  const auto load_keys = [&](int tile) {
    load_rows(kbase, rows.k, tile);
    const int ln = fresh(lane), slot = slots_of(tile)[ln & 31];
    const int64_t at = (int64_t)(slot < 0 ? 0 : slot) * a.b.n_kv + kh;
    const uint8_t* p = (kOut && (ln & 32) ? a.vs : a.ks) + (HD == 128 ? 4 * at : 2 * at & ~(int64_t)3);
    dma_to<4>(p, lds_address(rows.scales[tile & 1]));
  };
  // the scales of a row's blocks: of hd 64 half of a word
  const auto scales_of = [&](unsigned w, int tile, int row) -> unsigned {
    if constexpr (HD == 128) return w;
    const int slot = slots_of(tile)[row];
    return ((slot < 0 ? 0 : slot) * (a.b.n_kv & 1) + kh) & 1 ? w >> 16 : w & 0xffffu;
  };
  const unsigned key_at = Rows::key(c, g), value_at = Rows::value(c, g);

  int page[kPages];
  if (tiles) {
    look_up_pages(0, page);
    set_slots(0, page);
    load_keys(0);
    if constexpr (kOut) load_rows(vbase, rows.v, 0);
  }
  for (int tile = 0; tile < tiles; ++tile) {
    const int base = base0 + tile * stride;
    const uint32_t good = (uint32_t)__ballot(slots_of(tile)[lane & 31] >= 0);
    const bool masked = base + kRows > ctx || base + kRows > end || good != 0xffffffffu, more = tile + 1 < tiles;
    if (good != 0xffffffffu) page_err = 1;
    uint32_t there = good;                            // rows of this step that exist
    if (end - base < 32) there &= (1u << (end - base)) - 1u;

    dma_wait<kOut ? kLoads : 0>();                    // the keys and scales; the values may be under way
    f32x4 s[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    const unsigned* scales = rows.scales[tile & 1];
    const unsigned key0 = fresh(key_at);
    unsigned vscale[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const unsigned ks = scales_of(scales[16 * h + c], tile, 16 * h + c);
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(rows.k + (key0 ^ Rows::key_step(st)) + 16 * h * HD);
        const float f = scale_of(ks >> (8 * st) & 255u);
        const u32x2 x = values_of<kType>(w[0], f), y = values_of<kType>(w[1], f);
        s[h] = mfma16(__builtin_bit_cast(bf16x8, (u32x4{x[0], x[1], y[0], y[1]})), qf[st], s[h]);
      }
      if constexpr (kOut) {
        // of rows 16 h + 4 g .. + 3, this lane's block
        const u32x4 w = *reinterpret_cast<const u32x4*>(scales + 32 + 16 * h + 4 * g);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          vscale[4 * h + j] = scales_of(w[j], tile, 16 * h + 4 * g + j) >> (8 * (c * (HD / 16) / kBlock)) & 255u;
      }
    }
    reads_done();
    if (more) {
      if ((tile + 1) % kCodeTiles == 0) {
        look_up_pages(tile + 1, page);
        set_slots(tile + 1, page);
      }
      load_keys(tile + 1);
    }

    uint32_t seen = 0xffffffffu;                      // rows that this lane's query sees
    if (masked) {
      seen = there;
      if (base + kRows > ctx) seen &= seen_rows(word, base - ctx);
    }
    float x[8];
    {
      // rounded here, as the kernel of bf16 caches does, not joined with the subtraction below
#pragma clang fp contract(off)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = s[j / 4][j % 4] * scale2;
    }
    if (masked) {
      const uint32_t mine = seen >> (4 * (fresh(lane) >> 4));   // a branch: not what all steps would compute
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!(mine >> (16 * (j / 4) + j % 4) & 1)) x[j] = -INFINITY;
    }
    float top = x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) top = fmaxf(top, x[j]);
    top = fmaxf(top, other_sixteen(top));
    top = fmaxf(top, other_half(top));
    if (__any(top > m_run + kSlack)) {
      const float m_new = fmaxf(m_run, top);
      const float shrink = __builtin_amdgcn_exp2f(m_run - (m_new == -INFINITY ? 0.f : m_new));
      l_run *= shrink;
      if constexpr (kOut) {
#pragma unroll
        for (int f = 0; f < kFeat; ++f) o[f] *= shrink;
      }
      m_run = m_new;
    }
    const float zero = m_run == -INFINITY ? 0.f : m_run;
    float p[8], sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = __builtin_amdgcn_exp2f(x[j] - zero);
      sum += p[j];
    }
    l_run += sum;
    if constexpr (kOut) {
      u32x4 pw[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Weights w = split_weights(p[2 * i], p[2 * i + 1]);
        pw[0][i] = w.lead;
        pw[1][i] = w.rest;
      }
      if (more)
        dma_wait<kLoads + 1>();                       // only the next keys and scales may be under way
      else
        dma_wait<0>();
      unsigned w[8][HD / 64];
      const unsigned value0 = fresh(value_at);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const unsigned char* at = rows.v + (value0 ^ Rows::value_step(j % 4)) + j / 4 * 16 * HD;
        if constexpr (HD == 128) {
          const u32x2 y = *reinterpret_cast<const u32x2*>(at);
          w[j][0] = y[0];
          w[j][1] = y[1];
        } else {
          w[j][0] = *reinterpret_cast<const unsigned*>(at);
        }
      }
      reads_done();
      if (more) load_rows(vbase, rows.v, tile + 1);
      uint32_t lost = 0u;                             // rows whose block of this lane's outputs is NaN
      if (masked) {
        // 0 times what a query does not see has to be 0: rows that are not there and NaN blocks become 0;
        // queries that see such a block get its NaN below
        const int g = fresh(lane) >> 4;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = 16 * (j / 4) + 4 * g + j % 4;
          bool gone = !(there >> r & 1), nan = false;
#pragma unroll
          for (int i = 0; i < HD / 64; ++i) nan |= not_finite<kType>(w[j][i], vscale[j]);
          if (nan && !gone) lost |= 1u << r;
          gone |= nan;
          if (gone) vscale[j] = 127u;
#pragma unroll
          for (int i = 0; i < HD / 64; ++i)
            if (gone) w[j][i] = 0u;
        }
        if (__any(lost != 0u)) {
          // a block lies in 4 (hd 128) or 8 lanes c of all g; its outputs in the lanes of one or two g
#pragma unroll
          for (int d = 16; d < 64; d <<= 1) lost |= __shfl_xor(lost, d);
#pragma unroll
          for (int d = 1; d < 512 / HD; d <<= 1) lost |= __shfl_xor(lost, d);
          lost = __shfl(lost, HD == 128 ? 4 * g : 8 * (g / 2));
        }
      }
#pragma unroll
      for (int i = 0; i < kFeat / 2; ++i) {
        __builtin_amdgcn_sched_barrier(0);            // features 2 i and 2 i + 1 of every lane's eight
        unsigned row[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) row[j] = value_pair<kType>(w[j][i / 2], i & 1, scale_of(vscale[j]));
        u32x4 vf[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int q = 0; q < 4; ++q) vf[e][q] = half_pair(row[2 * q], row[2 * q + 1], e);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            o[2 * i + e] = mfma16(__builtin_bit_cast(bf16x8, vf[e]), __builtin_bit_cast(bf16x8, pw[n]), o[2 * i + e]);
      }
      if (__ballot(masked && (seen & lost)) && (seen & lost)) {
        asm volatile("");
#pragma unroll
        for (int f = 0; f < kFeat; ++f)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[f][r] = NAN;
      }
    }
  }
  if (page_err && a.report && lane == 0) atomicOr(a.status, kStatusRowsBit);
  __syncthreads();                                    // all waves are done with their rows
  const Row q = row_of_query();
  join_waves<HD, kOut>(a, pt, heads, q.m, q.in, first + q.qi, q.head, m_run, l_run, o, sh.join.o, sh.join.ml);
}

// More than 16 query rows: bound by the matrix cores and the exponentials, so K and V go
// through LDS and are shared by the workgroup's eight waves, each of which keeps 32 query rows
// (32x32x16 MFMAs, the same transposed products: lane (q, h) = (lane % 32, lane / 32) of S^T
// holds cache rows 8 (r / 4) + 4 h + r % 4, r < 16).  WM of the waves lie along the query rows, with
// WM = 4 two have the same ones, each with half of a step's cache rows, and are added at the end.
// The rows of a step (64) are copied into LDS as they are, by direct loads that hold no
// registers, two steps ahead of the products: four buffers, one barrier a step.  K^T's fragments
// are 16-byte reads, V^T's are transposing reads (four rows of one feature a lane).  The pieces of
// a row lie in another order in each of the rows that are read at a time (16 of K's 16 bytes, four
// of V's 64), so that these come from all 64 banks: no conflicts, where turns of eight and two
// rows gave as many cycles of them as of reads and 153 instead of 150 us for 65,536 rows.  The pool
// slots of the workgroup's rows are looked up beforehand: a table load between the direct loads
// would wait for those.
// Trees of up to 48 tokens on 4 sequences of up to 32,768 rows, 32 query and 8 key heads of 128: 173 us
// with the join's 9, 429 TFLOP/s; one of 64 tokens over 65,536 rows, 40 query heads: 175 us, 490 TFLOP/s;
// 32 query heads there: 112 and 9 us, 615 TFLOP/s.
// What bounds it are the matrix products (36 to 39% of the cycles) beside the vector instructions (50%,
// exponentials included) of two waves to a SIMD, at 1.6 to 1.9 GHz; and waves with no query rows: a step
// takes nearly as long with five busy (132 to 192 query rows, the trees) as with eight, and of 320 query
// rows the block of 64 keeps two of eight busy for as many parts of the cache as the block of 256.
// Blocks of 128 query rows that loaded through registers took 248 us, two workgroups for each compute
// unit 203 (139 with the present ones, all with one operand a weight).
constexpr int kTileRows = 64;
constexpr int kTileWaves = 8;
constexpr int kBufs = 4;
constexpr int kSlots = 4096;          // cache rows whose slots are looked up at a time

// Whether one of eight bf16 values is infinite or NaN.
__device__ __forceinline__ bool not_finite(u32x4 w) {
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) any |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
  return any;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
// Eight cache rows of one feature: two transposing reads of four rows, eight rows apart.
__device__ __forceinline__ bf16x8 read_transposed(const unsigned char* p, int apart) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  typedef const __attribute__((address_space(3))) unsigned char lds_byte;
  struct Pair {
    s16x4 a, b;
  } pr = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_byte*)p),
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds_byte*)(p + apart))};
  return __builtin_bit_cast(bf16x8, pr);
}

// How the pieces of an LDS row are turned: of K in 16 bytes, of V in 64.
template <int HD>
__device__ __forceinline__ unsigned k_turn(unsigned row) {
  return HD == 128 ? row & 15 : row >> 1 & 7;
}
template <int HD>
__device__ __forceinline__ unsigned v_turn(unsigned row) {
  return HD == 128 ? row & 3 : row >> 1 & 1;
}

// A thread's codes of a step: the eighth p of a row's, all in one block.  Trees of up to 48 tokens on 4 int8 sequences
// of up to 32,768 rows: 155 us a call (the same from bf16: 170); 8 trees of 24 after a prefix of 65,536 rows, 40
// query heads: 419 to 433, 605 to 620 TFLOP/s.
template <int HD>
struct Codes {
  unsigned w[HD / 32];
  unsigned scale;
  __device__ void load(const uint8_t* pool, const uint8_t* scales, int64_t at, int p) {
    if constexpr (HD == 128) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(pool + at * HD + 16 * p);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = x[i];
    } else {
      const u32x2 x = *reinterpret_cast<const u32x2*>(pool + at * HD + 8 * p);
      w[0] = x[0];
      w[1] = x[1];
    }
    scale = scales[at * (HD / kBlock) + p * (HD / 8) / kBlock];
  }
  // Their values into the row's pieces of 16 bytes, each where its turn puts it.
  template <int kType>
  __device__ void store(unsigned char* row, int p, unsigned turn) const {
    const float f = scale_of(scale);
#pragma unroll
    for (int i = 0; i < HD / 64; ++i) {
      const u32x2 x = values_of<kType>(w[2 * i], f), y = values_of<kType>(w[2 * i + 1], f);
      *reinterpret_cast<u32x4*>(row + (((HD / 64 * p + i) ^ turn) << 4)) = u32x4{x[0], x[1], y[0], y[1]};
    }
  }
};

// Eight values of a pool of codes, from feature `at` of it on.
template <int kType>
__device__ __forceinline__ u32x4 values_at(const uint16_t* pool, const uint8_t* scales, int64_t at) {
  const u32x2 w = *reinterpret_cast<const u32x2*>(reinterpret_cast<const uint8_t*>(pool) + at);
  const float f = scale_of(scales[at / kBlock]);
  const u32x2 x = values_of<kType>(w[0], f), y = values_of<kType>(w[1], f);
  return {x[0], x[1], y[0], y[1]};
}

template <int HD, int WM, bool kOut, int kType, bool kShared>
__global__ __launch_bounds__(64 * kTileWaves, 2) void attend_tile_kernel(AttendArgs a) {
  constexpr bool kCodes = kType != RF_CACHE_BF16;
  constexpr int kS = HD / 16;                 // MFMA steps over the features
  constexpr int kF = HD / 32;                 // feature tiles
  constexpr int kE = WM / 4;                  // groups of 32 cache rows of a step that a wave takes
  constexpr int kRowBytes = 2 * HD, kPieces = HD / 8;
  constexpr int kLoadRows = 64 / kPieces;     // rows of one direct load of a wave
  constexpr int kLoads = kTileRows / kLoadRows / kTileWaves;   // a wave's for K, and for V, of a step
  constexpr int kAhead = kLoads * (kOut ? 2 : 1);
  static_assert(kLoads >= 1 && kLoads * kLoadRows * kTileWaves == kTileRows, "rows of a step");
  constexpr int kBufBytes = kTileRows * kRowBytes;
  __shared__ __attribute__((aligned(256))) unsigned char sh_kv[kBufs * kBufBytes * (kOut ? 2 : 1)];
  __shared__ int sh_slot[kSlots];
  __shared__ unsigned long long sh_wild;      // drafts with a value that is not finite, a bit each
  if (a.scan && blockIdx.x == 0) return scan_status(a.b, a.q, a.status);
  int unit = blockIdx.x - a.scan, mb = 0;
  const bool prefix = kShared && unit >= a.own;
  if (!prefix) place_block(a, &unit, &mb);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h = lane >> 5;
  // this wave's query rows, and its first group.  Few query rows are spread over the SIMDs (wave % 4): for 32 and 64
  // of 4 int8 sequences of up to 32,768 rows 89 and 95 us; both groups of a row's on one SIMD: 116 and 119.
  const int wm = WM == 4 ? wave / 2 : wave, e0 = WM == 4 ? wave % 2 : 0;

  Part pt;
  if (prefix ? !find_prefix(a, unit - a.own, &pt, &mb) : !find_part<kShared>(a, unit, &pt)) return;
  // the end is the same in all lanes: the loop's counting is scalar (148 -> 145 us for 65,536 rows; the
  // kernel above loses 5 us of 200 by it)
  const int kh = pt.kh, first = pt.first, begin = pt.begin;
  const int end = __builtin_amdgcn_readfirstlane(pt.end);
  const int m_rows = pt.n * a.group, m0 = mb * 32 * WM;
  if (m0 >= m_rows) return;
  const int ctx = pt.ctx;

  // this wave's 32 query rows; a negative scale turns their sign, so that the largest product
  // is the largest score, and a scale of 0 makes them 0
  const int m = m0 + 32 * wm + c;
  const bool busy = m0 + 32 * wm < m_rows, in = m < m_rows;
  // Waves without query rows, where there are two of them or more, turn the codes into values for the others, who share
  // the SIMDs with them: 4 int8 sequences of up to 32,768 rows, trees of up to 48 (192 to 132 query rows) 174 -> 155
  // us.  (In workgroups of 128 query rows there are waves to spare: 64 rows 94 -> 110.)
  const int rest = m_rows - m0, workers = rest < 32 * WM ? (rest + 31) / 32 : WM, idle = kTileWaves - workers;
  const bool staged = kCodes && WM == 8 && idle >= 2;
  const int qi = in ? m / a.group : 0;
  const uint64_t word = prefix ? 0ull : draft_word(a.q, first + qi, qi);
  const float scale2 = (a.q.scale == 0.f ? 1.f : fabsf(a.q.scale)) * kLog2e;
  bf16x8 qf[kS];
  {
    const uint16_t* p = a.q.q + (int64_t)(first + qi) * a.q.q_stride + (kh * a.group + (in ? m % a.group : 0)) * HD + 8 * h;
    const uint32_t flip = a.q.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      u32x4 w = {0u, 0u, 0u, 0u};
      if (in && a.q.scale != 0.f) w = *reinterpret_cast<const u32x4*>(p + 16 * s) ^ flip;
      qf[s] = __builtin_bit_cast(bf16x8, w);
    }
  }
  f32x16 o[kOut ? kF : 1];
#pragma unroll
  for (int f = 0; f < (kOut ? kF : 1); ++f)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[f][r] = 0.f;
  float m_run = -INFINITY, l_run = 0.f;

  const int32_t* table = pt.table;
  const int64_t row_size = (int64_t)a.b.n_kv * HD;
  const unsigned row_bytes = 2u * a.b.n_kv * HD;
  const uint16_t* kbase = a.kp + kh * HD;
  const uint16_t* vbase = kOut ? a.vp + kh * HD : nullptr;
  // of 8 bits: a thread's share of a step's rows, 16 (hd 128) or 8 codes of one row of each, which
  // wait in registers for their place in LDS; a wave takes eight rows, its own or those that it is given
  struct Share {
    Codes<HD> k, v;
  };
  Share mine;
  const auto k_at = [&](int step) { return sh_kv + step % kBufs * kBufBytes; };
  const auto v_at = [&](int step) { return sh_kv + (kBufs + step % kBufs) * kBufBytes; };
  const auto load_codes = [&](int step, int eight, Share& to) {
    const int t = fresh(lane), slot = sh_slot[step * kTileRows + eight * 8 + (t >> 3)];
    const int64_t at = (int64_t)(slot < 0 ? 0 : slot) * a.b.n_kv + kh;
    to.k.load(reinterpret_cast<const uint8_t*>(a.kp), a.ks, at, t & 7);
    if constexpr (kOut) to.v.load(reinterpret_cast<const uint8_t*>(a.vp), a.vs, at, t & 7);
  };
  const auto store_codes = [&](int step, int eight, const Share& from) {
    const int t = fresh(lane), row = eight * 8 + (t >> 3), p = t & 7;
    from.k.template store<kType>(k_at(step) + row * kRowBytes, p, k_turn<HD>(row));
    if constexpr (kOut) from.v.template store<kType>(v_at(step) + row * kRowBytes, p, v_turn<HD>(row) << 2);
  };
  const auto load = [&](int step) {
    if constexpr (kCodes) {
      if (!staged) load_codes(step, wave, mine);
      return;
    }
    const unsigned ln = fresh(lane), at = ln % kPieces;   // where the lane's piece goes
    int slot[kLoads];                                     // together: no load waits between two of them
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      slot[i] = sh_slot[step * kTileRows + (wave * kLoads + i) * kLoadRows + ln / kPieces];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const unsigned block = wave * kLoads + i, row = block * kLoadRows + ln / kPieces;
      const uint64_t off = (uint64_t)(unsigned)(slot[i] < 0 ? 0 : slot[i]) * row_bytes;
      dma_row(kbase + (at ^ k_turn<HD>(row)) * 8, off, lds_address(k_at(step)) + block * 1024);
      if constexpr (kOut) dma_row(vbase + (at ^ v_turn<HD>(row) << 2) * 8, off, lds_address(v_at(step)) + block * 1024);
    }
  };

  const auto store = [&](int step) {
    if (!staged) store_codes(step, wave, mine);
  };

  // Looks the slots of up to kSlots rows up and returns the steps that they take.
  const auto look_up_slots = [&](int part) {
    const int rows = end - part < kSlots ? end - part : kSlots;
    const int steps = (rows + kTileRows - 1) / kTileRows;
    if (part > begin) __syncthreads();                    // the slots before are done with
    bool err = false;
    int page[kSlots / 64 / kTileWaves];                   // table loads together
#pragma unroll
    for (int i = 0; i < kSlots / 64 / kTileWaves; ++i) {
      const int x = tid + 64 * kTileWaves * i;
      page[i] = x < rows ? table[quotient((unsigned)(part + x), a.page)] : 0;
    }
#pragma unroll
    for (int i = 0; i < kSlots / 64 / kTileWaves; ++i) {
      const int x = tid + 64 * kTileWaves * i;
      const bool is = x < rows && page[i] >= 0 && page[i] < a.b.num_pages;
      if (x < rows && !is) err = true;
      if (x < steps * kTileRows)                          // -1: not there
        sh_slot[x] = is ? page[i] * a.b.page_size + (part + x - (int)quotient((unsigned)(part + x), a.page) * a.b.page_size) : -1;
    }
    if (a.report && __any(err) && lane == 0) atomicOr(a.status, kStatusRowsBit);
    if (tid == 0 && part == begin) sh_wild = 0ull;
    __builtin_amdgcn_s_waitcnt(0x0f70);                   // vmcnt(0): only direct loads from here on
    __syncthreads();
    return steps;
  };
  // rows of a step that exist, and whether some query does not see all 64
  const auto there_at = [&](int step) -> uint64_t { return __ballot(sh_slot[step * kTileRows + lane] >= 0); };
  const auto masked_at = [&](int part, int step, uint64_t there) { return ~there || part + (step + 1) * kTileRows > ctx; };
  // Hands a step's rows to all waves.
  const auto meet = [&](int part, int step) {
    __syncthreads();
    const uint64_t there = there_at(step);
    if (kOut && masked_at(part, step, there)) {
      // 0 times what a query does not see has to be 0: rows that are not there become 0, and so do
      // pieces of a draft's row with an infinity or NaN, which is remembered for the end
      for (int x = tid; x < kTileRows * kPieces; x += 64 * kTileWaves) {
        u32x4* p = reinterpret_cast<u32x4*>(v_at(step)) + x;
        const int r = x / kPieces, draft = part + step * kTileRows + r - ctx;
        const bool is = there >> r & 1, wild = is && draft >= 0 && not_finite(*p);
        if (!is || wild) *p = u32x4{0u, 0u, 0u, 0u};
        if (wild) atomicOr(&sh_wild, 1ull << draft);
      }
      __syncthreads();
    }
  };
  if constexpr (kCodes && WM == 8) {
    if (staged && !busy) {
      // up to four times eight rows of a step (rows past the last ones are loaded, and not stored)
      Share shares[4];
      const auto send = [&](int step) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int eight = wave - workers + i * idle;
          load_codes(step, eight < kTileRows / 8 ? eight : kTileRows / 8 - 1, shares[i]);
        }
      };
      const auto keep = [&](int step) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int eight = wave - workers + i * idle;
          if (eight < kTileRows / 8) store_codes(step, eight, shares[i]);
        }
      };
      for (int part = begin; part < end; part += kSlots) {
        const int steps = look_up_slots(part);
        send(0);
        keep(0);
        if (1 < steps) send(1);
        for (int step = 0; step < steps; ++step) {
          meet(part, step);
          if (step + 1 < steps) keep(step + 1);
          if (step + 2 < steps) send(step + 2);
        }
      }
      return;
    }
  }

  for (int part = begin; part < end; part += kSlots) {
    const int steps = look_up_slots(part);
    f32x16 s[kE];
    // The order of reads, products and exponentials is pinned: fragments are read four products
    // ahead, and between two products of V the exponentials of the next sixteen rows.
    const auto scores = [&](int step) {
      const int ln = fresh(lane);
      const unsigned char* row = k_at(step) + (32 * e0 + (ln & 31)) * kRowBytes;
      const auto fragment = [&](int i) {
        return *reinterpret_cast<const bf16x8*>(row + i % kE * 32 * kRowBytes + (((2 * (i / kE) + (ln >> 5)) ^ k_turn<HD>(ln & 31)) << 4));
      };
#pragma unroll
      for (int e = 0; e < kE; ++e)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[e][r] = 0.f;
      bf16x8 kf[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) kf[i] = fragment(i);
#pragma unroll
      for (int i = 0; i < kE * kS; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        s[i % kE] = mfma32(kf[i % 4], qf[i / kE], s[i % kE]);
        if (i + 4 < kE * kS) kf[i % 4] = fragment(i + 4);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    const auto finish = [&](int step) {
      const int ln = fresh(lane), base = part + step * kTileRows;
      const uint64_t there = there_at(step);
      if (masked_at(part, step, there)) {
        uint64_t seen = there;
        if (base + kTileRows > ctx) seen &= seen64(word, base - ctx);
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const uint32_t bits = (uint32_t)(seen >> (32 * (e0 + e) + 4 * h));
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (!(bits >> (8 * (r / 4) + r % 4) & 1)) s[e][r] = -INFINITY;
        }
      }
      // lane i of 16 reads row i / 4, features 4 (i % 4) .. and gets feature i of the four rows
      const int i16 = ln & 15, turn = (int)v_turn<HD>(i16 >> 2);
      const unsigned char* vs = v_at(step) + 32 * e0 * kRowBytes;
      const unsigned char* v = vs + (4 * (ln >> 5) + (i16 >> 2)) * kRowBytes + ((ln >> 4 & 1) * 2 + (i16 >> 1 & 1)) * 16 + 8 * (i16 & 1);
      const auto fragment = [&](int i) {
        return read_transposed(v + i / kF * 16 * kRowBytes + 64 * (i % kF ^ turn), 8 * kRowBytes);
      };
      bf16x8 vf[4];
      if constexpr (kOut) {
#pragma unroll
        for (int i = 0; i < 4; ++i) vf[i] = fragment(i);
        __builtin_amdgcn_sched_barrier(0);
      }
      float top = s[0][0];
#pragma unroll
      for (int e = 0; e < kE; ++e)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, s[e][r]);
      top = fmaxf(top, other_half(top));
      top *= scale2;
      if (__any(top > m_run + kSlack)) {
        const float m_new = fmaxf(m_run, top);
        const float shrink = __builtin_amdgcn_exp2f(m_run - (m_new == -INFINITY ? 0.f : m_new));
        l_run *= shrink;
        if constexpr (kOut) {
#pragma unroll
          for (int f = 0; f < kF; ++f) o[f] *= shrink;
        }
        m_run = m_new;
      }
      const float zero = m_run == -INFINITY ? 0.f : m_run;
      // exponentials of values 2 i and 2 i + 1 of the sixteen rows x, as operands; their sum is added once
      // a step (equal scores, added by twos, stood still at 2^25 in a lane: 2^26 rows of one workgroup)
      float sum = 0.f;
      const auto pair = [&](int x, int i) -> Weights {
        const float p0 = __builtin_amdgcn_exp2f(fmaf(s[x / 2][x % 2 * 8 + 2 * i], scale2, -zero));
        const float p1 = __builtin_amdgcn_exp2f(fmaf(s[x / 2][x % 2 * 8 + 2 * i + 1], scale2, -zero));
        sum += p0 + p1;
        return split_weights(p0, p1);
      };
      if constexpr (!kOut) {
#pragma unroll
        for (int x = 0; x < 2 * kE; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) pair(x, i);
      } else {
        u32x4 now[2], next[2] = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
        const auto weigh = [&](int x, int i, u32x4 (&to)[2]) {
          const Weights w = pair(x, i);
          to[0][i] = w.lead;
          to[1][i] = w.rest;
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) weigh(0, i, now);
#pragma unroll
        for (int x = 0; x < 2 * kE; ++x) {
#pragma unroll
          for (int u = 0; u < 2 * kF; ++u) {                // all features with the leading bits, then the rest
            const int f = u % kF, i = x * kF + f;
            __builtin_amdgcn_sched_barrier(0);
            o[f] = mfma32(vf[i % 4], __builtin_bit_cast(bf16x8, now[u / kF]), o[f]);
            if (u >= kF && i + 4 < 2 * kE * kF) vf[i % 4] = fragment(i + 4);
            if (x + 1 < 2 * kE && u % (kF / 2) == 0) weigh(x + 1, u / (kF / 2), next);
          }
          now[0] = next[0];
          now[1] = next[1];
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      l_run += sum;
    };

    load(0);
    if constexpr (kCodes) store(0);
    if (1 < steps) load(1);
    // Meets the others and sends for the rows of two steps on.
    const auto sync = [&](int step) {
      // the step's loads are done when only those of the next are under way
      if constexpr (!kCodes) {
        if (steps - step > 1)
          dma_wait<kAhead>();
        else
          dma_wait<0>();
      }
      meet(part, step);
      if constexpr (kCodes) {
        if (step + 1 < steps) store(step + 1);
      }
      if (step + 2 < steps) load(step + 2);
    };
    // Waves 0 to 3 meet the others before a step's scores, waves 4 to 7, on the same SIMDs, between
    // the scores of a step and its exponentials and second product: the products of one run
    // beside the exponentials of the other.
    const bool late = wave >= 4;
    if (late) sync(0);
    for (int step = 0; step < steps; ++step) {
      if (!late) sync(step);
      if (busy) scores(step);
      if (late && step + 1 < steps) sync(step + 1);
      if (busy) finish(step);
    }
  }

  l_run += __shfl_xor(l_run, 32);
  if constexpr (WM == 4) {
    // the second half's waves hand over to the first's
    float* sh_o = reinterpret_cast<float*>(sh_kv);        // [4][16 kF + 2][64]
    constexpr int kWords = (kOut ? 16 * kF : 0) + 2;
    static_assert(4 * kWords * 256 <= (int)sizeof(sh_kv), "room to hand over");
    __syncthreads();
    float* at = sh_o + wm * kWords * 64 + lane;
    if (e0 == 1 && busy) {
      at[0] = m_run;
      at[64] = l_run;
      if constexpr (kOut) {
#pragma unroll
        for (int f = 0; f < kF; ++f)
#pragma unroll
          for (int r = 0; r < 16; ++r) at[(2 + 16 * f + r) * 64] = o[f][r];
      }
    }
    __syncthreads();
    if (e0 == 1 || !busy) return;
    const float mo = at[0], m_new = fmaxf(m_run, mo), zero = m_new == -INFINITY ? 0.f : m_new;
    const float mine = __builtin_amdgcn_exp2f(m_run - zero), theirs = __builtin_amdgcn_exp2f(mo - zero);
    m_run = m_new;
    l_run = l_run * mine + at[64] * theirs;
    if constexpr (kOut) {
#pragma unroll
      for (int f = 0; f < kF; ++f)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[f][r] = o[f][r] * mine + at[(2 + 16 * f + r) * 64] * theirs;
    }
  }
  if (!busy) return;
  if constexpr (kOut) {
    // the pieces left out above, for the queries that see their rows
    for (uint64_t wild = sh_wild; wild; wild &= wild - 1) {
      const int draft = __ffsll((unsigned long long)wild) - 1, row = ctx + draft;
      const int pi = (int)quotient((unsigned)row, a.page);
      const int64_t off = ((int64_t)table[pi] * a.b.page_size + (row - pi * a.b.page_size)) * row_size;
      float dot = 0.f;
#pragma unroll
      for (int s = 0; s < kS; ++s) {
        const u32x4 x = kCodes ? values_at<kType>(a.kp, a.ks, off + kh * HD + 16 * s + 8 * h)
                               : *reinterpret_cast<const u32x4*>(kbase + off + 16 * s + 8 * h);
        const u32x4 y = __builtin_bit_cast(u32x4, qf[s]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dot += bf16_to_f32(x[i] & 0xffffu) * bf16_to_f32(y[i] & 0xffffu) + bf16_to_f32(x[i] >> 16) * bf16_to_f32(y[i] >> 16);
      }
      dot += other_half(dot);
      const float zero = m_run == -INFINITY ? 0.f : m_run;
      const float p = __builtin_amdgcn_exp2f(fmaf(dot, scale2, -zero));
      const bool sees = word >> draft & 1;
#pragma unroll
      for (int f = 0; f < kF; ++f)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const u32x4 x = kCodes ? values_at<kType>(a.vp, a.vs, off + kh * HD + 32 * f + 8 * b)
                                 : *reinterpret_cast<const u32x4*>(vbase + off + 32 * f + 8 * b);
          if (!sees || !not_finite(x)) continue;
          const uint32_t lo = h ? x[2] : x[0], hi = h ? x[3] : x[1];
          o[f][4 * b] += p * bf16_to_f32(lo & 0xffffu);
          o[f][4 * b + 1] += p * bf16_to_f32(lo >> 16);
          o[f][4 * b + 2] += p * bf16_to_f32(hi & 0xffffu);
          o[f][4 * b + 3] += p * bf16_to_f32(hi >> 16);
        }
    }
  }
  if (!in) return;
  const int head = kh * a.group + m % a.group;
  const int64_t row = first + qi, part = pt.at + m;
  if (pt.at >= 0) {
    if (h == 0) a.part_ml[part] = make_float2(m_run, l_run);
  } else if (a.lse && h == 0) {
    a.lse[row * a.q.n_heads + head] = l_run == 0.f ? -INFINITY : m_run * kLn2 + __logf(l_run);
  }
  if constexpr (kOut) {
    // lane (q, h) holds features 32 f + 8 b + 4 h + r for r < 4
    const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
#pragma unroll
    for (int f = 0; f < kF; ++f)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int d = 32 * f + 8 * b + 4 * h;
        const f32x4 w = {o[f][4 * b], o[f][4 * b + 1], o[f][4 * b + 2], o[f][4 * b + 3]};
        if (pt.at >= 0) {
          *reinterpret_cast<f32x4*>(a.part_o + part * HD + d) = w;
        } else {
          const u32x2 x = {pack_bf16x2(w[0] * inv, w[1] * inv), pack_bf16x2(w[2] * inv, w[3] * inv)};
          *reinterpret_cast<u32x2*>(a.out + row * a.out_stride + head * HD + d) = l_run == 0.f ? u32x2{0u, 0u} : x;
        }
      }
  }
}

// The first kernel of a call, by its query rows to a workgroup.
template <int HD, bool kOut, int kType, bool kShared>
void launch_form(const AttendArgs& a, int rows, unsigned grid, hipStream_t stream) {
  if (rows == 16) {
    if constexpr (kType == RF_CACHE_BF16)
      hipLaunchKernelGGL((attend_kernel<HD, kOut, kShared>), dim3(grid), dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((attend_codes_kernel<HD, kOut, kType>), dim3(grid), dim3(kThreads), 0, stream, a);
  } else if (rows == 128)
    hipLaunchKernelGGL((attend_tile_kernel<HD, 4, kOut, kType, kShared>), dim3(grid), dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((attend_tile_kernel<HD, 8, kOut, kType, kShared>), dim3(grid), dim3(512), 0, stream, a);
}
template <int kType, bool kShared>
void launch_rows(const AttendArgs& a, int rows, unsigned grid, hipStream_t stream) {
  const auto launch = a.b.hd == 128 ? (a.out ? launch_form<128, true, kType, kShared> : launch_form<128, false, kType, kShared>)
                                    : (a.out ? launch_form<64, true, kType, kShared> : launch_form<64, false, kType, kShared>);
  launch(a, rows, grid, stream);
}
// Each in a file of its own.
extern template void launch_rows<RF_CACHE_BF16, true>(const AttendArgs&, int, unsigned, hipStream_t);
extern template void launch_rows<RF_CACHE_FP8, true>(const AttendArgs&, int, unsigned, hipStream_t);
extern template void launch_rows<RF_CACHE_INT8, true>(const AttendArgs&, int, unsigned, hipStream_t);

}  // namespace rf
