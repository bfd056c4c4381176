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
#include "rf_cache_dev.h"
#include "rf_split.h"

namespace rf {

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 32;             // cache rows of one step of a wave
// The running maximum follows a larger score only when that is more than 2^8 times as heavy: the
// weights relative to it then stay below 2^8, which costs neither fp32 sums nor bf16 weights any
// precision, and the outputs are rescaled a few times in all instead of in every other step.
constexpr float kSlack = 8.f;

struct AttendArgs {
  Batch b;
  Queries q;
  const uint16_t* kp;
  const uint16_t* vp;
  uint16_t* out;
  float* lse;
  unsigned* status;
  unsigned* each;               // grains of a part, from the first launch to the join
  float* part_o;                // [parts][n_kv][max_q G][hd]
  float2* part_ml;              // [parts][n_kv][max_q G]: running maximum (log2), sum
  int64_t out_stride;
  Divide page;
  int parts, goal, least;       // parts of the grid; wanted of all sequences (0: one each), rows of one
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
__device__ int grains_of_part(const AttendArgs& a, const Seq& mine) {
  const int lane = threadIdx.x & 63;
  const auto sum = [](auto v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
  };
  long long total = mine.grains;
  for (int b = 64 + lane; b < a.b.batch; b += 64) total += look_up(a, b).grains;
  return part_grains(sum(total), a.b.batch, a.goal, a.least / kGrain, [&](int each) {
    int parts = (mine.grains + each - 1) / each;
    for (int b = 64 + lane; b < a.b.batch; b += 64) parts += (look_up(a, b).grains + each - 1) / each;
    return sum(parts);
  });
}

// What a workgroup computes: rows [begin, end) of a sequence, for one key head.
struct Part {
  int kh, seq, len, first, n, begin, end, id;
  bool whole;                           // the sequence's only part
};
__device__ bool find_part(const AttendArgs& a, int unit, Part* p) {
  const int lane = threadIdx.x & 63;
  p->kh = unit % a.b.n_kv;
  p->id = unit / a.b.n_kv;
  if (!a.goal) {
    p->seq = p->id;
    bool bad;
    const bool go = sequence_of(a.b, a.q, p->seq, &p->len, &p->first, &p->n, &bad);
    if (bad && a.report && threadIdx.x == 0) atomicOr(a.status, kStatusRowsBit);
    p->begin = 0;
    p->end = p->len;
    p->whole = true;
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
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(upto, d);
      if (lane >= d) upto += o;
    }
    const uint64_t past = __ballot(before + upto > p->id);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
      const int parts = of(mine), split = p->id - before - (of(upto) - parts);
      p->seq = b0 + l;
      p->len = of(s.len);
      p->first = of(s.first);
      p->n = of(s.n);
      p->begin = __builtin_amdgcn_readfirstlane((int)((int64_t)split * each * kGrain));
      p->end = p->len - p->begin < each * kGrain ? p->len : p->begin + each * kGrain;
      p->whole = parts == 1;
      return true;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
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

// kOut: with the product with V (else only the statistics).
// At most 16 query rows: bound by the read of K and V.  16 sequences of up to 16,384 rows, one token,
// 8 key heads of 128 (760 MB): 148 us of the call's 153, 5.1 TB/s, as a large copy.  (The tile kernel
// below took 187 us there; this one, with four tiles of 16 queries, 120 us for 64 query rows over 65,536
// where that took 70; both with one operand a weight.)
template <int HD, bool kOut>
__global__ __launch_bounds__(kThreads, 2) void attend_kernel(AttendArgs a) {
  constexpr int kSteps = HD / 32, kFeat = HD / 16;
  __shared__ float sh_o[kWaves / 2][16][HD + 4];
  __shared__ float2 sh_ml[kWaves / 2][16];
  if (a.scan && blockIdx.x == 0) return scan_status(a.b, a.q, a.status);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  Part pt;
  if (!find_part(a, blockIdx.x - a.scan, &pt)) return;
  const int kh = pt.kh, seq = pt.seq, len = pt.len, first = pt.first, n = pt.n, begin = pt.begin, end = pt.end;
  const int m_rows = n * a.group, ctx = len - n;

  // Q^T fragments: query row c, zero past the last
  const bool in = c < m_rows;
  const int qi = in ? c / a.group : 0, head = kh * a.group + (in ? c % a.group : 0);
  const uint64_t word = draft_word(a.q, first + qi, qi);
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

  const int32_t* table = a.b.tables + (int64_t)seq * a.b.table_stride;
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

  // sums over g, then the waves: 2 and 3 into 0 and 1, then 1 into 0
  l_run += __shfl_xor(l_run, 16);
  l_run += __shfl_xor(l_run, 32);
  for (int half = kWaves / 2; half; half /= 2) {
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
  if (wave != 0 || !in) return;
  if (!pt.whole) {
    const int64_t part = ((int64_t)pt.id * a.b.n_kv + kh) * (a.q.max_q * a.group) + c;
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
  const int64_t row = first + qi;
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

// More than 16 query rows: bound by the matrix cores and the exponentials, so K and V go
// through LDS and are shared by the workgroup's eight waves, each of which keeps 32 query rows
// (32x32x16 MFMAs, the same transposed products: lane (q, h) = (lane % 32, lane / 32) of S^T
// holds cache rows 8 (r / 4) + 4 h + r % 4, r < 16).  WM of the waves lie along the query rows, with
// WM = 4 the other four take the second half of a step's cache rows and are added at the end.
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

// Whether one of eight bf16 values is infinite or NaN.
__device__ __forceinline__ bool not_finite(u32x4 w) {
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) any |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
  return any;
}

// The value of lane ^ 32.
__device__ __forceinline__ float other_half(float v) {
  const int x = __builtin_bit_cast(int, v);
  const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return __builtin_bit_cast(float, (threadIdx.x & 32) ? r[0] : r[1]);
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

template <int HD, int WM, bool kOut>
__global__ __launch_bounds__(64 * kTileWaves, 2) void attend_tile_kernel(AttendArgs a) {
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
  place_block(a, &unit, &mb);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h = lane >> 5;
  const int wm = wave % WM, e0 = wave / WM;   // this wave's query rows; its first group

  Part pt;
  if (!find_part(a, unit, &pt)) return;
  // the end is the same in all lanes: the loop's counting is scalar (148 -> 145 us for 65,536 rows; the
  // kernel above loses 5 us of 200 by it)
  const int kh = pt.kh, seq = pt.seq, len = pt.len, first = pt.first, n = pt.n, begin = pt.begin;
  const int end = __builtin_amdgcn_readfirstlane(pt.end);
  const int m_rows = n * a.group, m0 = mb * 32 * WM;
  if (m0 >= m_rows) return;
  const int ctx = len - n;

  // this wave's 32 query rows; a negative scale turns their sign, so that the largest product
  // is the largest score, and a scale of 0 makes them 0
  const int m = m0 + 32 * wm + c;
  const bool busy = m0 + 32 * wm < m_rows, in = m < m_rows;
  const int qi = in ? m / a.group : 0;
  const uint64_t word = draft_word(a.q, first + qi, qi);
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

  const int32_t* table = a.b.tables + (int64_t)seq * a.b.table_stride;
  const int64_t row_size = (int64_t)a.b.n_kv * HD;
  const unsigned row_bytes = 2u * a.b.n_kv * HD;
  const uint16_t* kbase = a.kp + kh * HD;
  const uint16_t* vbase = kOut ? a.vp + kh * HD : nullptr;
  const auto k_at = [&](int step) { return sh_kv + step % kBufs * kBufBytes; };
  const auto v_at = [&](int step) { return sh_kv + (kBufs + step % kBufs) * kBufBytes; };
  const auto load = [&](int step) {
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

  for (int part = begin; part < end; part += kSlots) {
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
    f32x16 s[kE];
    // rows of a step that exist, and whether some query does not see all 64
    const auto there_at = [&](int step) -> uint64_t { return __ballot(sh_slot[step * kTileRows + lane] >= 0); };
    const auto masked_at = [&](int step, uint64_t there) { return ~there || part + (step + 1) * kTileRows > ctx; };
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
      if (masked_at(step, there)) {
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

#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i < steps) load(i);
    // Hands a step's rows to all waves and sends for those of two steps on.
    const auto sync = [&](int step) {
      // the step's loads are done when only those of the next are under way
      if (steps - step > 1)
        dma_wait<kAhead>();
      else
        dma_wait<0>();
      __syncthreads();
      const uint64_t there = there_at(step);
      if (kOut && masked_at(step, there)) {
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
        const u32x4 x = *reinterpret_cast<const u32x4*>(kbase + off + 16 * s + 8 * h), y = __builtin_bit_cast(u32x4, qf[s]);
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
          const u32x4 x = *reinterpret_cast<const u32x4*>(vbase + off + 32 * f + 8 * b);
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
  const int64_t row = first + qi, part = ((int64_t)pt.id * a.b.n_kv + kh) * (a.q.max_q * a.group) + m;
  if (!pt.whole) {
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
        if (!pt.whole) {
          *reinterpret_cast<f32x4*>(a.part_o + part * HD + d) = w;
        } else {
          const u32x2 x = {pack_bf16x2(w[0] * inv, w[1] * inv), pack_bf16x2(w[2] * inv, w[3] * inv)};
          *reinterpret_cast<u32x2*>(a.out + row * a.out_stride + head * HD + d) = l_run == 0.f ? u32x2{0u, 0u} : x;
        }
      }
  }
}

// Joins the parts of one output row by kPer waves: sixteen lanes hold the row, four parts to a
// wave at a time (and several of those in flight: one at a time, 128 parts took 80 us).  One token
// over 65,536 rows, 8 key heads: 64 us by four waves a row, 72 by one; one key head 26 and 40.
// Eight workgroups fit a compute unit (with more registers for the scan: five, 12.6 instead of 9.4
// us for the trees above).
template <int HD, int kPer>
__global__ __launch_bounds__(kThreads, 8) void join_kernel(AttendArgs a) {
  constexpr int kE = HD / 16;
  __shared__ float sh_o[kPer][HD + 1];
  const int rows = a.q.max_q * a.group;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = threadIdx.x >> 6, g0 = 4 * (wave % kPer) + g;
  const int scans = a.b.batch * a.scan_parts;
  if ((int)blockIdx.x < scans)
    return scan_sequence(a.b, a.q, blockIdx.x / a.scan_parts, blockIdx.x % a.scan_parts, a.scan_parts, a.status);
  const int64_t id = (int64_t)(blockIdx.x - scans) * (kWaves / kPer) + wave / kPer;
  const int sh = (int)(id / rows), m = (int)(id % rows);
  if (sh >= a.b.batch * a.b.n_kv) return;
  const int kh = sh % a.b.n_kv, seq = sh / a.b.n_kv;
  const Seq mine = look_up(a, lane), self = look_up(a, seq);
  const int n = self.n, first = self.first;
  if (!self.grains || m >= n * a.group) return;
  const int each = (int)*a.each, parts = (self.grains + each - 1) / each;
  if (parts == 1) return;                           // written by its workgroup
  int before = lane < seq ? (mine.grains + each - 1) / each : 0;
  for (int b = 64 + lane; b < seq; b += 64) before += (look_up(a, b).grains + each - 1) / each;
#pragma unroll
  for (int d = 32; d; d >>= 1) before += __shfl_xor(before, d);
  const int64_t at = ((int64_t)before * a.b.n_kv + kh) * rows + m, step = (int64_t)a.b.n_kv * rows;
  const float2* ml = a.part_ml + at;
  float top = -INFINITY;
  for (int s = lane; s < parts; s += 64) top = fmaxf(top, ml[s * step].x);
#pragma unroll
  for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  const float zero = top == -INFINITY ? 0.f : top;
  float sum = 0.f, o[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) o[e] = 0.f;
  if (a.out) {
    const float* po = a.part_o + at * HD + c * kE;
#pragma unroll 4
    for (int s = g0; s < parts; s += 4 * kPer) {
      const float2 v = ml[s * step];
      const float w = __builtin_amdgcn_exp2f(v.x - zero);
      sum += v.y * w;
#pragma unroll
      for (int e = 0; e < kE; e += 4) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(po + s * step * HD + e);
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
      const float2 v = ml[s * step];
      sum += v.y * __builtin_amdgcn_exp2f(v.x - zero);
    }
  }
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if constexpr (kPer > 1) {                         // one row to a workgroup: all its waves are here
    static_assert(kPer == kWaves, "a row is one workgroup's");
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
  int mblocks, group, parts, goal, least;
  size_t ml, o, total;
};
AttendPlan attend_plan(const Batch& b, int n_heads, int max_q) {
  AttendPlan p;
  p.group = n_heads / b.n_kv;
  const int rows = max_q * p.group;
  p.rows = rows <= 16 ? 16 : rows <= 128 ? 128 : 256;
  p.mblocks = (rows + p.rows - 1) / p.rows;
  // enough workgroups for the chip: up to four a compute unit with registers alone, one with LDS
  const int per_part = b.n_kv * p.mblocks, want = p.rows == 16 ? 1024 : 256;
  p.least = p.rows == 16 ? 256 : 128;
  p.goal = parts_goal(want, per_part);
  if (p.goal <= b.batch || b.max_len <= p.least) p.goal = 0;
  const int64_t most = (int64_t)b.batch * ((b.max_len + p.least - 1) / p.least);
  p.parts = p.goal == 0 ? b.batch : most < p.goal ? (int)most : p.goal;
  const size_t held = p.goal ? (size_t)p.parts * b.n_kv * rows : 0;
  p.ml = kStatusBytes;
  p.o = p.ml + align256(held * sizeof(float2));
  p.total = p.o + align256(held * b.hd * sizeof(float));
  return p;
}

template <int HD, bool kOut>
void launch_rows(const AttendArgs& a, int rows, unsigned grid, hipStream_t stream) {
  if (rows == 16)
    hipLaunchKernelGGL((attend_kernel<HD, kOut>), dim3(grid), dim3(kThreads), 0, stream, a);
  else if (rows == 128)
    hipLaunchKernelGGL((attend_tile_kernel<HD, 4, kOut>), dim3(grid), dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((attend_tile_kernel<HD, 8, kOut>), dim3(grid), dim3(512), 0, stream, a);
}

template <int HD>
void launch_head(const AttendArgs& a, const AttendPlan& p, unsigned grid, hipStream_t stream) {
  if (a.out)
    launch_rows<HD, true>(a, p.rows, grid, stream);
  else
    launch_rows<HD, false>(a, p.rows, grid, stream);
  if (p.goal) {
    const int64_t rows = (int64_t)a.b.batch * a.b.n_kv * a.q.max_q * a.group, scans = (int64_t)a.b.batch * a.scan_parts;
    if (p.goal > 32)                // a sequence can have more parts than a wave has under way
      hipLaunchKernelGGL((join_kernel<HD, kWaves>), dim3((unsigned)(rows + scans)), dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((join_kernel<HD, 1>), dim3((unsigned)((rows + kWaves - 1) / kWaves + scans)),
                         dim3(kThreads), 0, stream, a);
  }
}

}  // namespace

size_t attend_workspace(const Batch& b, int n_heads, int max_q) {
  return attend_plan(b, n_heads, max_q).total;
}

hipError_t launch_attend(const Batch& b, const uint16_t* kp, const uint16_t* vp, const Queries& q,
                         uint16_t* out, int64_t out_stride, float* lse, void* ws,
                         hipStream_t stream) {
  const AttendPlan p = attend_plan(b, q.n_heads, q.max_q);
  unsigned char* w = static_cast<unsigned char*>(ws);
  AttendArgs a = {};
  a.b = b;
  a.q = q;
  a.kp = kp;
  a.vp = vp;
  a.out = out;
  a.lse = lse;
  a.status = reinterpret_cast<unsigned*>(w);
  a.each = a.status + 1;
  a.part_ml = reinterpret_cast<float2*>(w + p.ml);
  a.part_o = reinterpret_cast<float*>(w + p.o);
  a.out_stride = out_stride;
  a.page = divide_by((unsigned)b.page_size);
  a.parts = p.parts;
  a.goal = p.goal;
  a.least = p.least;
  a.mblocks = p.mblocks;
  a.group = p.group;
  a.scan = !p.goal && scans(b) ? 1 : 0;
  a.report = !p.goal && !a.scan ? 1 : 0;
  a.scan_parts = scan_parts(b);
  if (a.report) {
    const hipError_t e = launch_clear_status(a.status, stream);
    if (e != hipSuccess) return e;
  }
  const int64_t grid = (int64_t)p.parts * b.n_kv * p.mblocks + a.scan;
  if (b.hd == 128)
    launch_head<128>(a, p, (unsigned)grid, stream);
  else
    launch_head<64>(a, p, (unsigned)grid, stream);
  return hipGetLastError();
}

}  // namespace rf
