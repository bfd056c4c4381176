// Norms of query and key heads with their rotation on gfx950: forward, backward, and as the append of
// rows to a cache of 16 or 8 bits (section "Hybrid layers and two corrections" of the English
// RidgeFill review: layers that norm their keys; the fill does the same to the rows that it writes).
// Rows that such a cache holds come back by read_kernel.
//
// For a head x of hd features with weight w, r = (mean x^2 + eps)^-1/2 and the rotation R:
//   y = R (w r x);    backward, with g = R^T gy and xh = r x:
//   gx = r (w g - xh mean(w g xh)),   gw = sum over rows and heads of g xh.
// One read of the inputs and one write of the outputs: bound by memory (8,191 rows of 40 heads
// of 128 in bf16: 35.8 us a call, 4.7 TB/s, in fp32 63, 5.3 TB/s; backward, 8,192 rows of 48 heads: 66 us,
// 4.6 TB/s, and 4.6 for the sum of the weights' gradients; 4,097 rows of 40 in fp32: 50 and 4.8), the append of
// codes by its instructions as well (4,096 rows of 48 heads into int8 or fp8: 22 us, 4.2 TB/s; into bf16 24,
// 4.2).  A thread holds a unit of a head, two 16-byte pieces that turn together; a head's units lie in
// neighbouring lanes, as many as the next power of two, so that its sums are a few lane exchanges, and a
// thread's place in a head stays the same from row to row (its weights stay in registers).  Everything is
// fp32 between the one load and the one rounding.
#include "rf_held_dev.h"
#include "rf_rope_dev.h"

namespace rf {

namespace {

constexpr int kThreads = 256;
// Heads that a thread takes in turn where there are rows for kBlocks workgroups, forward: for 8,191 rows of 40 heads
// of 128 features in bf16 (168 MB read and written) 37.5 us with 3, 39.3 with 4, 41.8 with 2, 57.7 with 2 under way
// at a time (timed side by side in one process).
constexpr int kRounds = 3, kBlocks = 2048;
// Backward, and its workgroups to a compute unit: 8,192 rows of 48 heads of 128 in bf16 (302 MB) 70.5 us with 4 and 3,
// 81 with 8 and 3, 80.5 with 2 workgroups, 128 with 4 (registers in scratch memory).
constexpr int kGradRounds = 4, kGradGroups = 3;

template <int kControl>
__device__ __forceinline__ float lanes(float v) {
  const int x = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(x, x, kControl, 0xf, 0xf, false));
}

// Sum and largest over the lanes of a head (lp of them, a power of two); every lane takes part.
template <typename Op>
__device__ __forceinline__ float over_lanes(float v, int lp, Op op) {
  if (lp >= 2) v = op(v, lanes<0xb1>(v));         // lane ^ 1
  if (lp >= 4) v = op(v, lanes<0x4e>(v));         // lane ^ 2
  if (lp >= 8) v = op(v, lanes<0x141>(v));        // mirrored in eight
  if (lp >= 16) v = op(v, lanes<0x140>(v));       // mirrored in sixteen
  if (lp >= 32) v = op(v, __shfl_xor(v, 16));
  return v;
}
__device__ __forceinline__ float sum_lanes(float v, int lp) {
  return over_lanes(v, lp, [](float a, float b) { return a + b; });
}

// How a workgroup's threads lie over the heads of its rows.
struct Layout {
  Divide heads;                 // of a row, and of each of its tensors
  Divide q_heads, k_heads;
  int lp, shift;                // lanes of a head: 2^shift
  int per;                      // rows of a workgroup
};

// turn_of with what the angle's rounding to fp32 takes off added back: cos and sin are then as near as
// their own rounding.  An fp32 angle of half a turn puts them up to 2^-23 off, and twice as many
// codes of 8 bits (of some in a million, next to a border) on the other side as need be.  For those, and
// for normed fp32 rows; rows that are only rotated are ridgefill_rope's, bit for bit.
__device__ __forceinline__ float2 near_turn_of(const RopeFreq& f, int j, int pos, float sign) {
  double t = (double)pos * f.turns[j];
  t -= rint(t);
  const float x = 2.0f * (float)t, rest = (float)((2.0 * t - (double)x) * 3.14159265358979323846);
  float s, c;
  sincospif(x, &s, &c);
  return make_float2(f.m * fmaf(-rest, s, c), sign * f.m * fmaf(rest, c, s));
}

// cos and sin of the rows from row0 on.
__device__ __forceinline__ void fill_turns(float2* cs, const RopeFreq& f, const int32_t* pos, int64_t row0, int rows,
                                           float sign, bool near) {
  const int pairs = f.rot / 2;
  for (int i = threadIdx.x; i < rows * pairs; i += kThreads) {
    const int p = pos[row0 + i / pairs];
    cs[i] = near ? near_turn_of(f, i % pairs, p, sign) : turn_of(f, i % pairs, p, sign);
  }
}

template <typename T>
__device__ __forceinline__ bool near_turns(const NormCall& c) {
  return sizeof(T) == 4 && (c.t[0].w || c.t[1].w);
}

template <int kN>
__device__ __forceinline__ float squares(const float (&a)[kN], const float (&b)[kN]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kN; ++i) s = fmaf(a[i], a[i], s);
#pragma unroll
  for (int i = 0; i < kN; ++i) s = fmaf(b[i], b[i], s);
  return s;
}

// m^-1/2 within half a place: a root and a division leave about one, which the residual 1 - m r^2, its product
// taken in two parts, puts right.  Of 0 and infinity (whose residual is NaN) infinity and 0.
__device__ __forceinline__ float inverse_root(float m) {
  const float r = 1.f / sqrtf(m), h = m * r;
  const float e = fmaf(-fmaf(m, r, -h), r, fmaf(-h, r, 1.f));
  return e == e ? fmaf(0.5f * e, r, r) : r;
}

// A thread's two pieces of a weight.
template <typename T>
struct Weight {
  Piece<T> lo, hi;
  __device__ void load(const void* w, const Unit& u) {
    lo.r = hi.r = u32x4{0u, 0u, 0u, 0u};
    if (!w) return;
    lo.r = *reinterpret_cast<const u32x4*>(static_cast<const T*>(w) + u.lo);
    hi.r = *reinterpret_cast<const u32x4*>(static_cast<const T*>(w) + u.hi);
  }
};

// A thread's place: its unit of a head, and which of the heads that the workgroup takes at a time.
template <typename T>
struct Seat {
  Unit u;
  int slot, slots;
  bool in_head;
  __device__ Seat(const RopeFreq& f, int hd, const Layout& l) {
    const int at = threadIdx.x & (l.lp - 1);
    slot = threadIdx.x >> l.shift;
    slots = kThreads >> l.shift;
    in_head = at < hd / (2 * Piece<T>::kN);
    u = unit_of<T>(f, hd, in_head ? at : 0);
  }
};

// q's heads of the rows first, then k's: a thread's weight and sums are one tensor's at a time.
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_rope_kernel(RopeFreq f, NormCall c, Layout l) {
  constexpr int kN = Piece<T>::kN;
  extern __shared__ float2 cs[];                    // [per][rot / 2]
  const int64_t row0 = (int64_t)blockIdx.x * l.per;
  const int rows = (int)(c.n - row0 < l.per ? c.n - row0 : l.per);
  const int pairs = f.rot / 2;
  const Seat<T> seat(f, c.hd, l);
  const Unit u = seat.u;
  const float inv_hd = 1.f / (float)c.hd;
  bool filled = false;
  const auto tensor = [&](const NormTensor& t, Divide by_heads) {
    Weight<T> w;
    w.load(t.w, u);
    const int total = rows * t.heads;
    for (int i0 = 0; i0 < total; i0 += seat.slots) {
      const int i = i0 + seat.slot;
      const bool in = i < total && seat.in_head;
      const int row = (int)quotient((unsigned)(in ? i : 0), by_heads), head = (in ? i : 0) - row * t.heads;
      Piece<T> lo, hi;
      lo.r = hi.r = u32x4{0u, 0u, 0u, 0u};
      if (in) {
        const T* x = static_cast<const T*>(t.x) + (row0 + row) * t.x_stride + head * c.hd;
        lo.r = *reinterpret_cast<const u32x4*>(x + u.lo);
        hi.r = *reinterpret_cast<const u32x4*>(x + u.hi);
      }
      if (!filled) {
        fill_turns(cs, f, c.pos, row0, rows, 1.f, near_turns<T>(c));
        __syncthreads();
        filled = true;
      }
      float a[kN], b[kN];
      lo.get(a);
      hi.get(b);
      const bool turned = u.pair_lo >= 0;
      if (t.w) {
        const float r = inverse_root(sum_lanes(squares(a, b), l.lp) * inv_hd + c.eps);
        float x[kN], y[kN];
        w.lo.get(x);
        w.hi.get(y);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          a[i] = a[i] * x[i] * r;                     // of two bf16 the first product is exact
          b[i] = b[i] * y[i] * r;
        }
      }
      if (turned) turn_values<kN>(a, b, cs + row * pairs, u, f.layout != RF_ROPE_HALF);
      if (t.w || turned) {
        lo.set(a);
        hi.set(b);
      }
      if (in) {
        T* out = static_cast<T*>(t.out) + (row0 + row) * t.out_stride + head * c.hd;
        *reinterpret_cast<u32x4*>(out + u.lo) = lo.r;
        *reinterpret_cast<u32x4*>(out + u.hi) = hi.r;
      }
    }
  };
  tensor(c.t[0], l.q_heads);
  tensor(c.t[1], l.k_heads);
}

// Backward.  A workgroup takes row blocks in turn and keeps its threads' share of both weights'
// gradients in fp32; what all of them hold goes to `part` [workgroups][2][hd], which a second launch
// adds in a fixed order.
template <typename T>
__global__ __launch_bounds__(kThreads, kGradGroups) void norm_grad_kernel(RopeFreq f, NormCall c, Layout l, float* part) {
  constexpr int kN = Piece<T>::kN;
  extern __shared__ float2 cs[];                    // [per][rot / 2]; at the end [4][2][hd] floats
  const int pairs = f.rot / 2;
  const Seat<T> seat(f, c.hd, l);
  const Unit u = seat.u;
  const float inv_hd = 1.f / (float)c.hd;
  Weight<T> w[2];
  float acc[2][2 * kN];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    w[t].load(c.t[t].w, u);
#pragma unroll
    for (int i = 0; i < 2 * kN; ++i) acc[t][i] = 0.f;
  }
  for (int64_t row0 = (int64_t)blockIdx.x * l.per; row0 < c.n; row0 += (int64_t)gridDim.x * l.per) {
    const int rows = (int)(c.n - row0 < l.per ? c.n - row0 : l.per);
    bool filled = false;
    __syncthreads();                                // the rows before are done with
    const auto tensor = [&](const NormTensor& t, Divide by_heads, const Weight<T>& weight, float (&sums)[2 * kN]) {
      const int total = rows * t.heads;
      for (int i0 = 0; i0 < total; i0 += seat.slots) {
        const int i = i0 + seat.slot;
        const bool in = i < total && seat.in_head;
        const int row = (int)quotient((unsigned)(in ? i : 0), by_heads), head = (in ? i : 0) - row * t.heads;
        Piece<T> xl, xh, gl, gh;
        xl.r = xh.r = gl.r = gh.r = u32x4{0u, 0u, 0u, 0u};
        if (in) {
          const T* g = static_cast<const T*>(t.g) + (row0 + row) * t.g_stride + head * c.hd;
          gl.r = *reinterpret_cast<const u32x4*>(g + u.lo);
          gh.r = *reinterpret_cast<const u32x4*>(g + u.hi);
          if (t.w) {
            const T* x = static_cast<const T*>(t.x) + (row0 + row) * t.x_stride + head * c.hd;
            xl.r = *reinterpret_cast<const u32x4*>(x + u.lo);
            xh.r = *reinterpret_cast<const u32x4*>(x + u.hi);
          }
        }
        if (!filled) {
          fill_turns(cs, f, c.pos, row0, rows, -1.f, near_turns<T>(c));
          __syncthreads();
          filled = true;
        }
        float ga[kN], gb[kN];
        gl.get(ga);
        gh.get(gb);
        if (u.pair_lo >= 0) turn_values<kN>(ga, gb, cs + row * pairs, u, f.layout != RF_ROPE_HALF);
        if (t.w) {
          float xa[kN], xb[kN], wa[kN], wb[kN], dot = 0.f;
          xl.get(xa);
          xh.get(xb);
          weight.lo.get(wa);
          weight.hi.get(wb);
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            wa[e] *= ga[e];
            wb[e] *= gb[e];
            dot = fmaf(wa[e], xa[e], dot);
            dot = fmaf(wb[e], xb[e], dot);
          }
          const float mean = sum_lanes(squares(xa, xb), l.lp) * inv_hd;
          dot = sum_lanes(in ? dot : 0.f, l.lp);
          // no head, no share (r may be infinite there)
          const float r = inverse_root(mean + c.eps), back = r * r * dot * inv_hd;
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            const float da = ga[e] * xa[e] * r, db = gb[e] * xb[e] * r;
            sums[e] += in ? da : 0.f;
            sums[kN + e] += in ? db : 0.f;
            ga[e] = r * (wa[e] - xa[e] * back);
            gb[e] = r * (wb[e] - xb[e] * back);
          }
        }
        if (t.w || u.pair_lo >= 0) {
          gl.set(ga);
          gh.set(gb);
        }
        if (in) {
          T* out = static_cast<T*>(t.out) + (row0 + row) * t.out_stride + head * c.hd;
          *reinterpret_cast<u32x4*>(out + u.lo) = gl.r;
          *reinterpret_cast<u32x4*>(out + u.hi) = gh.r;
        }
      }
    };
    tensor(c.t[0], l.q_heads, w[0], acc[0]);
    tensor(c.t[1], l.k_heads, w[1], acc[1]);
  }
  // the lanes that hold the same place of a head, then the waves
  float* sh = reinterpret_cast<float*>(cs);
  __syncthreads();
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 2 * kN; ++i) {
      float v = acc[t][i];
      for (int d = l.lp; d < 64; d <<= 1) v += __shfl_xor(v, d);
      if (lane < l.lp && seat.in_head) sh[(wave * 2 + t) * c.hd + (i < kN ? u.lo + i : u.hi + i - kN)] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * c.hd; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kThreads / 64; ++k) v += sh[k * 2 * c.hd + i];
    part[(int64_t)blockIdx.x * 2 * c.hd + i] = v;
  }
}

// Sixteen columns of [parts][2 hd] to a workgroup, 64 rows at a time (sixteen at a time took 16 us for 768 parts).
__global__ __launch_bounds__(1024) void norm_grad_sum_kernel(NormCall c, const float* part, int parts) {
  constexpr int kRowsAt = 64, kAhead = 4;
  __shared__ float sh[kRowsAt][17];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4, col = blockIdx.x * 16 + x;
  float v = 0.f;
  for (int p0 = y; p0 < parts; p0 += kRowsAt * kAhead) {
    float at[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int p = p0 + i * kRowsAt;
      at[i] = p < parts ? part[(int64_t)p * 2 * c.hd + col] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) v += at[i];
  }
  sh[y][x] = v;
  __syncthreads();
  if (y) return;
#pragma unroll
  for (int i = 1; i < kRowsAt; ++i) v += sh[i][x];
  const int t = col >= c.hd;
  if (c.t[t].dw && c.t[t].w) c.t[t].dw[col - t * c.hd] = v;
}

// Whether a block of 32 features is held by four neighbouring lanes' pieces: their low ones or their
// high ones.
__host__ __device__ inline bool aligned_blocks(int rot, int hd) { return rot / 2 % kBlock == 0 && (hd - rot) / 2 % kBlock == 0; }

// The append: heads 0 .. n_q-1 of a row are q (into q_out), then k, then v (into the pages).
template <int kType, bool kScan>
__global__ __launch_bounds__(kThreads) void hold_kernel(RopeFreq f, Batch b, HoldCall c, Layout l, Divide page) {
  constexpr int kN = 8;
  extern __shared__ float2 cs[];                    // [per][rot / 2], then the rows' slots
  if (kScan && blockIdx.x == 0) return scan_rows(b, page, c.a.seq, c.a.rows, c.a.n, c.a.status);
  const int64_t row0 = (int64_t)(blockIdx.x - kScan) * l.per;
  const int rows = (int)(c.a.n - row0 < l.per ? c.a.n - row0 : l.per);
  const int pairs = f.rot / 2, total = rows * (int)l.heads.d, slots = kThreads >> l.shift, hd = b.hd;
  int* places = reinterpret_cast<int*>(cs + l.per * pairs);
  const int32_t* pos = c.a.pos ? c.a.pos : c.a.rows;
  const int at = threadIdx.x & (l.lp - 1), slot = threadIdx.x >> l.shift;
  const bool in_head = at < hd / (2 * kN);
  const Unit u = unit_of<uint16_t>(f, hd, in_head ? at : 0);
  const float inv_hd = 1.f / (float)hd;
  Weight<uint16_t> w[2];
  w[0].load(c.q_w, u);
  w[1].load(c.k_w, u);
  for (int i0 = 0; i0 == 0 || i0 < total; i0 += slots) {
    const int i = i0 + slot;
    const bool in = i < total && in_head;
    const int row = (int)quotient((unsigned)(in ? i : 0), l.heads), h = (in ? i : 0) - row * (int)l.heads.d;
    Piece<uint16_t> lo, hi;
    lo.r = hi.r = u32x4{0u, 0u, 0u, 0u};
    if (in) {
      const int64_t r = row0 + row;
      const uint16_t* x = h < c.a.n_q ? c.a.q + r * c.a.q_stride + h * hd
                          : h < c.a.n_q + b.n_kv ? c.a.k + r * c.a.k_stride + (h - c.a.n_q) * hd
                                                 : c.a.v + r * c.a.v_stride + (h - c.a.n_q - b.n_kv) * hd;
      lo.r = *reinterpret_cast<const u32x4*>(x + u.lo);
      hi.r = *reinterpret_cast<const u32x4*>(x + u.hi);
    }
    if (i0 == 0) {
      for (int r = threadIdx.x; r < rows; r += kThreads) {
        const int s = c.a.seq ? c.a.seq[row0 + r] : 0;
        const int p = append_slot(b, page, s < 0 ? 0 : s, c.a.rows[row0 + r]);
        places[r] = s < 0 ? -2 : p;                   // -2: a padding row
        if (!kScan && s >= 0 && p < 0) atomicOr(c.a.status, kStatusRowsBit);
      }
      fill_turns(cs, f, pos, row0, rows, 1.f, kType != RF_CACHE_BF16);
      __syncthreads();
    }
    float x[kN], y[kN];
    lo.get(x);
    hi.get(y);
    const int kind = h < c.a.n_q ? 0 : h < c.a.n_q + b.n_kv ? 1 : 2;
    const bool normed = kind == 0 ? c.q_w != nullptr : kind == 1 && c.k_w, turned = kind < 2 && u.pair_lo >= 0;
    // A wave's heads are mostly of one kind: what none of them needs is left out (23.7 us for 4,096 rows of 32 + 16
    // heads of 128 into int8 with all of it for all, 22.2 without).
    if (__any(normed)) {
      const float r = inverse_root(sum_lanes(squares(x, y), l.lp) * inv_hd + c.eps);
      float s[kN], t[kN];
      Weight<uint16_t> one;                           // chosen, not indexed: they stay in registers
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        one.lo.r[i] = kind == 1 ? w[1].lo.r[i] : w[0].lo.r[i];
        one.hi.r[i] = kind == 1 ? w[1].hi.r[i] : w[0].hi.r[i];
      }
      one.lo.get(s);
      one.hi.get(t);
      if (normed) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          x[i] = x[i] * s[i] * r;
          y[i] = y[i] * t[i] * r;
        }
      }
    }
    if (turned) turn_values<kN>(x, y, cs + row * pairs, u, f.layout != RF_ROPE_HALF);
    const int place = places[row];
    if (normed || turned) {
      lo.set(x);
      hi.set(y);
    }
    if (kind == 0 || kType == RF_CACHE_BF16) {
      const int64_t base = kind == 0 ? 0 : ((int64_t)place * b.n_kv + (h - c.a.n_q - (kind == 2 ? b.n_kv : 0))) * hd;
      uint16_t* out = kind == 0 ? c.a.q_out + (row0 + row) * c.a.qo_stride + h * hd
                                : static_cast<uint16_t*>(kind == 1 ? c.pools.k : c.pools.v) + base;
      if (in && (kind == 0 ? place != -2 : place >= 0)) {
        *reinterpret_cast<u32x4*>(out + u.lo) = lo.r;
        *reinterpret_cast<u32x4*>(out + u.hi) = hi.r;
      }
    }
    if (kType != RF_CACHE_BF16 && __any(kind != 0)) {
      // magnitudes as whole numbers, which order NaN above infinity
      unsigned top[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const unsigned p = __float_as_uint(x[i]) & 0x7fffffffu, q = __float_as_uint(y[i]) & 0x7fffffffu;
        top[0] = top[0] > p ? top[0] : p;
        top[1] = top[1] > q ? top[1] : q;
      }
      const auto most = [](float p, float q) {
        const unsigned a = __float_as_uint(p), c = __float_as_uint(q);
        return __uint_as_float(a > c ? a : c);
      };
      if (aligned_blocks(f.rot, hd)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) top[e] = __float_as_uint(over_lanes(__uint_as_float(top[e]), 4, most));
      } else {
        const unsigned mine[2] = {top[0], top[1]};
        for (int k = 0; k < hd / kBlock; ++k) {
          unsigned t = u.lo / kBlock == k ? mine[0] : 0u;
          if (u.hi / kBlock == k) t = t > mine[1] ? t : mine[1];
          if (!in_head) t = 0u;
          t = __float_as_uint(over_lanes(__uint_as_float(t), l.lp, most));
          if (u.lo / kBlock == k) top[0] = t;
          if (u.hi / kBlock == k) top[1] = t;
        }
      }
      if (in && kind != 0 && place >= 0) {
        const int64_t at_head = (int64_t)place * b.n_kv + (h - c.a.n_q - (kind == 2 ? b.n_kv : 0));
        uint8_t* codes = static_cast<uint8_t*>(kind == 1 ? c.pools.k : c.pools.v) + at_head * hd;
        uint8_t* scales = (kind == 1 ? c.pools.ks : c.pools.vs) + at_head * (hd / kBlock);
        const int s0 = scale_byte<kType>(top[0]), s1 = scale_byte<kType>(top[1]);
        *reinterpret_cast<u32x2*>(codes + u.lo) = codes_of<kType>(x, s0);
        *reinterpret_cast<u32x2*>(codes + u.hi) = codes_of<kType>(y, s1);
        if (u.lo % kBlock == 0) scales[u.lo / kBlock] = (uint8_t)s0;
        if (u.hi % kBlock == 0) scales[u.hi / kBlock] = (uint8_t)s1;
      }
    }
  }
}

// Cached rows back: sixteen values to a thread, k's then v's of a row.
template <int kType, typename T, bool kScan>
__global__ __launch_bounds__(kThreads) void read_kernel(Batch b, ReadCall c, Divide row_units, Divide page) {
  if (kScan && blockIdx.x == 0) return scan_rows(b, page, c.seq, c.rows, c.n, c.status);
  const int64_t unit = (int64_t)(blockIdx.x - kScan) * kThreads + threadIdx.x;
  const int units = (int)row_units.d;
  // rows of a workgroup are few: the first one's number in 64 bits, the rest by multiplication
  const int64_t first = (int64_t)(blockIdx.x - kScan) * kThreads / units;
  const int rest = (int)quotient((unsigned)(unit - first * units), row_units);
  const int64_t row = first + rest;
  if (row >= c.n) return;
  const int at = (int)(unit - row * units), width = b.n_kv * b.hd;
  const bool both = c.k_out && c.v_out, is_v = both ? at >= width / 16 : c.v_out != nullptr;
  const int feature = (both && is_v ? at - width / 16 : at) * 16;
  const int s = c.seq ? c.seq[row] : 0;
  if (s < 0) return;
  const int slot = append_slot(b, page, s, c.rows[row]);
  if (slot < 0) {
    if (!kScan && at == 0) atomicOr(c.status, kStatusRowsBit);
    return;
  }
  const int64_t from = (int64_t)slot * width + feature;
  u32x4 v[2];                                         // sixteen bf16
  const void* pool = is_v ? c.pools.v : c.pools.k;
  if constexpr (kType == RF_CACHE_BF16) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(pool) + from);
    v[0] = p[0];
    v[1] = p[1];
  } else {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(pool) + from);
    const float scale = scale_of((is_v ? c.pools.vs : c.pools.ks)[from / kBlock]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x2 x = values_of<kType>(w[i], scale);
      v[i / 2][i % 2 * 2] = x[0];
      v[i / 2][i % 2 * 2 + 1] = x[1];
    }
  }
  T* out = static_cast<T*>(is_v ? c.v_out : c.k_out) + row * (is_v ? c.v_stride : c.k_stride) + feature;
  u32x4* o = reinterpret_cast<u32x4*>(out);
  if constexpr (sizeof(T) == 2) {
    o[0] = v[0];
    o[1] = v[1];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = u32x4{v[i / 2][i % 2 * 2] << 16, v[i / 2][i % 2 * 2] & 0xffff0000u, v[i / 2][i % 2 * 2 + 1] << 16,
                   v[i / 2][i % 2 * 2 + 1] & 0xffff0000u};
  }
}

Layout layout_of(int heads, int units) {
  Layout l = {divide_by((unsigned)heads), divide_by(1u), divide_by(1u), 1, 0, 1};
  while (l.lp < units) {
    l.lp *= 2;
    ++l.shift;
  }
  return l;
}

// Rows per workgroup: what its threads take in `rounds` where that makes `blocks` workgroups, else in one round; one
// row at least.
int rows_per_block(int per_row, int64_t n, int rounds, int blocks) {
  const auto rows = [&](int heads) {
    const int per = heads * kThreads / per_row;
    return per < 1 ? 1 : per > 32 ? 32 : per;
  };
  const int many = rows(rounds);
  return n >= (int64_t)many * blocks ? many : rows(1);
}

void set_heads(Layout& l, const NormCall& c) {
  l.q_heads = divide_by((unsigned)(c.t[0].heads ? c.t[0].heads : 1));
  l.k_heads = divide_by((unsigned)(c.t[1].heads ? c.t[1].heads : 1));
}

constexpr int kMostParts = 256 * kGradGroups;      // workgroups of a backward pass: all at a time

Layout grad_layout(int heads, int hd, bool f32, int64_t n) {
  Layout l = layout_of(heads, hd / (f32 ? 8 : 16));
  l.per = rows_per_block(heads << l.shift, n, kGradRounds, kMostParts);
  return l;
}

int grad_parts(int64_t n, const Layout& l) {
  const int64_t blocks = (n + l.per - 1) / l.per;
  return (int)(blocks < kMostParts ? blocks : kMostParts);
}

}  // namespace

hipError_t launch_norm_rope(const RopeFreq& f, const NormCall& c, bool f32, hipStream_t stream) {
  const int heads = c.t[0].heads + c.t[1].heads;
  Layout l = layout_of(heads, c.hd / (f32 ? 8 : 16));
  l.per = rows_per_block(heads << l.shift, c.n, kRounds, kBlocks);
  set_heads(l, c);
  const dim3 grid((unsigned)((c.n + l.per - 1) / l.per));
  const size_t lds = (size_t)l.per * (f.rot / 2) * sizeof(float2);
  hipLaunchKernelGGL(f32 ? norm_rope_kernel<float> : norm_rope_kernel<uint16_t>, grid, dim3(kThreads), lds, stream, f, c, l);
  return hipGetLastError();
}

size_t norm_grad_workspace(int64_t n, int hd) {
  const int64_t parts = n < kMostParts ? n : kMostParts;
  return align256((size_t)(parts > 0 ? parts : 1) * 2 * hd * sizeof(float));
}

hipError_t launch_norm_grad(const RopeFreq& f, const NormCall& c, bool f32, void* ws, hipStream_t stream) {
  Layout l = grad_layout(c.t[0].heads + c.t[1].heads, c.hd, f32, c.n);
  set_heads(l, c);
  const int parts = grad_parts(c.n, l);
  float* part = static_cast<float*>(ws);
  if (parts) {
    const size_t turns = (size_t)l.per * (f.rot / 2) * sizeof(float2), sums = (size_t)8 * c.hd * sizeof(float);
    hipLaunchKernelGGL(f32 ? norm_grad_kernel<float> : norm_grad_kernel<uint16_t>, dim3(parts), dim3(kThreads),
                       turns > sums ? turns : sums, stream, f, c, l, part);
  }
  hipLaunchKernelGGL(norm_grad_sum_kernel, dim3(2 * c.hd / 16), dim3(1024), 0, stream, c, part, parts);
  return hipGetLastError();
}

namespace {
// Whether a workgroup that looks all rows over beside the others keeps up with them (see rf_rope.hip).
bool scans_rows(int64_t n, int values) { return n <= 4096 || values >= 4096; }

template <int kType>
void launch_hold_type(bool scan, unsigned grid, size_t lds, hipStream_t stream, const RopeFreq& f, const Batch& b,
                      const HoldCall& c, const Layout& l, Divide page) {
  const auto kernel = scan ? hold_kernel<kType, true> : hold_kernel<kType, false>;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), lds, stream, f, b, c, l, page);
}

template <int kType, typename T>
void launch_read_type(bool scan, unsigned grid, hipStream_t stream, const Batch& b, const ReadCall& c, Divide units,
                      Divide page) {
  const auto kernel = scan ? read_kernel<kType, T, true> : read_kernel<kType, T, false>;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, stream, b, c, units, page);
}
}  // namespace

hipError_t launch_hold(const RopeFreq& f, const Batch& b, const HoldCall& c, hipStream_t stream) {
  const int heads = c.a.n_q + 2 * b.n_kv;
  Layout l = layout_of(heads, b.hd / 16);
  l.per = rows_per_block(heads << l.shift, c.a.n, kRounds, kBlocks);
  const bool scan = scans_rows(c.a.n, heads * b.hd);
  if (!scan) {
    const hipError_t e = launch_clear_status(c.a.status, stream);
    if (e != hipSuccess) return e;
  }
  const unsigned grid = (unsigned)((c.a.n + l.per - 1) / l.per + scan);
  const size_t lds = (size_t)l.per * ((f.rot / 2) * sizeof(float2) + sizeof(int));
  const Divide page = divide_by((unsigned)b.page_size);
  const auto launch = c.pools.type == RF_CACHE_BF16  ? launch_hold_type<RF_CACHE_BF16>
                      : c.pools.type == RF_CACHE_FP8 ? launch_hold_type<RF_CACHE_FP8>
                                                     : launch_hold_type<RF_CACHE_INT8>;
  launch(scan, grid, lds, stream, f, b, c, l, page);
  return hipGetLastError();
}

hipError_t launch_read(const Batch& b, const ReadCall& c, bool f32, hipStream_t stream) {
  const int units = b.n_kv * b.hd / 16 * (c.k_out && c.v_out ? 2 : 1);
  const bool scan = scans_rows(c.n, units * 16);
  if (!scan) {
    const hipError_t e = launch_clear_status(c.status, stream);
    if (e != hipSuccess) return e;
  }
  const unsigned grid = (unsigned)((c.n * units + kThreads - 1) / kThreads + scan);
  const Divide by = divide_by((unsigned)units), page = divide_by((unsigned)b.page_size);
  const auto launch = c.pools.type == RF_CACHE_BF16  ? (f32 ? launch_read_type<RF_CACHE_BF16, float> : launch_read_type<RF_CACHE_BF16, uint16_t>)
                      : c.pools.type == RF_CACHE_FP8 ? (f32 ? launch_read_type<RF_CACHE_FP8, float> : launch_read_type<RF_CACHE_FP8, uint16_t>)
                                                     : (f32 ? launch_read_type<RF_CACHE_INT8, float> : launch_read_type<RF_CACHE_INT8, uint16_t>);
  launch(scan, grid, stream, b, c, by, page);
  return hipGetLastError();
}

}  // namespace rf
