// Rotary positions on gfx950: rotation of any [rows][heads][head_dim] tensor, forward and
// transposed, and the append of rotated rows to the paged cache (the rows that the fill does
// not write: section "Two numbers set the skip range" of the English RidgeFill review).
//
// Pair j of a head turns by position * f_j.  A row's cos and sin are the same for all its
// heads, so a workgroup forms them once per row, in LDS: the angle in turns as an fp64
// product, its nearest integer taken off in fp64 (positions up to 2^31 keep an error below
// 1e-6 turns at f = 1/(2 pi)), then cos and sin of pi times the fp32 rest.
// Everything else is one read and one write of the data.  A thread turns units of two 16-byte
// pieces half the rotated width apart, in either layout, so that neighbouring lanes read
// neighbouring pieces; its first units are on their way while cos and sin are formed.  Measured:
// 8,191 rows of 32 fp32 heads of 128 in 48 us, 5.6 TB/s; 4,096 rows of 32 query and 8 key heads of
// 128 appended in 23 us, 4.4 TB/s (reads and writes of 100 MB, a large copy's rate 4.9 to 5.5).
#include "rf_cache_dev.h"
#include "ridgefill.h"

namespace rf {

namespace {

constexpr int kThreads = 256;

// 16 bytes of a head: 8 (bf16) or 4 (fp32) features.
template <typename T>
struct Piece;
template <>
struct Piece<uint16_t> {
  static constexpr int kN = 8;
  u32x4 r;
  __device__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_to_f32(r[i] & 0xffffu);
      f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
  __device__ void set(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  }
};
template <>
struct Piece<float> {
  static constexpr int kN = 4;
  u32x4 r;
  __device__ void get(float (&f)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(r[i]);
  }
  __device__ void set(const float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(f[i]);
  }
};

// cos and sin of `pos` at pair j, times m.
__device__ __forceinline__ float2 turn_of(const RopeFreq& f, int j, int pos, float sign) {
  double t = (double)pos * f.turns[j];
  t -= rint(t);
  float s, c;
  sincospif(2.0f * (float)t, &s, &c);
  return make_float2(f.m * c, sign * f.m * s);
}

// Where the two pieces of unit u of a head lie, and the first pair of each when they rotate.  Units
// past the rotated part pass unchanged (pair < 0).
struct Unit {
  int lo, hi, pair_lo, pair_hi;
};
template <typename T>
__device__ __forceinline__ Unit unit_of(const RopeFreq& f, int hd, int u) {
  constexpr int kN = Piece<T>::kN;
  const int turned = f.rot / (2 * kN), half = f.rot / 2;
  if (u >= turned) {
    const int lo = f.rot + (u - turned) * kN;
    return {lo, lo + (hd - f.rot) / 2, -1, -1};
  }
  if (f.layout == RF_ROPE_HALF) return {u * kN, half + u * kN, u * kN, u * kN};
  return {u * kN, half + u * kN, u * kN / 2, (half + u * kN) / 2};
}

template <typename T>
__device__ __forceinline__ void turn_unit(Piece<T>& lo, Piece<T>& hi, const float2* cs, const Unit& u,
                                          bool interleaved) {
  constexpr int kN = Piece<T>::kN;
  float a[kN], b[kN];
  lo.get(a);
  hi.get(b);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
      const float2 p = cs[u.pair_lo + i], q = cs[u.pair_hi + i];
      const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
      a[2 * i] = a0 * p.x - a1 * p.y;
      a[2 * i + 1] = a1 * p.x + a0 * p.y;
      b[2 * i] = b0 * q.x - b1 * q.y;
      b[2 * i + 1] = b1 * q.x + b0 * q.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float2 p = cs[u.pair_lo + i];
      const float x = a[i], y = b[i];
      a[i] = x * p.x - y * p.y;
      b[i] = y * p.x + x * p.y;
    }
  }
  lo.set(a);
  hi.set(b);
}

// Turns the units of a workgroup's rows, kUnits of them to a thread at a time.  place(i) says
// where unit i's data come from, dest(i) where they go to (null: nowhere); between() prepares what
// dest and the rotation take, with the first units' loads under way.
constexpr int kUnits = 2;
template <typename T>
struct Place {
  const T* x;                   // null: no such unit
  const float2* cs;
  Unit u;
};
template <typename T, typename Where, typename To, typename Between>
__device__ __forceinline__ void turn_rows(int total, bool interleaved, Where place, To dest, Between between) {
  for (int i0 = 0; i0 == 0 || i0 < total; i0 += kUnits * kThreads) {
    Place<T> p[kUnits];
    Piece<T> lo[kUnits], hi[kUnits];
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int i = i0 + j * kThreads + (int)threadIdx.x;
      p[j].x = nullptr;
      if (i < total) p[j] = place(i);
      if (p[j].x) {
        lo[j].r = *reinterpret_cast<const u32x4*>(p[j].x + p[j].u.lo);
        hi[j].r = *reinterpret_cast<const u32x4*>(p[j].x + p[j].u.hi);
      }
    }
    if (i0 == 0) {
      between();
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      if (!p[j].x) continue;
      if (p[j].u.pair_lo >= 0) turn_unit<T>(lo[j], hi[j], p[j].cs, p[j].u, interleaved);
      T* y = dest(i0 + j * kThreads + (int)threadIdx.x);
      if (!y) continue;
      *reinterpret_cast<u32x4*>(y + p[j].u.lo) = lo[j].r;
      *reinterpret_cast<u32x4*>(y + p[j].u.hi) = hi[j].r;
    }
  }
}

// Divisions of a unit's number in a workgroup into row, head and unit of the head; of a cache row
// into pages.
struct Units {
  Divide row, head, page;
};

// Rows [blockIdx.x * per, + per).
template <typename T>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeFreq f, RopeCall c, Units d, int per) {
  extern __shared__ float2 cs[];                    // [per][rot / 2]
  const int64_t row0 = (int64_t)blockIdx.x * per;
  const int rows = (int)(c.n - row0 < per ? c.n - row0 : per);
  const int pairs = f.rot / 2;
  turn_rows<T>(
      rows * (int)d.row.d, f.layout != RF_ROPE_HALF,
      [&](int i) -> Place<T> {
        const int r = (int)quotient((unsigned)i, d.row), w = i - r * (int)d.row.d, h = (int)quotient((unsigned)w, d.head);
        return {static_cast<const T*>(c.x) + (row0 + r) * c.x_stride + h * c.hd, cs + r * pairs,
                unit_of<T>(f, c.hd, w - h * (int)d.head.d)};
      },
      [&](int i) -> T* {
        const int r = (int)quotient((unsigned)i, d.row), w = i - r * (int)d.row.d, h = (int)quotient((unsigned)w, d.head);
        return static_cast<T*>(c.out) + (row0 + r) * c.out_stride + h * c.hd;
      },
      [&] {
        for (int i = threadIdx.x; i < rows * pairs; i += kThreads)
          cs[i] = turn_of(f, i % pairs, c.pos[row0 + i / pairs], c.transpose ? -1.f : 1.f);
      });
}

// Pool slot of cache row `row` of sequence `seq`, or -1 if any of them is out of range (then the
// table's first entry is looked at instead: no branch keeps several lookups from running together).
__device__ __forceinline__ int append_slot(const Batch& b, Divide by_page, int seq, int row) {
  const bool in = seq < b.batch && row >= 0 && row < b.max_len;
  const int pi = in ? (int)quotient((unsigned)row, by_page) : 0;
  const int page = b.tables[(int64_t)(in ? seq : 0) * b.table_stride + pi];
  return in && page >= 0 && page < b.num_pages ? page * b.page_size + (row - pi * b.page_size) : -1;
}

// The same for the append: heads 0 .. n_q-1 of a row are q, then k (rotated into the key
// pages), then v (copied).  With kScan the first workgroup writes the status word: it alone looks
// all rows over, beside the others' work, so that the word needs no clearing launch; else it is clear,
// and the workgroups report what they meet.
template <bool kScan>
__global__ __launch_bounds__(kThreads) void append_kernel(RopeFreq f, Batch b, AppendCall c,
                                                          Units d, int per) {
  extern __shared__ float2 cs[];                    // [per][rot / 2], then the rows' slots
  if (kScan && blockIdx.x == 0) {
    int bad = 0;
    for (int64_t i0 = threadIdx.x; i0 < c.n; i0 += 8 * kThreads) {   // eight lookups at a time
      int slot[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t i = i0 + j * kThreads < c.n ? i0 + j * kThreads : i0;
        const int s = c.seq ? c.seq[i] : 0;
        const int at = append_slot(b, d.page, s < 0 ? 0 : s, c.rows[i]);
        slot[j] = s < 0 ? 0 : at;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) bad |= slot[j] < 0;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *c.status = bad ? kStatusRowsBit : 0u;
    return;
  }
  const int64_t row0 = (int64_t)(blockIdx.x - kScan) * per;
  const int rows = (int)(c.n - row0 < per ? c.n - row0 : per);
  const int pairs = f.rot / 2;
  int* slots = reinterpret_cast<int*>(cs + per * pairs);
  const int32_t* pos = c.pos ? c.pos : c.rows;
  turn_rows<uint16_t>(
      rows * (int)d.row.d, f.layout != RF_ROPE_HALF,
      [&](int i) -> Place<uint16_t> {
        const int r = (int)quotient((unsigned)i, d.row), w = i - r * (int)d.row.d;
        const int h = (int)quotient((unsigned)w, d.head);
        const int64_t row = row0 + r;
        Place<uint16_t> p = {c.v + row * c.v_stride + (h - c.n_q - b.n_kv) * b.hd, cs + r * pairs,
                             unit_of<uint16_t>(f, b.hd, w - h * (int)d.head.d)};
        if (h < c.n_q)
          p.x = c.q + row * c.q_stride + h * b.hd;
        else if (h < c.n_q + b.n_kv)
          p.x = c.k + row * c.k_stride + (h - c.n_q) * b.hd;
        else
          p.u.pair_lo = -1;                             // v is copied
        return p;
      },
      [&](int i) -> uint16_t* {
        const int r = (int)quotient((unsigned)i, d.row), h = (int)quotient((unsigned)(i - r * (int)d.row.d), d.head);
        const int slot = slots[r];
        if (h < c.n_q) return slot == -2 ? nullptr : c.q_out + (row0 + r) * c.qo_stride + h * b.hd;
        if (slot < 0) return nullptr;
        const int kh = h - c.n_q;
        return kh < b.n_kv ? c.kp + ((int64_t)slot * b.n_kv + kh) * b.hd : c.vp + ((int64_t)slot * b.n_kv + kh - b.n_kv) * b.hd;
      },
      [&] {
        for (int r = threadIdx.x; r < rows; r += kThreads) {
          const int s = c.seq ? c.seq[row0 + r] : 0;
          const int at = append_slot(b, d.page, s < 0 ? 0 : s, c.rows[row0 + r]);
          slots[r] = s < 0 ? -2 : at;                   // -2: a padding row
          if (!kScan && s >= 0 && at < 0) atomicOr(c.status, kStatusRowsBit);
        }
        for (int i = threadIdx.x; i < rows * pairs; i += kThreads)
          cs[i] = turn_of(f, i % pairs, pos[row0 + i / pairs], 1.f);
      });
}

// Rows per workgroup: enough that its threads all have two units, one for wide rows.
int rows_per_block(int per_row) {
  const int per = kUnits * kThreads / per_row;
  return per < 1 ? 1 : per > 32 ? 32 : per;
}

}  // namespace

hipError_t launch_rope(const RopeFreq& f, const RopeCall& c, bool f32, hipStream_t stream) {
  const int units = c.hd / (f32 ? 8 : 16), per = rows_per_block(c.heads * units);
  const Units d = {divide_by((unsigned)(c.heads * units)), divide_by((unsigned)units), divide_by(1u)};
  const dim3 grid((unsigned)((c.n + per - 1) / per));
  const size_t lds = (size_t)per * (f.rot / 2) * sizeof(float2);
  if (f32)
    hipLaunchKernelGGL(rope_kernel<float>, grid, dim3(kThreads), lds, stream, f, c, d, per);
  else
    hipLaunchKernelGGL(rope_kernel<uint16_t>, grid, dim3(kThreads), lds, stream, f, c, d, per);
  return hipGetLastError();
}

hipError_t launch_append(const RopeFreq& f, const Batch& b, const AppendCall& c,
                         hipStream_t stream) {
  const int units = b.hd / 16, per_row = (c.n_q + 2 * b.n_kv) * units, per = rows_per_block(per_row);
  const Units d = {divide_by((unsigned)per_row), divide_by((unsigned)units), divide_by((unsigned)b.page_size)};
  // One workgroup looks 2,048 rows over in 3.4 us, which the others take for rows of 2,048 values: it
  // keeps up with rows of 4,096, and is done in two rounds where there are few.  (2^20 rows of 128 values:
  // 1,765 us with the scan, 140 without; 32,768 of 2,048: 66 and 51.)
  const bool scan = c.n <= 4096 || per_row * 16 >= 4096;
  if (!scan) {
    const hipError_t e = launch_clear_status(c.status, stream);
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)((c.n + per - 1) / per + scan));
  const size_t lds = (size_t)per * ((f.rot / 2) * sizeof(float2) + sizeof(int));
  hipLaunchKernelGGL(scan ? append_kernel<true> : append_kernel<false>, grid, dim3(kThreads), lds, stream, f, b, c, d, per);
  return hipGetLastError();
}

}  // namespace rf
