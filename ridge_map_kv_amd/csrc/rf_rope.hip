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
#include "rf_rope_dev.h"

namespace rf {

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void turn_unit(Piece<T>& lo, Piece<T>& hi, const float2* cs, const Unit& u,
                                          bool interleaved) {
  constexpr int kN = Piece<T>::kN;
  float a[kN], b[kN];
  lo.get(a);
  hi.get(b);
  turn_values<kN>(a, b, cs, u, interleaved);
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

// The same for the append: heads 0 .. n_q-1 of a row are q, then k (rotated into the key
// pages), then v (copied).  With kScan the first workgroup writes the status word: it alone looks
// all rows over, beside the others' work, so that the word needs no clearing launch; else it is clear,
// and the workgroups report what they meet.
template <bool kScan>
__global__ __launch_bounds__(kThreads) void append_kernel(RopeFreq f, Batch b, AppendCall c,
                                                          Units d, int per) {
  extern __shared__ float2 cs[];                    // [per][rot / 2], then the rows' slots
  if (kScan && blockIdx.x == 0) return scan_rows(b, d.page, c.seq, c.rows, c.n, c.status);
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
