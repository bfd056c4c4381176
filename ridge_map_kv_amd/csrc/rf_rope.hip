// Rotary positions on gfx950: rotation of any [rows][heads][head_dim] tensor, forward and
// transposed, and the append of rotated rows to the paged cache (the rows that the fill does
// not write: section "Two numbers set the skip range" of the English RidgeFill review).
//
// Pair j of a head turns by position * f_j.  A row's cos and sin are the same for all its
// heads, so a workgroup forms them once per row, in LDS: the angle in turns as an fp64
// product, its nearest integer taken off in fp64 (positions up to 2^31 keep an error below
// 1e-6 turns at f = 1/(2 pi)), then cos and sin of pi times the fp32 rest.
// Everything else is one read and one write of the data, 16 bytes per lane.
#include "rf_cache.h"
#include "rf_common.h"
#include "ridgefill.h"

namespace rf {

namespace {

constexpr int kThreads = 256;

// Sixteen features of a head: the first 8 and the last 8 are loaded 16 (bf16) or 32 (fp32)
// bytes at a time.
template <typename T>
struct Half8;
template <>
struct Half8<uint16_t> {
  u32x4 r;
  __device__ void load(const uint16_t* p) { r = *reinterpret_cast<const u32x4*>(p); }
  __device__ void store(uint16_t* p) const { *reinterpret_cast<u32x4*>(p) = r; }
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
struct Half8<float> {
  f32x4 a, b;
  __device__ void load(const float* p) {
    a = *reinterpret_cast<const f32x4*>(p);
    b = *reinterpret_cast<const f32x4*>(p + 4);
  }
  __device__ void store(float* p) const {
    *reinterpret_cast<f32x4*>(p) = a;
    *reinterpret_cast<f32x4*>(p + 4) = b;
  }
  __device__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a[i];
      f[4 + i] = b[i];
    }
  }
  __device__ void set(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = f[i];
      b[i] = f[4 + i];
    }
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

// Where unit u (16 features) of a head lies: the offsets of its two runs of 8 features and,
// when they rotate, its first pair.  Units past the rotated part pass unchanged (pair < 0).
struct Unit {
  int lo, hi, pair;
};
__device__ __forceinline__ Unit unit_of(const RopeFreq& f, int u) {
  Unit w;
  if (u * 16 >= f.rot) {
    w.lo = u * 16;
    w.hi = u * 16 + 8;
    w.pair = -1;
  } else if (f.layout == RF_ROPE_HALF) {
    w.lo = u * 8;
    w.hi = f.rot / 2 + u * 8;
    w.pair = u * 8;
  } else {
    w.lo = u * 16;
    w.hi = u * 16 + 8;
    w.pair = u * 8;
  }
  return w;
}

template <typename T>
__device__ __forceinline__ void turn_unit(Half8<T>& lo, Half8<T>& hi, const float2* cs,
                                          bool interleaved) {
  float a[8], b[8];
  lo.get(a);
  hi.get(b);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = cs[i], q = cs[4 + i];
      const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
      a[2 * i] = a0 * p.x - a1 * p.y;
      a[2 * i + 1] = a1 * p.x + a0 * p.y;
      b[2 * i] = b0 * q.x - b1 * q.y;
      b[2 * i + 1] = b1 * q.x + b0 * q.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 p = cs[i];
      const float x = a[i], y = b[i];
      a[i] = x * p.x - y * p.y;
      b[i] = y * p.x + x * p.y;
    }
  }
  lo.set(a);
  hi.set(b);
}

// Rows [blockIdx.x * per, + per): their cos and sin into LDS, then units in turn.
template <typename T>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeFreq f, RopeCall c, int per) {
  extern __shared__ float2 cs[];                    // [per][rot / 2]
  const int64_t row0 = (int64_t)blockIdx.x * per;
  const int rows = (int)(c.n - row0 < per ? c.n - row0 : per);
  const int pairs = f.rot / 2;
  for (int i = threadIdx.x; i < rows * pairs; i += kThreads)
    cs[i] = turn_of(f, i % pairs, c.pos[row0 + i / pairs], c.transpose ? -1.f : 1.f);
  __syncthreads();
  const int units = c.hd / 16, per_row = c.heads * units;
  for (int i = threadIdx.x; i < rows * per_row; i += kThreads) {
    const int r = i / per_row, w = i % per_row, h = w / units;
    const Unit u = unit_of(f, w % units);
    const T* x = static_cast<const T*>(c.x) + (row0 + r) * c.x_stride + h * c.hd;
    T* y = static_cast<T*>(c.out) + (row0 + r) * c.out_stride + h * c.hd;
    Half8<T> lo, hi;
    lo.load(x + u.lo);
    hi.load(x + u.hi);
    if (u.pair >= 0) turn_unit(lo, hi, cs + r * pairs + u.pair, f.layout != RF_ROPE_HALF);
    lo.store(y + u.lo);
    hi.store(y + u.hi);
  }
}

// Pool slot of cache row `row` of sequence `seq`, or -1 if any of them is out of range.
__device__ __forceinline__ int append_slot(const Batch& b, int seq, int row) {
  if (seq >= b.batch || row < 0 || row >= b.max_len) return -1;
  const int page = b.tables[(int64_t)seq * b.table_stride + row / b.page_size];
  if (page < 0 || page >= b.num_pages) return -1;
  return page * b.page_size + row % b.page_size;
}

// The same for the append: heads 0 .. n_q-1 of a row are q, then k (rotated into the key
// pages), then v (copied).  The last workgroup writes the status word: it alone looks all
// rows over, beside the others' work, so that the word needs no clearing launch.
__global__ __launch_bounds__(kThreads) void append_kernel(RopeFreq f, Batch b, AppendCall c,
                                                          int per) {
  extern __shared__ float2 cs[];
  if (blockIdx.x == gridDim.x - 1) {
    int bad = 0;
    for (int64_t i = threadIdx.x; i < c.n; i += kThreads) {
      const int s = c.seq ? c.seq[i] : 0;
      if (s >= 0 && append_slot(b, s, c.rows[i]) < 0) bad = 1;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *c.status = bad ? kStatusRowsBit : 0u;
    return;
  }
  const int64_t row0 = (int64_t)blockIdx.x * per;
  const int rows = (int)(c.n - row0 < per ? c.n - row0 : per);
  const int pairs = f.rot / 2;
  const int32_t* pos = c.pos ? c.pos : c.rows;
  for (int i = threadIdx.x; i < rows * pairs; i += kThreads)
    cs[i] = turn_of(f, i % pairs, pos[row0 + i / pairs], 1.f);
  __syncthreads();
  const int units = b.hd / 16, per_row = (c.n_q + 2 * b.n_kv) * units;
  for (int i = threadIdx.x; i < rows * per_row; i += kThreads) {
    const int r = i / per_row, w = i % per_row;
    int h = w / units;
    const int64_t row = row0 + r;
    const int s = c.seq ? c.seq[row] : 0;
    if (s < 0) continue;
    Unit u = unit_of(f, w % units);
    const uint16_t* x;
    uint16_t* y;
    if (h < c.n_q) {
      x = c.q + row * c.q_stride + h * b.hd;
      y = c.q_out + row * c.qo_stride + h * b.hd;
    } else {
      h -= c.n_q;
      const bool val = h >= b.n_kv;
      if (val) {
        h -= b.n_kv;
        u.pair = -1;
      }
      const int slot = append_slot(b, s, c.rows[row]);
      if (slot < 0) continue;
      x = (val ? c.v + row * c.v_stride : c.k + row * c.k_stride) + h * b.hd;
      y = (val ? c.vp : c.kp) + ((int64_t)slot * b.n_kv + h) * b.hd;
    }
    Half8<uint16_t> lo, hi;
    lo.load(x + u.lo);
    hi.load(x + u.hi);
    if (u.pair >= 0) turn_unit(lo, hi, cs + r * pairs + u.pair, f.layout != RF_ROPE_HALF);
    lo.store(y + u.lo);
    hi.store(y + u.hi);
  }
}

// Rows per workgroup: enough that its threads all have a unit, one for wide rows.
int rows_per_block(int per_row) {
  const int per = kThreads / per_row;
  return per < 1 ? 1 : per > 32 ? 32 : per;
}

}  // namespace

hipError_t launch_rope(const RopeFreq& f, const RopeCall& c, bool f32, hipStream_t stream) {
  const int per = rows_per_block(c.heads * c.hd / 16);
  const dim3 grid((unsigned)((c.n + per - 1) / per));
  const size_t lds = (size_t)per * (f.rot / 2) * sizeof(float2);
  if (f32)
    hipLaunchKernelGGL(rope_kernel<float>, grid, dim3(kThreads), lds, stream, f, c, per);
  else
    hipLaunchKernelGGL(rope_kernel<uint16_t>, grid, dim3(kThreads), lds, stream, f, c, per);
  return hipGetLastError();
}

hipError_t launch_append(const RopeFreq& f, const Batch& b, const AppendCall& c,
                         hipStream_t stream) {
  const int per = rows_per_block((c.n_q + 2 * b.n_kv) * b.hd / 16);
  const dim3 grid((unsigned)((c.n + per - 1) / per) + 1);
  const size_t lds = (size_t)per * (f.rot / 2) * sizeof(float2);
  hipLaunchKernelGGL(append_kernel, grid, dim3(kThreads), lds, stream, f, b, c, per);
  return hipGetLastError();
}

}  // namespace rf
