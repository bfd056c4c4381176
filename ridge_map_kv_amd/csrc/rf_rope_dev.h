// Device helpers shared by the kernels that rotate rows (rf_rope.hip, rf_norm.hip): cos and sin of a
// row's pairs, how a head is cut into units of two pieces that turn together, and the cache slots of
// appended rows.
#pragma once

#include "rf_cache_dev.h"
#include "ridgefill.h"

namespace rf {

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

// Turns the values of a unit's two pieces.
template <int kN>
__device__ __forceinline__ void turn_values(float (&a)[kN], float (&b)[kN], const float2* cs, const Unit& u,
                                            bool interleaved) {
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
}

// Pool slot of cache row `row` of sequence `seq`, or -1 if any of them is out of range (then the
// table's first entry is looked at instead: no branch keeps several lookups from running together).
__device__ __forceinline__ int append_slot(const Batch& b, Divide by_page, int seq, int row) {
  const bool in = seq < b.batch && row >= 0 && row < b.max_len;
  const int pi = in ? (int)quotient((unsigned)row, by_page) : 0;
  const int page = b.tables[(int64_t)(in ? seq : 0) * b.table_stride + pi];
  return in && page >= 0 && page < b.num_pages ? page * b.page_size + (row - pi * b.page_size) : -1;
}

// The status word of an append or a read, from one workgroup that looks all rows over, eight lookups
// of a thread at a time (`rows` and `seq` as the calls take them).
__device__ inline void scan_rows(const Batch& b, Divide by_page, const int32_t* seq, const int32_t* rows, int64_t n,
                                 unsigned* status) {
  const int threads = blockDim.x;
  int bad = 0;
  for (int64_t i0 = threadIdx.x; i0 < n; i0 += 8 * threads) {
    int slot[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t i = i0 + j * threads < n ? i0 + j * threads : i0;
      const int s = seq ? seq[i] : 0;
      const int at = append_slot(b, by_page, s < 0 ? 0 : s, rows[i]);
      slot[j] = s < 0 ? 0 : at;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) bad |= slot[j] < 0;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *status = bad ? kStatusRowsBit : 0u;
}

}  // namespace rf
