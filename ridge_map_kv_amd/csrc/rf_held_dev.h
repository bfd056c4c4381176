// How a cache holds its values (rf_cache.type): bf16 as they are, or codes of 8 bits in blocks of 32
// features that share a power of two, much as in the OCP microscaling formats.  For a block whose largest
// magnitude is top, the exponent e is the smallest with top <= M 2^e (M = 448 for e4m3, 127 for int8),
// kept to -110 .. 118; a code is the nearest value of its type (ties to even) to x 2^-e, and stands for
// code 2^e; the scale byte is e + 127.  These values have at most eight significant bits and are
// normal numbers of bf16, so that a bf16 operand of the matrix cores holds each exactly, and whatever
// reads such a cache computes what it would from a bf16 cache of them.  A block that holds an infinity
// or NaN is NaN altogether: scale byte 255, codes 0 (int8: 0 times infinity) or 0x7f (e4m3).
#pragma once

#include "rf_common.h"
#include "ridgefill.h"

namespace rf {

constexpr int kBlock = 32;
constexpr int kScaleLeast = 17, kScaleMost = 245, kScaleNan = 255;

// The scale byte of a block, from the bits of its largest magnitude.
template <int kType>
__device__ __forceinline__ int scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return kScaleNan;
  // top = (1 + m 2^-23) 2^k; 448 = 1.75 2^8, 127 = 1.984375 2^6
  const int k = (int)(top >> 23), m = (int)(top & 0x7fffffu);
  const int e = kType == RF_CACHE_FP8 ? k - 8 + (m > 0x600000) : k - 6 + (m > 0x7e0000);
  return e < kScaleLeast ? kScaleLeast : e > kScaleMost ? kScaleMost : e;
}

// Codes of eight values of a block with this scale byte.
template <int kType>
__device__ __forceinline__ u32x2 codes_of(const float (&x)[8], int byte) {
  const float inv = __uint_as_float((unsigned)(254 - byte) << 23);
  u32x2 w = {0u, 0u};
  if (byte == kScaleNan) return kType == RF_CACHE_FP8 ? u32x2{0x7f7f7f7fu, 0x7f7f7f7fu} : w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // values of a block whose exponent is cut to 118 stay finite
      const float most = kType == RF_CACHE_FP8 ? 448.f : 127.f;
      y[i] = __builtin_amdgcn_fmed3f(x[4 * h + i] * inv, -most, most);
    }
    if constexpr (kType == RF_CACHE_FP8) {
      int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
      c = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c, true);
      w[h] = (unsigned)c;
    } else {
      // beside 1.5 2^23 a value is rounded to a whole number, nearest even, in the last bits
      unsigned c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(y[i] + 12582912.f);
      const unsigned lo = __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(c[3], c[2], 0x0c0c0400u);
      w[h] = hi << 16 | lo;
    }
  }
  return w;
}

// The factor of a block's codes: 2^(byte - 127), infinity for a NaN block (which makes its codes NaN in both
// conversions below).
__device__ __forceinline__ float scale_of(unsigned byte) { return __uint_as_float(byte << 23); }

// The values of four codes as bf16 pairs.  e4m3: one instruction for two codes, exact for the scale
// bytes above.  int8: code and product as floats, exact too.
template <int kType>
__device__ __forceinline__ u32x2 values_of(unsigned w, float s) {
  if constexpr (kType == RF_CACHE_FP8) {
    return {__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false)),
            __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true))};
  } else {
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(w >> (8 * i)) * s;
    return {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
  }
}

// Whether one of four codes stands for NaN.
template <int kType>
__device__ __forceinline__ bool not_finite(unsigned w, unsigned byte) {
  if (byte == kScaleNan) return true;
  if (kType != RF_CACHE_FP8) return false;
  const unsigned x = ~w & 0x7f7f7f7fu;              // a byte 0 where the code is 0x7f or 0xff
  return ((x - 0x01010101u) & ~x & 0x80808080u) != 0u;
}

// Those of two codes of a word, the first two or the last.
template <int kType>
__device__ __forceinline__ unsigned value_pair(unsigned w, bool second, float s) {
  if constexpr (kType == RF_CACHE_FP8) {
    return second ? __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true))
                  : __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false));
  } else {
    const unsigned u = second ? w >> 16 : w;
    return pack_bf16x2((float)(int8_t)u * s, (float)(int8_t)(u >> 8) * s);
  }
}

}  // namespace rf
