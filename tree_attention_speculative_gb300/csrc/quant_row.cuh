// One row of the 8-bit KV cache: the D values of one token of one KV head as
// e4m3 codes and one scale byte s, value = code * 2^(s - 127).
//
// The scale is the smallest power of two that keeps the row's largest
// magnitude within 448, the largest code.  A power of two costs no precision
// (codes are floating point, so only up to one of their 17 binades is given
// up), scales without rounding, and fits a byte.
#pragma once

#include <cuda_fp8.h>

#include "internal.cuh"

namespace ts {

constexpr int Q8_MIN_SCALE = 1;    // 2^-126: smaller rows round towards zero codes
constexpr int Q8_MAX_SCALE = 247;  // 2^120: the scale of the largest finite bf16 (and of an infinity, stored as 448)
constexpr int Q8_NAN_SCALE = 255;  // a row with a NaN is NaN throughout

// The scale byte of a row whose largest magnitude has these bf16 bits.
__device__ __forceinline__ int q8_scale_byte(uint32_t abs_bits) {
  const int e = (int)(abs_bits >> 7) - 8 + ((abs_bits & 0x7f) > 0x60);  // 1.75 * 2^8 = 448
  return min(max(e, Q8_MIN_SCALE), Q8_MAX_SCALE);
}

// The larger of two bf16 pairs of magnitudes; a NaN loses to a number.
__device__ __forceinline__ uint32_t q8_max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// The same, but a NaN wins.
__device__ __forceinline__ uint32_t q8_max2_nan(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// Magnitudes of this lane's 8 values, folded to one pair.
__device__ __forceinline__ uint32_t q8_fold(const uint4& x) {
  return q8_max2_nan(q8_max2_nan(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), q8_max2_nan(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
}

// The bf16 bits of the largest magnitude of a row that LANES consecutive lanes
// hold, from their folded pairs.  All 32 lanes take part.
template <int LANES>
__device__ __forceinline__ uint32_t q8_row_max(uint32_t m) {
#pragma unroll
  for (int d = LANES / 2; d > 0; d >>= 1) m = q8_max2_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
  return q8_max2_nan(m, m >> 16) & 0x7fffu;
}

// The codes of 8 values in a row with scale byte s.
__device__ __forceinline__ uint2 q8_codes(const uint4& x, int s) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const float inv = __uint_as_float((uint32_t)(254 - s) << 23);  // 2^(127 - s)
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]));
    c[k] = __nv_cvt_float2_to_fp8x2(make_float2(f.x * inv, f.y * inv), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// LANES consecutive lanes hold a row, 8 values each: this lane's 8 codes, and
// the row's scale byte on each of them.  All 32 lanes take part.
template <int LANES>
__device__ __forceinline__ uint2 q8_row(const uint4& x, int* scale_byte) {
  const uint32_t m = q8_row_max<LANES>(q8_fold(x));
  if (m > 0x7f80u) {
    *scale_byte = Q8_NAN_SCALE;
    return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
  }
  *scale_byte = q8_scale_byte(m);
  return q8_codes(x, *scale_byte);
}

}  // namespace ts
