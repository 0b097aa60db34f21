// kv.cuh -- the 8-bit codes of the KV cache (e4m3 or int8) and their scales.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace idx {

constexpr int kMinScaleExp = -100;  // the smallest scale kv_append writes is 2^-100

// Two codes (the low 16 bits of w) as two fp32 values.
template <int FMT>
__device__ __forceinline__ float2 decode2(uint32_t w) {
  if (FMT == kKvE4m3) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
    return __half22float2(__half2(h));
  }
  return make_float2((float)(int8_t)(w & 0xFFu), (float)(int8_t)((w >> 8) & 0xFFu));
}

// Two fp32 values (in units of the scale) as two codes, rounded to nearest
// even and saturated.  NaN becomes the e4m3 NaN code; int8 has none: 0.
template <int FMT>
__device__ __forceinline__ uint32_t encode2(float x, float y) {
  if (FMT == kKvE4m3)
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
  auto one = [](float v) {
    const int i = __float2int_rn(fminf(fmaxf(v, -127.f), 127.f));
    return (uint32_t)(v == v ? i : 0) & 0xFFu;
  };
  return one(x) | (one(y) << 8);
}

// The exponent e of the least power of two with QMAX * 2^e >= a (QMAX = 448 =
// 0.875 * 2^9 for e4m3, 127 = (127/128) * 2^7 for int8), at least -100; a is
// given by its bf16 bits, finite and without sign.
template <int FMT>
__device__ __forceinline__ int scale_exp(uint32_t a_bits) {
  const int e = (int)(a_bits >> 7) - 126;  // a = m * 2^e, m in [0.5, 1)
  const uint32_t mant = a_bits & 127u;     // m = 0.5 + mant / 256
  const int s = FMT == kKvE4m3 ? e - 9 + (mant > 96u) : e - 7 + (mant > 126u);
  return s < kMinScaleExp ? kMinScaleExp : s;  // zero and subnormals end here too
}

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

}  // namespace idx
