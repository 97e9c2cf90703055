// 8-bit floating point (e4m3) with a scale for every 128 values: what the kernels that
// write it share.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace dflash {

namespace f8 {
constexpr int G = 128;                    // values per scale, and the product's k-block
constexpr float kMax = 448.f;             // largest finite e4m3
constexpr float kMinScale = 1.17549435e-38f;
}  // namespace f8

__device__ __forceinline__ float f8_scale(float amax) { return fmaxf(__fdiv_rn(amax, f8::kMax), f8::kMinScale); }

// Four values to a word of e4m3, rounded to nearest even, at most 448 (NaN stays NaN).
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

}  // namespace dflash
