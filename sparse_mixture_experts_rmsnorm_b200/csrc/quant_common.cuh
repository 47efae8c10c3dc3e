// Quantisation to e4m3 (4 exponent, 3 mantissa bits, largest finite value 448)
// with one fp32 scale per block of 128 columns, as every 8-bit operand of the
// library is held:
//   scale = max(fl32(amax / 448), 2^-126),  code = e4m3(x * fl32(1 / scale)),
// rounded to nearest even and saturated at +-448.  The floor keeps 1 / scale
// finite, so a block of zeros gives zero codes.  A NaN element stays NaN (and
// does not enter amax); a block with an infinity gets an infinite scale, and
// its products are NaN.
#pragma once

#include <cuda_fp8.h>

#include "moe_common.cuh"

namespace moe {

constexpr int Q_BLOCK = 128;

__device__ __forceinline__ float quant_scale(float amax) {
  return fmaxf(__fdiv_rn(amax, 448.f), 1.17549435e-38f);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

__device__ __forceinline__ uint8_t e4m3x1(float v) {
  return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

}  // namespace moe

namespace moe_host {
inline int q_blocks(int cols) { return cols / moe::Q_BLOCK + (cols % moe::Q_BLOCK != 0); }
}  // namespace moe_host
