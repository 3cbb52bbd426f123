// gg_f8.cuh — what the kernels of E4M3 products with scales per block of 128
// share: the block's scale and its codes.
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

namespace gg {
namespace {

constexpr int kF8Block = 128;  // columns (and rows of a weight) that share a scale

// Of a block's largest magnitude a (as bits; a NaN is above infinity): the
// factor that takes it to 448, the largest E4M3 value, and the scale of the
// codes. The floor keeps both finite; a block with a NaN or an infinity gets
// codes 0 and the scale NaN.
__device__ __forceinline__ void f8_scale(uint32_t top, float& inv, float& scale) {
  const bool finite = top < 0x7F800000u;
  const float a = fmaxf(__uint_as_float(finite ? top : 0u), 7.888609052210118e-31f);  // 2^-100
  inv = finite ? __fmul_rn(__frcp_rn(a), 448.0f) : 0.0f;
  scale = finite ? __fmul_rn(a, 1.0f / 448.0f) : __uint_as_float(0x7FC00000u);
}

// Codes of (lo, hi), to nearest even.
__device__ __forceinline__ uint32_t f8_codes2(float lo, float hi, float inv) {
  return __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(lo, inv), __fmul_rn(hi, inv)),
                                  __NV_SATFINITE, __NV_E4M3);
}

}  // namespace
}  // namespace gg
