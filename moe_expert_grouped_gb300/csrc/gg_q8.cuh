// gg_q8.cuh — what the 8-bit kernels share: exact widening of codes to FP16.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace gg {
namespace {

// Four 8-bit integers (bytes of w) -> four FP16 of the same value: byte + 128
// under the exponent of 1024 reads 1152 + value.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
  const uint32_t x = w ^ 0x80808080u;
  const uint32_t lo = __byte_perm(x, 0x64646464u, 0x4140);
  const uint32_t hi = __byte_perm(x, 0x64646464u, 0x4342);
  const __half2 bias = __half2half2(__ushort_as_half(static_cast<unsigned short>(0x6480)));
  const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), bias);
  const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), bias);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

}  // namespace
}  // namespace gg
