// gg_q8_quant.cu — 8-bit row quantiser: one scale per row (a token's
// activations, or an output channel of a weight),
//   a = max(max_c |x_c|, 2^-100),  q_c = rint(x_c * (127 / a)),  s = a / 127,
// in fp32. |x_c| <= a, so no code leaves [-127, 127]; the floor keeps 127 / a
// finite and gives an all-zero row codes 0 and a scale that is not 0. A row
// with a NaN or an infinity gets codes 0 and the scale NaN, so that every
// product with it is NaN.
//
// One warp per source row, held in registers up to K = 4096 (all its loads in
// flight together, 64 registers at most); longer rows are read twice. Memory
// bound (2 bytes read and 1 written per element and destination row): 131072 x
// 2048 in 121 us, 6.6 TB/s; read twice it took 142, and 65536 x 4096 took 183
// against 154.

#include <cuda_runtime.h>

#include "gg_internal.h"
#include "gg_launch.cuh"
#include "gg_ptx.cuh"

namespace gg {
namespace {

constexpr int kWarps = 8;
constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr float kAmaxFloor = 7.888609052210118e-31f;  // 2^-100

__device__ __forceinline__ uint32_t quantize4(float a, float b, float c, float d, float inv) {
  const int q0 = __float2int_rn(a * inv), q1 = __float2int_rn(b * inv);
  const int q2 = __float2int_rn(c * inv), q3 = __float2int_rn(d * inv);
  return (q0 & 0xFF) | ((q1 & 0xFF) << 8) | ((q2 & 0xFF) << 16) |
         (static_cast<uint32_t>(q3) << 24);
}

__device__ __forceinline__ uint32_t top_of(uint4 w) {  // largest |BF16|, as its bits
  const uint32_t a = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                              __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
  return max(a & 0xFFFFu, a >> 16);
}

// V: 16-byte pieces of a row per lane, 0 for any number of them.
template <int V>
__global__ void __launch_bounds__(32 * kWarps)
q8_quantize_kernel(const uint4* __restrict__ src, long long rows, int K,
                   const int32_t* __restrict__ offsets, int E,
                   const int32_t* __restrict__ row_of_slot, int k, int R_cap,
                   uint2* __restrict__ Q, float* __restrict__ S, int32_t* status) {
  grid_dependents_launch();  // the product's weight loads need not wait for the codes
  const int lane = threadIdx.x & 31;
  const int vec = K / 8;
  if (offsets != nullptr) {
    const int used = offsets[E];
    rows = used < 0 ? 0 : (used < rows ? used : rows);
  }
  for (long long r = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < rows;
       r += static_cast<long long>(gridDim.x) * kWarps) {
    const uint4* x = src + r * vec;
    uint32_t top = 0;  // largest magnitude, as BF16 bits (ordered, NaN above infinity)
    uint4 held[V > 0 ? V : 1];
    if constexpr (V > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = lane + 32 * i;
        held[i] = c < vec ? x[c] : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) top = max(top, top_of(held[i]));
    } else {
      for (int c = lane; c < vec; c += 32) top = max(top, top_of(x[c]));
    }
    top = __reduce_max_sync(kFull, top);
    const bool finite = top < 0x7F80u;
    const float a = fmaxf(__uint_as_float(top << 16), kAmaxFloor);
    const float inv = finite ? 127.0f / a : 0.0f;
    const float scale = finite ? a / 127.0f : __uint_as_float(0x7FC00000u);
    const int copies = row_of_slot != nullptr ? k : 1;
    int dst = 0;
    if (row_of_slot != nullptr && lane < k) {
      dst = row_of_slot[r * k + lane];
      if (dst < -1 || dst >= R_cap) {
        set_status(status, GG_ERR_DEVICE_BAD_ROW);
        dst = -1;
      }
    }
    const auto put = [&](int c, uint4 w) {
      uint2 q = make_uint2(0u, 0u);
      if (finite) {
        q.x = quantize4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y), inv);
        q.y = quantize4(bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w), inv);
      }
      for (int j = 0; j < copies; ++j) {
        const long long to = row_of_slot != nullptr ? __shfl_sync(kFull, dst, j) : r;
        if (to >= 0 && c < vec) Q[to * vec + c] = q;
      }
    };
    if constexpr (V > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (32 * i < vec) put(lane + 32 * i, held[i]);
    } else {
      for (int c = lane; c - lane < vec; c += 32)
        put(c, c < vec ? x[c] : make_uint4(0u, 0u, 0u, 0u));
    }
    if (row_of_slot == nullptr) {
      if (lane == 0) S[r] = scale;
    } else if (lane < k && dst >= 0) {
      S[dst] = scale;
    }
  }
}

}  // namespace

cudaError_t launch_q8_quantize(const gg_bf16* src, long long rows, int K, const int32_t* offsets,
                               int E, const int32_t* row_of_slot, int k, int R_cap, int8_t* Q,
                               float* S, int32_t* status, int sm_count, cudaStream_t stream) {
  if (rows <= 0) return cudaSuccess;
  long long blocks = (rows + kWarps - 1) / kWarps;
  const long long cap = static_cast<long long>(sm_count) * 8;
  if (blocks > cap) blocks = cap;
  const int pieces = (K / 8 + 31) / 32;  // per lane
  const auto go = [&](auto kernel) {
    kernel<<<static_cast<int>(blocks), 32 * kWarps, 0, stream>>>(
        reinterpret_cast<const uint4*>(src), rows, K, offsets, E, row_of_slot, k, R_cap,
        reinterpret_cast<uint2*>(Q), S, status);
  };
  if (pieces <= 1) go(q8_quantize_kernel<1>);
  else if (pieces <= 2) go(q8_quantize_kernel<2>);
  else if (pieces <= 4) go(q8_quantize_kernel<4>);
  else if (pieces <= 8) go(q8_quantize_kernel<8>);
  else if (pieces <= 16) go(q8_quantize_kernel<16>);
  else go(q8_quantize_kernel<0>);
  count_launch();
  return cudaGetLastError();
}

}  // namespace gg
