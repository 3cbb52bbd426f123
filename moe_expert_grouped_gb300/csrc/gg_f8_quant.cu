// gg_f8_quant.cu — E4M3 codes with one fp32 scale for every block of 128:
//   a = max(max |x|, 2^-100),  q = e4m3(x (448 / a)),  s = a / 448,
// the maximum over 128 columns of a row (activations), or over 128 x 128
// elements of a weight. Rounded to nearest even; |x| 448 / a is at most 448
// but for its rounding, and saturates there.
//
// Rows: one warp per source row, eight lanes per block (32 bytes each), the row
// in registers up to 4096 columns so that all its loads are in flight together. The scales
// of one block of columns lie together, S[ceil(K / 128)][R_cap]: the products'
// tiles take a block of rows for one block of columns at a time. Bound by memory:
// 131072 x 2048 in 134 us, 6.0 TB/s; 16384 tokens to their 8 rows each, 69 us.
//
// Weights: one block of 256 threads for each 128 x 128; 128 of 1536 x 2048 in
// 165 us, 7.3 TB/s.

#include <cuda_runtime.h>

#include "gg_f8.cuh"
#include "gg_internal.h"
#include "gg_launch.cuh"
#include "gg_ptx.cuh"

namespace gg {
namespace {

constexpr int kWarps = 8;
constexpr uint32_t kFull = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t top_of(uint4 w) {  // largest |BF16|, as its bits
  const uint32_t a = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                              __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
  return max(a & 0xFFFFu, a >> 16);
}

__device__ __forceinline__ uint2 codes8(uint4 w, float inv) {
  // a NaN times 0 stays one, and E4M3 has it: the codes of such a block are 0
  if (inv == 0.0f) return make_uint2(0u, 0u);
  uint2 q;
  q.x = f8_codes2(bf16_lo(w.x), bf16_hi(w.x), inv) |
        f8_codes2(bf16_lo(w.y), bf16_hi(w.y), inv) << 16;
  q.y = f8_codes2(bf16_lo(w.z), bf16_hi(w.z), inv) |
        f8_codes2(bf16_lo(w.w), bf16_hi(w.w), inv) << 16;
  return q;
}

// V: 32-byte pieces (16 columns) of a row per lane; eight lanes share a scale.
template <int V>
__global__ void __launch_bounds__(32 * kWarps)
f8_quantize_kernel(const uint4* __restrict__ src, long long rows, int K,
                   const int32_t* __restrict__ offsets, int E,
                   const int32_t* __restrict__ row_of_slot, int k, int R_cap,
                   uint4* __restrict__ Q, float* __restrict__ S, int32_t* status) {
  grid_dependents_launch();  // the product's set-up need not wait for the codes
  const int lane = threadIdx.x & 31;
  const int vec = K / 16;
  if (offsets != nullptr) {
    const int used = offsets[E];
    rows = used < 0 ? 0 : (used < rows ? used : rows);
  }
  for (long long r = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < rows;
       r += static_cast<long long>(gridDim.x) * kWarps) {
    int dst = 0;
    if (row_of_slot != nullptr && lane < k) {
      dst = row_of_slot[r * k + lane];
      if (dst < -1 || dst >= R_cap) {
        set_status(status, GG_ERR_DEVICE_BAD_ROW);
        dst = -1;
      }
    }
    const int copies = row_of_slot != nullptr ? k : 1;
    for (int c0 = 0; c0 < vec; c0 += 32 * V) {  // once, up to 512 V columns
      const uint4* x = src + 2 * (r * vec + c0 + lane);
      uint4 held[V][2];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool there = c0 + 32 * i + lane < vec;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          held[i][h] = there ? __ldcs(x + 64 * i + h) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = c0 + 32 * i + lane;
        if (c - lane >= vec) break;
        uint32_t top = max(top_of(held[i][0]), top_of(held[i][1]));
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(kFull, top, d));
        float inv, scale;
        f8_scale(top << 16, inv, scale);
        const uint2 lo = codes8(held[i][0], inv), hi = codes8(held[i][1], inv);
        const uint4 q = make_uint4(lo.x, lo.y, hi.x, hi.y);
        const int block = c >> 3;
        for (int j = 0; j < copies; ++j) {
          const long long to = row_of_slot != nullptr ? __shfl_sync(kFull, dst, j) : r;
          if (to < 0 || c >= vec) continue;
          Q[to * vec + c] = q;
          if ((lane & 7) == 0) S[static_cast<long long>(block) * R_cap + to] = scale;
        }
      }
    }
  }
}

constexpr int kTile = kF8Block;
__global__ void __launch_bounds__(256)
f8_weight_kernel(const uint4* __restrict__ W, int N, int K, int NB, int KB,
                 uint2* __restrict__ Wq, float* __restrict__ Ws) {
  __shared__ uint32_t tops[8];
  const int kb = blockIdx.x, nb = blockIdx.y;
  const long long e = blockIdx.z;
  const int vec = K / 8;
  const int col = kb * (kTile / 8) + (threadIdx.x & 15);
  const int row0 = nb * kTile + (threadIdx.x >> 4);
  const bool in = col < vec;
  uint4 held[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = row0 + 16 * i;
    held[i] = in && n < N ? W[(e * N + n) * vec + col] : make_uint4(0u, 0u, 0u, 0u);
    top = max(top, top_of(held[i]));
  }
  top = __reduce_max_sync(kFull, top);
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, tops[i]);
  float inv, scale;
  f8_scale(top << 16, inv, scale);
  if (threadIdx.x == 0) Ws[(e * NB + nb) * KB + kb] = scale;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = row0 + 16 * i;
    if (in && n < N) Wq[(e * N + n) * vec + col] = codes8(held[i], inv);
  }
}

}  // namespace

cudaError_t launch_f8_quantize(const gg_bf16* src, long long rows, int K, const int32_t* offsets,
                               int E, const int32_t* row_of_slot, int k, int R_cap, uint8_t* Q,
                               float* S, int32_t* status, int sm_count, cudaStream_t stream) {
  if (rows <= 0) return cudaSuccess;
  long long blocks = (rows + kWarps - 1) / kWarps;
  const long long cap = static_cast<long long>(sm_count) * 8;
  if (blocks > cap) blocks = cap;
  const int pieces = (K / 16 + 31) / 32;  // per lane
  const auto go = [&](auto kernel) {
    kernel<<<static_cast<int>(blocks), 32 * kWarps, 0, stream>>>(
        reinterpret_cast<const uint4*>(src), rows, K, offsets, E, row_of_slot, k, R_cap,
        reinterpret_cast<uint4*>(Q), S, status);
  };
  if (pieces <= 1) go(f8_quantize_kernel<1>);
  else if (pieces <= 2) go(f8_quantize_kernel<2>);
  else if (pieces <= 4) go(f8_quantize_kernel<4>);
  else go(f8_quantize_kernel<8>);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_f8_weight(const gg_bf16* W, int E, int N, int K, uint8_t* Wq, float* Ws,
                             cudaStream_t stream) {
  const int NB = (N + kTile - 1) / kTile, KB = (K + kTile - 1) / kTile;
  f8_weight_kernel<<<dim3(KB, NB, E), 256, 0, stream>>>(reinterpret_cast<const uint4*>(W), N, K,
                                                        NB, KB, reinterpret_cast<uint2*>(Wq), Ws);
  count_launch();
  return cudaGetLastError();
}

}  // namespace gg
