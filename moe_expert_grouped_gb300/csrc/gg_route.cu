// gg_route.cu — the router in front of the expert layer: the k largest of E
// logits per token with their probabilities, the tokens per expert, the
// balance and z losses, and the gradient of the logits.
//
// One warp holds one token's logits in registers (column c in lane c % 32),
// so every statistic of the row (maximum, sums of the scores, the picks) is a
// warp reduction and the row is read once. Selection works on the logits
// themselves, which both scores preserve the order of, as order-preserving
// 32-bit keys: the picks do not depend on how an exponential rounds, and
// equal logits go to the lower expert id. Everything is held in fp32; logits'
// gradients are rounded once to the logits' type.

#include <cuda_runtime.h>

#include <cmath>

#include "gg_internal.h"
#include "gg_launch.cuh"
#include "gg_ptx.cuh"

namespace gg {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kFull = 0xFFFFFFFFu;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(gg_bf16 v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
__device__ __forceinline__ void store_as(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_as(gg_bf16* p, float v) {
  *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Order-preserving key of a logit: larger logits have larger keys, both zeros
// the same one, NaN the largest of all, -inf a key above 0 (0 = "taken").
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  if (v != v) return 0xFFFFFFFFu;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key ^ 0x80000000u) : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

__device__ __forceinline__ float sigmoid_of(float v) { return 1.0f / (1.0f + expf(-v)); }

// A row's logits: v[i] is column lane + 32 i, -inf past the last one.
template <typename X, int V>
__device__ __forceinline__ void load_row(const X* row, int E, int lane, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = lane + 32 * i;
    v[i] = c < E ? to_f32(row[c]) : -INFINITY;
  }
}

struct RouteParams {
  int T, E, k;
  int sigmoid, renorm;
  float scale;
  int32_t* idx;
  float* prob;
  float* part_p;     // [blocks][E] sums over the block's rows of score / row sum, or null
  int32_t* part_n;   // [blocks][E] picks of each expert
  float* part_z;     // [blocks] sums of logsumexp^2
  int want_losses;
};

template <typename X, int V, bool kStats>
__global__ void __launch_bounds__(kThreads)
route_kernel(const X* __restrict__ x, const RouteParams p) {
  extern __shared__ float sh[];  // kStats: [kWarps][E] sums, then int [E] picks, [kWarps] z
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int E = p.E, k = p.k;
  int* hist = reinterpret_cast<int*>(sh + kWarps * E);
  float pacc[V];
  float zacc = 0.0f;
  if (kStats) {
#pragma unroll
    for (int i = 0; i < V; ++i) pacc[i] = 0.0f;
    for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
    __syncthreads();
  }
  for (long long t = static_cast<long long>(blockIdx.x) * kWarps + warp; t < p.T;
       t += static_cast<long long>(gridDim.x) * kWarps) {
    float v[V];
    uint32_t key[V];
    load_row<X, V>(x + t * E, E, lane, v);
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = lane + 32 * i < E ? key_of(v[i]) : 0u;
    int my_id = 0;
    uint32_t my_key = 0;
    for (int j = 0; j < k; ++j) {
      uint32_t best = 0;
      int bi = 0;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] > best) {
          best = key[i];
          bi = i;
        }
      const uint32_t top = __reduce_max_sync(kFull, best);
      const uint32_t c = __reduce_min_sync(
          kFull, best == top ? static_cast<uint32_t>(lane + 32 * bi) : 0xFFFFFFFFu);
      if ((c & 31u) == static_cast<uint32_t>(lane)) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (c >> 5 == static_cast<uint32_t>(i)) key[i] = 0;
      }
      if (lane == j) {
        my_id = static_cast<int>(c);
        my_key = top;
      }
    }
    const float mine = value_of(my_key);  // lanes < k: this pick's logit
    const float m = __shfl_sync(kFull, mine, 0);
    const bool dead = m == -INFINITY;     // no expert left: everything of the row is zero
    const bool pick = lane < k;
    float row_sum = 0.0f;                 // softmax: sum of exp(v - m)
    if (kStats || (!p.sigmoid && !p.renorm)) {
#pragma unroll
      for (int i = 0; i < V; ++i) row_sum += dead ? 0.0f : expf(v[i] - m);
      row_sum = warp_sum(row_sum);
    }
    float s = 0.0f;  // this pick's score, up to the softmax's common factor
    if (pick && !dead) s = p.sigmoid ? sigmoid_of(mine) : expf(mine - m);
    float denom = row_sum;
    if (p.renorm) denom = warp_sum(s);
    float w = s;
    if (p.renorm || !p.sigmoid) w = denom > 0.0f || denom != denom ? s / denom : 0.0f;
    if (pick) {
      p.idx[t * k + lane] = my_id;
      p.prob[t * k + lane] = p.scale * w;
    }
    if (kStats) {
      if (pick) atomicAdd(&hist[my_id], 1);
      if (p.want_losses && !dead) {
        const float lse = m + logf(row_sum);
        zacc += lse * lse;
        if (p.sigmoid) {
          float ss[V], tot = 0.0f;
#pragma unroll
          for (int i = 0; i < V; ++i) tot += ss[i] = sigmoid_of(v[i]);
          tot = warp_sum(tot);
#pragma unroll
          for (int i = 0; i < V; ++i) pacc[i] += tot > 0.0f ? ss[i] / tot : 0.0f;
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) pacc[i] += expf(v[i] - m) / row_sum;
        }
      }
    }
  }
  if (kStats) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i < E) sh[warp * E + lane + 32 * i] = pacc[i];
    float* zs = reinterpret_cast<float*>(hist + E);
    if (lane == 0) zs[warp] = zacc;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float a = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) a += sh[w * E + e];
      p.part_p[static_cast<long long>(blockIdx.x) * E + e] = a;
      p.part_n[static_cast<long long>(blockIdx.x) * E + e] = hist[e];
    }
    if (threadIdx.x == 0) {
      float a = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) a += zs[w];
      p.part_z[blockIdx.x] = a;
    }
  }
}

// Sums the blocks' partials in a fixed order: counts[e], and losses[0] =
// E sum_e f_e P_e with f_e = counts[e] / (T k) and P_e the mean share of e,
// losses[1] = mean logsumexp^2.
constexpr int kFinThreads = 1024;
__global__ void __launch_bounds__(kFinThreads)
route_finalise_kernel(const float* part_p, const int32_t* part_n, const float* part_z, int blocks,
                      int T, int E, int k, int32_t* counts, float* losses) {
  __shared__ float sp[kFinThreads];
  __shared__ int sn[kFinThreads];
  const int tid = threadIdx.x;
  int cols = 32;  // columns handled side by side, a power of two >= min(E, 1024)
  while (cols < E) cols *= 2;
  const int groups = kFinThreads / cols;
  const int e = tid & (cols - 1), g = tid / cols;
  float a = 0.0f;
  int n = 0;
  if (e < E)
    for (int b = g; b < blocks; b += groups) {
      a += part_p[static_cast<long long>(b) * E + e];
      n += part_n[static_cast<long long>(b) * E + e];
    }
  sp[tid] = a;
  sn[tid] = n;
  __syncthreads();
  float term = 0.0f;
  if (g == 0 && e < E) {
    for (int q = 1; q < groups; ++q) {
      a += sp[q * cols + e];
      n += sn[q * cols + e];
    }
    if (counts != nullptr) counts[e] = n;
    if (T > 0)
      term = static_cast<float>(n) / (static_cast<float>(T) * static_cast<float>(k)) *
             (a / static_cast<float>(T)) * static_cast<float>(E);
  }
  float z = 0.0f;
  for (int b = tid; b < blocks; b += kFinThreads) z += part_z[b];
  __syncthreads();
  term = warp_sum(term);
  z = warp_sum(z);
  if ((tid & 31) == 0) {
    sp[tid >> 5] = term;
    sp[32 + (tid >> 5)] = z;
  }
  __syncthreads();
  if (tid < 32 && losses != nullptr) {
    term = warp_sum(sp[tid]);
    z = warp_sum(sp[32 + tid]);
    if (tid == 0) {
      losses[0] = term;
      losses[1] = T > 0 ? z / static_cast<float>(T) : 0.0f;
    }
  }
}

struct RouteBwdParams {
  int T, E, k;
  int sigmoid, renorm;
  float scale;
  const int32_t* idx;
  const float* dprob;
  const int32_t* counts;  // null when aux is 0
  float aux, z;           // coefficients of the two losses
  int32_t* status;        // or null
};

template <typename X, int V>
__global__ void __launch_bounds__(kThreads)
route_bwd_kernel(const X* x, const RouteBwdParams p, X* dx) {
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int E = p.E, k = p.k;
  const float inv_T = 1.0f / static_cast<float>(p.T);
  float load[V];  // E f_e: what the balance loss weighs expert e's mean share with
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = lane + 32 * i;
    load[i] = p.counts != nullptr && c < E
                  ? static_cast<float>(E) * static_cast<float>(p.counts[c]) /
                        (static_cast<float>(p.T) * static_cast<float>(k))
                  : 0.0f;
  }
  for (long long t = static_cast<long long>(blockIdx.x) * kWarps + warp; t < p.T;
       t += static_cast<long long>(gridDim.x) * kWarps) {
    float v[V];
    const X* row = x + t * E;
    load_row<X, V>(row, E, lane, v);
    int id = -1;
    float g = 0.0f, picked = -INFINITY;
    if (lane < k) {
      id = p.idx[t * k + lane];
      if (id < 0 || id >= E) {
        set_status(p.status, GG_ERR_DEVICE_BAD_EXPERT_ID);
        id = -1;
      } else {
        g = p.dprob[t * k + lane];
        picked = to_f32(row[id]);
      }
    }
    float m = v[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, v[i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
    const bool dead = m == -INFINITY;
    float soft[V], mass = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) mass += soft[i] = dead ? 0.0f : expf(v[i] - m);
    mass = warp_sum(mass);
    const float inv_mass = dead ? 0.0f : 1.0f / mass;
#pragma unroll
    for (int i = 0; i < V; ++i) soft[i] *= inv_mass;
    const float zg = dead ? 0.0f : 2.0f * p.z * inv_T * (m + logf(mass));

    // gradient of this lane's pick: of its score, or (renormalised softmax) of its logit
    float ps = 0.0f;
    if (id >= 0 && !dead) ps = p.sigmoid ? sigmoid_of(picked) : expf(picked - m) * inv_mass;
    float gp = p.scale * g;
    if (p.renorm) {
      const float tot = warp_sum(ps);
      const float share = tot > 0.0f || tot != tot ? ps / tot : 0.0f;
      const float mean = warp_sum(g * share);
      gp = p.scale * (g - mean);
      if (p.sigmoid)
        gp = tot > 0.0f || tot != tot ? gp / tot : 0.0f;
      else
        gp *= share;
    }
    const float dot = !p.sigmoid && !p.renorm ? warp_sum(gp * ps) : 0.0f;
    float add[V];
#pragma unroll
    for (int i = 0; i < V; ++i) add[i] = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int c = __shfl_sync(kFull, id, j);
      const float gj = __shfl_sync(kFull, gp, j);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c == lane + 32 * i) add[i] += gj;
    }
    if (p.sigmoid) {
      float s[V], tot = 0.0f, cs = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[i] = sigmoid_of(v[i]);
        tot += s[i];
        cs += load[i] * s[i];
      }
      float ga = 0.0f, mean = 0.0f;
      if (p.aux != 0.0f) {
        tot = warp_sum(tot);
        mean = warp_sum(cs) / tot;
        ga = tot > 0.0f || tot != tot ? p.aux * inv_T / tot : 0.0f;
        if (ga == 0.0f) mean = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        soft[i] = (add[i] + ga * (load[i] - mean)) * s[i] * (1.0f - s[i]) + zg * soft[i];
    } else {
      float cs = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) cs += load[i] * soft[i];
      const float mean = p.aux != 0.0f ? warp_sum(cs) : 0.0f;
      const float ga = p.aux * inv_T;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float own = p.renorm ? add[i] : soft[i] * (add[i] - dot);
        soft[i] = own + soft[i] * (ga * (load[i] - mean) + zg);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i < E) store_as(dx + t * E + lane + 32 * i, soft[i]);
  }
}

template <typename X, bool kStats>
cudaError_t launch_route_t(const RouteArgs& a, const RouteParams& p, int blocks, size_t smem,
                           cudaStream_t stream) {
  const X* x = static_cast<const X*>(a.logits);
  const int v = (a.E + 31) / 32;
  if (v <= 1) route_kernel<X, 1, kStats><<<blocks, kThreads, smem, stream>>>(x, p);
  else if (v <= 2) route_kernel<X, 2, kStats><<<blocks, kThreads, smem, stream>>>(x, p);
  else if (v <= 4) route_kernel<X, 4, kStats><<<blocks, kThreads, smem, stream>>>(x, p);
  else if (v <= 8) route_kernel<X, 8, kStats><<<blocks, kThreads, smem, stream>>>(x, p);
  else if (v <= 16) route_kernel<X, 16, kStats><<<blocks, kThreads, smem, stream>>>(x, p);
  else route_kernel<X, 32, kStats><<<blocks, kThreads, smem, stream>>>(x, p);
  count_launch();
  return cudaGetLastError();
}

template <typename X>
cudaError_t launch_route_bwd_t(const RouteBwdArgs& a, const RouteBwdParams& p, int blocks,
                               cudaStream_t stream) {
  const X* x = static_cast<const X*>(a.logits);
  X* dx = static_cast<X*>(a.dlogits);
  const int v = (a.E + 31) / 32;
  if (v <= 1) route_bwd_kernel<X, 1><<<blocks, kThreads, 0, stream>>>(x, p, dx);
  else if (v <= 2) route_bwd_kernel<X, 2><<<blocks, kThreads, 0, stream>>>(x, p, dx);
  else if (v <= 4) route_bwd_kernel<X, 4><<<blocks, kThreads, 0, stream>>>(x, p, dx);
  else if (v <= 8) route_bwd_kernel<X, 8><<<blocks, kThreads, 0, stream>>>(x, p, dx);
  else if (v <= 16) route_bwd_kernel<X, 16><<<blocks, kThreads, 0, stream>>>(x, p, dx);
  else route_bwd_kernel<X, 32><<<blocks, kThreads, 0, stream>>>(x, p, dx);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

int route_blocks(long long T) {
  const long long b = (T + kWarps - 1) / kWarps;
  return static_cast<int>(b < kRouteMaxBlocks ? b : kRouteMaxBlocks);
}

cudaError_t launch_route(const RouteArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  RouteParams p{};
  p.T = a.T;
  p.E = a.E;
  p.k = a.k;
  p.sigmoid = a.sigmoid;
  p.renorm = a.renorm;
  p.scale = a.scale;
  p.idx = a.idx;
  p.prob = a.prob;
  const bool stats = a.counts != nullptr || a.losses != nullptr;
  const int blocks = route_blocks(a.T);
  cudaError_t e = cudaSuccess;
  if (stats) {
    p.part_p = a.scratch;
    p.part_n = reinterpret_cast<int32_t*>(a.scratch + static_cast<size_t>(blocks) * a.E);
    p.part_z = a.scratch + 2 * static_cast<size_t>(blocks) * a.E;
    p.want_losses = a.losses != nullptr;
    const size_t smem = (static_cast<size_t>(kWarps + 1) * a.E + kWarps) * sizeof(float);
    if (blocks > 0) {
      e = a.bf16 ? launch_route_t<gg_bf16, true>(a, p, blocks, smem, stream)
                 : launch_route_t<float, true>(a, p, blocks, smem, stream);
      if (e != cudaSuccess) return e;
    }
    route_finalise_kernel<<<1, kFinThreads, 0, stream>>>(p.part_p, p.part_n, p.part_z, blocks, a.T,
                                                         a.E, a.k, a.counts, a.losses);
    count_launch();
    return cudaGetLastError();
  }
  if (blocks == 0) return cudaSuccess;
  const long long want = (static_cast<long long>(a.T) + kWarps - 1) / kWarps;
  const long long cap = static_cast<long long>(dev.sm_count) * 8;
  const int grid = static_cast<int>(want < cap ? want : cap);
  return a.bf16 ? launch_route_t<gg_bf16, false>(a, p, grid, 0, stream)
                : launch_route_t<float, false>(a, p, grid, 0, stream);
}

cudaError_t launch_route_bwd(const RouteBwdArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  RouteBwdParams p{};
  p.T = a.T;
  p.E = a.E;
  p.k = a.k;
  p.sigmoid = a.sigmoid;
  p.renorm = a.renorm;
  p.scale = a.scale;
  p.idx = a.idx;
  p.dprob = a.dprob;
  p.counts = a.aux != 0.0f ? a.counts : nullptr;
  p.aux = a.aux;
  p.z = a.z;
  p.status = a.status;
  const long long want = (static_cast<long long>(a.T) + kWarps - 1) / kWarps;
  const long long cap = static_cast<long long>(dev.sm_count) * 8;
  const int grid = static_cast<int>(want < cap ? want : cap);
  return a.bf16 ? launch_route_bwd_t<gg_bf16>(a, p, grid, stream)
                : launch_route_bwd_t<float>(a, p, grid, stream);
}

}  // namespace gg
