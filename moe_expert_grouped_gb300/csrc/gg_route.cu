// gg_route.cu — the router in front of the expert layer: the k largest of E
// logits per token with their probabilities, the tokens per expert, the
// balance and z losses, and the gradient of the logits.
//
// A token's logits lie in the registers of 8 lanes (up to 256 experts) or 16
// (up to 512), four columns at a time, or of 32 where there are more of them
// or more than 16 picks. The row is read once. With 8 or 16 lanes the picks
// come from sorting networks: every lane keeps the largest of its own columns,
// block by block, and three or four exchanges merge the lanes.
// One warp per token, with a search and two reductions per pick, took 500
// instructions per token of 128 logits and 2.8 times as long.
//
// Bound by the networks' comparisons (integer ALU 72% of its rate; memory is
// at 2.1 TB/s). Measured (events on an empty queue, 4 us of them launch):
// forward of 121088 x 256 BF16, k 8, sigmoid 29 us, with statistics 89;
// gradient 85; 121088 x 128 fp32, k 8 54 and 68, gradient 42; 16384 x 128 fp32,
// k 8 15 and 21, gradient 13; 121088 x 32 fp32, k 2 23 and 31, gradient 21.
//
// Selection works on the logits themselves, which both scores preserve the
// order of, as order-preserving keys: the picks do not depend on how an
// exponential rounds, and equal logits go to the lower expert id. Everything
// is held in fp32; logits' gradients are rounded once to the logits' type.

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

__device__ __forceinline__ float larger(float a, float b) {  // NaN above all
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
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
  int pieces;        // rows are whole, aligned pieces of four logits
  int32_t* idx;
  float* prob;
  float* part_p;     // [blocks][E] sums over the block's rows of score / row sum, or null
  int32_t* part_n;   // [blocks][E] picks of each expert
  float* part_z;     // [blocks] sums of logsumexp^2
  int want_losses;
};

// A block's sums over its warps, as one row of the partials.
__device__ __forceinline__ void store_partials(const float* sums, const int* hist, const float* zs,
                                               const RouteParams& p) {
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    float a = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) a += sums[w * p.E + e];
    p.part_p[static_cast<long long>(blockIdx.x) * p.E + e] = a;
    p.part_n[static_cast<long long>(blockIdx.x) * p.E + e] = hist[e];
  }
  if (threadIdx.x == 0) {
    float a = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) a += zs[w];
    p.part_z[blockIdx.x] = a;
  }
}

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
    grid_dependents_launch();
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
          for (int i = 0; i < V; ++i)
            pacc[i] += tot > 0.0f || tot != tot ? ss[i] / tot : 0.0f;
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
    store_partials(sh, hist, zs, p);
  }
}

// Sums the blocks' partials in a fixed order: counts[e], and losses[0] =
// E sum_e f_e P_e with f_e = counts[e] / (T k) and P_e the mean share of e,
// losses[1] = mean logsumexp^2. One cluster: each of its blocks takes 32
// columns at a time, 32 threads to a column (one block alone waited 27 us for
// its loads at 256 experts).
constexpr int kFinThreads = 1024;
constexpr int kFinBlocks = 8;
__global__ void __cluster_dims__(kFinBlocks, 1, 1) __launch_bounds__(kFinThreads)
route_finalise_kernel(const float* part_p, const int32_t* part_n, const float* part_z, int blocks,
                      int T, int E, int k, int32_t* counts, float* losses) {
  __shared__ float sp[32][33];
  __shared__ int sn[32][33];
  __shared__ float terms[kFinBlocks];  // of block 0: every block's share of the balance loss
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(cluster_ctarank());
  cluster_arrive();
  grid_dependency_wait();
  float term = 0.0f;  // warp 0, by lane
  for (int e0 = rank * 32; e0 < E; e0 += 32 * kFinBlocks) {
    const int e = e0 + lane;
    float a = 0.0f;
    int n = 0;
    if (e < E)
#pragma unroll 5
      for (int b = warp; b < blocks; b += 32) {
        a += part_p[static_cast<long long>(b) * E + e];
        n += part_n[static_cast<long long>(b) * E + e];
      }
    sp[warp][lane] = a;
    sn[warp][lane] = n;
    __syncthreads();
    if (warp == 0 && e < E) {
      a = 0.0f;
      n = 0;
#pragma unroll
      for (int q = 0; q < 32; ++q) {
        a += sp[q][lane];
        n += sn[q][lane];
      }
      if (counts != nullptr) counts[e] = n;
      if (T > 0)
        term += static_cast<float>(n) / (static_cast<float>(T) * static_cast<float>(k)) *
                (a / static_cast<float>(T)) * static_cast<float>(E);
    }
    __syncthreads();
  }
  cluster_wait();  // block 0 has started: its shared memory may be written
  if (warp == 0) {
    term = warp_sum(term);
    if (lane == 0)
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(
                       smem_u32(&terms[rank]), 0)),
                   "f"(term)
                   : "memory");
  }
  cluster_sync();
  if (rank == 0 && warp == 0 && losses != nullptr) {
    float z = 0.0f;
    for (int b = lane; b < blocks; b += 32) z += part_z[b];
    z = warp_sum(z);
    if (lane == 0) {
      float sum = 0.0f;
#pragma unroll
      for (int r = 0; r < kFinBlocks; ++r) sum += terms[r];
      losses[0] = sum;
      losses[1] = T > 0 ? z / static_cast<float>(T) : 0.0f;
    }
  }
}

// --------------------------------------------------- several tokens per warp

template <int kL>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = kL / 2; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

// A lane's share of a row on kL lanes, V columns of it: of every 4 kL columns,
// lane l has columns 4 l to 4 l + 3; past the row's end it holds -inf. Their
// sort keys are the order-preserving key of the logit above the complement of
// its column, all different: those past the end come after the row's own, of
// which there are at least k. 0 is below every key.
template <typename X, int V, int kL>
struct Share;

template <int V, int kL>
struct ShareColumns {
  static __device__ __forceinline__ int column(int l, int i) {
    return 4 * (l + kL * (i / 4)) + i % 4;
  }
};

// fp32: 64-bit keys.
template <int V, int kL>
struct Share<float, V, kL> : ShareColumns<V, kL> {
  using K = unsigned long long;
  using ShareColumns<V, kL>::column;
  float v[V];
  __device__ __forceinline__ void load(const float* row, int E, int l, bool pieces) {
    if (pieces) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const int c = column(l, i);
        const float4 q = c < E ? *reinterpret_cast<const float4*>(row + c)
                               : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        v[i] = q.x;
        v[i + 1] = q.y;
        v[i + 2] = q.z;
        v[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = column(l, i) < E ? row[column(l, i)] : -INFINITY;
    }
  }
  __device__ __forceinline__ float value(int i) const { return v[i]; }
  static __device__ __forceinline__ K make(float value, int c) {
    return static_cast<K>(key_of(value)) << 32 | (0xFFFFFFFFu - c);
  }
  __device__ __forceinline__ K key(int i, int l) const { return make(v[i], column(l, i)); }
  // Of four columns from i on: the largest logit's, as column i's.
  __device__ __forceinline__ K lead(int i, int l) const {
    return make(larger(larger(v[i], v[i + 1]), larger(v[i + 2], v[i + 3])), column(l, i));
  }
  static __device__ __forceinline__ int column_of(K k) {
    return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k));
  }
  static __device__ __forceinline__ float value_of_key(K k) {
    return value_of(static_cast<uint32_t>(k >> 32));
  }
};

// BF16: two columns to a word, 32-bit keys, made two at a time: adding 0 to
// the pair turns -0 into +0 and every NaN into the positive one, then the
// sign's copies flip the bits.
template <int V, int kL>
struct Share<gg_bf16, V, kL> : ShareColumns<V, kL> {
  using K = uint32_t;
  using ShareColumns<V, kL>::column;
  uint32_t w[V / 2];
  __device__ __forceinline__ void load(const gg_bf16* row, int E, int l, bool pieces) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const int c = column(l, i);
      uint2 q = make_uint2(0xFF80FF80u, 0xFF80FF80u);
      if (pieces) {
        if (c < E) q = *reinterpret_cast<const uint2*>(row + c);
      } else {
        if (c < E) q.x = 0xFF800000u | row[c];
        if (c + 1 < E) q.x = (q.x & 0xFFFFu) | static_cast<uint32_t>(row[c + 1]) << 16;
        if (c + 2 < E) q.y = 0xFF800000u | row[c + 2];
        if (c + 3 < E) q.y = (q.y & 0xFFFFu) | static_cast<uint32_t>(row[c + 3]) << 16;
      }
      w[i / 2] = q.x;
      w[i / 2 + 1] = q.y;
    }
  }
  __device__ __forceinline__ float value(int i) const {
    return i % 2 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  }
  __device__ __forceinline__ uint32_t pair(int word) const {  // two logits' keys
    __nv_bfloat162 q = *reinterpret_cast<const __nv_bfloat162*>(&w[word]);
    q = __hadd2(q, __floats2bfloat162_rn(0.0f, 0.0f));
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&q);
    uint32_t signs;  // copies of each half's sign bit (selectors with their top bit set)
    asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(signs) : "r"(u));
    return u ^ (signs | 0x80008000u);
  }
  __device__ __forceinline__ K key(int i, int l) const {
    return __byte_perm(pair(i / 2), 0xFFFFu - column(l, i), i % 2 ? 0x3254 : 0x1054);
  }
  // Of four columns from i on: the largest logit's, as column i's.
  __device__ __forceinline__ K lead(int i, int l) const {
    const uint32_t two = __vmaxu2(pair(i / 2), pair(i / 2 + 1));
    const uint32_t low = 0xFFFFu - column(l, i);
    return max(__byte_perm(two, low, 0x3254), __byte_perm(two, low, 0x1054));
  }
  static __device__ __forceinline__ int column_of(K k) { return 0xFFFF - (k & 0xFFFFu); }
  static __device__ __forceinline__ float value_of_key(K k) {
    return __uint_as_float(__float_as_uint(value_of(k)) & 0xFFFF0000u);
  }
};

template <typename K>
__device__ __forceinline__ void order(K& a, K& b) {  // the larger first
  const K hi = a > b ? a : b;
  b = a > b ? b : a;
  a = hi;
}

// Odd-even merge sort (Batcher 1968), descending: the network's comparators.
template <int N>
struct Network {
  int n = 0;
  int a[N * N / 2] = {}, b[N * N / 2] = {};
  constexpr Network() {
    for (int p = 1; p < N; p *= 2)
      for (int k = p; k >= 1; k /= 2)
        for (int j = k % p; j + k < N; j += 2 * k)
          for (int i = 0; i < k; ++i)
            if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
              a[n] = i + j;
              b[n++] = i + j + k;
            }
  }
};

template <int N, int I = 0, typename K>
__device__ __forceinline__ void sort_down(K (&v)[N]) {
  constexpr Network<N> net;
  if constexpr (I < net.n) {
    order(v[net.a[I]], v[net.b[I]]);
    sort_down<N, I + 1>(v);
  }
}

template <int N, typename K>
__device__ __forceinline__ void sort_bitonic(K (&v)[N]) {
#pragma unroll
  for (int d = N / 2; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & d) == 0) order(v[i], v[i + d]);
}

// top = the N largest of top and v, both descending: the larger of each pair
// from opposite ends is one of them, and what results is bitonic.
template <int N, typename K>
__device__ __forceinline__ void larger_ones(K (&top)[N], const K (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) top[i] = top[i] > v[N - 1 - i] ? top[i] : v[N - 1 - i];
}

// top: the N largest of all kL lanes' v, each descending; where kSet,
// unordered, and the upper half of the lanes in the other half's order
// reversed. M < N: lanes' keys are joined until there are N.
template <int kL, bool kSet, int D = 1, int M, int N, typename K>
__device__ __forceinline__ void over_lanes(K (&v)[M], K (&top)[N]) {
  if constexpr (D == kL) {
    static_assert(M == N, "too few lanes for N keys");
#pragma unroll
    for (int i = 0; i < N; ++i) top[i] = v[i];
  } else {
    K other[M];
#pragma unroll
    for (int i = 0; i < M; ++i) other[i] = __shfl_xor_sync(kFull, v[i], D);
    if constexpr (M < N) {
      K both[2 * M];
#pragma unroll
      for (int i = 0; i < M; ++i) {
        both[i] = v[i];
        both[2 * M - 1 - i] = other[i];
      }
      sort_bitonic(both);
      over_lanes<kL, kSet, 2 * D>(both, top);
    } else {
      larger_ones(v, other);
      if constexpr (!kSet || 2 * D < kL) sort_bitonic(v);
      over_lanes<kL, kSet, 2 * D>(v, top);
    }
  }
}

// V: columns per lane; N: picks kept, at least k.
template <typename X, int kL, int V, int N, bool kStats>
__global__ void __launch_bounds__(kThreads)
route_group_kernel(const X* __restrict__ x, const RouteParams p) {
  using Key = Share<X, V, kL>;
  using K = typename Key::K;
  constexpr int B = V < N ? V : N;      // block of columns sorted at once
  // From 16 columns per lane on: no pick is outside the N pieces of four
  // columns with the largest leaders (of equal ones the first), since a better
  // piece's leader comes before all of this one. So the networks run on
  // leaders, and then on those pieces, one per lane, read once more:
  // 121088 x 256 BF16 40 -> 29 us, 121088 x 128 fp32 68 -> 54.
  constexpr bool kLead = V >= 16 && N <= kL;
  constexpr int kMine = N > kL ? N / kL : 1;  // picks per lane
  extern __shared__ float sh[];         // kStats: [kWarps][E] sums, int [E] picks, [kWarps] z
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int l = lane & (kL - 1);
  const int E = p.E, k = p.k;
  int* hist = reinterpret_cast<int*>(sh + kWarps * E);
  float pacc[kStats ? V : 1];
  float zacc = 0.0f;
  if (kStats) {
#pragma unroll
    for (int i = 0; i < (kStats ? V : 1); ++i) pacc[i] = 0.0f;
    grid_dependents_launch();
    for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
    __syncthreads();
  }
  constexpr int kTokens = 32 / kL;
  // With statistics there are two blocks per SM: too few warps to hide a row's
  // loads, so the next row's are on their way meanwhile (121088 x 32 fp32, k 2:
  // 35 -> 31 us; 16 columns per lane gain nothing by it).
  constexpr bool kAhead = kStats && V <= 8;
  const long long step = static_cast<long long>(gridDim.x) * kWarps * kTokens;
  const auto row_of = [&](long long t0) { return min(t0 + lane / kL, p.T - 1LL); };
  long long t0 = (static_cast<long long>(blockIdx.x) * kWarps + warp) * kTokens;
  Key own;
  if (kAhead) own.load(x + row_of(t0) * E, E, l, p.pieces);
  for (; t0 < p.T; t0 += step) {
    const bool here = t0 + lane / kL < p.T;
    const long long t = row_of(t0);
    Key next;
    if (kAhead)
      next.load(x + row_of(t0 + step) * E, E, l, p.pieces);
    else
      own.load(x + t * E, E, l, p.pieces);
    K top[N];
    if constexpr (kLead) {
      K lead[V / 4];
#pragma unroll
      for (int i = 0; i < V / 4; ++i) lead[i] = own.lead(4 * i, l);
      sort_down(lead);
      over_lanes<kL, true>(lead, top);
      // lane l's piece is l in the order of the first lanes
      const int at = l < kL / 2 ? l : N - 1 - l;
      K mine = top[0];
#pragma unroll
      for (int j = 1; j < (N < kL ? N : kL / 2); ++j)
        if (at == j) mine = top[j];
      const int piece = Key::column_of(mine) / 4;
      Share<X, 4, kL> four;
      four.load(x + t * E, E, piece, p.pieces);
      K key[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) key[i] = N < kL && l >= N ? K(0) : four.key(i, piece);
      sort_down(key);
      over_lanes<kL, false>(key, top);
    } else {
      K best[B];
#pragma unroll
      for (int b = 0; b < V; b += B) {
        K key[B];
#pragma unroll
        for (int i = 0; i < B; ++i) key[i] = own.key(b + i, l);
        sort_down(key);
        if (b == 0) {
#pragma unroll
          for (int i = 0; i < B; ++i) best[i] = key[i];
        } else {
          larger_ones(best, key);
          sort_bitonic(best);
        }
      }
      over_lanes<kL, false>(best, top);
    }
    const float m = Key::value_of_key(top[0]);
    const bool dead = m == -INFINITY;  // no expert left: everything of the row is zero
    float mass = 0.0f;                 // sum of exp(v - m)
    float e[kStats ? V : 1];
    if (kStats) {
#pragma unroll
      for (int i = 0; i < (kStats ? V : 1); ++i)
        mass += e[i] = dead ? 0.0f : expf(own.value(i) - m);
      mass = group_sum<kL>(mass);
    } else if (!p.sigmoid && !p.renorm) {
#pragma unroll
      for (int i = 0; i < V; ++i) mass += dead ? 0.0f : expf(own.value(i) - m);
      mass = group_sum<kL>(mass);
    }
    // lane l writes picks l, l + kL, ..
    int id[kMine];
    float s[kMine], picked = 0.0f;
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      K mine = top[q * kL];
#pragma unroll
      for (int j = 1; j < kL; ++j)
        if (q * kL + j < N && l == j) mine = top[q * kL + j < N ? q * kL + j : 0];
      const float mv = Key::value_of_key(mine);
      id[q] = Key::column_of(mine);
      s[q] = q * kL + l >= k || dead ? 0.0f : (p.sigmoid ? sigmoid_of(mv) : expf(mv - m));
      picked += s[q];
    }
    const float denom = p.renorm ? group_sum<kL>(picked) : mass;
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const int j = q * kL + l;
      if (j >= k || !here) continue;
      float w = s[q];
      if (p.renorm || !p.sigmoid) w = denom > 0.0f || denom != denom ? w / denom : 0.0f;
      p.idx[t * k + j] = id[q];
      p.prob[t * k + j] = p.scale * w;
      if (kStats) atomicAdd(&hist[id[q]], 1);
    }
    if constexpr (kStats) {
      if (p.want_losses) {
        if (p.sigmoid) {
          float tot = 0.0f;
#pragma unroll
          for (int i = 0; i < V; ++i) tot += e[i] = sigmoid_of(own.value(i));
          tot = group_sum<kL>(tot);
          const float inv = tot > 0.0f || tot != tot ? 1.0f / tot : 0.0f;
          if (here) {
#pragma unroll
            for (int i = 0; i < V; ++i) pacc[i] += e[i] * inv;
          }
        } else if (here && !dead) {
          const float inv = 1.0f / mass;
#pragma unroll
          for (int i = 0; i < V; ++i) pacc[i] += e[i] * inv;
        }
        const float lse = m + logf(mass);
        if (here && !dead && l == 0) zacc += lse * lse;
      }
    }
    if (kAhead) own = next;
  }
  if constexpr (kStats) {
    // the sums over the warp's tokens, then the block's warps
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float a = pacc[i];
#pragma unroll
      for (int d = kL; d < 32; d *= 2) a += __shfl_xor_sync(kFull, a, d);
      const int c = Key::column(l, i);
      if (lane < kL && c < E) sh[warp * E + c] = a;
    }
    float* zs = reinterpret_cast<float*>(hist + E);
    zacc = warp_sum(zacc);
    if (lane == 0) zs[warp] = zacc;
    __syncthreads();
    store_partials(sh, hist, zs, p);
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
  int pieces;             // both tensors' rows are whole, aligned pieces of four
  int32_t* status;        // or null
};

// The fast exponential and divide: a few units of fp32, times the size of the
// exponent, on gradients.
__device__ __forceinline__ float fast_sigmoid(float v) {
  return __fdividef(1.0f, 1.0f + __expf(-v));
}

// Four columns' gradients from column c on, as the logits' type.
__device__ __forceinline__ void store_piece(float* row, int c, int E, bool pieces,
                                            const float (&g)[4]) {
  if (pieces) {
    if (c < E) *reinterpret_cast<float4*>(row + c) = make_float4(g[0], g[1], g[2], g[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < E) row[c + j] = g[j];
  }
}
__device__ __forceinline__ void store_piece(gg_bf16* row, int c, int E, bool pieces,
                                            const float (&g)[4]) {
  if (pieces) {
    if (c < E)
      *reinterpret_cast<uint2*>(row + c) =
          make_uint2(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < E) store_as(row + c + j, g[j]);
  }
}

// kL lanes per token, at least k. Every column's gradient without its picks is
// written first, then the picks' lanes write theirs over it. The sums over the
// row are taken together, and the next row is on its way meanwhile.
template <typename X, int V, int kL>
__global__ void __launch_bounds__(kThreads)
route_bwd_kernel(const X* x, const RouteBwdParams p, X* dx) {
  using Row = Share<X, V, kL>;
  __shared__ float4 load[kL * V / 4];  // E f_e: what the balance loss weighs a mean share with
  const int lane = threadIdx.x % kL;
  const int base = threadIdx.x & 31 & ~(kL - 1);  // the token's first lane
  const int E = p.E, k = p.k;
  const float inv_T = 1.0f / static_cast<float>(p.T);
  const bool aux = p.aux != 0.0f, zl = p.z != 0.0f;
  const bool soft = !p.sigmoid || zl;  // the softmax is needed
  const float per_pick = static_cast<float>(E) / (static_cast<float>(p.T) * static_cast<float>(k));
  for (int c = threadIdx.x; c < kL * V; c += kThreads)
    reinterpret_cast<float*>(load)[c] =
        aux && c < E ? per_pick * static_cast<float>(p.counts[c]) : 0.0f;
  __syncthreads();
  constexpr int kTokens = kThreads / kL;  // per block
  const long long step = static_cast<long long>(gridDim.x) * kTokens;
  long long t = static_cast<long long>(blockIdx.x) * kTokens + threadIdx.x / kL;
  Row own{}, next{};
  int id = -1, next_id = -1;
  float g = 0.0f, next_g = 0.0f;
  const auto fetch = [&](long long at, Row& to, int& pick, float& grad) {
    pick = -1;
    grad = 0.0f;
    if (at >= p.T) return;
    to.load(x + at * E, E, lane, p.pieces);
    if (lane < k) {
      pick = p.idx[at * k + lane];
      grad = p.dprob[at * k + lane];
    }
  };
  fetch(t, own, id, g);
  // a warp's lanes stay together: tokens past the end do not load or store
  for (long long first = t - (base / kL); first < p.T; first += step, t += step) {
    const bool here = t < p.T;
    if (here && lane < k && (id < 0 || id >= E)) {
      set_status(p.status, GG_ERR_DEVICE_BAD_EXPERT_ID);
      id = -1;
      g = 0.0f;
    }
    const float picked = id >= 0 ? to_f32(x[t * E + id]) : -INFINITY;
    fetch(t + step, next, next_id, next_g);

    float m = own.value(0);
#pragma unroll
    for (int i = 1; i < V; ++i) m = larger(m, own.value(i));
    if constexpr (kL == 32) {
      m = value_of(__reduce_max_sync(kFull, key_of(m)));
    } else {
#pragma unroll
      for (int d = kL / 2; d > 0; d >>= 1) m = larger(m, __shfl_xor_sync(kFull, m, d));
    }
    const bool dead = m == -INFINITY;
    // e: exp(v - m); sums of e, of the scores, of load * score, of the picks'
    // scores and of gradient * score (softmax: all up to 1 / mass)
    float e[V], sc[V];
    float mass = 0.0f, st = 0.0f, cs = 0.0f;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 ld = load[Row::column(lane, i) / 4];
      const float four[4] = {ld.x, ld.y, ld.z, ld.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = own.value(i + j);
        e[i + j] = soft && !dead ? __expf(v - m) : 0.0f;
        sc[i + j] = p.sigmoid ? fast_sigmoid(v) : e[i + j];
        mass += e[i + j];
        st += sc[i + j];
        cs += four[j] * sc[i + j];
      }
    }
    float ps = 0.0f;
    if (id >= 0 && !dead) ps = p.sigmoid ? fast_sigmoid(picked) : __expf(picked - m);
    float tot = ps, gps = g * ps;
#pragma unroll
    for (int d = kL / 2; d > 0; d >>= 1) {
      if (soft) mass += __shfl_xor_sync(kFull, mass, d);
      if (aux) {
        if (p.sigmoid) st += __shfl_xor_sync(kFull, st, d);
        cs += __shfl_xor_sync(kFull, cs, d);
      }
      if (p.renorm) tot += __shfl_xor_sync(kFull, tot, d);
      gps += __shfl_xor_sync(kFull, gps, d);
    }
    const float inv_mass = soft && !dead ? 1.0f / mass : 0.0f;
    const float zg = dead || !zl ? 0.0f : 2.0f * p.z * inv_T * (m + logf(mass));
    // gradient of this lane's pick: of its score, or (renormalised softmax) of its logit
    float gp = p.scale * g, dot = 0.0f;
    if (p.renorm) {
      const bool some = tot > 0.0f || tot != tot;
      gp = some ? p.scale * (g - gps / tot) / tot : 0.0f;
      if (!p.sigmoid) gp *= ps;  // the factor 1 / mass of both scores cancels
      if (id < 0) gp = 0.0f;
    } else if (!p.sigmoid) {
      dot = p.scale * gps * inv_mass;
    }
    float ga = 0.0f, mean = 0.0f;  // balance loss: gradient ga (load - mean) of each share
    if (aux) {
      const float total = p.sigmoid ? st : mass;
      if (!dead && (total > 0.0f || total != total)) {
        ga = p.sigmoid ? p.aux * inv_T / total : p.aux * inv_T;
        mean = cs / total;
      }
    }
    // a column's gradient, add: from its picks
    const auto grad = [&](float sm, float score, float ld, float add) {
      if (p.sigmoid) return (add + ga * (ld - mean)) * score * (1.0f - score) + zg * sm;
      return (p.renorm ? add : sm * (add - dot)) + sm * (ga * (ld - mean) + zg);
    };
    X* out = dx + t * E;
    if (here) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const int c = Row::column(lane, i);
        const float4 ld = load[c / 4];
        const float four[4] = {ld.x, ld.y, ld.z, ld.w};
        float to[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) to[j] = grad(e[i + j] * inv_mass, sc[i + j], four[j], 0.0f);
        store_piece(out, c, E, p.pieces, to);
      }
    }
    float add = 0.0f;  // an expert named in several slots gets them all
    for (int j = 0; j < k; ++j) {
      const int other = __shfl_sync(kFull, id, base + j);
      const float gj = __shfl_sync(kFull, gp, base + j);
      if (other == id) add += gj;
    }
    __syncwarp();  // the picks' columns are written after the others
    if (here && id >= 0) {
      const float sm = soft && !dead ? __expf(picked - m) * inv_mass : 0.0f;
      const float ld = reinterpret_cast<const float*>(load)[id];
      store_as(out + id, grad(sm, p.sigmoid ? fast_sigmoid(picked) : 0.0f, ld, add));
    }
    own = next;
    id = next_id;
    g = next_g;
  }
}

// Lanes per token of the forward: eight or 16 hold a row and its picks, else a
// warp (121088 x 512 fp32, k 8: 167 us against 202).
inline int fwd_lanes(int E, int k) { return E > 512 || k > 16 ? 32 : E > 256 ? 16 : 8; }

template <typename X, bool kStats, int kL, int V>
void launch_route_group(const RouteArgs& a, const RouteParams& p, int blocks, size_t smem,
                        cudaStream_t stream) {
  const auto go = [&](auto kernel) {
    kernel<<<blocks, kThreads, smem, stream>>>(static_cast<const X*>(a.logits), p);
  };
  if constexpr (V <= 4) {
    if (a.k <= 4) return go(route_group_kernel<X, kL, V, 4, kStats>);
  }
  if (a.k <= 8) go(route_group_kernel<X, kL, V, 8, kStats>);
  else go(route_group_kernel<X, kL, V, 16, kStats>);
}

template <typename X, bool kStats>
cudaError_t launch_route_t(const RouteArgs& a, const RouteParams& p, int blocks, size_t smem,
                           cudaStream_t stream) {
  const int lanes = fwd_lanes(a.E, a.k);
  if (lanes < 32) {
    if (a.E <= 32) launch_route_group<X, kStats, 8, 4>(a, p, blocks, smem, stream);
    else if (a.E <= 64) launch_route_group<X, kStats, 8, 8>(a, p, blocks, smem, stream);
    else if (a.E <= 128) launch_route_group<X, kStats, 8, 16>(a, p, blocks, smem, stream);
    else if (lanes == 8) launch_route_group<X, kStats, 8, 32>(a, p, blocks, smem, stream);
    else launch_route_group<X, kStats, 16, 32>(a, p, blocks, smem, stream);
    count_launch();
    return cudaGetLastError();
  }
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

// Lanes per token of the backward: as few as hold the row at 16 columns each,
// and its picks (121088 x 128 fp32: 42 us, 52 at 8 columns each, 66 at 4;
// 121088 x 256 BF16, sigmoid: 85 us, 97 at 8 columns, 242 at 32).
inline int bwd_lanes(int E, int k) {
  if (E <= 128 && k <= 8) return 8;
  if (E <= 256 && k <= 16) return 16;
  return 32;
}

template <typename X, int kL, int V>
void launch_route_bwd_v(const RouteBwdArgs& a, const RouteBwdParams& p, int blocks,
                        cudaStream_t stream) {
  route_bwd_kernel<X, V, kL><<<blocks, kThreads, 0, stream>>>(
      static_cast<const X*>(a.logits), p, static_cast<X*>(a.dlogits));
}

template <typename X>
cudaError_t launch_route_bwd_t(const RouteBwdArgs& a, const RouteBwdParams& p, int blocks,
                               cudaStream_t stream) {
  const int lanes = bwd_lanes(a.E, a.k);
  const int v = (a.E + lanes - 1) / lanes;  // columns per lane
  if (lanes == 8) {
    if (v <= 4) launch_route_bwd_v<X, 8, 4>(a, p, blocks, stream);
    else if (v <= 8) launch_route_bwd_v<X, 8, 8>(a, p, blocks, stream);
    else launch_route_bwd_v<X, 8, 16>(a, p, blocks, stream);
  } else if (lanes == 16) {
    if (v <= 8) launch_route_bwd_v<X, 16, 8>(a, p, blocks, stream);
    else launch_route_bwd_v<X, 16, 16>(a, p, blocks, stream);
  } else if (v <= 8) launch_route_bwd_v<X, 32, 8>(a, p, blocks, stream);
  else if (v <= 16) launch_route_bwd_v<X, 32, 16>(a, p, blocks, stream);
  else launch_route_bwd_v<X, 32, 32>(a, p, blocks, stream);
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
  p.pieces =
      a.E % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % (a.bf16 ? 8 : 16) == 0;
  const bool stats = a.counts != nullptr || a.losses != nullptr;
  const int tokens = 32 / fwd_lanes(a.E, a.k);  // per warp
  const long long want =
      (static_cast<long long>(a.T) + kWarps * tokens - 1) / (kWarps * tokens);
  const int blocks = static_cast<int>(want < kRouteMaxBlocks ? want : kRouteMaxBlocks);
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
    e = launch_early(route_finalise_kernel, dim3(kFinBlocks), dim3(kFinThreads), 0, stream,
                     p.part_p, p.part_n, p.part_z, blocks, a.T, a.E, a.k, a.counts, a.losses);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  if (blocks == 0) return cudaSuccess;
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
  p.pieces = a.E % 4 == 0 && (reinterpret_cast<uintptr_t>(a.logits) |
                              reinterpret_cast<uintptr_t>(a.dlogits)) % (a.bf16 ? 8 : 16) == 0;
  const int tokens = kThreads / bwd_lanes(a.E, a.k);  // per block
  const long long want = (static_cast<long long>(a.T) + tokens - 1) / tokens;
  const long long cap = static_cast<long long>(dev.sm_count) * 8;
  const int grid = static_cast<int>(want < cap ? want : cap);
  return a.bf16 ? launch_route_bwd_t<gg_bf16>(a, p, grid, stream)
                : launch_route_bwd_t<float>(a, p, grid, stream);
}

}  // namespace gg
