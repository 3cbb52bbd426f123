// gg_adamw.cu — the optimizer step over many tensors in one launch, and the
// norm of all gradients that clips it.
//
// For each element, every operation rounded to fp32 (fused multiply-adds would
// move a result by an ulp, and a code of an 8-bit state at a border by a step):
//   g' = s g,  m' = b1 m + (1 - b1) g',  v' = b2 v + (1 - b2) g'^2,
//   w' = w (1 - lr wd) - (m' c1) / (sqrt(v') c2 + eps),
//   c1 = lr / (1 - b1^t),  c2 = 1 / sqrt(1 - b2^t).
//
// 8-bit states are E4M3 codes of m' and of sqrt(v') (half of v's range of
// exponents), with one fp32 scale a / 448 for each cell of 256 elements, a the
// cell's largest magnitude. A state moves by less than half a code's step in
// most steps (b2 near 1: 0.05 of a percent of sqrt(v), a step is 6 to 12), and
// rounding to nearest would leave it where it is. So what is kept from one
// step to the next in fewer than 32 bits, the states and BF16 weights, is
// rounded up with the probability of the part cut off, by bits of a hash
// (Wellons' two-multiplication mixer) of seed, step, tensor and element: 256 hashes
// of neighbouring numbers from a cell's key on. In a large list two cells' keys
// can lie closer than that, and then share words; each rounding stays unbiased. A
// sqrt(v') above 0 keeps at least the smallest code: as 0 it would divide m'
// by eps alone.
//
// A warp takes a cell of 256 elements, a block eight of them; the blocks go
// through all tensors' cells together, so that small tensors cost what they
// hold and not a launch each. The list of tensors travels in the launch's
// parameters: nothing is copied to the device ahead of it, and a captured
// launch keeps its own.
//
// What bounds it: memory with 32-bit states (120 M elements, fp32 weights, BF16
// gradients: 500 us, with BF16 copies 536, 6.2 TB/s; no array aligned 584 and
// 630), the issue of instructions with 8-bit ones, some 110 an element: a
// division and a square root, both rounded to nearest, the hash, two codes (their
// cells' two reciprocals serve eight elements of a lane). fp32 weights 404 us,
// BF16 ones 420, 79 % of the issue slots; no array aligned 485 and 456.

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>

#include "gg_internal.h"
#include "gg_launch.cuh"
#include "gg_ptx.cuh"

namespace gg {
namespace {

constexpr int kCell = 256;        // elements that share a scale
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kFew = 8, kSome = 64, kMany = 310;  // tensors in a launch's parameters (32 KB at most)
constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr uint32_t kInf = 0x7F800000u;
constexpr float kTop = 448.0f;                       // largest E4M3 value
constexpr float kAmaxFloor = 7.888609052210118e-31f; // 2^-100

struct Entry {
  void* w;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  gg_bf16* half;
  long long n;
  long long first;         // blocks' turns of kWarps cells before this tensor's
  double lr_scale, decay;
  float c1, kept;          // from the host's lr and step
  int position;            // in the caller's list
  int wide;                // every array aligned for four elements at a time
};
static_assert(sizeof(Entry) == 104, "parameter space");

template <int kCap>
struct List {
  Entry t[kCap];
};

struct StepParams {
  int count;
  long long turns;
  float b1, b2, ib1, ib2, c2, eps;
  uint32_t run_key;
  const float* grad_scale;
  // values that a captured launch reads anew
  const float* lr_dev;
  const int32_t* step_dev;
  double lr, beta1, beta2;
  long long step;
  uint32_t seed_key;
};

// ----------------------------------------------------- randomness and powers

__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

__host__ __device__ __forceinline__ double times(double a, double b) {
#ifdef __CUDA_ARCH__
  return __dmul_rn(a, b);
#else
  volatile double r = a * b;  // a rounded product on every host
  return r;
#endif
}

// beta^t by squaring: the same products, so the same bits, on host and device.
__host__ __device__ inline double power(double beta, long long t) {
  double r = 1.0, b = beta;
  for (; t > 0; t >>= 1) {
    if (t & 1) r = times(r, b);
    b = times(b, b);
  }
  return r;
}

struct Factors {
  double lr, per_step;  // lr / (1 - b1^t)
  float c2;
};

__host__ __device__ inline Factors factors(double lr, double beta1, double beta2, long long t) {
  Factors f;
  const double p1 = power(beta1, t), p2 = power(beta2, t);
  f.lr = lr;
  f.per_step = lr / (1.0 - p1);
  f.c2 = static_cast<float>(1.0 / sqrt(1.0 - p2));
  return f;
}

__host__ __device__ inline float c1_of(const Factors& f, double lr_scale) {
  return static_cast<float>(times(f.per_step, lr_scale));
}

__host__ __device__ inline float kept_of(const Factors& f, double lr_scale, double decay) {
  return static_cast<float>(1.0 - times(times(f.lr, lr_scale), decay));
}

// -------------------------------------------------------------- the elements

// Rounded products of two elements at a time, and their sums one by one: packed
// multiplications and additions came out fused, whatever rounding they named.
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 mul(float2 a, float b) { return mul(a, make_float2(b, b)); }
__device__ __forceinline__ float2 add(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// Values of four E4M3 codes.
__device__ __forceinline__ void e4m3_values(uint32_t codes, float2* to) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(codes >> (16 * h) & 0xFFFFu), __NV_E4M3);
    to[h] = __half22float2(__half2(r));
  }
}

// E4M3 code of y in [0, 448], rounded up where the part cut off exceeds
// 1 - r / 2^20, r the random bits (16 of them, times 16). Below 2^-6 codes are
// 2^-9 apart, as mantissas of 3 bits are from 2^-6 to 2^-5: y + 2^-6 is cut
// there. y 448 / a may exceed 448 by its rounding: at most code 126.
__device__ __forceinline__ uint32_t round_code(float y, uint32_t r) {
  const bool small = y < 0.015625f;
  const float z = small ? __fadd_rn(y, 0.015625f) : y;
  const uint32_t less = small ? 968u << 20 : 960u << 20;
  return min((__float_as_uint(z) + r - less) >> 20, 126u);
}

// The low bytes of a, b, c, d as one word.
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// How a cell is read and written: four neighbours of a lane at once or one by
// one (arrays that are not aligned), or those below its end (a tensor's last
// cell). One by one, a lane's neighbours are still the better ones: 552 us where
// an element of every 32 took 625 (120 M elements, fp32 states, weights and
// gradients unaligned).
enum Way : int { kWide = 0, kSingle = 1, kPartial = 2 };

__device__ __forceinline__ int place(int i, int lane) {
  return 128 * (i / 4) + 4 * lane + i % 4;
}

// A lane's eight elements of 32-bit or BF16 values.
template <Way kWay, typename T>
__device__ __forceinline__ void load8(float2 (&x)[4], const void* base, long long e0, int n,
                                      int lane) {
  const T* from = static_cast<const T*>(base) + e0;
  if constexpr (kWay == kWide) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = 128 * h + 4 * lane;
      if constexpr (sizeof(T) == 4) {
        const float4 v = *reinterpret_cast<const float4*>(from + j);
        x[2 * h] = make_float2(v.x, v.y);
        x[2 * h + 1] = make_float2(v.z, v.w);
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(from + j);
        x[2 * h] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
        x[2 * h + 1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = place(i, lane);
      float v = 0.0f;
      if (kWay == kSingle || j < n) {
        if constexpr (sizeof(T) == 4)
          v = from[j];
        else
          v = __uint_as_float(static_cast<uint32_t>(from[j]) << 16);
      }
      (i & 1 ? x[i / 2].y : x[i / 2].x) = v;
    }
  }
}

template <Way kWay>
__device__ __forceinline__ void load_codes(uint32_t (&w)[2], const void* base, long long e0, int n,
                                           int lane) {
  const uint8_t* from = static_cast<const uint8_t*>(base) + e0;
  if constexpr (kWay == kWide) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[h] = *reinterpret_cast<const uint32_t*>(from + 128 * h + 4 * lane);
  } else {
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = place(i, lane);
      c[i] = kWay == kSingle || j < n ? from[j] : 0u;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) w[h] = bytes4(c[4 * h], c[4 * h + 1], c[4 * h + 2], c[4 * h + 3]);
  }
}

template <Way kWay>
__device__ __forceinline__ void store8(const float2 (&x)[4], void* base, long long e0, int n,
                                       int lane) {
  float* to = static_cast<float*>(base) + e0;
  if constexpr (kWay == kWide) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float4*>(to + 128 * h + 4 * lane) =
          make_float4(x[2 * h].x, x[2 * h].y, x[2 * h + 1].x, x[2 * h + 1].y);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = place(i, lane);
      if (kWay == kSingle || j < n) to[j] = i & 1 ? x[i / 2].y : x[i / 2].x;
    }
  }
}

// Pairs of BF16.
template <Way kWay>
__device__ __forceinline__ void store8_bf16(const uint32_t (&x)[4], gg_bf16* base, long long e0,
                                            int n, int lane) {
  gg_bf16* to = base + e0;
  if constexpr (kWay == kWide) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<uint2*>(to + 128 * h + 4 * lane) = make_uint2(x[2 * h], x[2 * h + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = place(i, lane);
      if (kWay == kSingle || j < n)
        to[j] = static_cast<gg_bf16>(i & 1 ? x[i / 2] >> 16 : x[i / 2] & 0xFFFFu);
    }
  }
}

template <Way kWay>
__device__ __forceinline__ void store_codes(const uint32_t (&w)[2], void* base, long long e0,
                                            int n, int lane) {
  uint8_t* to = static_cast<uint8_t*>(base) + e0;
  if constexpr (kWay == kWide) {
#pragma unroll
    for (int h = 0; h < 2; ++h) *reinterpret_cast<uint32_t*>(to + 128 * h + 4 * lane) = w[h];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = place(i, lane);
      if (kWay == kSingle || j < n) to[j] = static_cast<uint8_t>(w[i / 4] >> (8 * (i % 4)));
    }
  }
}

// What the elements of a tensor share.
struct Shared {
  float gs, b1, b2, ib1, ib2, c1, c2, eps, kept;
  uint32_t key;  // of the cell
};

template <Way kWay, typename W, typename G, bool k8>
__device__ __forceinline__ void step_cell(const Entry& t, long long cell, int n, int lane,
                                          const Shared& k) {
  const long long e0 = cell * kCell;
  float2 w[4], g[4], m[4], v[4];
  float ms = 0.0f, vs = 0.0f;
  load8<kWay, W>(w, t.w, e0, n, lane);
  load8<kWay, G>(g, t.g, e0, n, lane);
  if constexpr (k8) {
    uint32_t mw[2], vw[2];
    load_codes<kWay>(mw, t.m, e0, n, lane);
    load_codes<kWay>(vw, t.v, e0, n, lane);
    ms = t.ms[cell];
    vs = t.vs[cell];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      e4m3_values(mw[h], m + 2 * h);
      e4m3_values(vw[h], v + 2 * h);
    }
  } else {
    load8<kWay, float>(m, t.m, e0, n, lane);
    load8<kWay, float>(v, t.v, e0, n, lane);
  }
  uint32_t mtop = 0, vtop = 0, wtop = 0;
  float2 r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 gi = mul(g[i], k.gs);
    if constexpr (k8) {
      m[i] = mul(m[i], ms);
      v[i] = mul(v[i], vs);
      v[i] = mul(v[i], v[i]);
    }
    m[i] = add(mul(m[i], k.b1), mul(gi, k.ib1));
    v[i] = add(mul(v[i], k.b2), mul(mul(gi, gi), k.ib2));
    r[i] = make_float2(__fsqrt_rn(v[i].x), __fsqrt_rn(v[i].y));
    const float2 up = mul(m[i], k.c1);
    const float2 down = add(mul(r[i], k.c2), make_float2(k.eps, k.eps));
    const float2 q = make_float2(-__fdiv_rn(up.x, down.x), -__fdiv_rn(up.y, down.y));
    w[i] = add(mul(w[i], k.kept), q);
    // as bits: ordered, a NaN above infinity. What is behind a tensor's end is
    // all 0 and stays 0 in m and v.
    if constexpr (k8) {
      mtop = max(mtop, max(magnitude(m[i].x), magnitude(m[i].y)));
      vtop = max(vtop, max(magnitude(r[i].x), magnitude(r[i].y)));
    }
    if constexpr (sizeof(W) == 2)
      wtop = max(wtop, max(magnitude(w[i].x), magnitude(w[i].y)));
  }
  uint32_t noise[8];
  if constexpr (k8 || sizeof(W) == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) noise[i] = mix(k.key + place(i, lane));
  }
  if constexpr (k8) {
    mtop = __reduce_max_sync(kFull, mtop);
    vtop = __reduce_max_sync(kFull, vtop);
    // a NaN or infinity makes the cell's scale NaN, and so all its values
    const bool mfine = mtop < kInf, vfine = vtop < kInf;
    const float ma = fmaxf(__uint_as_float(mtop), kAmaxFloor);
    const float va = fmaxf(__uint_as_float(vtop), kAmaxFloor);
    const float minv = __fmul_rn(__frcp_rn(ma), kTop);
    const float vinv = __fmul_rn(__frcp_rn(va), kTop);
    if (lane == 0) {
      t.ms[cell] = mfine ? __fmul_rn(ma, 1.0f / kTop) : __uint_as_float(0x7FC00000u);
      t.vs[cell] = vfine ? __fmul_rn(va, 1.0f / kTop) : __uint_as_float(0x7FC00000u);
    }
    uint32_t mo[2], vo[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t a[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * h + j;
        const float mi = i & 1 ? m[i / 2].y : m[i / 2].x, ri = i & 1 ? r[i / 2].y : r[i / 2].x;
        a[j] = round_code(__fmul_rn(fabsf(mi), minv), noise[i] << 4 & 0xFFFF0u);
        if (mi < 0.0f) a[j] |= 128u;
        b[j] = max(round_code(__fmul_rn(ri, vinv), noise[i] >> 12 & 0xFFFF0u),
                   min(__float_as_uint(ri), 1u));  // ri > 0
      }
      mo[h] = mfine ? bytes4(a[0], a[1], a[2], a[3]) : 0u;
      vo[h] = vfine ? bytes4(b[0], b[1], b[2], b[3]) : 0u;
    }
    store_codes<kWay>(mo, t.m, e0, n, lane);
    store_codes<kWay>(vo, t.v, e0, n, lane);
  } else {
    store8<kWay>(m, t.m, e0, n, lane);
    store8<kWay>(v, t.v, e0, n, lane);
  }
  if constexpr (sizeof(W) == 2) {
    uint32_t out[4];
    uint32_t bits[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bits[i] = __float_as_uint(i & 1 ? w[i / 2].y : w[i / 2].x);
      const uint32_t up = mix(noise[i] + 0x9E3779B9u) & 0xFFFFu;
      if (wtop < kInf) {
        bits[i] += up;
      } else if (magnitude(__uint_as_float(bits[i])) > kInf) {
        bits[i] = 0x7FC00000u;  // a NaN stays one
      } else if ((bits[i] & kInf) != kInf) {
        bits[i] += up;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = __byte_perm(bits[2 * i], bits[2 * i + 1], 0x7632);
    store8_bf16<kWay>(out, static_cast<gg_bf16*>(t.w), e0, n, lane);
  } else {
    store8<kWay>(w, t.w, e0, n, lane);
    if (t.half != nullptr) {
      uint32_t out[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i] = pack_bf16x2(w[i].x, w[i].y);
      store8_bf16<kWay>(out, t.half, e0, n, lane);
    }
  }
}

template <int kCap, typename W, typename G, bool k8>
__global__ void __launch_bounds__(kThreads, 4)
adamw_kernel(const __grid_constant__ List<kCap> list, const __grid_constant__ StepParams p) {
  Shared k;
  k.gs = 1.0f;
  if (p.grad_scale != nullptr) {
    k.gs = *p.grad_scale;
    if ((__float_as_uint(k.gs) & kInf) == kInf) return;  // the step is skipped
  }
  const bool on_device = p.lr_dev != nullptr || p.step_dev != nullptr;
  __shared__ Factors shared;
  uint32_t run_key = p.run_key;
  k.b1 = p.b1, k.b2 = p.b2, k.ib1 = p.ib1, k.ib2 = p.ib2, k.c2 = p.c2, k.eps = p.eps;
  if (on_device) {
    const long long t = p.step_dev != nullptr ? *p.step_dev : p.step;
    if (t < 1) return;
    if (threadIdx.x == 0)
      shared = factors(p.lr_dev != nullptr ? static_cast<double>(*p.lr_dev) : p.lr, p.beta1,
                       p.beta2, t);
    __syncthreads();
    k.c2 = shared.c2;
    run_key = mix(p.seed_key + static_cast<uint32_t>(t));
  }
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  int at = 0;
  for (long long turn = blockIdx.x; turn < p.turns; turn += gridDim.x) {
    while (at + 1 < p.count && list.t[at + 1].first <= turn) ++at;
    const Entry& t = list.t[at];
    const long long cell = (turn - t.first) * kWarps + warp;
    const long long left = t.n - cell * kCell;
    if (left <= 0) continue;
    k.c1 = on_device ? c1_of(shared, t.lr_scale) : t.c1;
    k.kept = on_device ? kept_of(shared, t.lr_scale, t.decay) : t.kept;
    k.key = mix(mix(run_key + static_cast<uint32_t>(t.position)) + static_cast<uint32_t>(cell));
    const int n = static_cast<int>(min(static_cast<long long>(kCell), left));
    if (n < kCell)
      step_cell<kPartial, W, G, k8>(t, cell, n, lane, k);
    else if (t.wide)
      step_cell<kWide, W, G, k8>(t, cell, n, lane, k);
    else
      step_cell<kSingle, W, G, k8>(t, cell, n, lane, k);
  }
}

template <int kCap, typename W, typename G, bool k8>
cudaError_t launch_step_t(const List<kMany>& all, const StepParams& p, int sm_count,
                          cudaStream_t stream) {
  List<kCap> list;  // entries from p.count on are not read
  for (int i = 0; i < p.count; ++i) list.t[i] = all.t[i];
  const long long most = static_cast<long long>(sm_count) * 8;
  const unsigned grid = static_cast<unsigned>(p.turns < most ? p.turns : most);
  adamw_kernel<kCap, W, G, k8><<<grid, kThreads, 0, stream>>>(list, p);
  count_launch();
  return cudaGetLastError();
}

template <int kCap, typename W, typename G>
cudaError_t launch_step_b(const List<kMany>& all, const StepParams& p, bool k8, int sm_count,
                          cudaStream_t stream) {
  return k8 ? launch_step_t<kCap, W, G, true>(all, p, sm_count, stream)
            : launch_step_t<kCap, W, G, false>(all, p, sm_count, stream);
}

template <int kCap>
cudaError_t launch_step_w(const List<kMany>& all, const StepParams& p, bool w32, bool g32, bool k8,
                          int sm_count, cudaStream_t stream) {
  if (w32)
    return g32 ? launch_step_b<kCap, float, float>(all, p, k8, sm_count, stream)
               : launch_step_b<kCap, float, gg_bf16>(all, p, k8, sm_count, stream);
  return g32 ? launch_step_b<kCap, gg_bf16, float>(all, p, k8, sm_count, stream)
             : launch_step_b<kCap, gg_bf16, gg_bf16>(all, p, k8, sm_count, stream);
}

// ------------------------------------------------------------------- the norm

constexpr int kNormEach = 32;                    // elements per thread and turn
constexpr int kNormTurn = kThreads * kNormEach;  // and per block
constexpr int kNormList = 1024;                  // tensors in a launch's parameters
constexpr int kNormBlocks = 1024;                // most blocks of a launch

struct NormEntry {
  const void* g;
  long long n;
  long long first;  // turns before this tensor's; its lowest bit: unaligned
};

template <int kCap>
struct NormList {
  NormEntry t[kCap];
};

__device__ __forceinline__ void put_norm(double sum, float max_norm, float* out) {
  const double norm = sqrt(sum);
  const float n = static_cast<float>(norm);
  out[0] = n;
  float scale = 1.0f;
  if ((__float_as_uint(n) & kInf) == kInf)
    scale = __uint_as_float(0x7FC00000u);
  else if (max_norm > 0.0f)
    scale = static_cast<float>(fmin(1.0, static_cast<double>(max_norm) / (norm + 1e-6)));
  out[1] = scale;
}

// Sum of a block's values in a fixed order, in thread 0.
__device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[kWarps];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(kFull, x, d);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += part[i];
  return s;
}

template <typename T>
__device__ __forceinline__ float load1(const void* from, long long at) {
  if constexpr (sizeof(T) == 4)
    return static_cast<const float*>(from)[at];
  else
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(from)[at]) << 16);
}

// Squares are added in fp32, 32 at a time, and those sums in 64 bits. Bound by
// memory: 604 M BF16 elements in 172 us, 7.0 TB/s (200 M: 60 us, not 16-byte
// aligned 105; fp32 115 and 124); small lists by the two launches, 9 to 16 us from
// the host (60 odd tensors, 3 M elements: 9.5 us of it on the device). One launch of
// a cluster that adds everything up was no faster from the host and slower on the
// device.
template <int kCap, typename G>
__global__ void __launch_bounds__(kThreads)
norm_kernel(const __grid_constant__ NormList<kCap> list, int count, long long turns,
            double* partial, float max_norm, float* out) {
  grid_dependents_launch();
  constexpr int kVec = 16 / static_cast<int>(sizeof(G));
  constexpr int kLoads = kNormEach / kVec;
  double sum = 0.0;
  int at = 0;
  for (long long turn = blockIdx.x; turn < turns; turn += gridDim.x) {
    while (at + 1 < count && (list.t[at + 1].first >> 1) <= turn) ++at;
    const NormEntry& t = list.t[at];
    const long long e0 = (turn - (t.first >> 1)) * kNormTurn;
    float s = 0.0f;
    if ((t.first & 1) == 0 && e0 + kNormTurn <= t.n) {
      const uint4* from =
          reinterpret_cast<const uint4*>(static_cast<const G*>(t.g) + e0) + threadIdx.x;
      uint4 x[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) x[i] = __ldcs(from + i * kThreads);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (sizeof(G) == 4) {
            s = fmaf(__uint_as_float(u[j]), __uint_as_float(u[j]), s);
          } else {
            s = fmaf(bf16_lo(u[j]), bf16_lo(u[j]), s);
            s = fmaf(bf16_hi(u[j]), bf16_hi(u[j]), s);
          }
        }
      }
    } else {
      // a thread's elements, and their order, as above: the same sum wherever
      // the array starts
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const long long e = e0 + (i * kThreads + threadIdx.x) * kVec;
        float x[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) x[j] = e + j < t.n ? load1<G>(t.g, e + j) : 0.0f;
#pragma unroll
        for (int j = 0; j < kVec; ++j) s = fmaf(x[j], x[j], s);
      }
    }
    sum += s;
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) {
    if (out != nullptr)
      put_norm(sum, max_norm, out);
    else
      partial[blockIdx.x] = sum;
  }
}

__global__ void __launch_bounds__(kThreads)
norm_join_kernel(const double* partial, int count, float max_norm, float* out) {
  grid_dependency_wait();
  double sum = 0.0;
  for (int i = threadIdx.x; i < count; i += kThreads) sum += partial[i];
  sum = block_sum(sum);
  if (threadIdx.x == 0) put_norm(sum, max_norm, out);
}

template <int kCap, typename G>
cudaError_t launch_norm_t(const NormList<kNormList>& all, int count, long long turns, int grid,
                          double* partial, float max_norm, float* out, cudaStream_t stream) {
  NormList<kCap> list;  // entries from count on are not read
  for (int i = 0; i < count; ++i) list.t[i] = all.t[i];
  norm_kernel<kCap, G><<<grid, kThreads, 0, stream>>>(list, count, turns, partial, max_norm, out);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(const gg_adamw_tensor* tensors, int n, const gg_adamw_options& o,
                         const DeviceInfo& dev, cudaStream_t stream) {
  const bool w32 = o.w_dtype == GG_DTYPE_F32, g32 = o.g_dtype == GG_DTYPE_F32;
  const bool k8 = o.state_bits == 8;
  StepParams p{};
  const Factors f = factors(o.lr, o.beta1, o.beta2, o.step > 0 ? o.step : 1);
  p.b1 = static_cast<float>(o.beta1);
  p.b2 = static_cast<float>(o.beta2);
  p.ib1 = static_cast<float>(1.0 - o.beta1);
  p.ib2 = static_cast<float>(1.0 - o.beta2);
  p.c2 = f.c2;
  p.eps = static_cast<float>(o.eps);
  p.seed_key = mix(o.seed);
  p.run_key = mix(p.seed_key + static_cast<uint32_t>(o.step));
  p.grad_scale = o.grad_scale;
  p.lr_dev = o.lr_dev;
  p.step_dev = o.step_dev;
  p.lr = o.lr;
  p.beta1 = o.beta1;
  p.beta2 = o.beta2;
  p.step = o.step;
  List<kMany> list;
  int i = 0;
  while (i < n) {
    p.count = 0;
    p.turns = 0;
    for (; i < n && p.count < kMany; ++i) {
      const gg_adamw_tensor& t = tensors[i];
      if (t.n == 0) continue;
      Entry& e = list.t[p.count++];
      e.w = t.w;
      e.g = t.g;
      e.m = t.m;
      e.v = t.v;
      e.ms = t.m_scale;
      e.vs = t.v_scale;
      e.half = t.half;
      e.n = t.n;
      e.first = p.turns;
      e.lr_scale = t.lr_scale;
      e.decay = t.weight_decay;
      e.c1 = c1_of(f, t.lr_scale);
      e.kept = kept_of(f, t.lr_scale, t.weight_decay);
      e.position = i;
      const auto fits = [](const void* q, size_t bytes) {
        return (reinterpret_cast<uintptr_t>(q) & (4 * bytes - 1)) == 0;
      };
      e.wide = fits(t.w, w32 ? 4 : 2) && fits(t.g, g32 ? 4 : 2) && fits(t.m, k8 ? 1 : 4) &&
               fits(t.v, k8 ? 1 : 4) && fits(t.half, 2);
      const long long cells = (t.n + kCell - 1) / kCell;
      p.turns += (cells + kWarps - 1) / kWarps;
    }
    if (p.count == 0) break;
    const auto go = [&](auto launch) {
      return launch(list, p, w32, g32, k8, dev.sm_count, stream);
    };
    const cudaError_t e = p.count <= kFew    ? go(launch_step_w<kFew>)
                          : p.count <= kSome ? go(launch_step_w<kSome>)
                                             : go(launch_step_w<kMany>);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

size_t grad_norm_scratch(int n) {
  const size_t launches = (static_cast<size_t>(n) + kNormList - 1) / kNormList;
  return sizeof(double) * kNormBlocks * (launches < 1 ? 1 : launches);
}

cudaError_t launch_grad_norm(const gg_grad_tensor* tensors, int n, bool f32, float max_norm,
                             float* out, double* partial, const DeviceInfo& dev,
                             cudaStream_t stream) {
  NormList<kNormList> list;
  int i = 0, written = 0;
  bool done = false;
  const long long most = static_cast<long long>(dev.sm_count) * 6 < kNormBlocks
                             ? static_cast<long long>(dev.sm_count) * 6
                             : kNormBlocks;
  do {
    int count = 0;
    long long turns = 0;
    for (; i < n && count < kNormList; ++i) {
      if (tensors[i].n == 0) continue;
      NormEntry& e = list.t[count++];
      e.g = tensors[i].g;
      e.n = tensors[i].n;
      e.first = 2 * turns + ((reinterpret_cast<uintptr_t>(e.g) & 15u) != 0 ? 1 : 0);
      turns += (e.n + kNormTurn - 1) / kNormTurn;
    }
    const int grid = static_cast<int>(turns < 1 ? 1 : (turns < most ? turns : most));
    done = i == n && written == 0 && grid == 1;  // one block: it writes the result
    float* to = done ? out : nullptr;
    const auto go = [&](auto launch) {
      return launch(list, count, turns, grid, partial + written, max_norm, to, stream);
    };
    cudaError_t e;
    if (count <= kFew)
      e = f32 ? go(launch_norm_t<kFew, float>) : go(launch_norm_t<kFew, gg_bf16>);
    else if (count <= kSome)
      e = f32 ? go(launch_norm_t<kSome, float>) : go(launch_norm_t<kSome, gg_bf16>);
    else
      e = f32 ? go(launch_norm_t<kNormList, float>) : go(launch_norm_t<kNormList, gg_bf16>);
    if (e != cudaSuccess) return e;
    written += grid;
  } while (i < n);
  if (done) return cudaSuccess;
  const cudaError_t e = launch_early(norm_join_kernel, dim3(1), dim3(kThreads), 0, stream,
                                     static_cast<const double*>(partial), written, max_norm, out);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gg
