// gg_f8_rows.cu — the forward product of gg_gemm_f8.cu for few rows per expert
// (tokens being decoded), where reading the weights is all that costs:
//   C[r][n] = sum_b s[b][r] t[e][n / 128][b] sum_{k in block b} q[r][k] w[e][n][k],
// gated activations fused, in one launch: BF16 rows are quantised where they
// are used.
//
// A tile is 32 rows of a live expert's weight (gated: 16 gate rows and the
// matching 16 up rows) and up to eight of the expert's rows: a hot expert's
// tiles find its weights in L2, on other SMs at the same time (one after the
// other by the same warps, 256 rows of 128 experts by Zipf's law took 98 us
// where even ones took 67). One block of 16 warps per SM; kParts warps share a
// tile, each taking every kParts-th block of 128 codes. Every warp has a ring
// of its own in shared memory that TMA fills with 32 x 128 weight codes and
// the same columns of up to eight tokens per stage, so 128 KB of weights per SM
// are always on their way, across tiles too.
//
// A lane reads 16 consecutive codes of four weight rows at a time, and makes
// the codes of 32 columns of one token in registers, with the block's maximum
// from the other three lanes of the token. Both then have the fragments of
// mma.m16n8k32 on E4M3: which k of a fragment a code stands for does not matter
// as long as both operands agree. A block's sums are held to 2^-19 of their
// terms' magnitudes, as the tensor-memory path's are. Widening to FP16 for
// mma.m16n8k16 instead was bound by the conversions, 16 a clock and SM (512 rows
// of 128 experts, 2048 x 768: 44 us from codes, 38 as it is). The sums of a
// block are scaled and added up in fp32; the other parts' go through shared
// memory to the first, which adds them in order.

#include <cuda_runtime.h>

#include <atomic>

#include "gg_f8.cuh"
#include "gg_internal.h"
#include "gg_launch.cuh"
#include "gg_ptx.cuh"

namespace gg {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kTurns = kMaxExperts / 32;  // groups of 32 experts
static_assert(kTurns <= 32 && kMaxExperts % kThreads == 0, "one warp scans the groups");
constexpr int kRows = 32;          // weight rows per tile
constexpr int kChunk = kF8Block;   // codes of K per stage
constexpr int kTokens = 8;         // tokens multiplied with each piece of weight
constexpr int kMostRows = 4;       // rows per expert, on average, that this is for
constexpr int kMaxUnits = kMaxExperts + kMostRows * kMaxExperts / kTokens;
constexpr uint32_t kWeightBytes = kRows * kChunk;
constexpr int kStages = 2;         // of a warp's ring
constexpr uint32_t kStageBytes = kWeightBytes + kTokens * kChunk * 2;  // tokens in BF16 at most
constexpr uint32_t kWarpBytes = kStages * kStageBytes;

struct SmemTail {
  uint64_t full[kWarps][kStages];
  int abort_flag;
  int bad;
  int n_units;
  int in_turn[kTurns];
  uint32_t unit[kMaxUnits];    // an expert and, times 65536, eight of its rows
  float part[kWarps][8][32];   // sums of the parts but the first, as their lanes hold them
};

constexpr size_t kSmemBytes = 1024 + kWarps * kWarpBytes + sizeof(SmemTail);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
static_assert(kStageBytes % 1024 == 0, "128-byte swizzle");

struct RowsParams {
  const float* As;      // of codes: [ceil(K / 128)][R_cap]
  const float* Bs;
  const int32_t* offsets;
  int E, R_cap, K, N, F;
  float alpha;
  const float* row_scale;
  gg_bf16* C;
  gg_bf16* H1_save;
  int32_t* status;
};

// D (+)= A[16 x 32] * B[32 x 8], E4M3 operands, fp32 sums.
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t top_of(uint4 w) {  // largest |BF16|, as its bits
  const uint32_t a = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                              __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
  return max(a & 0xFFFFu, a >> 16);
}

// Where a warp is in its stages: tile, block of K.
struct Cursor {
  int tile, chunk;
  int e, n0;       // the tile's expert and first weight row
  int row0, rows;  // and rows
};

template <bool kGated, bool kBf16, int kParts>
__global__ void __launch_bounds__(kThreads, 1)
f8_rows_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
               const RowsParams p) {
  constexpr int kGroups = kWarps / kParts;  // tiles at a time
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  SmemTail& st = *reinterpret_cast<SmemTail*>(smem + kWarps * kWarpBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  // The units, in order of their experts: 32 experts per warp and turn, so that
  // all offsets are on their way at once.
  if (threadIdx.x == 0) {
    st.abort_flag = 0;
    st.bad = 0;
    tma_prefetch_desc(&mapA);
    tma_prefetch_desc(&mapB);
  }
  for (int i = threadIdx.x; i < kWarps * kStages; i += kThreads)
    mbar_init(smem_u32(&st.full[i / kStages][i % kStages]), 1);
  mbar_fence_init();
  fence_proxy_async();
  __syncthreads();
  int units[kMaxExperts / kThreads], upto[kMaxExperts / kThreads];  // of this thread's experts
#pragma unroll
  for (int i = 0; i < kMaxExperts / kThreads; ++i) {
    const int e = i * kThreads + threadIdx.x;
    const int o0 = e < p.E ? p.offsets[e] : 0;
    const int o1 = e < p.E ? p.offsets[e + 1] : 0;
    const bool bad = o1 < o0 || o0 < 0 || o1 > p.R_cap || (e == 0 && o0 != 0);
    if (bad) st.bad = 1;
    units[i] = bad ? 0 : (o1 - o0 + kTokens - 1) / kTokens;
    upto[i] = units[i];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int n = __shfl_up_sync(0xFFFFFFFFu, upto[i], d);
      if (lane >= d) upto[i] += n;
    }
    if (lane == 31) st.in_turn[i * kWarps + warp] = upto[i];
  }
  __syncthreads();
  {
    // units of the turns before each of this warp's
    const int mine = lane < kTurns ? st.in_turn[lane] : 0;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int n = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += n;
    }
    // valid offsets give R_cap / 8 and one for every expert at most
    const int all = st.bad ? 0 : __shfl_sync(0xFFFFFFFFu, sum, 31);
#pragma unroll
    for (int i = 0; i < kMaxExperts / kThreads; ++i) {
      const int before = __shfl_sync(0xFFFFFFFFu, sum - mine, i * kWarps + warp);
      for (int u = 0; u < units[i]; ++u) {
        const int to = before + upto[i] - units[i] + u;
        if (to < all && to < kMaxUnits)
          st.unit[to] = static_cast<uint32_t>(i * kThreads + threadIdx.x) |
                        static_cast<uint32_t>(u) << 16;
      }
    }
    if (threadIdx.x == 0) {
      st.n_units = all;
      if (st.bad && blockIdx.x == 0) set_status(p.status, GG_ERR_DEVICE_BAD_OFFSETS);
    }
  }
  __syncthreads();

  volatile int* abort_flag = &st.abort_flag;
  constexpr int kOut = kGated ? kRows / 2 : kRows;  // outputs per tile and token
  const int per = (kGated ? p.F : p.N) / kOut;      // tiles per unit
  const int total = st.n_units * per;
  const int chunks = (p.K + kChunk - 1) / kChunk;
  const int NB = (p.N + kF8Block - 1) / kF8Block;
  const int group = warp / kParts, part_of = warp % kParts;
  const int first_tile = group * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
  const int tile_step = kGroups * static_cast<int>(gridDim.x);
  uint8_t* ring = smem + warp * kWarpBytes;
  const uint32_t ring_addr = raw_addr + pad + warp * kWarpBytes;

  const auto enter = [&](Cursor& c) {  // c.tile has changed
    if (c.tile >= total) return;
    const int a = c.tile / per;
    const uint32_t unit = st.unit[a];
    const int first = static_cast<int>(unit >> 16) * kTokens;
    c.e = static_cast<int>(unit & 0xFFFFu);
    c.n0 = (c.tile - a * per) * kOut;
    c.row0 = p.offsets[c.e] + first;
    c.rows = min(kTokens, p.offsets[c.e + 1] - c.row0);
  };
  const auto advance = [&](Cursor& c) {
    c.chunk += kParts;
    if (c.chunk < chunks) return;
    c.chunk = part_of;
    c.tile += tile_step;
    enter(c);
  };
  constexpr uint32_t kTokenBytes = kTokens * kChunk * (kBf16 ? 2 : 1);
  const auto load = [&](const Cursor& c, int s) {
    const uint32_t bar = smem_u32(&st.full[warp][s]);
    const uint32_t dst = ring_addr + s * kStageBytes;
    const int k0 = c.chunk * kChunk;
    mbar_arrive_expect_tx(bar, kWeightBytes + kTokenBytes);
    tma_load_3d(dst, &mapB, bar, k0, c.n0, c.e);
    if (kGated) tma_load_3d(dst + kWeightBytes / 2, &mapB, bar, k0, p.F + c.n0, c.e);
    tma_load_2d(dst + kWeightBytes, &mapA, bar, k0, c.row0);
    if (kBf16)  // 128 bytes of a row at a time
      tma_load_2d(dst + kWeightBytes + kTokenBytes / 2, &mapA, bar, k0 + kChunk / 2,
                  c.row0);
  };
  // the weight's scales of a block: of the first and of the second 16 rows
  const auto load_scales = [&](const Cursor& c, float& t0, float& t1, float& ts) {
    if (c.tile >= total) return;
    if (!kBf16)  // of codes: token g's too
      ts = g < c.rows ? __ldg(p.As + static_cast<long long>(c.chunk) * p.R_cap + c.row0 + g)
                      : 0.0f;
    const float* b = p.Bs + (static_cast<long long>(c.e) * NB + c.n0 / kF8Block) * chunks + c.chunk;
    t0 = __ldg(b);
    t1 = kGated ? __ldg(p.Bs +
                        (static_cast<long long>(c.e) * NB + (p.F + c.n0) / kF8Block) * chunks +
                        c.chunk)
                : t0;
  };

  Cursor at{first_tile, part_of, 0, 0, 0, 0};  // of the stage consumed next
  enter(at);
  Cursor ahead = at;                    // of the stage loaded next
  uint32_t pending = 0;                 // stages with a load that was not waited for
  const bool works = part_of < chunks;  // short K: the later parts have nothing
  if (works) {
    for (int s = 0; s < kStages && ahead.tile < total; ++s) {
      if (lane == 0) load(ahead, s);
      pending |= 1u << s;
      advance(ahead);
    }
  }
  // scales one block ahead of their use
  Cursor next = at;
  float t0 = 0.0f, t1 = 0.0f, ts = 0.0f;
  if (works) {
    load_scales(next, t0, t1, ts);
    advance(next);
  }

  bool ok = true;
  int s = 0;
  uint32_t phase = 0;
  int failed = 0;
  uint32_t failed_phase = 0;
  for (; at.tile < total; at.tile += tile_step, enter(at)) {
    float sum[2][4] = {};
    for (int chunk = part_of; chunk < chunks; chunk += kParts) {
      const float w0 = t0, w1 = t1;
      float scale = ts;
      load_scales(next, t0, t1, ts);
      advance(next);
      if (ok) {
        ok = mbar_wait_bounded(smem_u32(&st.full[warp][s]), phase, abort_flag, p.status);
        if (ok)
          pending &= ~(1u << s);
        else
          failed = s, failed_phase = phase;
      }
      const uint8_t* stage = ring + s * kStageBytes;
      // codes of this lane's columns 32 t .. + 31 of token g
      uint32_t b[8];
      if constexpr (kBf16) {
        const uint8_t* row = stage + kWeightBytes + (t >> 1) * (kTokenBytes / 2) + g * 128;
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = *reinterpret_cast<const uint4*>(row + (((4 * (t & 1) + i) ^ g) << 4));
        uint32_t top = max(max(top_of(x[0]), top_of(x[1])), max(top_of(x[2]), top_of(x[3])));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        float inv;
        f8_scale(top << 16, inv, scale);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t lo = (&x[i / 2].x)[2 * (i % 2)], hi = (&x[i / 2].x)[2 * (i % 2) + 1];
          b[i] = f8_codes2(bf16_lo(lo), bf16_hi(lo), inv) |
                 f8_codes2(bf16_lo(hi), bf16_hi(hi), inv) << 16;
          if (inv == 0.0f) b[i] = 0u;  // a block with a NaN: its codes are 0
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 x = *reinterpret_cast<const uint4*>(stage + kWeightBytes + g * kChunk +
                                                          (((2 * t + h) ^ g) << 4));
          b[4 * h] = x.x, b[4 * h + 1] = x.y, b[4 * h + 2] = x.z, b[4 * h + 3] = x.w;
        }
      }
      float acc[2][4] = {};
      // 16-byte piece 2t + h of the swizzled 128-byte rows: the eight lanes
      // of an access, two neighbouring rows, then hit all banks
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t piece = ((2 * t + h) ^ g) << 4;
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = *reinterpret_cast<const uint4*>(stage + (8 * i + g) * kChunk + piece);
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          const auto word = [&](int i, int k) { return (&w[i].x)[k]; };
          const uint32_t b0 = b[4 * h + q], b1 = b[4 * h + q + 1];
          mma_e4m3(acc[0], word(0, q), word(1, q), word(0, q + 1), word(1, q + 1), b0, b1);
          mma_e4m3(acc[1], word(2, q), word(3, q), word(2, q + 1), word(3, q + 1), b0, b1);
        }
      }
      __syncwarp();  // every lane has read the stage
      if (ok && ahead.tile < total) {
        if (lane == 0) {
          fence_proxy_async();
          load(ahead, s);
        }
        pending |= 1u << s;
        advance(ahead);
      }
      if (++s == kStages) {
        s = 0;
        phase ^= 1u;
      }
      // D fragment: rows g (values 0, 1) and g + 8 (2, 3), tokens 2t and 2t + 1
      const float s0 = __shfl_sync(0xFFFFFFFFu, scale, 8 * t);
      const float s1 = __shfl_sync(0xFFFFFFFFu, scale, 8 * t + 4);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float f = v & 1 ? s1 : s0;
        sum[0][v] = fmaf(acc[0][v], f * w0, sum[0][v]);
        sum[1][v] = fmaf(acc[1][v], f * w1, sum[1][v]);
      }
    }
    if (part_of != 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) st.part[warp][i][lane] = sum[i / 4][i % 4];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * kParts) : "memory");
    if (part_of == 0) {
#pragma unroll
      for (int w = 1; w < kParts; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i / 4][i % 4] += st.part[warp + w][i][lane];
      const int have = ok ? at.rows : 0;
      const long long width = kGated ? p.F : p.N;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int tok = 2 * t + (v & 1), c = g + (v & 2 ? 8 : 0);
        if (tok >= have) continue;
        const long long r = static_cast<long long>(at.row0) + tok;
        gg_bf16* out = p.C + r * width + at.n0 + c;
        const float lo = sum[0][v], hi = sum[1][v];
        if (kGated) {
          const bool scaled = p.row_scale != nullptr;
          *out = __bfloat16_as_ushort(__float2bfloat16_rn(
              glu_mul(lo, hi, p.alpha, scaled, scaled ? p.row_scale[r] : 1.0f)));
          if (p.H1_save != nullptr) {
            gg_bf16* h1 = p.H1_save + r * p.N + at.n0 + c;
            h1[0] = __bfloat16_as_ushort(__float2bfloat16_rn(lo));
            h1[p.F] = __bfloat16_as_ushort(__float2bfloat16_rn(hi));
          }
        } else {
          out[0] = __bfloat16_as_ushort(__float2bfloat16_rn(lo));
          out[16] = __bfloat16_as_ushort(__float2bfloat16_rn(hi));
        }
      }
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * kParts) : "memory");
  }
  // after a wait that ran out: no load may still be on its way at the exit
  if (!ok)
    for (int i = 0; i < kStages; ++i)
      if (pending & (1u << i))
        (void)mbar_wait_bounded(smem_u32(&st.full[warp][i]),
                                i >= failed ? failed_phase : failed_phase ^ 1u, nullptr,
                                p.status);
}

template <bool kGated, bool kBf16, int kParts>
cudaError_t launch_rows_t(const CUtensorMap& ma, const CUtensorMap& mb, const RowsParams& p,
                          int grid, const DeviceInfo& dev, cudaStream_t stream) {
  static std::atomic<int> opted[kMaxDevices];
  if (opted[dev.device].load(std::memory_order_relaxed) == 0) {
    const cudaError_t o = cudaFuncSetAttribute(f8_rows_kernel<kGated, kBf16, kParts>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kSmemBytes));
    if (o != cudaSuccess) return o;
    opted[dev.device].store(1, std::memory_order_relaxed);
  }
  f8_rows_kernel<kGated, kBf16, kParts><<<grid, kThreads, kSmemBytes, stream>>>(ma, mb, p);
  count_launch();
  return cudaGetLastError();
}

template <bool kGated, bool kBf16>
cudaError_t launch_rows_p(const CUtensorMap& ma, const CUtensorMap& mb, const RowsParams& p,
                          const DeviceInfo& dev, cudaStream_t stream) {
  const int experts = p.R_cap < p.E ? p.R_cap : p.E;  // that can have rows
  // units at most; the parts go by the usual number, one for each expert
  const long long tiles = static_cast<long long>(p.N / kRows) * experts;
  const long long most = static_cast<long long>(p.N / kRows) * (experts + p.R_cap / kTokens);
  const int grid = static_cast<int>(most < dev.sm_count ? most : dev.sm_count);
  // as many warps to a tile as leave every tile its own
  const long long warps = static_cast<long long>(dev.sm_count) * kWarps;
  if (tiles * 8 <= warps) return launch_rows_t<kGated, kBf16, 8>(ma, mb, p, grid, dev, stream);
  if (tiles * 4 <= warps) return launch_rows_t<kGated, kBf16, 4>(ma, mb, p, grid, dev, stream);
  return launch_rows_t<kGated, kBf16, 2>(ma, mb, p, grid, dev, stream);
}

}  // namespace

// us here : quantiser and gg_gemm_f8.cu, rows dealt evenly, and by Zipf's law (1.2):
//   rows per expert                     1                2               4               8
//   128 experts, 1536 x 2048 gated  53:63   33:42    66:78   46:53   72:85   71:66  106:95  108:74
//   128 experts, 2048 x 768         29:37   19:25    35:45   25:28   40:49   39:39   54:53   56:45
//   32 experts, 4096 x 4096 gated   71:81   50:56    78:94   70:70   98:108  94:83  143:115 144:100
bool f8_rows_fits(int R_cap, int E) {
  const int experts = R_cap < E ? R_cap : E;
  return R_cap <= kMostRows * experts;
}

cudaError_t launch_f8_rows(const F8GemmArgs& a, const gg_bf16* x, const DeviceInfo& dev,
                           cudaStream_t stream) {
  const bool gated = a.alpha != 0.0f;
  CUtensorMap mb;
  const cuuint64_t bd[3] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.N),
                            static_cast<cuuint64_t>(a.E)};
  const cuuint64_t bs[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.K) * a.N};
  const cuuint32_t bbox[3] = {kChunk, gated ? kRows / 2u : static_cast<cuuint32_t>(kRows), 1};
  if (!encode_map(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.B, 3, bd, bs, bbox,
                  CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  CUtensorMap ma;
  const cuuint64_t ad[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.R_cap)};
  const cuuint64_t as[1] = {static_cast<cuuint64_t>(a.K) * (x != nullptr ? 2 : 1)};
  const cuuint32_t abox[2] = {x != nullptr ? kChunk / 2u : static_cast<cuuint32_t>(kChunk),
                              kTokens};
  if (!encode_map(&ma, x != nullptr ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                  x != nullptr ? static_cast<const void*>(x) : a.A, 2, ad, as, abox,
                  CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  RowsParams p{};
  p.As = a.As;
  p.Bs = a.Bs;
  p.offsets = a.offsets;
  p.E = a.E;
  p.R_cap = a.R_cap;
  p.K = a.K;
  p.N = a.N;
  p.F = a.N / 2;
  p.alpha = a.alpha;
  p.row_scale = a.row_scale;
  p.C = a.C;
  p.H1_save = a.H1_save;
  p.status = a.status;
  if (x != nullptr)
    return gated ? launch_rows_p<true, true>(ma, mb, p, dev, stream)
                 : launch_rows_p<false, true>(ma, mb, p, dev, stream);
  return gated ? launch_rows_p<true, false>(ma, mb, p, dev, stream)
               : launch_rows_p<false, false>(ma, mb, p, dev, stream);
}

}  // namespace gg
