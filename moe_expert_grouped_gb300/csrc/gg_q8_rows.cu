// gg_q8_rows.cu — 8-bit grouped linear layers for few rows per expert (tokens
// being decoded), where reading the weights is all that costs:
//   C[r][n] = s_r * t_en * sum_c qa[r][c] * qb[e][n][c],
// gated activations fused, as gg_gemm_q8.cu computes for many rows.
//
// A tile is 32 rows of one live expert's weight (gated: 16 gate rows and the
// matching 16 up rows). One block of 16 warps per SM; two warps share a tile,
// each taking every other 128-code chunk of K, and go from tile to tile.
// Every warp has a ring of its own in shared memory that TMA fills with 32 x
// 128 weight codes and the 128 codes of up to eight tokens per stage, so
// 128 KB of weights per SM are always on their way, across tiles too; the
// first are asked for before the kernel waits for the quantiser that makes the
// token codes. Measured at 4 rows for each of 128 experts, 1536 x 2048 gated
// (403 MB): 70 us; with 8 warps and twice the stages 76; with four or eight
// warps to a tile 83 and 95; loading the weights into registers instead, 16
// loads of 16 bytes per lane ahead, 99.
//
// A lane reads 16 consecutive codes of four weight rows and of its token,
// widens them to FP16 (exact) and has the fragments of mma.m16n8k16: which k
// of a fragment a code stands for does not matter as long as both operands
// agree, so nothing is shuffled. The second warp's partial sums go through
// shared memory to the first, which writes the tile.
//
// Bound by HBM: at the measured copy rate 22 weight bytes per clock and SM
// arrive, which take 1.2 instructions per clock, of 4, to widen and multiply.

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "gg_internal.h"
#include "gg_launch.cuh"
#include "gg_ptx.cuh"
#include "gg_q8.cuh"

namespace gg {
namespace {

constexpr int kWarps = 16;
constexpr int kPairs = kWarps / 2;
constexpr int kThreads = 32 * kWarps;
constexpr int kTurns = kMaxExperts / 32;  // groups of 32 experts
static_assert(kTurns <= 32 && kMaxExperts % kThreads == 0, "one warp scans the groups");
constexpr int kRows = 32;    // weight rows per tile
constexpr int kChunk = 128;  // codes of K per stage
constexpr int kTokens = 8;   // tokens multiplied with each piece of weight
constexpr uint32_t kWeightBytes = kRows * kChunk;
constexpr int kStages = 2;   // of a warp's ring
constexpr uint32_t kStageBytes = kWeightBytes + kTokens * kChunk;
constexpr uint32_t kWarpBytes = kStages * kStageBytes;

struct SmemTail {
  uint64_t full[kWarps][kStages];
  int abort_flag;
  int bad;
  int n_live;
  int in_turn[kTurns];
  uint16_t live[kMaxExperts];  // experts that have rows
  float part[kPairs][2 * 4][32];  // the second warp's sums, as its lanes hold them
};

constexpr size_t kSmemBytes = 1024 + kWarps * kWarpBytes + sizeof(SmemTail);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

struct RowsParams {
  const float* As;
  const float* Bs;
  const int32_t* offsets;
  int E, R_cap, K, N, F;
  float alpha;
  const float* row_scale;
  gg_bf16* C;
  int32_t* status;
  int early;  // launched behind the quantiser, which may still run
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Where a warp is in its stages: tile, first token of the pass, chunk of K.
struct Cursor {
  int tile, first, chunk;
  int e, n0;       // the tile's expert and first weight row
  int row0, rows;  // the expert's rows
};

template <bool kGated>
__global__ void __launch_bounds__(kThreads, 1)
q8_rows_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
               const RowsParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  SmemTail& st = *reinterpret_cast<SmemTail*>(smem + kWarps * kWarpBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  // The live experts, in order: 32 experts per warp and turn, so that all
  // offsets are on their way at once.
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
  uint32_t live[kMaxExperts / kThreads];  // of the warp's turns: lanes with rows
#pragma unroll
  for (int i = 0; i < kMaxExperts / kThreads; ++i) {
    const int e = i * kThreads + threadIdx.x;
    const int o0 = e < p.E ? p.offsets[e] : 0;
    const int o1 = e < p.E ? p.offsets[e + 1] : 0;
    if (o1 < o0 || o0 < 0 || o1 > p.R_cap || (e == 0 && o0 != 0)) st.bad = 1;
    live[i] = __ballot_sync(0xFFFFFFFFu, o1 > o0);
    if (lane == 0) st.in_turn[i * kWarps + warp] = __popc(live[i]);
  }
  __syncthreads();
  {
    // experts of the turns before each of this warp's
    const int mine = lane < kTurns ? st.in_turn[lane] : 0;
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int n = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if (lane >= d) upto += n;
    }
#pragma unroll
    for (int i = 0; i < kMaxExperts / kThreads; ++i) {
      const int before = __shfl_sync(0xFFFFFFFFu, upto - mine, i * kWarps + warp);
      if (live[i] >> lane & 1u)
        st.live[before + __popc(live[i] & ((1u << lane) - 1u))] =
            static_cast<uint16_t>(i * kThreads + threadIdx.x);
    }
    const int all = __shfl_sync(0xFFFFFFFFu, upto, 31);
    if (threadIdx.x == 0) {
      st.n_live = st.bad ? 0 : all;
      if (st.bad && blockIdx.x == 0) set_status(p.status, GG_ERR_DEVICE_BAD_OFFSETS);
    }
  }
  __syncthreads();

  volatile int* abort_flag = &st.abort_flag;
  constexpr int kOut = kGated ? kRows / 2 : kRows;  // outputs per tile and token
  const int per = (kGated ? p.F : p.N) / kOut;      // tiles per expert
  const int total = st.n_live * per;
  const int chunks = (p.K + kChunk - 1) / kChunk;
  const int pair = warp >> 1, part_of = warp & 1;
  const int first_tile = pair * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
  const int tile_step = kPairs * static_cast<int>(gridDim.x);
  uint8_t* ring = smem + warp * kWarpBytes;
  const uint32_t ring_addr = raw_addr + pad + warp * kWarpBytes;

  const auto enter = [&](Cursor& c) {  // c.tile has changed
    if (c.tile >= total) return;
    const int a = c.tile / per;
    c.e = st.live[a];
    c.n0 = (c.tile - a * per) * kOut;
    c.row0 = p.offsets[c.e];
    c.rows = p.offsets[c.e + 1] - c.row0;
  };
  const auto advance = [&](Cursor& c) {
    c.chunk += 2;
    if (c.chunk < chunks) return;
    c.chunk = part_of;
    c.first += kTokens;
    if (c.first < c.rows) return;
    c.first = 0;
    c.tile += tile_step;
    enter(c);
  };
  const auto load_weights = [&](const Cursor& c, int s) {
    const uint32_t bar = smem_u32(&st.full[warp][s]);
    const uint32_t dst = ring_addr + s * kStageBytes;
    mbar_arrive_expect_tx(bar, kStageBytes);
    tma_load_3d(dst, &mapB, bar, c.chunk * kChunk, c.n0, c.e);
    if (kGated)
      tma_load_3d(dst + kWeightBytes / 2, &mapB, bar, c.chunk * kChunk, p.F + c.n0, c.e);
  };
  const auto load_tokens = [&](const Cursor& c, int s) {
    tma_load_2d(ring_addr + s * kStageBytes + kWeightBytes, &mapA, smem_u32(&st.full[warp][s]),
                c.chunk * kChunk, c.row0 + c.first);
  };

  Cursor at{first_tile, 0, part_of, 0, 0, 0, 0};  // of the stage consumed next
  enter(at);
  Cursor ahead = at;                    // of the stage loaded next
  uint32_t pending = 0;                 // stages with a load that was not waited for
  const bool works = part_of < chunks;  // K <= 128: the second warp has nothing
  if (works) {
    for (int s = 0; s < kStages && ahead.tile < total; ++s) {
      if (lane == 0) load_weights(ahead, s);
      pending |= 1u << s;
      advance(ahead);
    }
  }
  if (p.early) grid_dependency_wait();
  if (works && lane == 0) {
    Cursor c = at;
    for (int s = 0; s < kStages && c.tile < total; ++s) {
      load_tokens(c, s);
      advance(c);
    }
  }

  bool ok = true;
  int s = 0;
  uint32_t phase = 0;
  int failed = 0;
  uint32_t failed_phase = 0;
  for (; at.tile < total; at.tile += tile_step, enter(at)) {
    for (int first = 0; first < at.rows; first += kTokens) {
      float acc[2][4] = {};
      for (int chunk = part_of; chunk < chunks; chunk += 2) {
        if (ok) {
          ok = mbar_wait_bounded(smem_u32(&st.full[warp][s]), phase, abort_flag, p.status);
          if (ok)
            pending &= ~(1u << s);
          else
            failed = s, failed_phase = phase;
        }
        const uint8_t* stage = ring + s * kStageBytes;
        // 16-byte piece 2t + h of the swizzled 128-byte rows: the eight lanes
        // of an access, two neighbouring rows, then hit all banks
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t piece = ((2 * t + h) ^ g) << 4;
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = *reinterpret_cast<const uint4*>(stage + (8 * i + g) * kChunk + piece);
          const uint4 x =
              *reinterpret_cast<const uint4*>(stage + kWeightBytes + g * kChunk + piece);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint2 r0 = widen4((&w[0].x)[q]), r1 = widen4((&w[1].x)[q]);
            const uint2 r2 = widen4((&w[2].x)[q]), r3 = widen4((&w[3].x)[q]);
            const uint32_t a0[4] = {r0.x, r1.x, r0.y, r1.y};
            const uint32_t a1[4] = {r2.x, r3.x, r2.y, r3.y};
            const uint2 b = widen4((&x.x)[q]);
            mma_f16(acc[0], a0, b.x, b.y);
            mma_f16(acc[1], a1, b.x, b.y);
          }
        }
        __syncwarp();  // every lane has read the stage
        if (ok && ahead.tile < total) {
          if (lane == 0) {
            fence_proxy_async();
            load_weights(ahead, s);
            load_tokens(ahead, s);
          }
          pending |= 1u << s;
          advance(ahead);
        }
        if (++s == kStages) {
          s = 0;
          phase ^= 1u;
        }
      }
      // D fragment: rows g (values 0, 1) and g + 8 (2, 3), tokens 2t and 2t + 1
      float(*sums)[32] = st.part[pair];
      if (part_of == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[i][lane] = acc[i / 4][i % 4];
      }
      asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory");
      if (part_of == 0) {
        const int have = ok ? min(kTokens, at.rows - first) : 0;
        const long long width = kGated ? p.F : p.N;
        const float* bs = p.Bs + static_cast<long long>(at.e) * p.N + at.n0;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int tok = 2 * t + (v & 1), c = g + (v & 2 ? 8 : 0);
          if (tok >= have) continue;
          const int r = at.row0 + first + tok;
          const float sr = p.As[r];
          gg_bf16* out = p.C + r * width + at.n0 + c;
          // one scale after the other: their product alone may leave fp32's range.
          // The probability goes with the token's scale of the up half, as
          // gg_gemm_q8.cu has it: a row's bits are the same there.
          const float up = kGated && p.row_scale != nullptr ? sr * p.row_scale[r] : sr;
          const float lo = (acc[0][v] + sums[v][lane]) * __ldg(bs + c) * sr;
          const float hi =
              (acc[1][v] + sums[4 + v][lane]) * __ldg(bs + (kGated ? p.F : 16) + c) * up;
          if (kGated) {
            *out = __bfloat16_as_ushort(
                __float2bfloat16_rn(glu_mul(lo, hi, p.alpha, false, 1.0f)));
          } else {
            out[0] = __bfloat16_as_ushort(__float2bfloat16_rn(lo));
            out[16] = __bfloat16_as_ushort(__float2bfloat16_rn(hi));
          }
        }
      }
      asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory");  // the sums were read
    }
  }
  // after a wait that ran out: no load may still be on its way at the exit
  if (!ok)
    for (int i = 0; i < kStages; ++i)
      if (pending & (1u << i))
        (void)mbar_wait_bounded(smem_u32(&st.full[warp][i]),
                                i >= failed ? failed_phase : failed_phase ^ 1u, nullptr,
                                p.status);
}

template <bool kGated>
cudaError_t launch_rows_t(const CUtensorMap& ma, const CUtensorMap& mb, const RowsParams& p,
                          const DeviceInfo& dev, cudaStream_t stream) {
  static std::atomic<int> opted[kMaxDevices];
  if (opted[dev.device].load(std::memory_order_relaxed) == 0) {
    const cudaError_t o =
        cudaFuncSetAttribute(q8_rows_kernel<kGated>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes));
    if (o != cudaSuccess) return o;
    opted[dev.device].store(1, std::memory_order_relaxed);
  }
  const int experts = p.R_cap < p.E ? p.R_cap : p.E;  // that can have rows
  const long long tiles = static_cast<long long>(p.N / kRows) * experts;
  const dim3 grid(static_cast<unsigned>(tiles < dev.sm_count ? tiles : dev.sm_count));
  cudaError_t e = cudaSuccess;
  if (p.early)
    e = launch_early(q8_rows_kernel<kGated>, grid, dim3(kThreads), kSmemBytes, stream, ma, mb, p);
  else
    q8_rows_kernel<kGated><<<grid, kThreads, kSmemBytes, stream>>>(ma, mb, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// Up to four rows per expert that can have any. The offsets are on the device,
// so the rule cannot see a hot expert, whose rows take a pass over its weights
// for every eight, one after the other in each tile. us here : many-row kernel,
// rows dealt evenly, and by Zipf's law (1.2, at most an eighth to one expert):
//   rows per expert                     1                2               4
//   128 experts, 1536 x 2048 gated  72:92   39:49    72:92  57:57   72:92  98:78
//   128 experts, 2048 x 768         41:51   23:29    41:51  33:35   41:51  45:43
//   32 experts, 4096 x 4096 gated   90:111  49:68    90:111 72:96   91:111 92:109
// At eight rows, passes of 16 tokens took 77:92, 45:51 and 96:111, by Zipf's law
// 113:87, 63:49 and 120:111; at 16 rows 80:93 and 180:100 on the first.
bool q8_rows_fits(int R_cap, int E) {
  const int experts = R_cap < E ? R_cap : E;
  return R_cap <= 4 * experts;
}

cudaError_t launch_q8_rows(const Q8GemmArgs& a, bool early, const DeviceInfo& dev,
                           cudaStream_t stream) {
  const bool gated = a.alpha != 0.0f;
  CUtensorMap ma, mb;
  const cuuint64_t ad[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.R_cap)};
  const cuuint64_t as[1] = {static_cast<cuuint64_t>(a.K)};
  const cuuint32_t abox[2] = {kChunk, kTokens};
  const cuuint64_t bd[3] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.N),
                            static_cast<cuuint64_t>(a.E)};
  const cuuint64_t bs[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.K) * a.N};
  const cuuint32_t bbox[3] = {kChunk, gated ? kRows / 2u : static_cast<cuuint32_t>(kRows), 1};
  if (!encode_map(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.A, 2, ad, as, abox,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.B, 3, bd, bs, bbox,
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
  p.status = a.status;
  p.early = early ? 1 : 0;
  return gated ? launch_rows_t<true>(ma, mb, p, dev, stream)
               : launch_rows_t<false>(ma, mb, p, dev, stream);
}

}  // namespace gg
