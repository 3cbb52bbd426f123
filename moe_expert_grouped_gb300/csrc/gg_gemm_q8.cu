// gg_gemm_q8.cu — grouped linear layers on 8-bit integers with a scale per row
// of A (token) and per row of B (output channel), on sm_103a:
//   C[r][n] = s_r * t_en * sum_c qa[r][c] * qb[e][n][c]
// with the gated activations fused.
//
// This chip has no fast integer tensor path (its INT8 rate is far below the
// 16-bit floating-point one), and FP16 holds every 8-bit integer exactly. So
// the codes travel and lie in memory as 8 bits and are widened to FP16 in
// shared memory, right before the FP16 tensor cores: products are exact, and
// fp32 sums of them are too below 2^24 (any K up to 1040; longer sums of
// larger magnitude round to fp32).
//
// One CTA per SM in clusters of two (one tcgen05 MMA pair, 448 threads per
// CTA, warp-specialised):
//   warp 0       TMA producer: 128 rows x 64 codes of A and of B per step into
//                a ring of raw steps (16 KB each);
//   warp 1       allocates TMEM; in the even CTA one lane issues
//                tcgen05.mma.cta_group::2 (M = 256, N = 256, K = 16);
//   warps 2-5    epilogue: one TMEM lane = one row of C;
//   warps 6-13   widen: raw step -> FP16 step (32 KB, K-major with the
//                128-byte swizzle the descriptors name), passed to the even
//                CTA's MMA issuer.
// Work items are (expert, 256-row pair of row blocks, 256-column block; gated:
// 128 gate and the matching 128 up columns) as in the BF16 grouped GEMM; rows
// past an expert's end are computed from whatever codes lie there (any 8 bits
// are a finite integer) and not stored.
//
// Every wait is bounded (gg_ptx.cuh); a wait that runs out records
// GG_ERR_DEVICE_TIMEOUT, raises a CTA-wide abort flag, and the CTA drains
// what is in flight, frees TMEM and exits after a final cluster barrier.

#include <cuda_runtime.h>

#include <atomic>

#include "gg_epilogue.cuh"
#include "gg_internal.h"
#include "gg_launch.cuh"
#include "gg_ptx.cuh"
#include "gg_q8.cuh"

namespace gg {
namespace {

constexpr int BM = 128;
constexpr int BN = 256;
constexpr int BK = 64;
constexpr int RAW = 4;     // raw steps in flight
constexpr int WIDE = 4;    // widened steps
constexpr uint16_t kPairMask = 0x3;
constexpr int kEpiWarps = 4;
constexpr int kWideWarps = 8;
constexpr int kFirstWide = 2 + kEpiWarps;
constexpr int kThreads = 32 * (kFirstWide + kWideWarps);
constexpr uint32_t RAW_HALF = BM * BK;              // 8 KB: 128 rows of codes
constexpr uint32_t RAW_BYTES = 2 * RAW_HALF;        // A rows, B rows
constexpr uint32_t WIDE_HALF = 2 * RAW_HALF;        // the same as FP16
constexpr uint32_t WIDE_BYTES = 2 * WIDE_HALF;
constexpr uint32_t TMEM_COLS = 512;

struct SmemTail {
  uint64_t raw_full[RAW];
  uint64_t raw_empty[RAW];
  uint64_t ready[WIDE];    // even CTA: both CTAs widened the step
  uint64_t empty[WIDE];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int total_tiles;
  int tiles_before[kMaxExperts + 1];
  int row_start[kMaxExperts + 1];
};

constexpr uint32_t kWarpStagingBytes = 32 * 64;
constexpr uint32_t kStagingBytes = kEpiWarps * kWarpStagingBytes;
constexpr uint32_t kWideAt = RAW * RAW_BYTES;
constexpr uint32_t kStagingAt = kWideAt + WIDE * WIDE_BYTES;
constexpr size_t kSmemBytes = 1024 + kStagingAt + kStagingBytes + sizeof(SmemTail);
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

struct QParams {
  const int32_t* offsets;
  int E, R_cap, K, N;
  int F;               // gated: N / 2
  int NT;
  const float* As;     // [R_cap]
  const float* Bs;     // [E][N]
  const float* row_scale;
  gg_bf16* C;
  int32_t* status;
};

// FP16 operands, fp32 sums: format fields 0.
constexpr uint32_t kIdesc = (1u << 4) | ((static_cast<uint32_t>(BN) >> 3) << 17) |
                            ((static_cast<uint32_t>(2 * BM) >> 4) << 24);

template <bool kGated>
__global__ void __launch_bounds__(kThreads, 1)
q8_gemm_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
               const QParams p, const float alpha) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_addr + pad;
  SmemTail& st = *reinterpret_cast<SmemTail*>(smem + kStagingAt + kStagingBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int E = p.E;
  const int NT = p.NT;
  const int KB = p.K / BK;
  const uint32_t crank = cluster_ctarank();
  const bool leader = crank == 0;

  if (warp == 0) {
    bool bad = false;
    int carry = 0;
    for (int base = 0; base < E; base += 32) {
      const int e = base + lane;
      int tiles = 0;
      if (e < E) {
        const int o0 = p.offsets[e];
        const int o1 = p.offsets[e + 1];
        if (o1 < o0) bad = true;
        tiles = o1 > o0 ? (o1 - o0 + 2 * BM - 1) / (2 * BM) * NT : 0;
        st.row_start[e] = o0;
      }
      int incl = tiles;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int n = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += n;
      }
      if (e < E) st.tiles_before[e] = carry + incl - tiles;
      carry += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (lane == 0) {
      const int o_last = p.offsets[E];
      if (p.offsets[0] != 0 || o_last > p.R_cap || o_last < 0) bad = true;
      st.row_start[E] = o_last;
      st.tiles_before[E] = carry;
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (lane == 0) {
      st.total_tiles = bad ? 0 : carry;
      st.abort_flag = 0;
      if (bad && blockIdx.x == 0) set_status(p.status, GG_ERR_DEVICE_BAD_OFFSETS);
      for (int s = 0; s < RAW; ++s) {
        mbar_init(smem_u32(&st.raw_full[s]), 1);
        mbar_init(smem_u32(&st.raw_empty[s]), kWideWarps);
      }
      for (int s = 0; s < WIDE; ++s) {
        mbar_init(smem_u32(&st.ready[s]), 2 * kWideWarps);
        mbar_init(smem_u32(&st.empty[s]), 1);
      }
      for (int a = 0; a < 2; ++a) {
        mbar_init(smem_u32(&st.tfull[a]), 1);
        mbar_init(smem_u32(&st.tempty[a]), 2 * kEpiWarps);
      }
      mbar_init(smem_u32(&st.mma_done), 1);
      mbar_fence_init();
      fence_proxy_async();
    }
  } else if (warp == 1) {
    tmem_alloc_pair(smem_u32(&st.tmem_base), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // both CTAs' barriers exist before anything can arrive on them

  const int first = static_cast<int>(blockIdx.x) / 2;
  const int step = static_cast<int>(gridDim.x) / 2;
  const uint32_t tmem_base = st.tmem_base;
  const int total = st.total_tiles;
  volatile int* abort_flag = &st.abort_flag;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------- TMA producer
      tma_prefetch_desc(&mapA);
      tma_prefetch_desc(&mapB);
      const int h = static_cast<int>(crank);
      int stage = 0;
      uint32_t phase = 0, used = 0, last_phase = 0;
      bool ok = true;
      for (int tile = first; tile < total && ok; tile += step) {
        int e, mp, nt;
        decode_tile(tile, st.tiles_before, E, NT, e, mp, nt);
        const int row0 = st.row_start[e] + (2 * mp + h) * BM;
        // half 0 of a gated block: gate rows, half 1: the matching up rows
        const int n0 = kGated ? h * p.F + nt * (BN / 2) : nt * BN + h * (BN / 2);
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait_bounded(smem_u32(&st.raw_empty[stage]), phase ^ 1u, abort_flag,
                                 p.status)) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_u32(&st.raw_full[stage]);
          const uint32_t sa = sbase + stage * RAW_BYTES;
          mbar_arrive_expect_tx(bar, RAW_BYTES);
          tma_load_2d(sa, &mapA, bar, kb * BK, row0);
          tma_load_3d(sa + RAW_HALF, &mapB, bar, kb * BK, n0, e);
          used |= 1u << stage;
          last_phase = (last_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == RAW) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // the CTA may not exit before its loads have landed
      for (int s = 0; s < RAW; ++s)
        if (used & (1u << s))
          (void)mbar_wait_bounded(smem_u32(&st.raw_full[s]), (last_phase >> s) & 1u, nullptr,
                                  p.status);
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ------------------------------------------------ MMA issuer (even CTA)
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int tile = first; tile < total && ok; tile += step) {
        if (!mbar_wait_bounded(smem_u32(&st.tempty[acc]), acc_phase ^ 1u, abort_flag, p.status))
          break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait_bounded(smem_u32(&st.ready[stage]), phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = sbase + kWideAt + stage * WIDE_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            tc_mma_bf16_pair(d_tmem, make_sdesc(sa + kk * 32, 16, 1024),
                             make_sdesc(sa + WIDE_HALF + kk * 32, 16, 1024), kIdesc,
                             (kb | kk) != 0 ? 1u : 0u);
          tc_commit_pair_mc(smem_u32(&st.empty[stage]), kPairMask);
          if (++stage == WIDE) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit_pair_mc(smem_u32(&st.tfull[acc]), kPairMask);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      tc_commit_pair(smem_u32(&st.mma_done));
      (void)mbar_wait_bounded(smem_u32(&st.mma_done), 0, nullptr, p.status);
    }
  } else if (warp >= kFirstWide) {
    // -------------------------------------------------------------- widen
    // 1024 pieces of 16 codes per step, A rows then B rows, four per row: a
    // warp reads 512 consecutive bytes and writes two swizzled 16-byte
    // pieces per lane, both free of bank conflicts.
    const int t = threadIdx.x - 32 * kFirstWide;
    int rs = 0, ws = 0;
    uint32_t rp = 0, wp = 0, used = 0, last_phase = 0;
    bool ok = true;
    for (int tile = first; tile < total && ok; tile += step) {
      for (int kb = 0; kb < KB; ++kb) {
        if (!mbar_wait_bounded(smem_u32(&st.raw_full[rs]), rp, abort_flag, p.status) ||
            !mbar_wait_bounded(smem_u32(&st.empty[ws]), wp ^ 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        const uint4* raw = reinterpret_cast<const uint4*>(smem + rs * RAW_BYTES);
        uint8_t* wide = smem + kWideAt + ws * WIDE_BYTES;
#pragma unroll
        for (int j = 0; j < 1024 / (32 * kWideWarps); ++j) {
          const int i = t + j * 32 * kWideWarps;
          const uint4 q = raw[i];
          const int row = i >> 2;  // 0..255: A rows, then B rows
          uint8_t* line = wide + row * 128;
          const uint2 a = widen4(q.x), b = widen4(q.y), c = widen4(q.z), d = widen4(q.w);
          const int piece = (i & 3) * 2;
          *reinterpret_cast<uint4*>(line + ((piece ^ (row & 7)) << 4)) =
              make_uint4(a.x, a.y, b.x, b.y);
          *reinterpret_cast<uint4*>(line + (((piece + 1) ^ (row & 7)) << 4)) =
              make_uint4(c.x, c.y, d.x, d.y);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&st.raw_empty[rs]));
          mbar_arrive_cluster_cta(mapa_shared(smem_u32(&st.ready[ws]), 0));
        }
        used |= 1u << ws;
        last_phase = (last_phase & ~(1u << ws)) | (wp << ws);
        if (++rs == RAW) {
          rs = 0;
          rp ^= 1u;
        }
        if (++ws == WIDE) {
          ws = 0;
          wp ^= 1u;
        }
      }
    }
    // the pair's MMAs read both CTAs' shared memory: wait for the last ones
    if (lane == 0)
      for (int s = 0; s < WIDE; ++s)
        if (used & (1u << s))
          (void)mbar_wait_bounded(smem_u32(&st.empty[s]), (last_phase >> s) & 1u, nullptr,
                                  p.status);
  } else {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    const int r = q * 32 + lane;
    int acc = 0;
    uint32_t acc_phase = 0;
    uint4* stg = reinterpret_cast<uint4*>(smem + kStagingAt + (warp - 2) * kWarpStagingBytes);
    for (int tile = first; tile < total; tile += step) {
      int e, mp, nt;
      decode_tile(tile, st.tiles_before, E, NT, e, mp, nt);
      const long long grow =
          static_cast<long long>(st.row_start[e]) + (2 * mp + static_cast<int>(crank)) * BM + r;
      const long long row_end = st.row_start[e + 1];
      const long long grow0 = grow - lane;
      const int nvalid = static_cast<int>(max(0LL, min(32LL, row_end - grow0)));
      const float sr = grow < row_end ? p.As[grow] : 0.0f;
      const float pr = kGated && p.row_scale != nullptr && grow < row_end ? p.row_scale[grow]
                                                                          : 1.0f;
      const int width = kGated ? p.F : p.N;
      const int n0 = nt * (kGated ? BN / 2 : BN);
      constexpr int kCols = (kGated ? BN / 2 : BN) / (kEpiWarps / 4);  // of the block's, per warp
      const int c0 = half * kCols;
      const float* bs = p.Bs + static_cast<long long>(e) * p.N + n0;
      gg_bf16* crow0 = p.C + grow0 * width + n0;
      if (!mbar_wait_bounded(smem_u32(&st.tfull[acc]), acc_phase, abort_flag, p.status)) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * BN;
#pragma unroll 1
      for (int c = c0; c < c0 + kCols; c += 32) {
        if (n0 + c >= width) break;
        float v[32];
        tmem_ld32(tbase + c, v);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 s = __ldg(reinterpret_cast<const float4*>(bs + c + i));
          v[i] *= sr * s.x;
          v[i + 1] *= sr * s.y;
          v[i + 2] *= sr * s.z;
          v[i + 3] *= sr * s.w;
        }
        if (kGated) {
          float u[32];
          tmem_ld32(tbase + BN / 2 + c, u);
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 s = __ldg(reinterpret_cast<const float4*>(bs + p.F + c + i));
            v[i] = glu_mul(v[i], u[i] * (sr * s.x), alpha, true, pr);
            v[i + 1] = glu_mul(v[i + 1], u[i + 1] * (sr * s.y), alpha, true, pr);
            v[i + 2] = glu_mul(v[i + 2], u[i + 2] * (sr * s.z), alpha, true, pr);
            v[i + 3] = glu_mul(v[i + 3], u[i + 3] * (sr * s.w), alpha, true, pr);
          }
        }
        uint4 w[4];
        pack_bf16x32(v, 1.0f, w);
        store_chunk(stg, w, crow0 + c, width, nvalid);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&st.tempty[acc]), 0));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
  cluster_sync();
}

template <bool kGated>
cudaError_t launch_q8_gemm_t(const CUtensorMap& ma, const CUtensorMap& mb, const QParams& p,
                             float alpha, const DeviceInfo& dev, cudaStream_t stream) {
  static std::atomic<int> resident[kMaxDevices];
  // no more clusters than there can be work items
  const long long items =
      (static_cast<long long>(p.R_cap) / (2 * BM) + (p.R_cap < p.E ? p.R_cap : p.E)) * p.NT;
  const int most = static_cast<int>(items < 1 ? 1 : (items < 0x7FFFFFFF ? items : 0x7FFFFFFF));
  return launch_pairs(q8_gemm_kernel<kGated>, resident, kThreads, kSmemBytes, most, dev, stream,
                      ma, mb, p, alpha);
}

}  // namespace

cudaError_t launch_q8_gemm(const Q8GemmArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  CUtensorMap ma, mb;
  const cuuint64_t ad[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.R_cap)};
  const cuuint64_t as[1] = {static_cast<cuuint64_t>(a.K)};
  const cuuint32_t abox[2] = {BK, BM};
  const cuuint64_t bd[3] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.N),
                            static_cast<cuuint64_t>(a.E)};
  const cuuint64_t bs[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.K) * a.N};
  const cuuint32_t bbox[3] = {BK, BN / 2, 1};
  if (!encode_map(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.A, 2, ad, as, abox,
                  CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !encode_map(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.B, 3, bd, bs, bbox,
                  CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  QParams p{};
  p.offsets = a.offsets;
  p.E = a.E;
  p.R_cap = a.R_cap;
  p.K = a.K;
  p.N = a.N;
  p.F = a.N / 2;
  p.As = a.As;
  p.Bs = a.Bs;
  p.row_scale = a.row_scale;
  p.C = a.C;
  p.status = a.status;
  if (a.alpha != 0.0f) {
    p.NT = (p.F + BN / 2 - 1) / (BN / 2);
    return launch_q8_gemm_t<true>(ma, mb, p, a.alpha, dev, stream);
  }
  p.NT = (a.N + BN - 1) / BN;
  return launch_q8_gemm_t<false>(ma, mb, p, 1.0f, dev, stream);
}

}  // namespace gg
