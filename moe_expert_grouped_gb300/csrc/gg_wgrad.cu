// gg_wgrad.cu — the weight gradient of a grouped linear layer on sm_103a:
// dB[e] = dC_e^T A_e for every expert e in one persistent launch, the
// reduction running over the expert's own (ragged) rows.
//
// One CTA per SM in clusters of two (one tcgen05 MMA pair, 352 threads per
// CTA, warp-specialised):
//   warp 0      TMA producer: per 64-row step its CTA's 128 columns of dC and
//               its half (128 columns) of A, 64 x 64 boxes of BF16 with
//               128-byte swizzle. Both operands are used as they lie in
//               memory, rows outermost ("MN-major"): the reduction index is
//               the row, so neither tensor is transposed;
//   warp 1      allocates TMEM; in the even CTA one lane issues
//               tcgen05.mma.cta_group::2 (M = 256 columns of dC, N = 256
//               columns of A, K = 16 rows);
//   warps 2-9   epilogue: one TMEM lane = one row of dB;
//   warp 10     passes each landed step on to the MMA issuer and, at the last
//               step of an expert, first zeroes the rows behind the expert's
//               end in both operands: they are the next expert's, and even
//               multiplied by zero an infinity or NaN there would reach the
//               sum.
// Work items are (expert, 256 x 256 block of dB); an expert without rows gets
// zeros (or the base).
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

namespace gg {
namespace {

constexpr int BM = 128;            // rows of dB per CTA (columns of dC)
constexpr int BN = 256;            // columns of dB per work item (columns of A)
constexpr int BK = 64;             // rows of dC and A per step
constexpr int STAGES = 6;
constexpr uint16_t kPairMask = 0x3;
constexpr int kEpiWarps = 8;
constexpr int kPassWarp = 2 + kEpiWarps;
constexpr int kThreads = 32 * (kPassWarp + 1);
constexpr uint32_t BOX_BYTES = BK * 64 * 2;            // 64 rows x 64 columns
constexpr uint32_t A_BYTES = 2 * BOX_BYTES;            // this CTA's 128 columns of dC
constexpr uint32_t STAGE_BYTES = A_BYTES + 2 * BOX_BYTES;  // and its 128 columns of A
constexpr uint32_t TMEM_COLS = 512;

struct SmemTail {
  uint64_t full[STAGES];   // this CTA's loads have landed
  uint64_t ready[STAGES];  // even CTA: both CTAs passed the step on
  uint64_t empty[STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int total_tiles;
  int row_start[kMaxExperts + 1];
};

constexpr uint32_t kWarpStagingBytes = 32 * 64;
constexpr uint32_t kStagingBytes = kEpiWarps * kWarpStagingBytes;
constexpr size_t kSmemBytes = 1024 + STAGES * STAGE_BYTES + kStagingBytes + sizeof(SmemTail);
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

struct WParams {
  const int32_t* offsets;
  int E, R_cap;
  int N, K;      // dB is [E][N][K]
  int MT, NT;    // 256-row and 256-column blocks of one expert's dB
  const void* base;
  void* dB;
  int32_t* status;
};

// A work item: expert, block of its dB, rows of the expert.
struct Item {
  int e, mt, nt, row0, rows;
};

__device__ __forceinline__ Item item_of(int tile, const WParams& p, const int* row_start) {
  Item it;
  const int per = p.MT * p.NT;
  it.e = tile / per;
  const int local = tile - it.e * per;
  it.mt = local / p.NT;
  it.nt = local - it.mt * p.NT;
  it.row0 = row_start[it.e];
  it.rows = row_start[it.e + 1] - it.row0;
  return it;
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
wgrad_kernel(const __grid_constant__ CUtensorMap mapD, const __grid_constant__ CUtensorMap mapA,
             const WParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_addr + pad;
  SmemTail& st = *reinterpret_cast<SmemTail*>(smem + STAGES * STAGE_BYTES + kStagingBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const bool leader = crank == 0;

  if (warp == 0) {
    bool bad = false;
    for (int e = lane; e <= p.E; e += 32) {
      const int o = p.offsets[e];
      st.row_start[e] = o;
      if (e < p.E ? p.offsets[e + 1] < o : o > p.R_cap) bad = true;
      if (e == 0 && o != 0) bad = true;
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (lane == 0) {
      st.total_tiles = bad ? 0 : p.E * p.MT * p.NT;
      st.abort_flag = 0;
      if (bad && blockIdx.x == 0) set_status(p.status, GG_ERR_DEVICE_BAD_OFFSETS);
      for (int s = 0; s < STAGES; ++s) {
        mbar_init(smem_u32(&st.full[s]), 1);
        mbar_init(smem_u32(&st.ready[s]), 2);
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
      tma_prefetch_desc(&mapD);
      tma_prefetch_desc(&mapA);
      const int h = static_cast<int>(crank);
      int stage = 0;
      uint32_t phase = 0, used = 0, last_phase = 0;
      bool ok = true;
      for (int tile = first; tile < total && ok; tile += step) {
        const Item it = item_of(tile, p, st.row_start);
        const int n0 = it.mt * (2 * BM) + h * BM;
        const int k0 = it.nt * BN + h * (BN / 2);
        for (int r = 0; r < it.rows; r += BK) {
          if (!mbar_wait_bounded(smem_u32(&st.empty[stage]), phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_u32(&st.full[stage]);
          const uint32_t sa = sbase + stage * STAGE_BYTES;
          mbar_arrive_expect_tx(bar, STAGE_BYTES);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            tma_load_2d(sa + j * BOX_BYTES, &mapD, bar, n0 + 64 * j, it.row0 + r);
            tma_load_2d(sa + A_BYTES + j * BOX_BYTES, &mapA, bar, k0 + 64 * j, it.row0 + r);
          }
          used |= 1u << stage;
          last_phase = (last_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // the CTA may not exit before its loads have landed and been consumed
      for (int s = 0; s < STAGES; ++s)
        if (used & (1u << s)) {
          (void)mbar_wait_bounded(smem_u32(&st.full[s]), (last_phase >> s) & 1u, nullptr,
                                  p.status);
          (void)mbar_wait_bounded(smem_u32(&st.empty[s]), (last_phase >> s) & 1u, nullptr,
                                  p.status);
        }
    }
  } else if (warp == kPassWarp) {
    // ------------------------------------------------ pass on, zero the tail
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tile = first; tile < total && ok; tile += step) {
      const Item it = item_of(tile, p, st.row_start);
      for (int r = 0; r < it.rows; r += BK) {
        int landed = 0;
        if (lane == 0)
          landed = mbar_wait_bounded(smem_u32(&st.full[stage]), phase, abort_flag, p.status);
        landed = __shfl_sync(0xFFFFFFFFu, landed, 0);
        if (!landed) {
          ok = false;
          break;
        }
        const int held = it.rows - r;  // rows of this step that are the expert's
        if (held < BK && (held & 15) != 0) {
          (void)mbar_try_wait(smem_u32(&st.full[stage]), phase);  // every lane sees the data
          // the MMAs read rows up to the next multiple of 16; each row is 128
          // bytes in each of the four boxes (the swizzle stays inside a row)
          const int pieces = (16 - (held & 15)) * 8;
          uint8_t* box = smem + stage * STAGE_BYTES + held * 128;
          for (int i = lane; i < 4 * pieces; i += 32)
            *reinterpret_cast<uint4*>(box + (i / pieces) * BOX_BYTES + (i % pieces) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive_cluster_cta(mapa_shared(smem_u32(&st.ready[stage]), 0));
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ------------------------------------------------ MMA issuer (even CTA)
      constexpr uint32_t idesc = make_idesc_bf16(2 * BM, BN, true, true);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int tile = first; tile < total && ok; tile += step) {
        const Item it = item_of(tile, p, st.row_start);
        if (it.rows == 0) continue;
        if (!mbar_wait_bounded(smem_u32(&st.tempty[acc]), acc_phase ^ 1u, abort_flag, p.status))
          break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int r = 0; r < it.rows; r += BK) {
          if (!mbar_wait_bounded(smem_u32(&st.ready[stage]), phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = sbase + stage * STAGE_BYTES;
          const int groups = min(BK / 16, (it.rows - r + 15) / 16);
          for (int kk = 0; kk < groups; ++kk) {
            const uint64_t adesc = make_sdesc(sa + kk * 2048, BOX_BYTES, 1024);
            const uint64_t bdesc = make_sdesc(sa + A_BYTES + kk * 2048, BOX_BYTES, 1024);
            tc_mma_bf16_pair(d_tmem, adesc, bdesc, idesc, (r | kk) != 0 ? 1u : 0u);
          }
          tc_commit_pair_mc(smem_u32(&st.empty[stage]), kPairMask);
          if (++stage == STAGES) {
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
  } else {
    // ---------------------------------------------------------- epilogue
    // Warp w may only read TMEM lanes 32*(w%4) .. +31: two warps share each
    // lane quadrant and split the block's columns in halves.
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    int acc = 0;
    uint32_t acc_phase = 0;
    uint4* stg =
        reinterpret_cast<uint4*>(smem + STAGES * STAGE_BYTES + (warp - 2) * kWarpStagingBytes);
    for (int tile = first; tile < total; tile += step) {
      const Item it = item_of(tile, p, st.row_start);
      const int n0 = it.mt * (2 * BM) + static_cast<int>(crank) * BM + q * 32;
      const int k0 = it.nt * BN + half * (BN / 2);
      const int nvalid = max(0, min(32, p.N - n0));
      const int cols = max(0, min(BN / 2, p.K - k0));  // a multiple of 64
      const long long at = (static_cast<long long>(it.e) * p.N + n0) * p.K + k0;
      if (it.rows > 0) {
        if (!mbar_wait_bounded(smem_u32(&st.tfull[acc]), acc_phase, abort_flag, p.status)) break;
        tc_fence_after();
      }
      const uint32_t tbase =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * BN + half * (BN / 2);
#pragma unroll 1
      for (int c = 0; c < cols; c += 32) {
        float v[32];
        if (it.rows > 0) {
          tmem_ld32(tbase + c, v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.0f;
        }
        if (kF32) {
          float* out = static_cast<float*>(p.dB) + at + c;
          const float* base = static_cast<const float*>(p.base) + at + c;
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {  // 16 columns at a time through the staging buffer
#pragma unroll
            for (int g = 0; g < 4; ++g)
              stg[stage_slot(lane, g)] = make_uint4(
                  __float_as_uint(v[16 * hh + 4 * g]), __float_as_uint(v[16 * hh + 4 * g + 1]),
                  __float_as_uint(v[16 * hh + 4 * g + 2]), __float_as_uint(v[16 * hh + 4 * g + 3]));
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r = 8 * j + (lane >> 2);
              const int g = lane & 3;
              const uint4 w = stg[stage_slot(r, g)];
              float4 f = make_float4(__uint_as_float(w.x), __uint_as_float(w.y),
                                     __uint_as_float(w.z), __uint_as_float(w.w));
              if (r < nvalid) {
                const long long o = static_cast<long long>(r) * p.K + 16 * hh + 4 * g;
                if (p.base != nullptr) {
                  const float4 b = *reinterpret_cast<const float4*>(base + o);
                  f.x += b.x;
                  f.y += b.y;
                  f.z += b.z;
                  f.w += b.w;
                }
                *reinterpret_cast<float4*>(out + o) = f;
              }
            }
            __syncwarp();
          }
        } else {
          gg_bf16* out = static_cast<gg_bf16*>(p.dB) + at + c;
          uint4 w[4];
          if (p.base != nullptr) {
            uint4 raw[4];
            load_chunk_raw(raw, static_cast<const gg_bf16*>(p.base) + at + c, p.K, nvalid);
            transpose_chunk(stg, raw, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] += bf16_lo(u[j]);
                v[8 * i + 2 * j + 1] += bf16_hi(u[j]);
              }
            }
          }
          pack_bf16x32(v, 1.0f, w);
          store_chunk(stg, w, out, p.K, nvalid);
        }
      }
      if (it.rows > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&st.tempty[acc]), 0));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
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

template <bool kF32>
cudaError_t launch_wgrad_t(const CUtensorMap& md, const CUtensorMap& ma, const WParams& p,
                           const DeviceInfo& dev, cudaStream_t stream) {
  static std::atomic<int> resident[kMaxDevices];
  return launch_pairs(wgrad_kernel<kF32>, resident, kThreads, kSmemBytes, p.E * p.MT * p.NT, dev,
                      stream, md, ma, p);
}

}  // namespace

cudaError_t launch_wgrad(const WgradArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  CUtensorMap md, ma;
  const cuuint32_t box[2] = {64, BK};
  const cuuint64_t rows = static_cast<cuuint64_t>(a.R_cap > 0 ? a.R_cap : 1);
  const cuuint64_t dd[2] = {static_cast<cuuint64_t>(a.N), rows};
  const cuuint64_t ds[1] = {static_cast<cuuint64_t>(a.N) * 2};
  const cuuint64_t ad[2] = {static_cast<cuuint64_t>(a.K), rows};
  const cuuint64_t as[1] = {static_cast<cuuint64_t>(a.K) * 2};
  if (!encode_map(&md, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.dC, 2, dd, ds, box,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map(&ma, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.A, 2, ad, as, box,
                  CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  WParams p{};
  p.offsets = a.offsets;
  p.E = a.E;
  p.R_cap = a.R_cap;
  p.N = a.N;
  p.K = a.K;
  p.MT = (a.N + 2 * BM - 1) / (2 * BM);
  p.NT = (a.K + BN - 1) / BN;
  p.base = a.base;
  p.dB = a.dB;
  p.status = a.status;
  return a.f32 ? launch_wgrad_t<true>(md, ma, p, dev, stream)
               : launch_wgrad_t<false>(md, ma, p, dev, stream);
}

}  // namespace gg
