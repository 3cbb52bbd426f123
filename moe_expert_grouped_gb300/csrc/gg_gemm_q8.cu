// gg_gemm_q8.cu — grouped linear layers on 8-bit integers with a scale per row
// of A (token) and per row of B (output channel), on sm_103a:
//   C[r][n] = s_r * t_en * sum_c qa[r][c] * qb[e][n][c]
// with the gated activations fused.
//
// This chip has no fast integer tensor path (its INT8 rate is far below the
// 16-bit floating-point one), and FP16 holds every 8-bit integer exactly. So
// the codes travel and lie in memory as 8 bits and are widened to FP16 on the
// SM, right before the FP16 tensor cores: products are exact, and fp32 sums of
// them are too below 2^24 (any K up to 1040; longer sums of larger magnitude
// round to fp32).
//
// The weights are the tensor core's A operand (M = 256 weight rows per pair
// of CTAs), the tokens its B operand (N = up to 256 tokens, in steps of 32):
// an expert's ragged token count then costs what it has, not a multiple of 256.
// Shared-memory bandwidth is what widening strains, so the widened weights go
// to tensor memory, which MMAs read as well (tcgen05.st, A in TMEM), and only
// the widened tokens to shared memory.
//
// Large products run at 0.9 of the rate the FP16 pipe reaches elsewhere: 65536
// rows, 4096 x 4096, one expert 1255 to 1300 us (1690 to 1750 TFLOP/s); 131072
// rows of 128 experts, 1536 x 2048 gated, 541 us (1523 TFLOP/s); 32768 rows of
// 32 experts, 4096 x 4096 gated, 615 us (1788 TFLOP/s). With blocks of up to
// 192 tokens these took 1397, 650 and 791: every block widens its weights anew;
// with the activation in the gate rows' warps alone the last two 592 and 660.
// Below about 128 rows per expert the weights bound it (4096 rows of those 128
// experts: 92 us, 4.5 TB/s), and the way of a step through its two widened
// places: widening, arrival at the issuer, MMAs, release.
//
// One CTA per SM in clusters of two (one tcgen05 MMA pair, 768 threads per
// CTA, warp-specialised):
//   warp 0       TMA producer: 128 weight rows (gated: 64 gate rows and the
//                matching 64 up rows) and half the tokens, 128 codes deep, into
//                a ring of raw steps (rows of 64 bytes cost TMA as much as
//                rows of 128 and held the kernel at 0.55 of the MMA rate);
//   warp 1       allocates TMEM; in the even CTA one lane issues
//                tcgen05.mma.cta_group::2 (M = 256, K = 16);
//   warp 2       finds the work items ahead of the others;
//   warps 4-11   widen the weights into TMEM, one thread per row;
//   warps 12-19  widen the tokens into shared memory (K-major, 128-byte
//                swizzle). Both in two groups, for the two halves of a step;
//   warps 20-23  epilogue: one TMEM lane = one weight row, one column = one
//                token. Gated: of every two chunks of 32 tokens the up rows'
//                warps hand the first one's values to the gate rows' warps and
//                get the gate values of the second, through shared memory.
// TMEM: 384 columns of sums, given to the items in turn, and two steps of
// weights (64 columns each). A step is 128 deep so that the issuer, whose loop
// costs it about 300 cycles, keeps ahead of the MMAs (256 tokens: 512 cycles
// per 64 codes). Work items are (expert, block of weight rows, block of
// tokens), the token block fastest, so that neighbours share their weights in
// L2.
//
// Every wait is bounded (gg_ptx.cuh); a wait that runs out records
// GG_ERR_DEVICE_TIMEOUT, raises a CTA-wide abort flag, and the CTA drains
// what is in flight, frees TMEM and exits after a final cluster barrier.

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <type_traits>

#include "gg_epilogue.cuh"
#include "gg_internal.h"
#include "gg_launch.cuh"
#include "gg_ptx.cuh"
#include "gg_q8.cuh"

namespace gg {
namespace {

constexpr int BM = 128;     // weight rows per CTA
constexpr int BN = 256;     // most tokens per work item
constexpr int BK = 64;      // half a step: what a group of widening warps takes
constexpr int RK = 128;     // codes of K per step
constexpr int RAW = 4;      // raw steps in flight
constexpr int WIDE = 2;     // widened steps
constexpr int UNITS = 6;    // TMEM for sums, in units of 64 columns
constexpr int kUnit = 64;
constexpr uint16_t kPairMask = 0x3;
constexpr int kItemWarp = 2;
constexpr int kFirstA = 4, kFirstB = 12, kFirstEpi = 20;  // first warps of the roles
constexpr int kGroups = 2;     // groups of widening warps, one for each half of a step:
constexpr int kAWarps = 4;     // warps of a group for the weights
constexpr int kBWarps = 4;     // and for the tokens, eight rows at a time each
constexpr int kFew = 2;        // turns of a token warp that have code of their own
constexpr int kEpiWarps = 4;
constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
constexpr int kItems = 4;      // work items found ahead
constexpr int kBoxes = 3;      // heights of token boxes: 64, 32 and 16 rows
constexpr uint32_t RAW_A = BM * RK;                  // 16 KB of weight codes
constexpr uint32_t RAW_BYTES = RAW_A + BN / 2 * RK;  // and up to 16 KB of token codes
constexpr uint32_t WIDE_HALF = BN / 2 * BK * 2;      // half a step's tokens as FP16
constexpr uint32_t WIDE_BYTES = 2 * WIDE_HALF;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t kTmemA = UNITS * kUnit;           // TMEM column of the first weight step
constexpr uint32_t kStepCols = RK / 2;               // two FP16 per column

// A work item: expert, block of weight rows, its tokens (first row, number;
// rows < 0: there are no more items). Its sums take `cols` columns of TMEM, a
// multiple of 32: `first` from column `col` on, and any others from column 0
// on, by MMAs of their own.
struct alignas(16) Item {
  int e, nt, row0, rows;
  int col, cols, first;
  int pad_;
};

struct SmemTail {
  Item item[kItems];
  uint64_t item_full[kItems];
  uint64_t item_empty[kItems];
  uint64_t raw_full[RAW];
  uint64_t raw_empty[RAW];
  uint64_t ready[WIDE];    // even CTA: both CTAs widened the step
  uint64_t empty[WIDE];
  uint64_t tfull[UNITS];   // of the item that starts in this unit
  uint64_t tempty[UNITS];
  // a chunk of values handed on, per pair of epilogue warps: to the gate rows'
  // warp, to the up rows' warp
  uint64_t hand_full[2][2];
  uint64_t hand_empty[2][2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int total_tiles;
  alignas(16) float scale[kEpiWarps][32];  // of the chunk's tokens, read as float4
  int tiles_before[kMaxExperts + 1];
  int row_start[kMaxExperts + 1];
};

constexpr uint32_t kWideAt = RAW * RAW_BYTES;
constexpr uint32_t kStagingAt = kWideAt + WIDE * WIDE_BYTES;
constexpr uint32_t kWarpStagingBytes = 32 * 64;
constexpr uint32_t kHandAt = kStagingAt + kEpiWarps * kWarpStagingBytes;
constexpr uint32_t kHandBytes = 32 * 32 * 4;         // a chunk of values, two per pair of warps
constexpr uint32_t kTailAt = kHandAt + 4 * kHandBytes;
constexpr size_t kSmemBytes = 1024 + kTailAt + sizeof(SmemTail);
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
static_assert(offsetof(SmemTail, scale) % 16 == 0 && kTailAt % 16 == 0, "float4 reads");
static_assert(kTmemA + WIDE * kStepCols <= TMEM_COLS, "tensor memory budget");
static_assert(kWideAt % 1024 == 0 && WIDE_BYTES % 1024 == 0, "128-byte swizzle");

struct QParams {
  const int32_t* offsets;
  int E, R_cap, K, N;
  int F;               // gated: N / 2
  int NT;              // blocks of weight rows
  const float* As;     // [R_cap]
  const float* Bs;     // [E][N]
  const float* row_scale;
  float alpha;
  gg_bf16* C;
  int32_t* status;
};

__device__ __forceinline__ int token_blocks(int rows) { return (rows + BN - 1) / BN; }

__device__ __forceinline__ Item item_of(int tile, const QParams& p, const SmemTail& st) {
  Item it;
  int lo = 0, hi = p.E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (st.tiles_before[mid] <= tile)
      lo = mid;
    else
      hi = mid;
  }
  it.e = lo;
  const int first = st.row_start[lo];
  const int rows = st.row_start[lo + 1] - first;
  const int blocks = token_blocks(rows);
  const int local = tile - st.tiles_before[lo];
  it.nt = local / blocks;
  const int tb = local - it.nt * blocks;
  const int each = ((rows + blocks - 1) / blocks + 31) / 32 * 32;  // as even as 32s allow
  it.row0 = first + tb * each;
  it.rows = min(each, rows - tb * each);  // each <= BN: no block is empty
  return it;
}

// The reader's side of the item ring (a whole warp or one thread; `arriver`
// reports the slot free, once per reader). False: no more items.
struct ItemReader {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ bool next(SmemTail& st, Item& it, bool warp, bool arriver,
                                       volatile int* abort_flag, int32_t* status) {
    if (!mbar_wait_bounded(smem_u32(&st.item_full[slot]), phase, abort_flag, status)) return false;
    it = st.item[slot];
    if (warp) __syncwarp();
    if (arriver) mbar_arrive(smem_u32(&st.item_empty[slot]));
    if (++slot == kItems) {
      slot = 0;
      phase ^= 1u;
    }
    return it.rows >= 0;
  }
};

// Gives the items their columns in turn. Up to 192 lie together (narrow MMAs
// cost what one of 128 columns does: two of 96 took 1.2 times as long as one
// of 192). More than that take four units from an even one on: two such items
// do not fit, so every third one goes over the end in two halves, and the next
// item's MMAs can start as the first units are read out.
struct Columns {
  int at = 0;  // unit
  __device__ __forceinline__ void give(Item& it) {
    it.cols = (it.rows + 31) & ~31;
    it.first = it.cols;
    const int units = (it.cols + kUnit - 1) / kUnit;
    if (units > UNITS / 2) {
      at = (at + 1) & ~1;
      if (at == UNITS) at = 0;
      it.first = min(it.cols, (UNITS - at) * kUnit);
    } else if (at + units > UNITS) {
      at = 0;
    }
    it.col = at * kUnit;
    at = (at + units) % UNITS;
  }
};

// FP16 operands (format fields 0), fp32 sums, M = 256, N = n; both K-major.
__device__ __forceinline__ uint32_t idesc_f16(int n) {
  return (1u << 4) | ((static_cast<uint32_t>(n) >> 3) << 17) |
         ((static_cast<uint32_t>(2 * BM) >> 4) << 24);
}

// D[tmem of both CTAs] (+)= A[256 x 16, tensor memory] * B[N x 16, N/2 rows per
// CTA, shared memory]^T.
__device__ __forceinline__ void tc_mma_f16_pair_ta(uint32_t d_tmem, uint32_t a_tmem,
                                                   uint64_t bdesc, uint32_t idesc,
                                                   uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Thread i of the warp writes 16 consecutive columns of lane (quadrant + i).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(taddr)
      : "memory");
}

struct TokenMaps {
  CUtensorMap box[kBoxes];
};

template <bool kGated>
__global__ void __launch_bounds__(kThreads, 1)
q8_gemm_kernel(const __grid_constant__ TokenMaps mapT, const __grid_constant__ CUtensorMap mapW,
               const QParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_addr + pad;
  SmemTail& st = *reinterpret_cast<SmemTail*>(smem + kTailAt);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int E = p.E;
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
        if (o1 < o0 || o0 < 0 || o1 > p.R_cap) bad = true;
        tiles = o1 > o0 ? token_blocks(o1 - o0) * p.NT : 0;
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
        mbar_init(smem_u32(&st.raw_empty[s]), kGroups * (kAWarps + kBWarps));
      }
      for (int s = 0; s < WIDE; ++s) {
        mbar_init(smem_u32(&st.ready[s]), 2 * kGroups * (kAWarps + kBWarps));
        mbar_init(smem_u32(&st.empty[s]), 1);
      }
      for (int a = 0; a < UNITS; ++a) {
        mbar_init(smem_u32(&st.tfull[a]), 1);
        mbar_init(smem_u32(&st.tempty[a]), 2 * kEpiWarps);
      }
      for (int a = 0; a < 2; ++a) {
        for (int d = 0; d < 2; ++d) {
          mbar_init(smem_u32(&st.hand_full[a][d]), 1);
          mbar_init(smem_u32(&st.hand_empty[a][d]), 1);
        }
      }
      for (int i = 0; i < kItems; ++i) {
        mbar_init(smem_u32(&st.item_full[i]), 1);
        // readers: producer, widening and epilogue warps, and the even CTA's issuer
        mbar_init(smem_u32(&st.item_empty[i]),
                  1 + kGroups * (kAWarps + kBWarps) + kEpiWarps + (leader ? 1 : 0));
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
      for (int i = 0; i < kBoxes; ++i) tma_prefetch_desc(&mapT.box[i]);
      tma_prefetch_desc(&mapW);
      const int h = static_cast<int>(crank);
      int stage = 0;
      uint32_t phase = 0, used = 0, last_phase = 0;
      bool ok = true;
      Item it;
      ItemReader items;
      while (ok && items.next(st, it, false, true, abort_flag, p.status)) {
        // two boxes of 64 weight rows: gated, gate rows and the matching up rows
        const int n0 = kGated ? it.nt * BM + h * (BM / 2) : it.nt * 2 * BM + h * BM;
        const int n1 = kGated ? p.F + n0 : n0 + BM / 2;
        // this CTA's half of the tokens of either MMA, multiples of 16
        const int half = it.cols / 2;
        const int half0 = it.first / 2;
        const int r0 = it.row0 + h * half0;
        const int r1 = it.row0 + half0 + h * (half - half0);  // of token half0 on
        for (int c = 0; c < p.K; c += RK) {
          if (!mbar_wait_bounded(smem_u32(&st.raw_empty[stage]), phase ^ 1u, abort_flag,
                                 p.status)) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_u32(&st.raw_full[stage]);
          const uint32_t sa = sbase + stage * RAW_BYTES;
          mbar_arrive_expect_tx(bar, RAW_A + half * RK);
          tma_load_3d(sa, &mapW, bar, c, n0, it.e);
          tma_load_3d(sa + RAW_A / 2, &mapW, bar, c, n1, it.e);
          // few boxes: 16 rows at a time, this thread held the others up
          const auto rows = [&](int i, int end, int from) {
            for (; i + 64 <= end; i += 64)
              tma_load_2d(sa + RAW_A + i * RK, &mapT.box[0], bar, c, from + i);
            if (i + 32 <= end) {
              tma_load_2d(sa + RAW_A + i * RK, &mapT.box[1], bar, c, from + i);
              i += 32;
            }
            if (i < end) tma_load_2d(sa + RAW_A + i * RK, &mapT.box[2], bar, c, from + i);
          };
          rows(0, half0, r0);
          if (half > half0) rows(half0, half, r1);
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
  } else if (warp == kItemWarp) {
    if (lane == 0) {
      // ------------------------------------------------------ work items
      int slot = 0;
      uint32_t phase = 0;
      Columns columns;
      for (int i = first;; i += step) {
        Item it{0, 0, 0, -1};
        if (i < total) {
          it = item_of(i, p, st);
          columns.give(it);
        }
        if (!mbar_wait_bounded(smem_u32(&st.item_empty[slot]), phase ^ 1u, abort_flag, p.status))
          break;
        st.item[slot] = it;
        mbar_arrive(smem_u32(&st.item_full[slot]));
        if (i >= total) break;
        if (++slot == kItems) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    if ((blockIdx.x & 1u) == 0) {
      // ------------------------------------------------ MMA issuer (even CTA)
      // The whole warp runs the loop and one lane issues: in a branch of one
      // lane the compiler moves every operand of every MMA to a uniform
      // register anew, 70 cycles an MMA. All of TMEM is ours, so it starts at
      // column 0.
      int stage = 0;
      uint32_t phase = 0;
      uint32_t unit_phase = 0;  // one bit per unit
      bool ok = tmem_base == 0;
      const uint64_t desc0 = make_sdesc(sbase + kWideAt, 16, 1024);
      Item it;
      ItemReader items;
      while (ok && items.next(st, it, true, lane == 0, abort_flag, p.status)) {
        // reductions, for their results are in uniform registers
        const int n = __reduce_max_sync(0xFFFFFFFFu, it.cols);
        const int n0 = __reduce_max_sync(0xFFFFFFFFu, it.first);
        const uint32_t d0 = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(it.col));
        const uint32_t idesc0 = idesc_f16(n0), idesc1 = idesc_f16(n - n0);
        const uint64_t second = (n0 / 2 * 128) >> 4;  // where the others' tokens begin
        for (int i = 0; i < n && ok; i += kUnit) {
          const int u = i < n0 ? d0 / kUnit + i / kUnit : (i - n0) / kUnit;
          ok = mbar_wait_bounded(smem_u32(&st.tempty[u]), (unit_phase >> u & 1u) ^ 1u, abort_flag,
                                 p.status);
          unit_phase ^= 1u << u;
        }
        if (!ok) break;
        tc_fence_after();
        for (int c = 0; c < p.K; c += RK) {
          if (!mbar_wait_bounded(smem_u32(&st.ready[stage]), phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t desc = desc0 + stage * (WIDE_BYTES >> 4);
          const uint32_t ta = kTmemA + stage * kStepCols;
          const auto half_step = [&](uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                     uint32_t more) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              tc_mma_f16_pair_ta(d, a + kk * 8, b + kk * 2, idesc, (more | kk) != 0 ? 1u : 0u);
          };
          if (n == n0) {
            if (elect_one()) {
              half_step(d0, ta, desc, idesc0, c);
              if (c + BK < p.K)
                half_step(d0, ta + BK / 2, desc + (WIDE_HALF >> 4), idesc0, 1u);
              tc_commit_pair_mc(smem_u32(&st.empty[stage]), kPairMask);
            }
          } else if (elect_one()) {
            half_step(d0, ta, desc, idesc0, c);
            half_step(0, ta, desc + second, idesc1, c);
            if (c + BK < p.K) {
              half_step(d0, ta + BK / 2, desc + (WIDE_HALF >> 4), idesc0, 1u);
              half_step(0, ta + BK / 2, desc + second + (WIDE_HALF >> 4), idesc1, 1u);
            }
            tc_commit_pair_mc(smem_u32(&st.empty[stage]), kPairMask);
          }
          __syncwarp();
          if (++stage == WIDE) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (elect_one()) tc_commit_pair_mc(smem_u32(&st.tfull[d0 / kUnit]), kPairMask);
        __syncwarp();
      }
      if (elect_one()) {
        tc_commit_pair(smem_u32(&st.mma_done));
        (void)mbar_wait_bounded(smem_u32(&st.mma_done), 0, nullptr, p.status);
      }
      __syncwarp();
    }
  } else if (warp >= kFirstA && warp < kFirstEpi) {
    // -------------------------------------------------------------- widen
    const bool weights = warp < kFirstB;
    const int q = warp & 3;
    const int group = weights ? (warp - kFirstA) / kAWarps : (warp - kFirstB) / kBWarps;
    // Raw rows are 128 bytes, their 16-byte pieces swizzled by TMA: eight lanes
    // that read the same piece of eight rows hit all banks. A weight lane takes
    // its row's four pieces of the group's half; a token warp widens eight rows
    // at a time, a lane one piece of 16 codes into two swizzled 16-byte pieces,
    // kBWarps * 8 rows further every turn. All offsets are set here: the loop
    // is bound by its instructions.
    const int row = weights ? q * 32 + lane
                            : (warp - kFirstB - group * kBWarps) * 8 + (lane & 7);
    const int piece = weights ? 0 : lane >> 3;
    const uint8_t* from = smem + (weights ? 0 : RAW_A) + row * RK +
                          (((4 * group + piece) ^ (row & 7)) << 4);
    const uint32_t flip = reinterpret_cast<uintptr_t>(from) & 0x70u;  // piece i is at ^ i << 4
    uint8_t* to = smem + kWideAt + group * WIDE_HALF + row * 128;
    const uint32_t to0 = ((2 * piece) ^ (row & 7)) << 4, to1 = ((2 * piece + 1) ^ (row & 7)) << 4;
    const uint32_t ta0 = tmem_base + kTmemA + (static_cast<uint32_t>(q * 32) << 16) +
                         group * (BK / 2);
    const uint32_t bars = smem_u32(&st.raw_full[0]);
    const uint32_t empty_raw = smem_u32(&st.raw_empty[0]);
    const uint32_t empty_bar = smem_u32(&st.empty[0]);
    const uint32_t ready_bar = mapa_shared(smem_u32(&st.ready[0]), 0);
    int rs = 0, ws = 0;
    uint32_t rp = 0, wp = 0, used = 0, last_phase = 0;
    bool ok = true;
    Item it;
    ItemReader items;
    while (ok && items.next(st, it, true, lane == 0, abort_flag, p.status)) {
      // of a token warp: turns of eight rows, 8 kBWarps rows apart
      const int turns =
          (it.cols / 2 - 8 * ((warp - kFirstB) % kBWarps) + 8 * kBWarps - 1) / (8 * kBWarps);
      for (int k0 = 0; k0 < p.K; k0 += RK) {
        // K an odd multiple of 64: the last step has one half
        const bool there = k0 + group * BK < p.K;
        if (!mbar_wait_bounded(bars + 8 * rs, rp, abort_flag, p.status)) {
          ok = false;
          break;
        }
        const uint8_t* raw = from + rs * RAW_BYTES;
        if (weights) {
          uint4 c[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            c[i] = *reinterpret_cast<const uint4*>(raw - flip + (flip ^ (i << 4)));
          __syncwarp();
          if (lane == 0) mbar_arrive(empty_raw + 8 * rs);
          uint32_t w[2][16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint2 f = widen4((&c[i / 4].x)[i % 4]);
            w[i / 8][2 * (i % 8)] = f.x;
            w[i / 8][2 * (i % 8) + 1] = f.y;
          }
          if (!mbar_wait_bounded(empty_bar + 8 * ws, wp ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (there) {
#pragma unroll
            for (int h = 0; h < 2; ++h) tmem_st16(ta0 + ws * kStepCols + 16 * h, w[h]);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tc_fence_before();
        } else {
          // the codes are read ahead of the wait for the place they go to
          const auto tokens = [&](auto most) {
            constexpr int kTurns = decltype(most)::value;
            uint4 c[kTurns];
#pragma unroll
            for (int j = 0; j < kTurns; ++j)
              if (j < turns) c[j] = *reinterpret_cast<const uint4*>(raw + j * 8 * kBWarps * RK);
            __syncwarp();
            if (lane == 0) mbar_arrive(empty_raw + 8 * rs);
            if (!mbar_wait_bounded(empty_bar + 8 * ws, wp ^ 1u, abort_flag, p.status))
              return false;
            if (!there) return true;
            uint8_t* wide = to + ws * WIDE_BYTES;
#pragma unroll
            for (int j = 0; j < kTurns; ++j)
              if (j < turns) {
                uint8_t* line = wide + j * 8 * kBWarps * 128;
                const uint2 a = widen4(c[j].x), b = widen4(c[j].y);
                const uint2 d = widen4(c[j].z), e = widen4(c[j].w);
                *reinterpret_cast<uint4*>(line + to0) = make_uint4(a.x, a.y, b.x, b.y);
                *reinterpret_cast<uint4*>(line + to1) = make_uint4(d.x, d.y, e.x, e.y);
              }
            return true;
          };
          // few turns have code of their own: masked ones are not free (4096 rows
          // of 128 experts: 99 us with the one code, 91)
          constexpr int kMost = BN / 2 / (8 * kBWarps);
          ok = turns <= kFew ? tokens(std::integral_constant<int, kFew>())
                             : tokens(std::integral_constant<int, kMost>());
          if (!ok) break;
          fence_proxy_async();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_cta(ready_bar + 8 * ws);
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
    // the pair's MMAs read both CTAs' memory: wait for the last ones
    if (lane == 0)
      for (int s = 0; s < WIDE; ++s)
        if (used & (1u << s))
          (void)mbar_wait_bounded(smem_u32(&st.empty[s]), (last_phase >> s) & 1u, nullptr,
                                  p.status);
  } else if (warp >= kFirstEpi) {
    // ---------------------------------------------------------- epilogue
    // One warp per lane quadrant, 32 tokens at a time. Gated: quadrants 0 and 1
    // are gate rows, 2 and 3 the matching up rows.
    const int q = warp & 3;
    const int w = warp - kFirstEpi;
    const bool up = kGated && q >= 2;
    constexpr int kChunks = kGated ? 2 : 1;  // a turn's
    const int pair = q & 1;
    const int width = kGated ? p.F : p.N;
    uint4* stg = reinterpret_cast<uint4*>(smem + kStagingAt + w * kWarpStagingBytes);
    // what this warp hands on, and what it is handed
    float* given = reinterpret_cast<float*>(smem + kHandAt + (2 * pair + up) * kHandBytes);
    const float* taken =
        reinterpret_cast<const float*>(smem + kHandAt + (2 * pair + !up) * kHandBytes);
    uint32_t unit_phase = 0;  // one bit per unit
    uint32_t give_phase = 0, take_phase = 0;
    bool ok = true;
    Item it;
    ItemReader items;
    while (ok && items.next(st, it, true, lane == 0, abort_flag, p.status)) {
      const int n0 = kGated ? it.nt * BM + static_cast<int>(crank) * (BM / 2) + (q & 1) * 32
                            : it.nt * 2 * BM + static_cast<int>(crank) * BM + q * 32;
      const bool exists = n0 < width;  // 32 channels exist together: widths are multiples of 64
      const float tn =
          exists ? __ldg(p.Bs + static_cast<long long>(it.e) * p.N + (up ? p.F : 0) + n0 + lane)
                 : 0.0f;
      const float2 tn2 = make_float2(tn, tn);
      // the tokens' scales, lane by lane for every chunk, ahead of the sums
      float sc[BN / 32];
#pragma unroll
      for (int i = 0; i < BN / 32; ++i) {
        const int r = 32 * i + lane;
        sc[i] = r < it.rows ? p.As[it.row0 + r] : 0.0f;
        if (up && p.row_scale != nullptr && r < it.rows) sc[i] *= p.row_scale[it.row0 + r];
      }
      const int start = it.col / kUnit;
      if (!mbar_wait_bounded(smem_u32(&st.tfull[start]), unit_phase >> start & 1u, abort_flag,
                             p.status))
        break;
      unit_phase ^= 1u << start;
      tc_fence_after();
      const uint32_t lanes = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      const auto column = [&](int c) { return c < it.first ? it.col + c : c - it.first; };
      // a chunk's scaled sums; scale: of the lane's token; done: with it the
      // unit's sums are in registers
      const auto load = [&](int c, float scale, bool done, float(&v)[32]) {
        st.scale[w][lane] = scale;
        tmem_ld32(lanes + column(c), v);
        if (done) tc_fence_before();
        __syncwarp();
        if (done && lane == 0)
          mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&st.tempty[column(c) / kUnit]), 0));
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&st.scale[w][i]);
          // one scale after the other: their product alone may leave fp32's range
          const float2 a = __fmul2_rn(__fmul2_rn(make_float2(v[i], v[i + 1]), tn2),
                                      make_float2(f.x, f.y));
          const float2 b = __fmul2_rn(__fmul2_rn(make_float2(v[i + 2], v[i + 3]), tn2),
                                      make_float2(f.z, f.w));
          v[i] = a.x;
          v[i + 1] = a.y;
          v[i + 2] = b.x;
          v[i + 3] = b.y;
        }
      };
      // [token][channel] through the staging buffer: four lanes then write each
      // token's 64-byte segment
      const auto store = [&](int c, const float(&v)[32]) {
        const int have = min(32, it.rows - c);
        const long long r0 = static_cast<long long>(it.row0) + c;
        uint16_t* cell = reinterpret_cast<uint16_t*>(stg);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          cell[stage_slot(i, lane >> 3) * 8 + (lane & 7)] =
              __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 8 * j + (lane >> 2);
          const uint4 x = stg[stage_slot(i, lane & 3)];
          if (exists && i < have)
            reinterpret_cast<uint4*>(p.C + (r0 + i) * width + n0)[lane & 3] = x;
        }
        __syncwarp();
      };
#pragma unroll 1
      for (int c = 0; c < it.rows; c += 32 * kChunks) {
        const bool second = c + 32 < it.rows;
        float v[32];
        if constexpr (kGated) {
          const bool keep = !up || second;
          if (up || second) {
            load(up ? c : c + 32, up ? sc[0] : sc[1], !keep, v);
            if (!mbar_wait_bounded(smem_u32(&st.hand_empty[pair][up]), give_phase ^ 1u, abort_flag,
                                   p.status)) {
              ok = false;
              break;
            }
            give_phase ^= 1u;
#pragma unroll
            for (int i = 0; i < 32; ++i) given[i * 32 + lane] = v[i];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&st.hand_full[pair][up]));
          }
          if (keep) {
            const int at = up ? c + 32 : c;
            load(at, up ? sc[1] : sc[0], true, v);
            if (!mbar_wait_bounded(smem_u32(&st.hand_full[pair][!up]), take_phase, abort_flag,
                                   p.status)) {
              ok = false;
              break;
            }
            take_phase ^= 1u;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float other = taken[i * 32 + lane];
              v[i] = glu_mul(up ? other : v[i], up ? v[i] : other, p.alpha, false, 1.0f);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&st.hand_empty[pair][!up]));
            store(at, v);
          }
        } else {
          load(c, sc[0], (c & 32) != 0 || !second, v);
          store(c, v);
        }
#pragma unroll
        for (int i = 0; i + kChunks < BN / 32; ++i) sc[i] = sc[i + kChunks];
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

template <bool kGated>
cudaError_t launch_q8_gemm_t(const TokenMaps& mt, const CUtensorMap& mw, const QParams& p,
                             const DeviceInfo& dev, cudaStream_t stream) {
  static std::atomic<int> resident[kMaxDevices];
  // no more clusters than there can be work items
  const long long items =
      (static_cast<long long>(p.R_cap) / BN + (p.R_cap < p.E ? p.R_cap : p.E)) * p.NT;
  const int most = static_cast<int>(items < 1 ? 1 : (items < 0x7FFFFFFF ? items : 0x7FFFFFFF));
  return launch_pairs(q8_gemm_kernel<kGated>, resident, kThreads, kSmemBytes, most, dev, stream,
                      mt, mw, p);
}

}  // namespace

cudaError_t launch_q8_gemm(const Q8GemmArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  TokenMaps mt;
  CUtensorMap mw;
  const cuuint64_t td[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.R_cap)};
  const cuuint64_t ts[1] = {static_cast<cuuint64_t>(a.K)};
  const cuuint64_t wd[3] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.N),
                            static_cast<cuuint64_t>(a.E)};
  const cuuint64_t ws[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.K) * a.N};
  const cuuint32_t wbox[3] = {RK, BM / 2, 1};
  for (int i = 0; i < kBoxes; ++i) {
    const cuuint32_t tbox[2] = {RK, 64u >> i};
    if (!encode_map(&mt.box[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, a.A, 2, td, ts, tbox,
                    CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  if (!encode_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.B, 3, wd, ws, wbox,
                  CU_TENSOR_MAP_SWIZZLE_128B))
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
  p.alpha = a.alpha;
  p.C = a.C;
  p.status = a.status;
  if (a.alpha != 0.0f) {
    p.NT = (p.F + BM - 1) / BM;
    return launch_q8_gemm_t<true>(mt, mw, p, dev, stream);
  }
  p.NT = (a.N + 2 * BM - 1) / (2 * BM);
  return launch_q8_gemm_t<false>(mt, mw, p, dev, stream);
}

}  // namespace gg
