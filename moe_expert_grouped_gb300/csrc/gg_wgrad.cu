// gg_wgrad.cu — the weight gradient of a grouped linear layer on sm_103a:
// dB[e] = dC_e^T A_e for every expert e in one persistent launch, the
// reduction running over the expert's own (ragged) rows.
//
// One CTA per SM in clusters of two (one tcgen05 MMA pair, 384 threads
// per CTA, warp-specialised):
//   warp 0      TMA producer: per 64-row step its CTA's 128 columns of dC and
//               its half of up to 256 columns of A, 64 x 64 boxes of BF16
//               with 128-byte swizzle. Both operands are used as they lie in
//               memory, rows outermost ("MN-major"): the reduction index is
//               the row, so neither tensor is transposed;
//   warp 1      allocates TMEM; in the even CTA one lane issues
//               tcgen05.mma.cta_group::2 (M = 256 columns of dC, N = up to
//               256 columns of A, K = 16 rows);
//   warp 2      passes each landed step on to the MMA issuer and, at the last
//               step of an expert, first zeroes the rows behind the expert's
//               end in both operands: they are the next expert's, and even
//               multiplied by zero an infinity or NaN there would reach the
//               sum;
//   warp 3      finds the work items (a search and divisions) ahead of the
//               others and hands them on through a ring: found by the MMA
//               issuer itself, each item cost it 1.5 us of idle tensor core;
//   the others  epilogue (8 warps): one TMEM lane = one row of dB.
//
// Work items are (expert, slice of its rows, block of dB), expert-major with
// the block fastest: the blocks that share rows run side by side and find
// them in L2. Every expert has the same number of blocks, so where there are
// few of them, or rows pile up in one expert, whole blocks would leave
// clusters idle. Then the rows of an expert are cut into slices whose fp32
// partial blocks go to the workspace, and a second kernel adds them in slice
// order (the slice length is chosen at the kernel's start; results depend on
// the offsets and sizes alone). 60000 rows, 768 x 320 fp32: one expert 46 us,
// whole blocks 229; 4 experts 46 and 70; 8 experts, whole blocks, 46, slices 51.
//
// The tensor core truncates each of its additions, by up to 2^-23 of the
// running sum and always towards zero, so a sum over 7500 rows (469 additions)
// is 8e-6 off. fp32 results are therefore carried in fp32 registers every
// kChunk steps (256 rows, 16 additions: 3e-7 off), which the epilogue warps do
// while the next chunk runs. BF16 results, rounded by up to 2^-9 in the end,
// are carried every kChunkBf16 steps (8192 rows, 512 additions: at most 2^-14;
// 131072 rows of one sign left in TMEM were 3e-4 low on average).
//
// An fp32 base is loaded by TMA into shared memory, piece by piece ahead of
// the sums: held in registers it spilled, and the loads then waited for each
// other (2048 x 768 over 128 experts, 32768 rows: 587 us, as it is 320).
//
// Bound by the tensor pipe where experts have rows enough: 131072 rows, 4096 x
// 4096, one expert 1840 TFLOP/s; 128 experts, 1536 x 2048 482 us (1710), 2048 x
// 768 255 us. fp32 results over few rows are bound by memory: 32768 rows of 128
// experts, 2048 x 768 with a base 320 us (5.6 TB/s), without one 216.
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
constexpr int BN = 256;            // most columns of dB per work item (columns of A)
constexpr int BK = 64;             // rows of dC and A per step
constexpr int kChunk = 4;          // fp32 results: steps summed inside TMEM
constexpr int kChunkBf16 = 128;    // and BF16 results
constexpr int kMaxStages = 6;
constexpr uint16_t kPairMask = 0x3;
constexpr int kItems = 4;          // work items found ahead
constexpr int kPassWarp = 2;
constexpr int kItemWarp = 3;
constexpr int kFirstEpi = 4;       // first epilogue warp
constexpr int kEpiWarps = 8;
constexpr int kCols = BN / (kEpiWarps / 4);  // columns of a block per epilogue warp
constexpr int kBaseBufs = 2;       // fp32 base: pieces per epilogue warp
constexpr uint32_t kPieceBytes = 32 * 32 * 4;
constexpr uint32_t BOX_BYTES = BK * 64 * 2;            // 64 rows x 64 columns
constexpr uint32_t A_BYTES = 2 * BOX_BYTES;            // this CTA's 128 columns of dC
constexpr uint32_t STAGE_BYTES = A_BYTES + 2 * BOX_BYTES;  // and up to 128 columns of A
constexpr uint32_t TMEM_COLS = 512;
constexpr long long kSlotFloats = 2LL * BM * BN;       // one partial block, [256][256]

// Numbers of slices tried for the expert with the most rows, and the fewest
// steps a slice may have.
constexpr int kTried = 11;
__constant__ const int kSlices[kTried] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 40, 76};
constexpr int kMinSlice = 8;
// What a partial block costs, in steps: writing 256 KB per pair and reading it
// back take about as long as 10 steps of MMAs. The second kernel takes 24.
constexpr int kPartialCost = 10;
constexpr int kJoinCost = 24;

// A work item: block (row block mt, column block nt) of expert e's dB over a
// slice of its rows; slot: its partial block, -1 for the whole sum. rows < 0:
// there are no more items.
struct alignas(16) Item {
  int e, mt, nt;
  int row0, rows;
  int slot;
  int pad_[2];
};

struct SmemTail {
  Item item[kItems];
  uint64_t item_full[kItems];
  uint64_t item_empty[kItems];
  uint64_t full[kMaxStages];   // this CTA's loads have landed
  uint64_t ready[kMaxStages];  // even CTA: both CTAs passed the step on
  uint64_t empty[kMaxStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t base_full[kEpiWarps][kBaseBufs];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int total_items;
  int most_steps;
  int slice;                          // most steps of a slice
  float cost[kTried];
  int row_start[kMaxExperts + 1];
  int items_before[kMaxExperts + 1];  // work items of earlier experts
  int slots_before[kMaxExperts + 1];  // partial blocks of earlier experts
};

constexpr uint32_t kWarpStagingBytes = 32 * 64;

// The layout of a CTA. An fp32 base comes through shared memory, two pieces of
// 32 rows x 32 columns per epilogue warp, and takes the place of two stages.
template <bool kBase32>
struct Layout {
  static constexpr int kStages = kBase32 ? 4 : kMaxStages;
  static constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
  static constexpr uint32_t kBaseAt = kStages * STAGE_BYTES;
  static constexpr uint32_t kStagingAt =
      kBaseAt + (kBase32 ? kEpiWarps * kBaseBufs * kPieceBytes : 0);
  static constexpr uint32_t kTailAt = kStagingAt + kEpiWarps * kWarpStagingBytes;
  static constexpr size_t kSmemBytes = 1024 + kTailAt + sizeof(SmemTail);
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

struct WParams {
  const int32_t* offsets;
  int E, R_cap;
  int N, K;       // dB is [E][N][K]
  int MT, NT;     // row and column blocks of one expert's dB
  int width;      // columns of a block (the last may be narrower)
  int min_cost;   // steps that writing a block takes at least
  int clusters;
  int slots;      // partial blocks the workspace holds; 0: no slices
  const void* base;
  void* dB;
  float* partial;
  int* plan;      // device word: the slice length that was chosen, 0 where nothing was cut
  int32_t* status;
};

__device__ __forceinline__ int steps_of(int rows) { return (rows + BK - 1) / BK; }

__device__ __forceinline__ int slices_of(int steps, int slice) {
  return steps > slice ? (steps + slice - 1) / slice : 1;
}

// Warp-collective: items_before and slots_before for slices of at most `slice`
// steps.
__device__ void fill_tables(const int* row_start, int E, int per, int slice, int* items_before,
                            int* slots_before) {
  const int lane = threadIdx.x & 31;
  int items = 0, slots = 0;
  for (int b = 0; b < E; b += 32) {
    const int e = b + lane;
    const int n =
        e < E ? per * slices_of(steps_of(row_start[e + 1] - row_start[e]), slice) : 0;
    const int m = n > per ? n : 0;
    int ni = n, mi = m;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, ni, d);
      const int y = __shfl_up_sync(0xFFFFFFFFu, mi, d);
      if (lane >= d) {
        ni += x;
        mi += y;
      }
    }
    if (e < E) {
      items_before[e] = items + ni - n;
      slots_before[e] = slots + mi - m;
    }
    items += __shfl_sync(0xFFFFFFFFu, ni, 31);
    slots += __shfl_sync(0xFFFFFFFFu, mi, 31);
  }
  if (lane == 0) {
    items_before[E] = items;
    slots_before[E] = slots;
  }
}

// Warp-collective: the estimated time, in steps, of slices of at most `slice`
// steps: the rounds of items every cluster takes times their mean length, at
// least the longest, plus the partial blocks. Infinite where these do not fit.
__device__ float cost_of(const WParams& p, const int* row_start, int slice) {
  const int lane = threadIdx.x & 31;
  const int per = p.MT * p.NT;
  float items = 0.0f, slots = 0.0f, work = 0.0f, longest = 0.0f;
  for (int e = lane; e < p.E; e += 32) {
    const int steps = steps_of(row_start[e + 1] - row_start[e]);
    const int n = slices_of(steps, slice);
    const float len = static_cast<float>(max((steps + n - 1) / n, p.min_cost));
    items += static_cast<float>(per) * n;
    slots += n > 1 ? static_cast<float>(per) * n : 0.0f;
    work += static_cast<float>(per) * n * len;
    longest = fmaxf(longest, len);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    items += __shfl_xor_sync(0xFFFFFFFFu, items, d);
    slots += __shfl_xor_sync(0xFFFFFFFFu, slots, d);
    work += __shfl_xor_sync(0xFFFFFFFFu, work, d);
    longest = fmaxf(longest, __shfl_xor_sync(0xFFFFFFFFu, longest, d));
  }
  if (slots > static_cast<float>(p.slots)) return INFINITY;
  const float c = static_cast<float>(p.clusters);
  return fmaxf(ceilf(items / c) * (work / items), longest) + slots * kPartialCost / c +
         (slots > 0.0f ? kJoinCost : 0.0f);
}

__device__ __forceinline__ Item item_of(int i, const WParams& p, const SmemTail& st) {
  Item it;
  int lo = 0, hi = p.E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (st.items_before[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  it.e = lo;
  const uint32_t per = p.MT * p.NT;
  const uint32_t local = i - st.items_before[lo];
  const int r0 = st.row_start[lo];
  it.row0 = r0;
  it.rows = st.row_start[lo + 1] - r0;
  it.slot = -1;
  uint32_t block = local;
  if (local >= per || st.slots_before[lo + 1] != st.slots_before[lo]) {
    const uint32_t slice = local / per;
    block = local - slice * per;
    // 2^31 rows are 2^25 steps, of at most kSlices[last] = 76 slices: 32 bits do
    const uint32_t steps = steps_of(it.rows);
    const uint32_t n = slices_of(steps, st.slice);
    const int s0 = steps * slice / n * BK;
    const int s1 = steps * (slice + 1) / n * BK;
    it.row0 = r0 + s0;
    it.rows = min(it.rows, s1) - s0;
    it.slot = st.slots_before[lo] + local;
  }
  it.mt = block / static_cast<uint32_t>(p.NT);
  it.nt = block - it.mt * p.NT;
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

// Warp-collective store of 32 rows x 16 columns of fp32 (lane i holds row i in
// v[]) through the warp's staging buffer, so that four lanes write each
// 64-byte row segment; rows r < nvalid only.
__device__ __forceinline__ void store_f32x16(uint4* stg, const float* v, float* row0,
                                             long long ld, int nvalid) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int g = 0; g < 4; ++g)
    stg[stage_slot(lane, g)] =
        make_uint4(__float_as_uint(v[4 * g]), __float_as_uint(v[4 * g + 1]),
                   __float_as_uint(v[4 * g + 2]), __float_as_uint(v[4 * g + 3]));
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = 8 * j + (lane >> 2);
    const uint4 w = stg[stage_slot(r, lane & 3)];
    if (r < nvalid) *reinterpret_cast<uint4*>(row0 + r * ld + 4 * (lane & 3)) = w;
  }
  __syncwarp();
}

template <bool kF32, bool kBase>
__global__ void __launch_bounds__(32 * (kFirstEpi + kEpiWarps), 1)
wgrad_kernel(const __grid_constant__ CUtensorMap mapD, const __grid_constant__ CUtensorMap mapA,
             const __grid_constant__ CUtensorMap mapBase, const WParams p) {
  using L = Layout<kF32 && kBase>;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_addr + pad;
  SmemTail& st = *reinterpret_cast<SmemTail*>(smem + L::kTailAt);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const bool leader = crank == 0;

  if (warp == 0) {
    bool bad = false;
    int most = 0;
    for (int e = lane; e <= p.E; e += 32) {
      const int o = p.offsets[e];
      st.row_start[e] = o;
      const int next = e < p.E ? p.offsets[e + 1] : o;
      if (next < o || o > p.R_cap || o < 0) bad = true;
      if (e == 0 && o != 0) bad = true;
      most = max(most, steps_of(next - o));
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) {
      st.most_steps = bad ? -1 : most;
      st.abort_flag = 0;
      if (bad && blockIdx.x == 0) set_status(p.status, GG_ERR_DEVICE_BAD_OFFSETS);
      for (int s = 0; s < kStages; ++s) {
        mbar_init(smem_u32(&st.full[s]), 1);
        mbar_init(smem_u32(&st.ready[s]), 2);
        mbar_init(smem_u32(&st.empty[s]), 1);
      }
      for (int i = 0; i < kItems; ++i) {
        mbar_init(smem_u32(&st.item_full[i]), 1);
        // readers: producer, pass warp, epilogue warps, and the even CTA's issuer
        mbar_init(smem_u32(&st.item_empty[i]), 2 + kEpiWarps + (leader ? 1 : 0));
      }
      for (int a = 0; a < 2; ++a) {
        mbar_init(smem_u32(&st.tfull[a]), 1);
        mbar_init(smem_u32(&st.tempty[a]), 2 * kEpiWarps);
      }
      for (int w = 0; w < kEpiWarps; ++w)
        for (int b = 0; b < kBaseBufs; ++b) mbar_init(smem_u32(&st.base_full[w][b]), 1);
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
  // slice length: one warp per candidate, the cheapest wins (ties: fewest)
  const int most_steps = st.most_steps;
  const bool may_slice = p.slots > 0 && most_steps >= 2 * kMinSlice;
  if (may_slice && warp < kTried) {
    const int slice = (most_steps + kSlices[warp] - 1) / kSlices[warp];
    const float c = slice >= kMinSlice ? cost_of(p, st.row_start, slice) : INFINITY;
    if (lane == 0) st.cost[warp] = c;
  }
  __syncthreads();
  if (warp == 0) {
    int slice = most_steps > 0 ? most_steps : 1;
    if (may_slice) {
      int best = 0;
      for (int i = 1; i < kTried; ++i)
        if (st.cost[i] < st.cost[best]) best = i;
      slice = (most_steps + kSlices[best] - 1) / kSlices[best];
    }
    if (most_steps >= 0)
      fill_tables(st.row_start, p.E, p.MT * p.NT, slice, st.items_before, st.slots_before);
    __syncwarp();
    if (lane == 0) {
      st.slice = slice;
      st.total_items = most_steps >= 0 ? st.items_before[p.E] : 0;
      if (blockIdx.x == 0 && p.plan != nullptr)
        *p.plan = most_steps >= 0 && st.slots_before[p.E] > 0 ? slice : 0;
    }
  }
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // both CTAs' barriers exist before anything can arrive on them
  // the join's blocks may take the SMs that run out of items first
  grid_dependents_launch();

  const int first = static_cast<int>(blockIdx.x) / 2;
  const int step = static_cast<int>(gridDim.x) / 2;
  const uint32_t tmem_base = st.tmem_base;
  const int total = st.total_items;
  volatile int* abort_flag = &st.abort_flag;

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    // The whole warp runs the loop and one lane issues, as the MMA issuer's
    // does: its values go into uniform registers (by reductions) once per item.
    if (elect_one()) {
      tma_prefetch_desc(&mapD);
      tma_prefetch_desc(&mapA);
    }
    __syncwarp();
    const int h = static_cast<int>(crank);
    int stage = 0;
    uint32_t phase = 0, used = 0, last_phase = 0;
    bool ok = true;
    Item it;
    ItemReader items;
    while (ok && items.next(st, it, true, lane == 0, abort_flag, p.status)) {
      const int nt = __reduce_max_sync(0xFFFFFFFFu, it.nt);
      const int n0 = __reduce_max_sync(0xFFFFFFFFu, it.mt) * (2 * BM) + h * BM;
      const int half = min(p.width, p.K - nt * p.width) / 2;  // a multiple of 32
      const int k0 = nt * p.width + h * half;
      const int boxes = (half + 63) / 64;
      const int row0 = __reduce_max_sync(0xFFFFFFFFu, it.row0);
      const int rows = __reduce_max_sync(0xFFFFFFFFu, it.rows);
      for (int r = 0; r < rows; r += BK) {
        if (!mbar_wait_bounded(smem_u32(&st.empty[stage]), phase ^ 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        const uint32_t bar = smem_u32(&st.full[stage]);
        const uint32_t sa = sbase + stage * STAGE_BYTES;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, A_BYTES + boxes * BOX_BYTES);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            tma_load_2d(sa + j * BOX_BYTES, &mapD, bar, n0 + 64 * j, row0 + r);
            if (j < boxes)
              tma_load_2d(sa + A_BYTES + j * BOX_BYTES, &mapA, bar, k0 + 64 * j, row0 + r);
          }
        }
        __syncwarp();
        used |= 1u << stage;
        last_phase = (last_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // the CTA may not exit before its loads have landed and been consumed
    for (int s = 0; s < kStages; ++s)
      if (used & (1u << s)) {
        (void)mbar_wait_bounded(smem_u32(&st.full[s]), (last_phase >> s) & 1u, nullptr, p.status);
        (void)mbar_wait_bounded(smem_u32(&st.empty[s]), (last_phase >> s) & 1u, nullptr,
                                p.status);
      }
  } else if (warp == kPassWarp) {
    // ------------------------------------------------ pass on, zero the tail
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    Item it;
    ItemReader items;
    while (ok && items.next(st, it, true, lane == 0, abort_flag, p.status)) {
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
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == kItemWarp) {
    if (lane == 0) {
      // ------------------------------------------------------ work items
      int slot = 0;
      uint32_t phase = 0;
      for (int i = first;; i += step) {
        Item it;
        if (i < total)
          it = item_of(i, p, st);
        else
          it.e = it.mt = it.nt = it.row0 = 0, it.rows = it.slot = -1;
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
      // register anew. All of TMEM is ours, so it starts at column 0.
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = tmem_base == 0;
      const uint64_t desc_d = make_sdesc(sbase, BOX_BYTES, 1024);
      Item it;
      ItemReader items;
      while (ok && items.next(st, it, true, lane == 0, abort_flag, p.status)) {
        const int rows = __shfl_sync(0xFFFFFFFFu, it.rows, 0);
        const uint32_t idesc = make_idesc_bf16(
            2 * BM, __shfl_sync(0xFFFFFFFFu, min(p.width, p.K - it.nt * p.width), 0), true, true);
        const int chunk = (kF32 ? kChunk : kChunkBf16) * BK;
        for (int c0 = 0; c0 < rows && ok; c0 += chunk) {
          if (!mbar_wait_bounded(smem_u32(&st.tempty[acc]), acc_phase ^ 1u, abort_flag,
                                 p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = acc * BN;
          const int c1 = min(rows, c0 + chunk);
          for (int r = c0; r < c1; r += BK) {
            if (!mbar_wait_bounded(smem_u32(&st.ready[stage]), phase, abort_flag, p.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t desc = desc_d + stage * (STAGE_BYTES >> 4);
            if (elect_one()) {
              const int groups = min(BK / 16, (rows - r + 15) / 16);
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk)
                if (kk < groups)
                  tc_mma_bf16_pair(d_tmem, desc + kk * (2048 >> 4),
                                   desc + ((A_BYTES + kk * 2048) >> 4), idesc,
                                   (r - c0) | kk ? 1u : 0u);
              tc_commit_pair_mc(smem_u32(&st.empty[stage]), kPairMask);
            }
            __syncwarp();
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          if (elect_one()) tc_commit_pair_mc(smem_u32(&st.tfull[acc]), kPairMask);
          __syncwarp();
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        }
      }
      if (elect_one()) {
        tc_commit_pair(smem_u32(&st.mma_done));
        (void)mbar_wait_bounded(smem_u32(&st.mma_done), 0, nullptr, p.status);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------- epilogue
    // Warp w may only read TMEM lanes 32*(w%4) .. +31: the warps of a lane
    // quadrant share the block's columns.
    const int q = warp & 3;
    const int c0 = ((warp - kFirstEpi) >> 2) * kCols;
    int acc = 0;
    uint32_t acc_phase = 0;
    uint4* stg =
        reinterpret_cast<uint4*>(smem + L::kStagingAt + (warp - kFirstEpi) * kWarpStagingBytes);
    const uint32_t piece_at = L::kBaseAt + (warp - kFirstEpi) * kBaseBufs * kPieceBytes;
    uint32_t piece_phase = 0, pending = 0;
    bool ok = true;
    Item it;
    ItemReader items;
    while (ok && items.next(st, it, true, lane == 0, abort_flag, p.status)) {
      const int row = static_cast<int>(crank) * BM + q * 32;  // of the block
      const int n0 = it.mt * (2 * BM) + row;
      const int nvalid = max(0, min(32, p.N - n0));
      const int width = min(p.width, p.K - it.nt * p.width);
      const int cols = max(0, min(kCols, width - c0));  // a multiple of 64
      const long long at =
          (static_cast<long long>(it.e) * p.N + n0) * p.K + it.nt * p.width + c0;
      float* part = it.slot >= 0
                        ? p.partial + it.slot * kSlotFloats + static_cast<long long>(row) * BN + c0
                        : nullptr;
      const bool add = kBase && it.slot < 0;
      const uint32_t lanes = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + c0;
      // fp32 base, one piece = 32 rows x 32 columns: its load by lane 0, and its
      // addition to a chunk that has one row per lane (the piece's 128-byte
      // rows are swizzled, so eight lanes' reads hit all banks)
      const auto load_piece = [&](int i) {
        if (32 * i >= cols) return;
        pending |= 1u << (i % kBaseBufs);
        if (lane != 0) return;
        const uint32_t bar = smem_u32(&st.base_full[warp - kFirstEpi][i % kBaseBufs]);
        mbar_arrive_expect_tx(bar, kPieceBytes);
        tma_load_3d(sbase + piece_at + (i % kBaseBufs) * kPieceBytes, &mapBase, bar,
                    it.nt * p.width + c0 + 32 * i, n0, it.e);
      };
      const auto add_piece = [&](int i, float* v) {
        const int buf = i % kBaseBufs;
        if (!mbar_wait_bounded(smem_u32(&st.base_full[warp - kFirstEpi][buf]),
                               (piece_phase >> buf) & 1u, abort_flag, p.status))
          return false;
        piece_phase ^= 1u << buf;
        pending &= ~(1u << buf);
        const uint8_t* line = smem + piece_at + buf * kPieceBytes + lane * 128;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const float4 f = *reinterpret_cast<const float4*>(line + ((g ^ (lane & 7)) << 4));
          v[4 * g] += f.x;
          v[4 * g + 1] += f.y;
          v[4 * g + 2] += f.z;
          v[4 * g + 3] += f.w;
        }
        fence_proxy_async();  // the buffer's next load comes behind these reads
        __syncwarp();
        load_piece(i + kBaseBufs);
        return true;
      };
      if (kF32) {
        float* out = part != nullptr ? part : static_cast<float*>(p.dB) + at;
        const long long ld = part != nullptr ? BN : p.K;
        // the first pieces of the base, on their way while the MMAs run
        if (add)
          for (int i = 0; i < kBaseBufs; ++i) load_piece(i);
        if (it.rows <= kChunk * BK) {
          // one chunk (or none): from TMEM straight to memory
          if (it.rows > 0) {
            if (!mbar_wait_bounded(smem_u32(&st.tfull[acc]), acc_phase, abort_flag, p.status))
              break;
            tc_fence_after();
          }
#pragma unroll 1
          for (int c = 0; c < cols; c += 32) {
            float v[32] = {};
            if (it.rows > 0) tmem_ld32(lanes + acc * BN + c, v);
            if (add && !(ok = add_piece(c / 32, v))) break;
            store_f32x16(stg, v, out + c, ld, nvalid);
            store_f32x16(stg, v + 16, out + c + 16, ld, nvalid);
          }
          if (it.rows > 0) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&st.tempty[acc]), 0));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
          }
          continue;
        }
        // several chunks: their sums are added up in registers
        float sum[kCols];
#pragma unroll
        for (int i = 0; i < kCols; ++i) sum[i] = 0.0f;
        for (int r = 0; r < it.rows; r += kChunk * BK) {
          if (!mbar_wait_bounded(smem_u32(&st.tfull[acc]), acc_phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kCols; c += 16) {
            if (c < cols) {
              float v[16];
              tmem_ld16(lanes + acc * BN + c, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) sum[c + i] += v[i];
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&st.tempty[acc]), 0));
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          if (c < cols && ok) {
            if (add) ok = add_piece(c / 32, sum + c);
            store_f32x16(stg, sum + c, out + c, ld, nvalid);
            store_f32x16(stg, sum + c + 16, out + c + 16, ld, nvalid);
          }
        }
      } else {
        // 32 columns of dB; raw: the base's
        const auto put = [&](int c, float(&v)[32], const uint4(&raw)[4]) {
          uint4 w[4];
          if (add) {
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
          store_chunk(stg, w, static_cast<gg_bf16*>(p.dB) + at + c, p.K, nvalid);
        };
        if (it.rows > kChunkBf16 * BK) {
          // several chunks, carried in registers; with a base in local memory, that
          // is in L2 (registers spilled what shorter items load ahead: 128 experts,
          // 1536 x 2048 onto a BF16 base 568 -> 703 us; in local memory one expert of
          // 131072 rows, 4096 x 4096, takes 2770 us, left in TMEM 2600)
          float4 sum[kCols / 4];
          constexpr int kUnroll = kBase ? 1 : kCols / 32;
#pragma unroll
          for (int i = 0; i < kCols / 4; ++i) sum[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int r = 0; r < it.rows; r += kChunkBf16 * BK) {
            if (!mbar_wait_bounded(smem_u32(&st.tfull[acc]), acc_phase, abort_flag, p.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll kUnroll * 2
            for (int c = 0; c < kCols; c += 16) {
              if (c >= cols) continue;
              float v[16];
              tmem_ld16(lanes + acc * BN + c, v);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float4& f = sum[c / 4 + i];
                f.x += v[4 * i];
                f.y += v[4 * i + 1];
                f.z += v[4 * i + 2];
                f.w += v[4 * i + 3];
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&st.tempty[acc]), 0));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
          }
          if (!ok) break;
#pragma unroll kUnroll
          for (int c = 0; c < kCols; c += 32) {
            if (c >= cols) continue;
            float v[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 f = sum[c / 4 + i];
              v[4 * i] = f.x;
              v[4 * i + 1] = f.y;
              v[4 * i + 2] = f.z;
              v[4 * i + 3] = f.w;
            }
            if (part != nullptr) {
              store_f32x16(stg, v, part + c, BN, nvalid);
              store_f32x16(stg, v + 16, part + c + 16, BN, nvalid);
            } else {
              uint4 raw[4];
              if (add)
                load_chunk_raw(raw, static_cast<const gg_bf16*>(p.base) + at + c, p.K, nvalid);
              put(c, v, raw);
            }
          }
          continue;
        }
        // one chunk: straight from TMEM
        uint4 raw[BN / 64][4];  // the base's 32-column chunks, loaded ahead of the sums
        if (add) {
#pragma unroll
          for (int b = 0; b < BN / 64; ++b)
            if (32 * b < cols)
              load_chunk_raw(raw[b], static_cast<const gg_bf16*>(p.base) + at + 32 * b, p.K,
                             nvalid);
        }
        if (it.rows > 0) {
          if (!mbar_wait_bounded(smem_u32(&st.tfull[acc]), acc_phase, abort_flag, p.status)) break;
          tc_fence_after();
        }
#pragma unroll
        for (int b = 0; b < BN / 64; ++b) {
          const int c = 32 * b;
          if (c < cols) {
            float v[32];
            if (it.rows > 0) {
              tmem_ld32(lanes + acc * BN + c, v);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0.0f;
            }
            if (part != nullptr) {
              store_f32x16(stg, v, part + c, BN, nvalid);
              store_f32x16(stg, v + 16, part + c + 16, BN, nvalid);
            } else {
              put(c, v, raw[b]);
            }
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
    // after a wait that ran out: no load may still be on its way at the exit
    for (int b = 0; b < kBaseBufs; ++b)
      if (pending & (1u << b))
        (void)mbar_wait_bounded(smem_u32(&st.base_full[warp - kFirstEpi][b]),
                                (piece_phase >> b) & 1u, nullptr, p.status);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
  cluster_sync();
}

// Adds the partial blocks of the experts whose rows were cut: dB = (base +) the
// slices' sums, in slice order. One warp per row of a block, a lane eight
// columns, all slices' loads in flight together: latency bound.
constexpr int kJoinThreads = 256;
constexpr int kJoinAhead = 4;  // slices loaded together
template <bool kF32>
__global__ void __launch_bounds__(kJoinThreads)
wgrad_join_kernel(const WParams p) {
  __shared__ int row_start[kMaxExperts + 1];
  __shared__ int cut[kWgradMaxSlots / 2 + 1];        // the experts whose rows were cut
  __shared__ int slot_of[kWgradMaxSlots / 2 + 1];    // and their first partial blocks
  __shared__ int n_cut;
  // the offsets are older than the kernel ahead of this one: read them early
  for (int e = threadIdx.x; e <= p.E; e += kJoinThreads) row_start[e] = p.offsets[e];
  __syncthreads();
  grid_dependency_wait();
  const int slice = *p.plan;
  if (slice == 0) return;  // nothing was cut
  const int per = p.MT * p.NT;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int found = 0, slots = 0;
    for (int b = 0; b < p.E; b += 32) {
      const int e = b + lane;
      const int n = e < p.E ? slices_of(steps_of(row_start[e + 1] - row_start[e]), slice) : 1;
      const uint32_t is_cut = __ballot_sync(0xFFFFFFFFu, n > 1);
      int before = n > 1 ? n : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, before, d);
        if (lane >= d) before += x;
      }
      if (n > 1) {  // at most kWgradMaxSlots / 2: each has two slices or more
        const int at = found + __popc(is_cut & ((1u << lane) - 1u));
        cut[at] = e;
        slot_of[at] = slots + (before - n) * per;
      }
      found += __popc(is_cut);
      slots += __shfl_sync(0xFFFFFFFFu, before, 31) * per;
    }
    if (lane == 0) n_cut = found;
  }
  __syncthreads();
  const int col = (threadIdx.x & 31) * 8;
  const int rows = n_cut * per * (2 * BM);
  for (int u = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5); u < rows;
       u += gridDim.x * (kJoinThreads / 32)) {
    const int row = u % (2 * BM);
    const int which = u / (2 * BM) / per;
    const int block = u / (2 * BM) - which * per;
    const int lo = cut[which];
    const int slot = slot_of[which] + block;
    const int mt = block / p.NT, nt = block - mt * p.NT;
    const int n = slices_of(steps_of(row_start[lo + 1] - row_start[lo]), slice);
    const int out_row = mt * 2 * BM + row;
    if (col >= min(p.width, p.K - nt * p.width) || out_row >= p.N) continue;
    const long long at = (static_cast<long long>(lo) * p.N + out_row) * p.K + nt * p.width + col;
    const float* src = p.partial + slot * kSlotFloats + static_cast<long long>(row) * BN + col;
    const long long next = static_cast<long long>(per) * kSlotFloats;  // the following slice's
    float4 v0 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v1 = v0;
    if (p.base != nullptr) {
      if (kF32) {
        const float4* b = reinterpret_cast<const float4*>(static_cast<const float*>(p.base) + at);
        v0 = b[0];
        v1 = b[1];
      } else {
        const uint4 b = *reinterpret_cast<const uint4*>(static_cast<const gg_bf16*>(p.base) + at);
        v0 = make_float4(bf16_lo(b.x), bf16_hi(b.x), bf16_lo(b.y), bf16_hi(b.y));
        v1 = make_float4(bf16_lo(b.z), bf16_hi(b.z), bf16_lo(b.w), bf16_hi(b.w));
      }
    }
    for (int s0 = 0; s0 < n; s0 += kJoinAhead) {
      float4 f[kJoinAhead][2];
#pragma unroll
      for (int s = 0; s < kJoinAhead; ++s) {
        const float4* q = reinterpret_cast<const float4*>(src + min(s0 + s, n - 1) * next);
        f[s][0] = q[0];
        f[s][1] = q[1];
      }
#pragma unroll
      for (int s = 0; s < kJoinAhead; ++s)
        if (s0 + s < n) {
          v0.x += f[s][0].x;
          v0.y += f[s][0].y;
          v0.z += f[s][0].z;
          v0.w += f[s][0].w;
          v1.x += f[s][1].x;
          v1.y += f[s][1].y;
          v1.z += f[s][1].z;
          v1.w += f[s][1].w;
        }
    }
    if (kF32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.dB) + at);
      o[0] = v0;
      o[1] = v1;
    } else {
      *reinterpret_cast<uint4*>(static_cast<gg_bf16*>(p.dB) + at) =
          make_uint4(pack_bf16x2(v0.x, v0.y), pack_bf16x2(v0.z, v0.w), pack_bf16x2(v1.x, v1.y),
                     pack_bf16x2(v1.z, v1.w));
    }
  }
}

template <bool kF32, bool kBase>
cudaError_t launch_wgrad_t(const CUtensorMap& md, const CUtensorMap& ma, const CUtensorMap& mb,
                           const WParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  static std::atomic<int> resident[kMaxDevices];
  // work items: the blocks, and with slices whatever the clusters can share
  const int most = p.slots > 0 ? p.clusters : p.E * p.MT * p.NT;
  using L = Layout<kF32 && kBase>;
  cudaError_t e = launch_pairs(wgrad_kernel<kF32, kBase>, resident, L::kThreads, L::kSmemBytes,
                               most, dev, stream, md, ma, mb, p);
  if (e != cudaSuccess || p.slots == 0) return e;
  e = launch_early(wgrad_join_kernel<kF32>, dim3(5 * dev.sm_count), dim3(kJoinThreads), 0, stream,
                   p);
  count_launch();
  return e;
}

}  // namespace

int wgrad_slots(int R_cap, int N, int K) {
  // no expert can have two slices' rows
  if (R_cap < 2 * kMinSlice * BK) return 0;
  const long long per = static_cast<long long>((N + 2 * BM - 1) / (2 * BM)) * ((K + BN - 1) / BN);
  // every slice but an expert's last has kMinSlice steps, each block a partial per slice
  const long long most = per * (R_cap / (kMinSlice * BK) + 1);
  return static_cast<int>(most < kWgradMaxSlots ? most : kWgradMaxSlots);
}

size_t wgrad_slot_bytes() { return static_cast<size_t>(kSlotFloats) * sizeof(float); }

cudaError_t launch_wgrad(const WgradArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  CUtensorMap md, ma, mb;
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
  mb = md;
  if (a.f32 && a.base != nullptr) {
    const cuuint64_t bd[3] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.N),
                              static_cast<cuuint64_t>(a.E)};
    const cuuint64_t bs[2] = {static_cast<cuuint64_t>(a.K) * 4,
                              static_cast<cuuint64_t>(a.K) * a.N * 4};
    const cuuint32_t bbox[3] = {32, 32, 1};
    if (!encode_map(&mb, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.base, 3, bd, bs, bbox,
                    CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  WParams p{};
  p.offsets = a.offsets;
  p.E = a.E;
  p.R_cap = a.R_cap;
  p.N = a.N;
  p.K = a.K;
  p.MT = (a.N + 2 * BM - 1) / (2 * BM);
  p.NT = (a.K + BN - 1) / BN;
  // columns in 64s, as even as the blocks allow (320: 192 + 128)
  p.width = (a.K / 64 + p.NT - 1) / p.NT * 64;
  // 128 KB of BF16 or 256 KB of fp32 per block and pair, again to read a base;
  // a pair moves about as much as 5 steps of MMAs take per 128 KB
  p.min_cost = 5 * (a.f32 ? 2 : 1) * (a.base != nullptr ? 2 : 1);
  p.clusters = dev.sm_count / 2;
  p.slots = a.slots;
  p.base = a.base;
  p.dB = a.dB;
  p.partial = a.partial;
  p.plan = a.plan;
  p.status = a.status;
  if (a.base != nullptr)
    return a.f32 ? launch_wgrad_t<true, true>(md, ma, mb, p, dev, stream)
                 : launch_wgrad_t<false, true>(md, ma, mb, p, dev, stream);
  return a.f32 ? launch_wgrad_t<true, false>(md, ma, mb, p, dev, stream)
               : launch_wgrad_t<false, false>(md, ma, mb, p, dev, stream);
}

}  // namespace gg
