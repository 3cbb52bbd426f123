// gg_gemm_f8.cu — grouped linear layers on E4M3 codes with an fp32 scale for
// every 128 columns of a token's row and every 128 x 128 block of a weight, on
// sm_103a; forward and input gradient on the same codes:
//   C[r][n]  = sum_b s[b][r] t[e][n / 128][b] sum_{k in block b} q[r][k] w[e][n][k]
//   dA[r][c] = sum_b s[b][r] t[e][b][c / 128] sum_{n in block b} d[r][n] w[e][n][c]
// with the gated activations, and their gradients, fused.
//
// Scales change every 128 of the reduction, so the tensor cores sum 128 codes
// (four MMAs) into one of two TMEM buffers, and eight warps add each buffer,
// scaled, to fp32 sums in registers while the other one is filled. Products of
// two E4M3 codes are exact in fp32.
//
// A work item is a block of 256 channels (gated forward: 128, gate and up) and
// up to 256 tokens of an expert, in one of two orientations:
//   - more than 128 tokens: tokens are the MMA's rows (M = 256, 128 per CTA),
//     channels its columns (N = 256). A TMEM lane is a token, so a step's scale
//     is one number per thread and 64 columns, a gate value and its up value
//     meet in one thread, and a thread has its row's channels together;
//   - up to 128 tokens (an expert's last ones, or all it has): channels are the
//     rows, tokens the columns, in steps of 32, so that a ragged count costs
//     what it has. The tokens' scales then differ by column, and reading them
//     from shared memory is what a step costs: with 256 tokens 750 ns of it
//     where the MMAs take 290, which is why long blocks are not done this way.
// Both find the same tiles in shared memory; the MMA's operands change places.
// For the input gradient the weights are read as they lie, reduction outermost
// ("MN-major"): one set of codes serves both directions.
//
// One CTA per SM in clusters of two (one tcgen05 MMA pair, 384 threads per
// CTA, warp-specialised):
//   warp 0      TMA producer: per step of 128 its half of the channels (gated
//               forward: 64 gate rows and the matching up rows) and half the
//               tokens, 128-byte swizzle;
//   warp 1      allocates TMEM; in the even CTA one lane issues
//               tcgen05.mma.cta_group::2.kind::f8f6f4 (M = 256, K = 32);
//   warp 2      finds the work items ahead of the others;
//   warp 3      writes each step's scales, token times weight block, into a
//               ring;
//   warps 4-11  sums and epilogue; two groups of four take half the columns
//               each.
// The epilogues pass their chunks through shared memory: pieces of 32 rows go
// out by TMA (few tokens: as 64-byte pieces of rows), while the next products
// run. The gated gradient's H1 comes in the same way. The quantiser ahead lets
// this kernel set itself up while it runs; loads wait for its end.
//
// What bounds it: a step is 517 cycles of MMAs, 750 of L2-to-SM loads (64 KB a
// pair), and about 970 of the round that one of the two TMEM buffers makes: MMA,
// wake-up, two TMEM loads and 128 additions a thread, release, wake-up. TMEM
// holds no third buffer of 256 columns, and 128-column MMAs read shared memory
// at its limit. 131072 rows, 128 experts, 1536 x 2048: 397 us forward (2080
// TFLOP/s), 463 gated with H1 kept, 400 input gradient; one expert, 65536 rows,
// 4096 x 4096: 2550 TFLOP/s. Gated gradient, 131072 rows, 2048 x 768: 340 us,
// 0.8 GB of H1 and its gradient among them.
//
// Every wait is bounded (gg_ptx.cuh); a wait that runs out records
// GG_ERR_DEVICE_TIMEOUT, raises a CTA-wide abort flag, and the CTA drains
// what is in flight, frees TMEM and exits after a final cluster barrier.

#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "gg_epilogue.cuh"
#include "gg_f8.cuh"
#include "gg_internal.h"
#include "gg_launch.cuh"
#include "gg_ptx.cuh"

namespace gg {
namespace {

enum F8Mode : int { kFwd = 0, kFwdGated = 1, kGrad = 2, kGradGated = 3 };

constexpr int BM = 128;       // channels per CTA
constexpr int BN = 256;       // most tokens per work item
constexpr int BK = kF8Block;  // codes per step
constexpr int kStages = 4;
constexpr int kScales = 4;    // steps of scales ready
constexpr int kItems = 4;     // work items found ahead
constexpr int kRaster = 8;    // token blocks that go through the channels together
constexpr int kItemWarp = 2, kFirstSum = 4;
constexpr int kSumWarps = 8;
constexpr int kThreads = 32 * (kFirstSum + kSumWarps);
constexpr int kChunks = 4;    // of 32 columns, that a summing warp has at most
constexpr int kFewTokens = 128;  // tokens up to which they are the columns
constexpr uint16_t kPairMask = 0x3;
constexpr uint32_t A_BYTES = BM * BK;
constexpr uint32_t STAGE_BYTES = A_BYTES + BN / 2 * BK;
constexpr uint32_t TMEM_COLS = 512;
constexpr int kBoxes = 4;     // heights of token boxes: 128, 64, 32 and 16 rows
// Registers per thread of the two roles. The launch has 168 for each of 384
// threads; either split, of the first four warps and the other eight, is three
// times that.
// And the steps of scales on their way (registers of the warp that loads them).
template <int MODE>
struct Regs {
  static constexpr int kAhead = MODE == kGradGated ? 2 : 4;
  static constexpr int kFew = MODE == kGradGated ? 56 : 72;
  static constexpr int kMany = MODE == kGradGated ? 224 : 216;
  static_assert(128 * (kFew + 2 * kMany) <= kThreads * 168, "register split");
};

// A work item: expert, block of channels, its tokens (first row, number; rows
// < 0: there are no more items); few: channels are the MMA's rows and the
// tokens its columns, in `cols` of them, a multiple of 32.
struct alignas(16) Item {
  int e, nt, row0, rows;
  int few, cols;
  int pad_[2];
};

struct SmemTail {
  Item item[kItems];
  uint64_t item_full[kItems];
  uint64_t item_empty[kItems];
  uint64_t full[kStages];    // even CTA: both CTAs' loads have landed
  uint64_t empty[kStages];
  uint64_t scale_full[kScales];
  uint64_t scale_empty[kScales];
  uint64_t tfull[2];
  uint64_t tempty[2];        // even CTA
  uint64_t pair[2][2];       // per group: warps of gate rows and of the matching up rows
  uint64_t group[2];         // the four warps of a group
  uint64_t h1_full[kSumWarps];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int total_tiles;
  // row sums of each lane quadrant's 32 channels, for a group's own tokens: which
  // those are differs from item to item, and the groups are not at the same one
  float dots[2][4][kFewTokens / 2];
  int tiles_before[kMaxExperts + 1];
  int row_start[kMaxExperts + 1];
};

constexpr uint32_t kScaleAt = kStages * STAGE_BYTES;
// A step's scales: [64 channels][this CTA's 128 tokens], or, few tokens, [this
// CTA's half of 64 channels][128 tokens].
constexpr uint32_t kScaleBytes = 4 * BM * 4;
constexpr uint32_t kStagingAt = kScaleAt + kScales * kScaleBytes;
constexpr uint32_t kWarpStaging = 2 * 32 * 64 * 2;  // two buffers of 32 rows x 64 BF16
constexpr uint32_t kTailAt = kStagingAt + kSumWarps * kWarpStaging;
constexpr size_t kSmemBytes = 1024 + kTailAt + sizeof(SmemTail);
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
static_assert(kTailAt % 16 == 0 && kScaleAt % 16 == 0, "16-byte reads");
static_assert(kStagingAt % 1024 == 0 && kWarpStaging % 1024 == 0, "128-byte swizzle");

struct F8Params {
  const int32_t* offsets;
  int E, R_cap;
  int red;             // length of the reduction
  int width;           // channels of an output half: N, F, K or F
  int F;               // gated: channels from gate to up
  int NT;              // blocks of channels
  const float* S;      // [ceil(red / 128)][R_cap]
  const float* T;      // weight scales of an expert: [.. channel block .. reduction block ..]
  int t_expert, t_chan, t_red;  // their strides
  const float* row_scale;
  float alpha;
  gg_bf16* C;
  gg_bf16* H1_save;    // gated forward, or null
  const gg_bf16* H1;   // gated gradient
  float* rowdot;       // gated gradient, or null
  int rowdot_stride;
  int32_t* status;
};

__device__ __forceinline__ int token_blocks(int rows) { return (rows + BN - 1) / BN; }

__device__ __forceinline__ Item item_of(int tile, const F8Params& p, const SmemTail& st) {
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
  // eight token blocks at a time, the token block fastest: what runs side by
  // side shares its weights and its tokens
  const int local = tile - st.tiles_before[lo];
  const int from = local / (kRaster * p.NT) * kRaster;
  const int wide = min(kRaster, blocks - from);
  const int at = local - from * p.NT;
  it.nt = at / wide;
  const int tb = from + at - it.nt * wide;
  it.row0 = first + tb * BN;
  it.rows = min(BN, rows - tb * BN);
  it.few = it.rows <= kFewTokens;
  it.cols = it.few ? (it.rows + 31) & ~31 : BN;
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

// E4M3 operands (format fields 0), fp32 sums, M = 256, N = n.
__device__ __forceinline__ uint32_t idesc_f8(int n, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((static_cast<uint32_t>(n) >> 3) << 17) | ((static_cast<uint32_t>(2 * BM) >> 4) << 24);
}

// 32 lanes x 32 columns: a thread gets its lane's 32. Valid after tmem_wait().
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// Names the registers that the loads write, so that no use moves ahead of it.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

// acc += v * (s, s), pairs of columns.
__device__ __forceinline__ void add_scaled(float (&acc)[32], const uint32_t (&v)[32], float s) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float2* to = reinterpret_cast<float2*>(&acc[i]);
    *to = __ffma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])),
                     make_float2(s, s), *to);
  }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// 16-byte piece c of row r in a buffer of 32 rows x 64 BF16 (8 pieces) or 32 x
// 32 (4): TMA's 128-byte and 64-byte swizzles, which also spread eight lanes
// that touch one piece of eight rows over all banks. stage_slot() is the
// latter.
__device__ __forceinline__ int wide_slot(int r, int c) { return r * 8 + (c ^ (r & 7)); }

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}

// The lane, made anew: address arithmetic on it is done where it is used, not
// kept in registers over the loops, where it spilled their sums.
__device__ __forceinline__ int lane_here() {
  int lane = threadIdx.x & 31;
  asm volatile("" : "+r"(lane));
  return lane;
}

// A warp's results on their way to memory: two buffers, filled in turn, each
// written by one TMA store where all 32 rows belong to the expert. Stores of
// the warp's own held it up behind those of all other SMs, which reach their
// epilogues together (131072 x 1536 x 2048: 362 us of 299 without any).
struct Outbox {
  uint8_t* at;   // the warp's buffers
  int turn = 0;
  // The buffer to fill next, once the store that read it last is done.
  __device__ __forceinline__ uint4* open() {
    if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
    uint4* buf = reinterpret_cast<uint4*>(at + turn * (kWarpStaging / 2));
    turn ^= 1;
    return buf;
  }
  // No store reads a buffer any more.
  __device__ __forceinline__ void drain() {
    if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
  }
};

// Every store of a buffer, or of none, is a group of its own.
__device__ __forceinline__ void end_group() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Warp-collective: 32 rows x 64 columns, lane i with row i in lo and hi, to
// rows row.. and columns col.. of out (ld wide). Rows below `have` exist, and
// columns below ld - col or `cols`, a multiple of 64.
__device__ __forceinline__ void send_wide(Outbox& box, const CUtensorMap* map,
                                          const float (&lo)[32], const float (&hi)[32],
                                          gg_bf16* out, long long ld, int row, int col, int have,
                                          int cols) {
  const int lane = lane_here();
  uint4* buf = box.open();
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    buf[wide_slot(lane, c)] = pack8(&lo[8 * c]);
    buf[wide_slot(lane, 4 + c)] = pack8(&hi[8 * c]);
  }
  if (have >= 32) {
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      if (cols > 0) tma_store_2d(map, smem_u32(buf), col, row);
      end_group();
    }
    return;
  }
  __syncwarp();
  if (cols > 0) {
#pragma unroll 2
    for (int j = 0; j < 8; ++j) {
      const int r = 4 * j + (lane >> 3);
      if (r < have)
        reinterpret_cast<uint4*>(out + (row + r) * ld + col)[lane & 7] =
            buf[wide_slot(r, lane & 7)];
    }
  }
  __syncwarp();
  if (lane == 0) end_group();
}

// Gradient of act(g) u at acc * w, act(g) = g s with s = sigmoid(alpha g), and
// dot + acc * act(g) u.
__device__ __forceinline__ void glu_grad(float acc, float w, float g, float u, float alpha,
                                         float& dg, float& du, float& dot) {
  const float ag = alpha * g;
  const float s = __fdividef(1.0f, 1.0f + __expf(-ag));
  const float gs = g * s;
  const float d = acc * w;
  dg = (d * u) * (s * fmaf(ag, 1.0f - s, 1.0f));
  du = d * gs;
  dot = fmaf(acc, gs * u, dot);
}

// sigmoid(alpha g) of two channels; to_exp = -alpha log2(e).
__device__ __forceinline__ float2 sigmoid2(float2 g, float2 to_exp) {
  const float2 t = __fmul2_rn(g, to_exp);
  float2 e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = __fadd2_rn(e, make_float2(1.0f, 1.0f));
  float2 s;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(e.y));
  return s;
}

__device__ __forceinline__ float2 exp_factor(float alpha) {
  const float x = -1.4426950408889634f * alpha;
  return make_float2(x, x);
}

// The same for two channels, in packed multiplications and additions, which
// take half the issue slots (77824 rows, 512 channels, reduction 256: 95 us
// where one by one took 107).
__device__ __forceinline__ void glu_grad2(float2 acc, float2 w, float2 g, float2 u, float2 alpha,
                                          float2 to_exp, float2& dg, float2& du, float2& dot) {
  const float2 one = make_float2(1.0f, 1.0f);
  const float2 s = sigmoid2(g, to_exp);
  const float2 gs = __fmul2_rn(g, s);
  const float2 d = __fmul2_rn(acc, w);
  const float2 rest = __ffma2_rn(s, make_float2(-1.0f, -1.0f), one);
  const float2 slope = __fmul2_rn(s, __ffma2_rn(__fmul2_rn(alpha, g), rest, one));
  dg = __fmul2_rn(__fmul2_rn(d, u), slope);
  du = __fmul2_rn(d, gs);
  dot = __ffma2_rn(acc, __fmul2_rn(gs, u), dot);
}

__device__ __forceinline__ void tc_mma_f8_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi,
                                               uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                               bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

struct F8Maps {
  CUtensorMap tokens[kBoxes];
  CUtensorMap weights;
  CUtensorMap out;  // C: 32 rows x 64 columns, gated gradient x 32
  CUtensorMap h1;   // H1_save: 32 x 64; gated gradient's H1: 32 x 32
};

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
f8_gemm_kernel(const __grid_constant__ F8Maps maps, const F8Params p) {
  constexpr bool kGated = MODE == kFwdGated;
  constexpr bool kMN = MODE == kGrad || MODE == kGradGated;
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
      for (int s = 0; s < kStages; ++s) {
        mbar_init(smem_u32(&st.full[s]), 1);
        mbar_init(smem_u32(&st.empty[s]), 1);
      }
      for (int s = 0; s < kScales; ++s) {
        mbar_init(smem_u32(&st.scale_full[s]), 1);
        mbar_init(smem_u32(&st.scale_empty[s]), kSumWarps);
      }
      for (int a = 0; a < 2; ++a) {
        mbar_init(smem_u32(&st.tfull[a]), 1);
        mbar_init(smem_u32(&st.tempty[a]), 2 * kSumWarps);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&st.pair[a][i]), 2);
        mbar_init(smem_u32(&st.group[a]), 4);
      }
      for (int w = 0; w < kSumWarps; ++w) mbar_init(smem_u32(&st.h1_full[w]), 1);
      for (int i = 0; i < kItems; ++i) {
        mbar_init(smem_u32(&st.item_full[i]), 1);
        // readers: producer, scale and summing warps, and the even CTA's issuer
        mbar_init(smem_u32(&st.item_empty[i]), 2 + kSumWarps + (leader ? 1 : 0));
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
  const int KB = (p.red + BK - 1) / BK;
  volatile int* abort_flag = &st.abort_flag;

  if (warp < kFirstSum) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<MODE>::kFew));
    if (warp == 0) {
      if (lane == 0) {
        // -------------------------------------------------- TMA producer
        for (int i = 0; i < kBoxes; ++i) tma_prefetch_desc(&maps.tokens[i]);
        grid_dependency_wait();  // the quantiser's codes
        tma_prefetch_desc(&maps.weights);
        tma_prefetch_desc(&maps.out);
        const int h = static_cast<int>(crank);
        int stage = 0;
        uint32_t phase = 0, used = 0, last_phase = 0;
        bool ok = true;
        Item it;
        ItemReader items;
        while (ok && items.next(st, it, false, true, abort_flag, p.status)) {
          // 128 channels; gated forward: 64 gate rows and the matching up rows
          const int n0 = it.nt * (kGated ? BM : 2 * BM) + h * (kGated ? 64 : BM);
          const int half = it.cols / 2;  // this CTA's tokens, a multiple of 16
          const int r0 = it.row0 + h * half;
          for (int kb = 0; kb < KB; ++kb) {
            if (!mbar_wait_bounded(smem_u32(&st.empty[stage]), phase ^ 1u, abort_flag,
                                   p.status)) {
              ok = false;
              break;
            }
            const uint32_t fb = mapa_shared(smem_u32(&st.full[stage]), 0);
            const uint32_t sa = sbase + stage * STAGE_BYTES;
            const int c = kb * BK;
            // the even CTA's barrier counts the bytes of both CTAs' loads
            if (leader)
              mbar_arrive_expect_tx(smem_u32(&st.full[stage]), 2 * (A_BYTES + half * BK));
            if (kMN) {
              tma_load_3d_pair(sa, &maps.weights, fb, n0, c, it.e);
            } else {
              tma_load_3d_pair(sa, &maps.weights, fb, c, n0, it.e);
              if (kGated)
                tma_load_3d_pair(sa + A_BYTES / 2, &maps.weights, fb, c, p.F + n0, it.e);
            }
            // few boxes: each costs this thread about 100 cycles of a step's 520
            int i = 0;
#pragma unroll
            for (int k = 0; k < kBoxes; ++k) {
              if (half & (BM >> k)) {
                tma_load_2d_pair(sa + A_BYTES + i * BK, &maps.tokens[k], fb, c, r0 + i);
                i += BM >> k;
              }
            }
            used |= 1u << stage;
            last_phase = (last_phase & ~(1u << stage)) | (phase << stage);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        // Before the CTA may exit, the pair's MMAs must have consumed (and so
        // the loads must have landed in) every stage this producer filled.
        for (int s = 0; s < kStages; ++s)
          if (used & (1u << s)) {
            if (leader)
              (void)mbar_wait_bounded(smem_u32(&st.full[s]), (last_phase >> s) & 1u, nullptr,
                                      p.status);
            (void)mbar_wait_bounded(smem_u32(&st.empty[s]), (last_phase >> s) & 1u, nullptr,
                                    p.status);
          }
      }
    } else if (warp == 1) {
      if (leader) {
        // ------------------------------------------ MMA issuer (even CTA)
        // The whole warp runs the loop and one lane issues. All of TMEM is
        // ours, so it starts at column 0.
        int stage = 0, buf = 0;
        uint32_t phase = 0, buf_phase = 0;
        bool ok = tmem_base == 0;
        // One group of 128 channels: the MN-major leading offset is not used.
        // Of a descriptor only the address, in the lower half, changes.
        const uint64_t wdesc = make_sdesc(sbase, kMN ? A_BYTES : 16, 1024);
        const uint64_t tdesc = make_sdesc(sbase + A_BYTES, 16, 1024);
        constexpr uint32_t kWStep = (kMN ? 32 * BM : 32) >> 4, kTStep = 32 >> 4;
        // waits end in a vote: what depends on them stays in uniform registers
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
          return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(bar), parity, abort_flag,
                                                           p.status)) != 0;
        };
        const auto run = [&](auto few, uint32_t idesc) {
          constexpr bool kFew = decltype(few)::value;
          const uint64_t a = kFew ? wdesc : tdesc, b = kFew ? tdesc : wdesc;
          constexpr uint32_t kA = kFew ? kWStep : kTStep, kB = kFew ? kTStep : kWStep;
          const uint32_t a_hi = static_cast<uint32_t>(a >> 32);
          const uint32_t b_hi = static_cast<uint32_t>(b >> 32);
          for (int kb = 0; kb < KB; ++kb) {
            if (!wait(&st.full[stage], phase)) return false;
            if (!wait(&st.tempty[buf], buf_phase ^ 1u)) return false;
            tc_fence_after();
            const uint32_t at = stage * (STAGE_BYTES >> 4);
            const uint32_t a_lo = static_cast<uint32_t>(a) + at;
            const uint32_t b_lo = static_cast<uint32_t>(b) + at;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < BK / 32; ++kk)
                tc_mma_f8_pair(buf * BN, a_lo + kk * kA, a_hi, b_lo + kk * kB, b_hi, idesc,
                               kk != 0);
              tc_commit_pair_mc(smem_u32(&st.tfull[buf]), kPairMask);
              tc_commit_pair_mc(smem_u32(&st.empty[stage]), kPairMask);
            }
            __syncwarp();
            buf ^= 1;
            if (buf == 0) buf_phase ^= 1u;
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          return true;
        };
        Item it;
        ItemReader items;
        while (ok && items.next(st, it, true, lane == 0, abort_flag, p.status)) {
          // a reduction, for its result is in a uniform register
          const int n = __reduce_max_sync(0xFFFFFFFFu, it.cols);
          if (__any_sync(0xFFFFFFFFu, it.few))
            ok = run(std::true_type{}, idesc_f8(n, kMN, false));
          else
            ok = run(std::false_type{}, idesc_f8(BN, false, kMN));
        }
        // All MMAs of the pair must retire before TMEM is freed.
        if (elect_one()) {
          tc_commit_pair(smem_u32(&st.mma_done));
          (void)mbar_wait_bounded(smem_u32(&st.mma_done), 0, nullptr, p.status);
        }
        __syncwarp();
      }
    } else if (warp == kItemWarp) {
      if (lane == 0) {
        // ---------------------------------------------------- work items
        int slot = 0;
        uint32_t phase = 0;
        for (int i = first;; i += step) {
          Item it{0, 0, 0, -1, 0, 0};
          if (i < total) it = item_of(i, p, st);
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
    } else {
      // ------------------------------------------------------------ scales
      grid_dependency_wait();  // the quantiser's scales
      // Loaded kAhead steps ahead of their use: their latency is 1000 cycles and more.
      struct Ahead {
        float s[BM / 32];
        float t[4];  // of 64 channels each; few tokens: two
      };
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      Item it;
      ItemReader items;
      while (ok && items.next(st, it, true, lane == 0, abort_flag, p.status)) {
        const int h = static_cast<int>(crank);
        const bool few = it.few != 0;
        const int own = few ? 0 : h * BM;  // first token
        const int most = (kGated ? 2 * p.F : p.width) - 1;
        const float* t = p.T + static_cast<long long>(it.e) * p.t_expert;
        const float* ts[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          int n;
          if (few)  // this CTA's halves of 64
            n = kGated ? (k & 1) * p.F + it.nt * BM + h * (BM / 2)
                       : it.nt * 2 * BM + h * BM + (k & 1) * (BM / 2);
          else
            n = kGated ? (k >> 1) * p.F + it.nt * BM + (k & 1) * (BM / 2)
                       : it.nt * 2 * BM + k * (BM / 2);
          // channels that do not exist are zeros in the tile, or past F another
          // half's, and are not stored: any scale will do
          ts[k] = t + static_cast<long long>(min(n, most) / kF8Block) * p.t_chan;
        }
        const auto load = [&](int kb, Ahead& a) {
          if (kb >= KB) return;
          const float* s = p.S + static_cast<long long>(kb) * p.R_cap + it.row0 + own;
#pragma unroll
          for (int j = 0; j < BM / 32; ++j) {
            const int i = 32 * j + lane;
            // plain loads: the quantiser writes while this kernel already runs
            a.s[j] = own + i < it.rows ? s[i] : 0.0f;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < 2 || !few) a.t[k] = __ldg(ts[k] + static_cast<long long>(kb) * p.t_red);
        };
        const auto put = [&](int kb, const Ahead& a) {
          if (!ok || kb >= KB) return;
          if (!mbar_wait_bounded(smem_u32(&st.scale_empty[slot]), phase ^ 1u, abort_flag,
                                 p.status)) {
            ok = false;
            return;
          }
          float* to = reinterpret_cast<float*>(smem + kScaleAt + slot * kScaleBytes);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= 2 && few) break;
#pragma unroll
            for (int j = 0; j < BM / 32; ++j) to[k * BM + 32 * j + lane] = a.s[j] * a.t[k];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&st.scale_full[slot]));
          if (++slot == kScales) {
            slot = 0;
            phase ^= 1u;
          }
        };
        constexpr int kAhead = Regs<MODE>::kAhead;
        Ahead a[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) load(j, a[j]);
        for (int kb = 0; kb < KB && ok; kb += kAhead) {
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            put(kb + j, a[j]);
            load(kb + j + kAhead, a[j]);
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<MODE>::kMany));
    // ---------------------------------------------------- sums and epilogue
    const int q = warp & 3;
    const int group = (warp - kFirstSum) >> 2;
    const int half = q >> 1;  // of the CTA's channels
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    uint8_t* staging = smem + kStagingAt + (warp - kFirstSum) * kWarpStaging;
    Outbox box;
    box.at = staging;
    int h1_chunks = 0;  // gated gradient: the item's chunks
    bool h1_pending = false;
    uint32_t h1_phase = 0;
    const uint32_t tempty = mapa_shared(smem_u32(&st.tempty[0]), 0);
    // What these warps wait for each other at: a barrier that a warp whose wait
    // ran out does not leave the others in.
    const uint32_t meet = smem_u32(kGated ? &st.pair[group][q & 1] : &st.group[group]);
    uint32_t meet_phase = 0;
    const auto met = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(meet);
      const bool in_time = mbar_wait_bounded(meet, meet_phase, abort_flag, p.status);
      meet_phase ^= 1u;
      return in_time;
    };
    int slot = 0, buf = 0;
    uint32_t slot_phase = 0, buf_phase = 0;
    bool ok = true;
    Item it;
    ItemReader items;
    const auto scales_there = [&]() {
      ok = mbar_wait_bounded(smem_u32(&st.scale_full[slot]), slot_phase, abort_flag, p.status);
      return reinterpret_cast<const float*>(smem + kScaleAt + slot * kScaleBytes);
    };
    const auto scales_read = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&st.scale_empty[slot]));
      if (++slot == kScales) {
        slot = 0;
        slot_phase ^= 1u;
      }
    };
    const auto sums_there = [&]() {
      ok = mbar_wait_bounded(smem_u32(&st.tfull[buf]), buf_phase, abort_flag, p.status);
      tc_fence_after();
      return lanes + buf * BN;
    };
    // they are in registers: the next MMAs may have the buffer
    const auto sums_read = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(tempty + 8 * buf);
      buf ^= 1;
      if (buf == 0) buf_phase ^= 1u;
    };
    while (ok && items.next(st, it, true, lane == 0, abort_flag, p.status)) {
      if (it.few == 0) {
        // Lane: token; registers: 128 channels of the CTA `group`, in four
        // chunks of 32; gated forward: 64 gate values, then their up values.
        if constexpr (MODE == kGradGated) {
          // H1 of the first two chunks into the idle buffers while the products
          // run: the epilogue read it from memory chunk by chunk, 13 us an item
          const int row = it.row0 + static_cast<int>(crank) * BM + q * 32;
          const int ch = it.nt * 2 * BM + group * BM;
          h1_chunks = row < it.row0 + it.rows ? max(0, min(kChunks, (p.width - ch) / 32)) : 0;
          if (h1_chunks > 0) {
            box.drain();
            if (lane == 0) {
              const uint32_t bar = smem_u32(&st.h1_full[warp - kFirstSum]);
              fence_proxy_async();
              mbar_arrive_expect_tx(bar, kWarpStaging);  // widths are multiples of 64
              for (int c = 0; c < 2; ++c) {
                const uint32_t to = smem_u32(staging) + c * (kWarpStaging / 2);
                tma_load_2d(to, &maps.h1, bar, ch + 32 * c, row);
                tma_load_2d(to + kWarpStaging / 4, &maps.h1, bar, p.F + ch + 32 * c, row);
              }
            }
            h1_pending = true;
          }
        }
        float acc[kChunks][32];
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[c][i] = 0.0f;
        for (int kb = 0; kb < KB; ++kb) {
          // the token's scales for either 64 channels
          const float* own = scales_there() + q * 32 + lane;
          if (!ok) break;
          const float s[2] = {own[(kGated ? group : 2 * group) * BM],
                              own[(kGated ? 2 + group : 2 * group + 1) * BM]};
          scales_read();
          const uint32_t from = sums_there() + BM * group;
          if (!ok) break;
          // The buffer is free as soon as the last loads are done. The branch
          // between the halves keeps the second one's loads behind the first
          // one's sums: moved ahead, they spilled them.
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            uint32_t v0[32], v1[32];
            tmem_ld32_start(from + 64 * hb, v0);
            tmem_ld32_start(from + 64 * hb + 32, v1);
            tmem_wait(v0);
            tmem_wait(v1);
            if (hb == 1) sums_read();
            add_scaled(acc[2 * hb], v0, s[hb]);
            add_scaled(acc[2 * hb + 1], v1, s[hb]);
            if (hb == 0 && *abort_flag) ok = false;
            if (!ok) break;
          }
          if (!ok) break;
        }
        if (!ok) break;
        const int lane = lane_here();
        const int row = it.row0 + static_cast<int>(crank) * BM + q * 32;  // the warp's first
        const int have = it.row0 + it.rows - row;
        const bool there = lane < have;
        if constexpr (kGated) {
          const int ch = it.nt * BM + group * 64;
          const int cols = p.width - ch;
          if (p.H1_save != nullptr) {
            send_wide(box, &maps.h1, acc[0], acc[1], p.H1_save, 2LL * p.F, row, ch, have, cols);
            send_wide(box, &maps.h1, acc[2], acc[3], p.H1_save, 2LL * p.F, row, p.F + ch, have,
                      cols);
          }
          const float w = p.row_scale != nullptr && there ? __ldg(p.row_scale + row + lane) : 1.0f;
          const float2 w2 = make_float2(w, w), to_exp = exp_factor(p.alpha);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 g = make_float2(acc[c][i], acc[c][i + 1]);
              const float2 u = make_float2(acc[2 + c][i], acc[2 + c][i + 1]);
              *reinterpret_cast<float2*>(&acc[c][i]) =
                  __fmul2_rn(__fmul2_rn(__fmul2_rn(g, sigmoid2(g, to_exp)), u), w2);
            }
          send_wide(box, &maps.out, acc[0], acc[1], p.C, p.width, row, ch, have, cols);
        } else if constexpr (MODE == kGradGated) {
          const float w = p.row_scale != nullptr && there ? __ldg(p.row_scale + row + lane) : 1.0f;
          float2 dot = make_float2(0.0f, 0.0f);
          const float2 w2 = make_float2(w, w), alpha2 = make_float2(p.alpha, p.alpha);
          const float2 to_exp = exp_factor(p.alpha);
          const int ch0 = it.nt * 2 * BM + group * BM;
          const gg_bf16* h1 = p.H1 + static_cast<long long>(row) * (2LL * p.F) + ch0;
          if (h1_chunks > 0) {
            if (!(ok = mbar_wait_bounded(smem_u32(&st.h1_full[warp - kFirstSum]), h1_phase,
                                         abort_flag, p.status)))
              break;
            h1_phase ^= 1u;
            h1_pending = false;
          }
          uint4 rg[4], ru[4];  // a later chunk's rows as loads bring them
          if (h1_chunks > 2) {
            load_chunk_raw(rg, h1 + 64, 2LL * p.F, have);
            load_chunk_raw(ru, h1 + p.F + 64, 2LL * p.F, have);
          }
          box.turn = 0;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const int ch = ch0 + 32 * c;
            if (c >= h1_chunks) continue;
            // gate and up rows lie in a buffer's halves, and are replaced there
            // by their gradients
            uint4* gs = box.open();
            uint4* us = gs + 32 * 4;
            if (c >= 2) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int to = stage_slot(8 * j + (lane >> 2), lane & 3);
                gs[to] = rg[j];
                us[to] = ru[j];
              }
              __syncwarp();
              if (c == 2 && h1_chunks > 3) {
                load_chunk_raw(rg, h1 + 96, 2LL * p.F, have);
                load_chunk_raw(ru, h1 + p.F + 96, 2LL * p.F, have);
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int own = stage_slot(lane, k);
              uint4 g = gs[own], u = us[own];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t& gw = (&g.x)[i];
                uint32_t& uw = (&u.x)[i];
                float2 dg, du;
                glu_grad2(make_float2(acc[c][8 * k + 2 * i], acc[c][8 * k + 2 * i + 1]), w2,
                          make_float2(bf16_lo(gw), bf16_hi(gw)),
                          make_float2(bf16_lo(uw), bf16_hi(uw)), alpha2, to_exp, dg, du, dot);
                gw = pack_bf16x2(dg.x, dg.y);
                uw = pack_bf16x2(du.x, du.y);
              }
              gs[own] = g;
              us[own] = u;
            }
            if (have >= 32) {
              fence_proxy_async();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d(&maps.out, smem_u32(gs), ch, row);
                tma_store_2d(&maps.out, smem_u32(us), p.F + ch, row);
                end_group();
              }
            } else {
              __syncwarp();
              gg_bf16* to = p.C + static_cast<long long>(row) * (2LL * p.F) + ch;
              for (int j = 0; j < 4; ++j) {
                const int i = 8 * j + (lane >> 2);
                if (i < have) {
                  reinterpret_cast<uint4*>(to + i * (2LL * p.F))[lane & 3] =
                      gs[stage_slot(i, lane & 3)];
                  reinterpret_cast<uint4*>(to + i * (2LL * p.F) + p.F)[lane & 3] =
                      us[stage_slot(i, lane & 3)];
                }
              }
              __syncwarp();
              if (lane == 0) end_group();
            }
          }
          // the group's 128 channels are one block of the row sums
          if (p.rowdot != nullptr && there)
            p.rowdot[static_cast<long long>(row + lane) * p.rowdot_stride + 2 * it.nt + group] =
                dot.x + dot.y;
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int ch = it.nt * 2 * BM + group * BM + c * 64;
            send_wide(box, &maps.out, acc[2 * c], acc[2 * c + 1], p.C, p.width, row, ch, have,
                      p.width - ch);
          }
        }
        continue;
      }
      // Few tokens. Lane: channel; registers: tokens, in chunks [mine0, mine0 + mine).
      const int at = lane_here();
      float* stg = reinterpret_cast<float*>(staging);
      const float* other = reinterpret_cast<const float*>(
          smem + kStagingAt + ((warp - kFirstSum) ^ 2) * kWarpStaging);
      const int chunks = it.cols / 32;
      const int mine0 = group == 0 ? 0 : (chunks + 1) / 2;
      const int mine = group == 0 ? (chunks + 1) / 2 : chunks / 2;
      float acc[kFewTokens / 64][32];
#pragma unroll
      for (int c = 0; c < kFewTokens / 64; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[c][i] = 0.0f;
      // a loop for each number of chunks: loads under a condition made v live
      // over the whole kernel, and spilled the other loop's sums
      const auto add_steps = [&](auto of) {
        constexpr int kMine = decltype(of)::value;
        for (int kb = 0; kb < KB; ++kb) {
          const float4* f =
              reinterpret_cast<const float4*>(scales_there() + half * BM + 32 * mine0);
          if (!ok) break;
          const uint32_t from = sums_there() + 32 * mine0;
          if (!ok) break;
          uint32_t v[kMine + 1][32];
#pragma unroll
          for (int c = 0; c < kMine; ++c) tmem_ld32_start(from + 32 * c, v[c]);
#pragma unroll
          for (int c = 0; c < kMine; ++c) tmem_wait(v[c]);
          sums_read();
#pragma unroll
          for (int c = 0; c < kMine; ++c) {
            if (kMN && c >= mine) continue;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 s = f[8 * c + i / 4];
              float2* to = reinterpret_cast<float2*>(&acc[c][i]);
              const uint32_t* x = &v[c][i];
              to[0] = __ffma2_rn(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                                 make_float2(s.x, s.y), to[0]);
              to[1] = __ffma2_rn(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])),
                                 make_float2(s.z, s.w), to[1]);
            }
          }
          scales_read();
        }
      };
      // (gradients: one loop, for three made the one of many tokens slower: gated,
      // 131072 rows, 2048 x 768, 352 us instead of 339)
      if (kMN || mine == 2)
        add_steps(std::integral_constant<int, 2>{});
      else if (mine == 1)
        add_steps(std::integral_constant<int, 1>{});
      else
        add_steps(std::integral_constant<int, 0>{});
      if (!ok) break;
      box.drain();
      // Chunk by chunk through the warp's staging buffer, token i's 16-byte
      // piece s at s ^ (i & 7): a lane then has channels 8 (lane % 4) .. + 7 of
      // tokens 8 j + lane / 4.
      const int ch0 = kGated ? it.nt * BM + static_cast<int>(crank) * (BM / 2) + (q & 1) * 32
                             : it.nt * 2 * BM + static_cast<int>(crank) * BM + q * 32;
      const bool exists = ch0 < p.width;  // 32 channels exist together: multiples of 64
      const int ch = ch0 + 8 * (at & 3);
      const auto read8 = [&](const float* from, int i, float(&x)[8]) {
        const float4* row = reinterpret_cast<const float4*>(from + 32 * i);
        const int s = 2 * (at & 3);
        const float4 a = row[s ^ (i & 7)], b = row[(s + 1) ^ (i & 7)];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
      };
#pragma unroll
      for (int c = 0; c < kFewTokens / 64; ++c) {
        if (c >= mine || !ok) continue;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          stg[32 * i + (((at >> 2) ^ (i & 7)) << 2) + (at & 3)] = acc[c][i];
        const int t0 = 32 * (mine0 + c);
        if constexpr (kGated) {
          // gate and up rows' warps (two lane quadrants apart) take half the
          // chunk's tokens each, from both buffers
          if (!(ok = met())) continue;
          const float* gates = q < 2 ? stg : other;
          const float* ups = q < 2 ? other : stg;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int i = 16 * half + 8 * j + (at >> 2);
            if (exists && t0 + i < it.rows) {
              float g[8], u[8], v[8];
              read8(gates, i, g);
              read8(ups, i, u);
              const long long r = static_cast<long long>(it.row0) + t0 + i;
              const bool scaled = p.row_scale != nullptr;
              const float w = scaled ? __ldg(p.row_scale + r) : 1.0f;
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] = glu_mul(g[k], u[k], p.alpha, scaled, w);
              *reinterpret_cast<uint4*>(p.C + r * p.width + ch) = pack8(v);
              if (p.H1_save != nullptr) {
                gg_bf16* h1 = p.H1_save + r * (2LL * p.F) + ch;
                *reinterpret_cast<uint4*>(h1) = pack8(g);
                *reinterpret_cast<uint4*>(h1 + p.F) = pack8(u);
              }
            }
          }
          ok = met();
        } else {
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = 8 * j + (at >> 2);
            const bool there = exists && t0 + i < it.rows;
            const long long r = static_cast<long long>(it.row0) + t0 + i;
            float v[8];
            read8(stg, i, v);
            if constexpr (MODE == kGradGated) {
              float dot = 0.0f;
              if (there) {
                const gg_bf16* h1 = p.H1 + r * (2LL * p.F) + ch;
                const uint4 gw = __ldg(reinterpret_cast<const uint4*>(h1));
                const uint4 uw = __ldg(reinterpret_cast<const uint4*>(h1 + p.F));
                const float w = p.row_scale != nullptr ? __ldg(p.row_scale + r) : 1.0f;
                const uint32_t gx[4] = {gw.x, gw.y, gw.z, gw.w};
                const uint32_t ux[4] = {uw.x, uw.y, uw.z, uw.w};
                float dg[8], du[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const float g = k & 1 ? bf16_hi(gx[k / 2]) : bf16_lo(gx[k / 2]);
                  const float u = k & 1 ? bf16_hi(ux[k / 2]) : bf16_lo(ux[k / 2]);
                  glu_grad(v[k], w, g, u, p.alpha, dg[k], du[k], dot);
                }
                gg_bf16* to = p.C + r * (2LL * p.F) + ch;
                *reinterpret_cast<uint4*>(to) = pack8(dg);
                *reinterpret_cast<uint4*>(to + p.F) = pack8(du);
              }
              dot += __shfl_xor_sync(0xFFFFFFFFu, dot, 1);
              dot += __shfl_xor_sync(0xFFFFFFFFu, dot, 2);
              if ((at & 3) == 0) st.dots[group][q][32 * c + i] = dot;
            } else {
              if (there) *reinterpret_cast<uint4*>(p.C + r * p.width + ch) = pack8(v);
            }
          }
          __syncwarp();
        }
      }
      if constexpr (MODE == kGradGated) {
        if (p.rowdot != nullptr) {
          // the CTA's 128 channels are one block of the row sums
          if (!(ok = met())) break;
          const int i = 32 * mine0 + 32 * q + lane;
          if (q < mine && i < it.rows) {
            const auto& d = st.dots[group];
            const int own = 32 * q + lane;
            const float sum = (d[0][own] + d[1][own]) + (d[2][own] + d[3][own]);
            p.rowdot[(static_cast<long long>(it.row0) + i) * p.rowdot_stride + 2 * it.nt +
                     static_cast<int>(crank)] = sum;
          }
          ok = met();
        }
      }
    }
    // (after an abort) H1 that is still on its way to shared memory
    if (h1_pending)
      (void)mbar_wait_bounded(smem_u32(&st.h1_full[warp - kFirstSum]), h1_phase, nullptr,
                              p.status);
  }

  // (after an abort) no load of TMEM is under way when it is freed
  if (warp >= kFirstSum) asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  // shared memory stays until the last stores have read it
  if (warp >= kFirstSum && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
  cluster_sync();
}

template <int MODE>
cudaError_t launch_f8_t(const F8Maps& maps, const F8Params& p, bool early, const DeviceInfo& dev,
                        cudaStream_t stream) {
  static std::atomic<int> resident[kMaxDevices];
  // no more clusters than there can be work items
  const long long items =
      (static_cast<long long>(p.R_cap) / BN + (p.R_cap < p.E ? p.R_cap : p.E)) * p.NT;
  const int most = static_cast<int>(items < 1 ? 1 : (items < 0x7FFFFFFF ? items : 0x7FFFFFFF));
  return launch_pairs_early(early, f8_gemm_kernel<MODE>, resident, kThreads, kSmemBytes, most, dev,
                            stream, maps, p);
}

}  // namespace

cudaError_t launch_f8_gemm(const F8GemmArgs& a, bool early, const DeviceInfo& dev,
                           cudaStream_t stream) {
  const int red = a.grad ? a.N : a.K;
  const int out = a.grad ? a.K : a.N;
  F8Maps maps;
  const cuuint64_t td[2] = {static_cast<cuuint64_t>(red), static_cast<cuuint64_t>(a.R_cap)};
  const cuuint64_t ts[1] = {static_cast<cuuint64_t>(red)};
  for (int i = 0; i < kBoxes; ++i) {
    const cuuint32_t tbox[2] = {BK, static_cast<cuuint32_t>(BM) >> i};
    if (!encode_map(&maps.tokens[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, a.A, 2, td, ts, tbox,
                    CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  const cuuint64_t wd[3] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.N),
                            static_cast<cuuint64_t>(a.E)};
  const cuuint64_t ws[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.K) * a.N};
  // 128 channels x 128 codes (gated forward 64); gradient: 128 rows of 128 channels
  const cuuint32_t wbox[3] = {BK, !a.grad && a.alpha != 0.0f ? 64u : 128u, 1};
  if (!encode_map(&maps.weights, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.B, 3, wd, ws, wbox,
                  CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  // results, in pieces of 32 rows
  const bool gated = a.alpha != 0.0f;
  const bool narrow = a.grad && gated;
  const cuuint64_t width = narrow ? 2ull * a.K : a.grad ? a.K : gated ? a.N / 2 : a.N;
  const cuuint64_t od[2] = {width, static_cast<cuuint64_t>(a.R_cap)};
  const cuuint64_t os[1] = {2 * width};
  const cuuint32_t obox[2] = {narrow ? 32u : 64u, 32u};
  if (!encode_map(&maps.out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.C, 2, od, os, obox,
                  narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  maps.h1 = maps.out;
  if (narrow && !encode_map(&maps.h1, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.H1, 2, od, os, obox,
                            CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  if (a.H1_save != nullptr) {
    const cuuint64_t hd[2] = {static_cast<cuuint64_t>(a.N), static_cast<cuuint64_t>(a.R_cap)};
    const cuuint64_t hs[1] = {2ull * a.N};
    if (!encode_map(&maps.h1, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.H1_save, 2, hd, hs, obox,
                    CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  const int NB = (a.N + kF8Block - 1) / kF8Block, KB = (a.K + kF8Block - 1) / kF8Block;
  F8Params p{};
  p.offsets = a.offsets;
  p.E = a.E;
  p.R_cap = a.R_cap;
  p.red = red;
  p.S = a.As;
  p.T = a.Bs;
  p.t_expert = NB * KB;
  p.t_chan = a.grad ? 1 : KB;
  p.t_red = a.grad ? KB : 1;
  p.row_scale = a.row_scale;
  p.alpha = a.alpha;
  p.C = a.C;
  p.H1_save = a.H1_save;
  p.H1 = a.H1;
  p.rowdot = a.rowdot;
  p.status = a.status;
  if (!a.grad && gated) {
    p.F = a.N / 2;
    p.width = p.F;
    p.NT = (p.F + BM - 1) / BM;
    return launch_f8_t<kFwdGated>(maps, p, early, dev, stream);
  }
  p.width = out;
  p.NT = (out + 2 * BM - 1) / (2 * BM);
  if (!a.grad) return launch_f8_t<kFwd>(maps, p, early, dev, stream);
  if (!gated) return launch_f8_t<kGrad>(maps, p, early, dev, stream);
  p.F = a.K;
  p.rowdot_stride = (2 * p.NT + 7) / 8 * 8;
  return launch_f8_t<kGradGated>(maps, p, early, dev, stream);
}

}  // namespace gg
