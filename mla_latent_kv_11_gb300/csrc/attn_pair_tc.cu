// Windowed attention on the tensor cores (tcgen05 + TMEM + TMA): split-KV decode and
// causal prefill limited to a sliding window and sinks, bf16, kv_lora_rank 512, rope 64
// or 0, up to 128 heads.
//
// Mathematics. A query at position p attends the rows t <= p with t < sinks or
// t > p - window. Rows come in blocks of 64; a row tile's visible blocks are those of
// the sinks and those of the window, listed one behind the other and taken two at a time.
// One pass with the running maximum and sum of a softmax: m the reference maximum (raised
// only when a tile's maximum exceeds it by more than 8 in base 2, so P stays below 2^8),
// l = sum of the float32 weights, O += bf16(P) V in float32. The weights' rounding to bf16
// is the only rounding between the inputs and the output's own: the tensor cores take them
// no wider. l sums them unrounded, so that the log-sum-exp is float32's; an output that one key
// dominates is off by its weight's rounding then, up to 2^-8 of itself, which the sum of the
// rounded weights would cancel there and carry into the log-sum-exp instead.
//
// Tile. 128 query rows (heads of one token, or several tokens' heads) x 128 keys, by a
// cluster of two CTAs. The rows are split: each CTA owns 64 of them, so that its output
// accumulator, 64 x 512 float32, takes half its tensor memory and every row's scores lie
// whole in one CTA (nothing is exchanged between the two). Each MMA is a
// cta_group::2 MMA with M = 128: it takes its A rows from both CTAs and half of B from
// each, at the full rate of both SMs (measured: 32 cycles for N = 128, K = 16, 64 for
// N = 256; with 64-key tiles, N = 64, shared memory bounds it to 26 instead of 16).
// Tensor memory per CTA (row r in lanes r and r + 64):
//   O  [0, 256): lane r columns 0..255 of the row, lane r + 64 columns 256..511
//   S  [256, 320) and [320, 384), of even and odd tiles: lane r keys 0..63, lane r + 64 keys 64..127
//   the finished output [384, 512): as O, bf16 pairs
//
// Shared memory per CTA: Q 64 x 576 (72 KB), P 64 x 128 (16 KB), two key tiles of 64 KB and
// one rope box of 8 KB. Q K^T needs, in each CTA, its 64 keys' whole rows (boxes H0: latent
// columns 0..255, H1: 256..511, R: rope); P V needs all 128 keys' columns of its half. CTA r
// keeps H_r of its keys for both; the other half is done with after Q K^T, and the other
// CTA's keys' columns (box W) are loaded into its place. So a cache row crosses HBM once and
// L2 1.44 times, and keys 64k .. 64k + 63 sit in H_k of both CTAs when P V runs.
//
// Order on the tensor pipe: QK(g+1), PV(g), so the softmax of tile g runs under QK(g+1);
// at a row tile's end PV comes first. 384 threads: warps 0 and 2 load the keys, a quarter (two column
// groups) a barrier, warp 3 the W boxes, rope and queries (TMA; with one warp for all, issuing the
// loads took longer than the MMAs); warp 1 of the first CTA issues every MMA; warp 2 owns the tensor
// memory; warps 4..11 run the softmax, the rescaling of O and the epilogue, two threads a lane. A row
// tile's output is parked in tensor memory as bf16 and stored under the next tiles' MMAs, in whole
// lines: its 64 KB take an SM 2100 cycles at its 31 bytes a cycle.
//
// Work. A row tile's key tiles are cut over the clusters where that shortens the longest one's list
// (window_sched.cu); the pieces' float32 outputs and log-sum-exps are joined by a second kernel.
//
// What bounds it and what it measured (152 SMs, 76 clusters; device times of replayed graphs):
//   prefill of 4 x 1024 tokens, 128 heads, window 2048: 1.40 ms, 1.6 PFLOP/s, in a short run, 84% of a
//     dense library product's rate; 1.5 ms a call, 1.45 PFLOP/s, under the power cap. A tile takes some
//     3200 cycles a cluster, its MMAs 2176 of them. Shared memory holds two tiles of keys, so the next
//     but one waits for PV to leave its place, for its load (1400 cycles: the 64 KB a CTA come at 50
//     bytes a cycle), for its QK, which PV then follows.
//   decode of 64 sequences of 1K to 16K rows, 128 heads, window 4096: 69.4 us, 4.2 TB/s; 6 TB/s between
//     a start of 11 us (schedule, first loads) and the last outputs.
//   prefill of ragged prompts, 64 heads, window 777: 106 us for 82 GFLOP, bounded by what a row tile
//     costs beside its 1 to 8 tiles (its queries' load, the pipeline's filling, its output: 4500 cycles
//     against 2350 a tile).
//   7 tokens over 16K rows, 128 heads: 37 us for 31 GFLOP: 11 to 12 tiles a cluster, the rest schedule,
//     start, float32 pieces and their merge.
//
// Every wait is bounded; one that gives up winds both CTAs down and is reported.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>
#include <mutex>
#include <vector>

#include "mla_internal.h"
#include "sm100_ptx.cuh"
#include "window_sched.cuh"

namespace mla {
namespace {

using namespace ptx;

__device__ unsigned g_pair_err = 0;

// a block of 64 cache rows (kBlk): the keys of one CTA
constexpr int kTileKeys = 2 * kBlk;          // keys per tile
constexpr int kBox = kBlk * 128;             // 64 rows x 64 bf16 columns, 128-byte swizzle
constexpr int kThreads = 384;
constexpr int kSoftmaxWarp0 = 4;
constexpr int kSoftmaxThreads = 256;
constexpr int kSoftmaxBar = 1;
constexpr float kLazyRescale = 8.f;
constexpr uint32_t kTmemS = 256, kTmemOut = 384, kTmemCols = 512;

template <int kRope>
struct PairCfg {
  static constexpr int kQBoxes = 8 + (kRope ? 1 : 0);
  static constexpr int kOffQ = 0;
  static constexpr int kOffP = kQBoxes * kBox;
  static constexpr int kOffKV = kOffP + 2 * kBox;          // [2 tiles][H0, H1][4 boxes]
  static constexpr int kOffR = kOffKV + 2 * 8 * kBox;
  static constexpr int kOffMisc = kOffR + (kRope ? kBox : 0);
  static constexpr int kMiscBytes = 3 * 1024;
  static constexpr int kSmemAlloc = kOffMisc + kMiscBytes;
};

// Offset of column group c (0..3) of half h of key tile b.
__host__ __device__ constexpr int kv_box(int b, int h, int c) { return (b * 8 + h * 4 + c) * kBox; }

struct PairShared {
  uint64_t full_k[2][4];   // [tile][quarter] first CTA: two boxes of H0 (quarters 0, 1) or H1 of both CTAs
  uint64_t full_r, full_q; // first CTA: the rope box, the queries, of both CTAs
  uint64_t full_w[2];      // own W boxes
  uint64_t s_full[2];      // scores of a tile are in tensor memory (and its Q, R and short half are read)
  uint64_t pv_done[2][4];  // [tile][quarter] the values in the place of that quarter are read; the last:
                           // and P is, O is updated
  uint64_t p_full;         // first CTA: P of both CTAs is written, O rescaled
  uint64_t fin;
  uint32_t tmem_base;
  int abort_flag;
  // exchanges between the four threads of a row, in turn in two places, [columns 0..31 / 32..63 of S]
  // [lane]: the maxima of a tile, at a segment's end the weights' sums
  float red[2][2][128];
};
static_assert(sizeof(PairShared) <= PairCfg<64>::kMiscBytes, "barrier block overflows its slot");

struct PairParams {
  int H, tptc;               // heads, tokens of a row tile per CTA (heads split when H > 64: tptc 0)
  int window, sinks;
  float scale_log2;
  WindowSched sched;
  WindowOut out;             // partial rows of a slot: 64 * CTA + row
  int page, num_blocks;
  const int32_t* block_table;
  int64_t bt_stride;
  int o_32B;                 // output rows lie on 32-byte boundaries: whole sectors a store
  int q_whole;               // the queries' column groups come in one load
  int prefetch;              // bring the tile after the next into L2 (rows come from HBM, each read once)
};


// The walker's next segment for a role that issues from a whole warp: its tiles [first, return
// value), none (0, 0) behind the last. Values that come from memory are not uniform to the compiler,
// and under a branch on them it forms every operand of the MMAs and loads in vector registers (an MMA
// then took 75 cycles to issue, a load 300); the results of a reduction over the warp are.
template <bool kDirect>
__device__ __forceinline__ int open_segment(const WindowSched& sched, Walker<2, kDirect>& wk, Seg& s, int& first) {
  const bool any = wk.next(sched, s, &g_pair_err);
  first = __reduce_max_sync(0xffffffffu, any ? s.t0 : 0);
  return __reduce_max_sync(0xffffffffu, any ? s.t1 : 0);
}

// The wait behind a first look, kept out of line: the roles' loops have to stay in the instruction
// cache together. The timer, slow to read, is read only every 256 looks.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort) {
  uint64_t since = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_test_cluster(bar, parity)) return true;
    if ((i & 255u) == 0) {
      if (*abort) return false;
      const uint64_t now = globaltimer_ns();
      if (since == 0) {
        since = now;
      } else if (now - since > kWaitLimitNs) {
        *abort = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_test_cluster(bar, parity) || wait_slow(bar, parity, abort);
}

// The lowest n bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

__device__ __forceinline__ void alloc_pair(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Four MMAs of the pair (K = 64), issued by the first CTA's converged warp (an elected lane). The
// operands' descriptors are given by their low words, which advance by kAs and kBs 16-byte units; the
// high words (stride 1024, 128-byte swizzle) are constant, so that a descriptor costs one move into
// the uniform registers instead of two. The first MMA replaces D where `fresh`.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
template <uint32_t kAs, uint32_t kBs, uint32_t kIdesc>
__device__ __forceinline__ void umma_pair4(uint32_t d, uint32_t a, uint32_t b, bool fresh) {
  asm volatile(
      "{\n .reg .pred p, t, e;\n .reg .b32 r, x, y;\n .reg .b64 a, b;\n"
      " elect.sync r|e, 0xffffffff;\n setp.eq.b32 p, %3, 0;\n setp.eq.b32 t, 0, 0;\n"
      " mov.b64 a, {%1, %7};\n mov.b64 b, {%2, %7};\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %6, p;\n"
      " add.u32 x, %1, %4;\n add.u32 y, %2, %5;\n mov.b64 a, {x, %7};\n mov.b64 b, {y, %7};\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %6, t;\n"
      " add.u32 x, x, %4;\n add.u32 y, y, %5;\n mov.b64 a, {x, %7};\n mov.b64 b, {y, %7};\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %6, t;\n"
      " add.u32 x, x, %4;\n add.u32 y, y, %5;\n mov.b64 a, {x, %7};\n mov.b64 b, {y, %7};\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %6, t;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"((uint32_t)fresh), "n"(kAs), "n"(kBs), "n"(kIdesc), "n"(kDescHi)
      : "memory");
}
// Low word of a descriptor: address and leading-dimension offset in 16-byte units.
__device__ __forceinline__ uint32_t desc_lo(const void* p, uint32_t lbo) {
  return (smem_u32(p) >> 4) | ((lbo >> 4) << 16);
}
// Arrive on `bar` of both CTAs once every MMA issued so far is complete.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .b32 r;\n elect.sync r|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// The loader's operations, each run by its whole converged warp and issued by an elected lane:
// the operands then stay warp-uniform and a TMA load issues in 28 cycles. Behind a branch on one
// lane it takes 147 (measured), which made the loads the pair's bottleneck.
#define MLA_ELECT "{\n .reg .pred e;\n .reg .b32 r;\n elect.sync r|e, 0xffffffff;\n @e "

__device__ __forceinline__ void expect_bytes(uint64_t* bar, uint32_t bytes) {
  asm volatile(MLA_ELECT "mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(smem_u32(bar)), "r"(bytes)
               : "memory");
}
// Loads into this CTA whose bytes are counted on `bar`, a shared::cluster address (the first CTA's
// barrier).
__device__ __forceinline__ void load_pair_3d(void* dst, const void* map, uint32_t bar, int32_t c0, int32_t c1,
                                             int32_t c2) {
  asm volatile(MLA_ELECT
               "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
               " [%0], [%1, {%3, %4, %5}], [%2];\n}\n" ::"r"(smem_u32(dst)),
               "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
__device__ __forceinline__ void load_pair_4d(void* dst, const void* map, uint32_t bar, int32_t c1, int32_t c2,
                                             int32_t c3) {
  asm volatile(MLA_ELECT
               "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
               " [%0], [%1, {%3, %4, %5, %6}], [%2];\n}\n" ::"r"(smem_u32(dst)),
               "l"(map), "r"(bar), "r"(0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
// The same counted on a barrier of this CTA.
__device__ __forceinline__ void load_own_3d(void* dst, const void* map, uint64_t* bar, int32_t c0, int32_t c1,
                                            int32_t c2) {
  asm volatile(MLA_ELECT
               "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
               " [%0], [%1, {%3, %4, %5}], [%2];\n}\n" ::"r"(smem_u32(dst)),
               "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
__device__ __forceinline__ void load_own_4d(void* dst, const void* map, uint64_t* bar, int32_t c1, int32_t c2,
                                            int32_t c3) {
  asm volatile(MLA_ELECT
               "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
               " [%0], [%1, {%3, %4, %5, %6}], [%2];\n}\n" ::"r"(smem_u32(dst)),
               "l"(map), "r"(smem_u32(bar)), "r"(0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
// Bring a box into L2 without waiting.
__device__ __forceinline__ void prefetch_3d(const void* map, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(MLA_ELECT "cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];\n}\n" ::"l"(map),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
__device__ __forceinline__ void prefetch_4d(const void* map, int32_t c1, int32_t c2, int32_t c3) {
  asm volatile(MLA_ELECT "cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];\n}\n" ::"l"(map),
               "r"(0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
#undef MLA_ELECT

// 32 bytes to a 32-byte aligned address in one store: a whole sector.
__device__ __forceinline__ void st_global_32B(void* dst, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Two float32 in one register pair, and arithmetic on both at once.
__device__ __forceinline__ uint64_t pair_f32(float a, float b) {
  return (uint64_t)__float_as_uint(b) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 16 lanes x 32 columns of tensor memory: w[4 k + 2 j + i] of lane t is row 8 j + t / 4, column
// 8 k + 2 (t % 4) + i.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t addr, uint32_t* w) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]), "=r"(w[8]),
        "=r"(w[9]), "=r"(w[10]), "=r"(w[11]), "=r"(w[12]), "=r"(w[13]), "=r"(w[14]), "=r"(w[15])
      : "r"(addr));
}

// kSmall: pages of less than 64 rows. kDirect: a direct schedule.
template <int kRope, bool kSmall, bool kDirect>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    window_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap qmap,
                       const PairParams p) {
  using C = PairCfg<kRope>;
  static_assert(C::kSmemAlloc <= 232448, "shared memory beyond the 227 KB a CTA may hold");
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw;
  PairShared& sh = *reinterpret_cast<PairShared*>(smem + C::kOffMisc);
  unsigned char *sQ = smem + C::kOffQ, *sP = smem + C::kOffP, *sKV = smem + C::kOffKV, *sR = smem + C::kOffR;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // clusters are pairs along x; unlike the cluster's own registers blockIdx is uniform to the compiler
  const uint32_t rank = blockIdx.x & 1;
  const int unit = blockIdx.x >> 1, units = gridDim.x >> 1;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      for (int q = 0; q < 4; ++q) {
        mbar_init(&sh.full_k[i][q], 1);
        mbar_init(&sh.pv_done[i][q], 1);
      }
      mbar_init(&sh.full_w[i], 1);
      mbar_init(&sh.s_full[i], 1);
    }
    mbar_init(&sh.full_r, 1);
    mbar_init(&sh.full_q, 1);
    mbar_init(&sh.p_full, 2 * kSoftmaxThreads / 32);   // the softmax warps of both CTAs
    mbar_init(&sh.fin, 1);
    sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) alloc_pair(&sh.tmem_base, kTmemCols);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&kvmap);
    tma_prefetch_desc(&qmap);
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers initialised, both tensor memories allocated
  tc_fence_after();
  pdl_enter();      // queries, cache and schedule come from the kernels before
  constexpr uint32_t tmem = 0;   // all 512 columns are allocated: they begin at 0
  volatile int* abort = &sh.abort_flag;
  auto give_up = [&]() {   // tell both CTAs
    sh.abort_flag = 1;
    const uint32_t remote = map_to_rank(&sh.abort_flag, rank ^ 1u);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(1) : "memory");
  };

  if (warp == 0 || warp == 2 || warp == 3) {
    // ------------------------------------------------------------ loads, in both CTAs: warps 0 and 2 the
    // keys, which the tensor pipe waits for (two quarters of a tile each), warp 3 the rest. The whole
    // warp walks the tiles. Lane h looks up the block id of a tile's block h (small pages: lanes
    // 8h .. 8h + 7 the ids of its pages).
    const int rows_box = kSmall ? p.page : kBlk, subs = kBlk / rows_box;
    Walker<2, kDirect> wk;
    wk.init(p.sched, unit, units, &g_pair_err);
    Seg sg;
    bool ok = true;
    int j = 0, nt = 0;   // next tile of the open segment, its end; both warp-uniform
    bool fresh = true;
    auto open = [&]() {
      nt = open_segment(p.sched, wk, sg, j);
      fresh = true;
    };
    open();
    // a tile to load: this lane's block id (and page row of its block), whether it starts a segment
    struct Tile {
      int id, row;
      bool seen, first;
      int tok0;
    };
    // the next tile: its block id is asked for here and used a tile later (settle)
    auto fetch = [&](Tile& t) -> bool {
      if (j >= nt) return false;
      const int h = kSmall ? (lane >> 3) & 1 : lane & 1;
      const int base = block_row(sg, 2 * j + h);
      const int key = kSmall ? base + (lane & 7) * rows_box : base;
      // a box with rows that some token attends (of a listed block of 64 rows: always)
      t.seen = base >= 0 && lane < (kSmall ? 16 : 2) &&
               (!kSmall || ((lane & 7) < subs && key <= sg.hi && (key < p.sinks || key + rows_box > sg.lo)));
      int page = 0;
      t.row = 0;
      if (t.seen) {
        page = key / kBlk;   // pages of 64 rows: the block itself
        if (p.page != kBlk) {
          page = key / p.page;
          t.row = key - page * p.page;
        }
      }
      t.id = t.seen ? p.block_table[(int64_t)sg.b * p.bt_stride + page] : -1;
      t.first = fresh;
      t.tok0 = sg.tok0;
      fresh = false;
      if (++j == nt) open();
      return true;
    };
    // an id outside the cache, and boxes nobody attends, load from outside the tensor map: zeros
    auto settle = [&](Tile& t) {
      if (t.id < 0 || t.id >= p.num_blocks) {
        if (t.seen) atomicOr(&g_pair_err, kErrDeviceData);
        t.id = p.num_blocks;
      }
    };
    auto wait = [&](uint64_t* bar, int parity) { ok = ok && __all_sync(0xffffffffu, wait_for(bar, parity, abort)); };
    // column groups c .. c + n - 1 of 64 of block h of a tile, one under the other from dst on; counted
    // on the first CTA's barrier `pair`, or on `own`. Small pages: box by box.
    auto load_small = [&](const Tile& t, int h, int c, int n, unsigned char* dst, uint32_t pair, uint64_t* own) {
#pragma unroll 1
      for (int i = 0; i < subs; ++i) {
        const int id = __shfl_sync(0xffffffffu, t.id, 8 * h + i);
#pragma unroll 1
        for (int k = 0; k < n; ++k) {
          unsigned char* d = dst + k * kBox + i * rows_box * 128;
          if (own != nullptr)
            load_own_3d(d, &kvmap, own, 64 * (c + k), 0, id);
          else
            load_pair_3d(d, &kvmap, pair, 64 * (c + k), 0, id);
        }
      }
    };
    // a tile whose id is settled, the next, and one whose id is on its way
    Tile cur, t1, t2;
    bool have_cur = fetch(cur), have1 = fetch(t1), have2 = fetch(t2);
    if (have_cur) settle(cur);
    if (have1) settle(t1);
    auto advance = [&]() {
      cur = t1;
      t1 = t2;
      have_cur = have1;
      have1 = have2;
      if (have1) settle(t1);
      have2 = fetch(t2);
    };
    if (warp != 3) {
      const uint32_t bar0 = map_to_rank(&sh.full_k[0][0], 0);
#pragma unroll 1
      for (int g = 0; ok && have_cur; ++g) {
        const int b = g & 1;
        const int id = __shfl_sync(0xffffffffu, cur.id, (int)rank), r = __shfl_sync(0xffffffffu, cur.row, (int)rank);
        // a quarter as soon as PV(g - 2) has read what lies there; QK(g) takes them in the same order
#pragma unroll 1
        for (int q = warp >> 1; ok && q < 4; q += 2) {
          if (g > 1) wait(&sh.pv_done[b][q], ((g >> 1) & 1) ^ 1);
          if (!ok) break;
          unsigned char* d = sKV + (8 * b + 2 * q) * kBox;
          const uint32_t bar = bar0 + (4 * b + q) * 8;
          if (kSmall)
            load_small(cur, (int)rank, 2 * q, 2, d, bar, nullptr);
          else
            load_pair_4d(d, &kmap, bar, r, 2 * q, id);
          if (rank == 0) expect_bytes(&sh.full_k[b][q], 2 * 2 * kBox);
        }
        advance();
      }
    } else {
      const uint32_t bar_r = map_to_rank(&sh.full_r, 0), bar_q = map_to_rank(&sh.full_q, 0);
      const int own_h = (int)rank, other = 1 - own_h;
      auto load_rope = [&](const Tile& t) {
        if (kRope == 0) return;
        if (kSmall)
          load_small(t, own_h, 8, 1, sR, bar_r, nullptr);
        else
          load_pair_3d(sR, &kvmap, bar_r, 512, __shfl_sync(0xffffffffu, t.row, own_h),
                       __shfl_sync(0xffffffffu, t.id, own_h));
        if (rank == 0) expect_bytes(&sh.full_r, 2 * kBox);
      };
      auto load_q = [&](const Tile& t) {
        const int hb = min(p.H, 64), toks = max(p.tptc, 1), h0 = p.tptc ? 0 : 64 * (int)rank;
        const int t0 = t.tok0 + p.tptc * (int)rank;
        const int n = p.q_whole ? 1 : C::kQBoxes;
#pragma unroll 1
        for (int c = 0; c < n; ++c) load_pair_4d(sQ + c * kBox, &qmap, bar_q, h0, t0, c);
        if (rank == 0) expect_bytes(&sh.full_q, 2u * C::kQBoxes * hb * toks * 128);
      };
      auto prefetch_keys = [&](const Tile& t) {   // this CTA's keys into L2
        if (kSmall) return;
        const int id = __shfl_sync(0xffffffffu, t.id, own_h), r = __shfl_sync(0xffffffffu, t.row, own_h);
#pragma unroll 1
        for (int c = 0; c < 8; c += 2) prefetch_4d(&kmap, r, c, id);
        if (kRope) prefetch_3d(&kvmap, 512, r, id);
      };
      if (have_cur) {
        load_q(cur);
        load_rope(cur);
      }
      if (have1 && p.prefetch) prefetch_keys(t1);
#pragma unroll 1
      for (int g = 0; ok && have_cur; ++g) {
        const int b = g & 1;
        wait(&sh.s_full[b], (g >> 1) & 1);
        if (!ok) break;
        // QK(g) is done with the rope box, with Q at a segment's end, and with its keys' columns of the
        // other CTA's half: the other CTA's keys' columns of this CTA's half take their place
        if (have1) load_rope(t1);
        unsigned char* d = sKV + kv_box(b, other, 0);
        const int id = __shfl_sync(0xffffffffu, cur.id, other), r = __shfl_sync(0xffffffffu, cur.row, other);
#pragma unroll 1
        for (int c = 0; c < 4; c += 2) {
          if (kSmall)
            load_small(cur, other, 4 * own_h + c, 2, d + c * kBox, 0, &sh.full_w[b]);
          else
            load_own_4d(d + c * kBox, &kmap, &sh.full_w[b], r, 4 * own_h + c, id);
        }
        expect_bytes(&sh.full_w[b], 4 * kBox);
        if (have1 && t1.first) load_q(t1);
        advance();
        if (have1 && p.prefetch) prefetch_keys(t1);
      }
    }
    if (!ok) {
      // copies in flight land within microseconds: wait well beyond that before the CTA ends
      if (lane == 0) {
        give_up();
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
      }
      __syncwarp();
    }
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------ MMA issuer of the pair. Its loops
    // stay loops (four MMAs a round, descriptors advanced by additions): unrolled over a tile they
    // would not stay in the instruction cache beside the other warps' code
    constexpr uint32_t id_qk = idesc_bf16(128, kTileKeys, false, false);
    constexpr uint32_t id_pv = idesc_bf16(128, 256, false, true);
    const uint32_t dq = desc_lo(sQ, 16), dp = desc_lo(sP, 16), dk = desc_lo(sKV, 16), dv = desc_lo(sKV, kBox),
                   dr = desc_lo(sR, 16);
    constexpr int kStep = kBox / 16;   // one box, in a descriptor's 16-byte units
    Walker<2, kDirect> wk;
    wk.init(p.sched, unit, units, &g_pair_err);
    Seg sg;
    int g = 0, seg_i = 0;
    bool ok = true, pv_first = true;   // pv_first: the pending PV starts its segment's O
    // A barrier is looked at before the MMAs that precede its wait are issued, so that the look's
    // latency passes under them; looked at behind them it cost the tensor pipe 80 cycles each time
    bool seen = false;
    auto look = [&](uint64_t* bar, int parity) { seen = mbar_test_cluster(bar, parity); };
    auto wait = [&](uint64_t* bar, int parity) {
      ok = ok && (__all_sync(0xffffffffu, seen) || __all_sync(0xffffffffu, wait_slow(bar, parity, abort)));
      return ok;
    };
    auto qk = [&](int x) {
      const int b = x & 1;
      const uint32_t d = __reduce_max_sync(0xffffffffu, kTmemS + 64 * b);
      const uint32_t k = __reduce_max_sync(0xffffffffu, dk + 8 * b * kStep);
      const int ph = (x >> 1) & 1;
      look(&sh.full_k[b][0], ph);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (!wait(&sh.full_k[b][q], ph)) return;
        tc_fence_after();
        if (q < 3)
          look(&sh.full_k[b][q + 1], ph);
        else if (kRope)
          look(&sh.full_r, x & 1);
#pragma unroll
        for (int i = 2 * q; i < 2 * q + 2; ++i) umma_pair4<2, 2, id_qk>(d, dq + i * kStep, k + i * kStep, i == 0);
      }
      if (kRope) {   // last: the one box that has no second buffer
        if (!wait(&sh.full_r, x & 1)) return;
        tc_fence_after();
        umma_pair4<2, 2, id_qk>(d, dq + 8 * kStep, dr, false);
      }
      commit_pair(&sh.s_full[b]);
    };
    auto pv = [&](int x) {
      const int b = x & 1;
      look(&sh.p_full, b);
      const uint32_t v = __reduce_max_sync(0xffffffffu, dv + 8 * b * kStep);
      if (!wait(&sh.p_full, b)) return;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 4; ++i) {   // keys 64 (i / 2) .., columns 128 (i % 2) .. of each half
        umma_pair4<2, 128, id_pv>(128 * (i & 1), dp + (i >> 1) * kStep, v + 2 * i * kStep, pv_first && i < 2);
        commit_pair(&sh.pv_done[b][i]);
      }
    };
    int t0 = 0, t1 = open_segment(p.sched, wk, sg, t0);
    while (ok && t0 < t1) {
      for (int j = t0; ok && j < t1; ++j, ++g) {
        if (j == t0) {
          if (g > 0) pv(g - 1);
          look(&sh.full_q, seg_i & 1);
          if (!ok || !wait(&sh.full_q, seg_i & 1)) break;
          pv_first = true;
          qk(g);
        } else {
          qk(g);
          if (!ok) break;
          pv(g - 1);
          pv_first = false;
        }
      }
      ++seg_i;
      t1 = open_segment(p.sched, wk, sg, t0);
    }
    if (ok && g > 0) pv(g - 1);
    if (!ok && lane == 0) give_up();
    __syncwarp();
    commit_pair(&sh.fin);
  } else if (warp >= kSoftmaxWarp0) {
    // ------------------------------------------------------------ softmax, rescaling, epilogue: two
    // threads a lane, each with half of the lane's columns
    const int st = tid - kSoftmaxWarp0 * 32;
    const int ln = st & 127, part = st >> 7;            // tensor memory lane; columns of this thread
    const int row = ln & 63, half = ln >> 6;            // this CTA's row; keys (S) and columns (O) of this lane
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t bar_p = map_to_rank(&sh.p_full, 0);
    // the row's token within the tile and its head
    const int tok = p.tptc ? p.tptc * (int)rank + row / p.H : 0;
    const int head = p.tptc ? row % p.H : 64 * (int)rank + row;
    const bool real = p.tptc ? row < p.tptc * p.H : head < p.H;
    auto group_all = [](bool v) { return named_bar_and(kSoftmaxBar, kSoftmaxThreads, v); };
    Walker<2, kDirect> wk;
    wk.init(p.sched, unit, units, &g_pair_err);
    Seg sg;
    // The output that waits in tensor memory: quarters left of this warp's 32 rows x 128 columns, this
    // lane's row. A quarter is 16 rows x 64 columns, whole lines of 128 bytes: an SM stores those at 31
    // bytes a cycle, a sector of 32 a row at 17. The words are parked in the order that gives each lane
    // 32 bytes of a row: lanes 4 a .. 4 a + 3 rows a and a + 8
    int left = 0;
    __nv_bfloat16* to = nullptr;
    auto store_quarter = [&]() {
      const int r = 4 - left--, h = r & 1, c = r >> 1;
      uint32_t w[16];
      tmem_ld_16x32(tmem + lane_addr + ((16u * h) << 16) + kTmemOut + 64 * part + 32 * c, w);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        __nv_bfloat16* const o = reinterpret_cast<__nv_bfloat16*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), 16 * h + 8 * j + (lane >> 2)));
        if (o == nullptr) continue;
        uint32_t y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = w[4 * (k >> 1) + 2 * j + (k & 1)];
        __nv_bfloat16* const d = o + 64 * c + 16 * (lane & 3);
        if (p.o_32B) {
          st_global_32B(d, y);
        } else {
          *reinterpret_cast<uint4*>(d) = make_uint4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4*>(d + 8) = make_uint4(y[4], y[5], y[6], y[7]);
        }
      }
      __syncwarp();
    };
    int g = 0, x = 0;              // x: which of the two places the next exchange between the rows' threads takes
    bool ok = true, mine = true;   // ok: the group's decision; mine: this thread's waits so far
    bool more = wk.next(p.sched, sg, &g_pair_err);
    while (ok && more) {
      const bool valid = real && tok < sg.ntok;
      const int pos = valid ? sg.pos0 + tok : -1;       // -1 attends nothing
      float m = -CUDART_INF_F, l = 0.f;
      for (int j = sg.t0; j < sg.t1; ++j, ++g) {
        const int b = g & 1, ph = (g >> 1) & 1;
        mine = mine && wait_for(&sh.s_full[b], ph, abort);
        tc_fence_after();
        float sv[32];
        tmem_ld32(tmem + lane_addr + kTmemS + 64 * b + 32 * part, sv);
        tmem_ld_wait();
        const int blk = block_row(sg, 2 * j + half);
        const int kb = blk + 32 * part;                 // this thread's first key
        const bool whole = blk >= 0 && kb + 31 <= pos && (kb + 32 <= p.sinks || kb > pos - p.window);
        if (!__all_sync(0xffffffffu, whole)) {
          // bit k: key kb + k is attended: [0, sinks) and (pos - window, ..) up to pos
          const uint32_t m32 = blk < 0 ? 0u
                                       : (bits_below(p.sinks - kb) | ~bits_below(pos - p.window + 1 - kb)) &
                                             bits_below(pos + 1 - kb);
#pragma unroll
          for (int k = 0; k < 32; ++k) sv[k] = (m32 >> k) & 1u ? sv[k] : -CUDART_INF_F;
        }
        float mx[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = max3(sv[k], sv[4 + 2 * k], sv[5 + 2 * k]);
#pragma unroll
        for (int k = 12; k < 28; k += 2) mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], sv[k], sv[k + 1]);
        const float top = max3(max3(mx[0], mx[1], sv[28]), max3(mx[2], mx[3], sv[29]), fmaxf(sv[30], sv[31]));
        sh.red[x][part][ln] = top;
        ok = group_all(mine);                // the one group decision of a tile; the row's four maxima
        if (!ok) break;
        const float mt = fmaxf(fmaxf(top, sh.red[x][part ^ 1][ln]),
                               fmaxf(sh.red[x][0][ln ^ 64], sh.red[x][1][ln ^ 64])) * p.scale_log2;
        x ^= 1;   // every thread is done with the place of the exchange before
        float alpha = 1.f;
        if (mt > m + kLazyRescale || (m == -CUDART_INF_F && mt > -CUDART_INF_F)) {
          alpha = m == -CUDART_INF_F ? 0.f : ex2_approx(m - mt);
          m = mt;
        }
        const float ref = m == -CUDART_INF_F ? 0.f : -m;
        l *= alpha;
        uint32_t pk[16];
        const uint64_t by = pair_f32(p.scale_log2, p.scale_log2), from = pair_f32(ref, ref);
        uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          const uint64_t x = fma_pair(pair_f32(sv[k], sv[k + 1]), by, from);
          const float e0 = ex2_approx(__uint_as_float((uint32_t)x)), e1 = ex2_approx(__uint_as_float((uint32_t)(x >> 32)));
          sum[(k >> 1) & 3] = add_pair(sum[(k >> 1) & 3], pair_f32(e0, e1));
          const __nv_bfloat162 h = __floats2bfloat162_rn(e0, e1);
          pk[k >> 1] = *reinterpret_cast<const uint32_t*>(&h);
        }
        const uint64_t all = add_pair(add_pair(sum[0], sum[1]), add_pair(sum[2], sum[3]));
        l += __uint_as_float((uint32_t)all) + __uint_as_float((uint32_t)(all >> 32));
        // P(g) takes P(g - 1)'s place and O is rescaled once PV(g - 1) is done
        if (g > 0) mine = mine && wait_for(&sh.pv_done[b ^ 1][3], ((g - 1) >> 1) & 1, abort);
        tc_fence_after();
        if (__any_sync(0xffffffffu, alpha != 1.f && j > sg.t0)) {
          for (int c = 128 * part; c < 128 * part + 128; c += 32) {
            float v[32];
            tmem_ld32(tmem + lane_addr + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= alpha;
            tmem_st32(tmem + lane_addr + c, v);
          }
          tmem_st_wait();
        }
#pragma unroll
        for (int ch = 0; ch < 4; ++ch)
          *reinterpret_cast<uint4*>(sP + half * kBox + row * 128 + (((4 * part + ch) ^ (row & 7)) << 4)) =
              make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
        // the other CTA's keys' values are here (the issuer does not wait for them itself)
        mine = mine && wait_for(&sh.full_w[b], ph, abort);
        // rows that no token attends: their weights are zero, and so must their values be,
        // whatever the cache holds there
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int base = block_row(sg, 2 * j + h);
          if (base < 0 || (base + kBlk - 1 <= sg.hi && (base + kBlk <= p.sinks || base >= sg.lo))) continue;
          const int t = base + row;
          if (!(t <= sg.hi && (t < p.sinks || t >= sg.lo))) {
            unsigned char* v = sKV + kv_box(b, h, 2 * half + part) + row * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i)   // lanes in different banks
              *reinterpret_cast<uint4*>(v + ((i ^ (row & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        // The lanes' shared-memory writes (P, cleared values) are ordered before this arrive by the warp's
        // barrier and a release; their tensor memory accesses by the fence before. Across the two CTAs the
        // release is one of shared memory alone: one of everything (an arrive with .release.cluster) waits
        // for the output's stores and the copies in flight too, 2200 to 3500 cycles a tile
        if (lane == 0) {
          if (rank == 0)
            mbar_arrive(&sh.p_full);
          else
            mbar_arrive_smem_released(bar_p);
        }
        if (left > 0) store_quarter();
      }
      if (!ok) break;
      // ---- O / l. The weights' sums are exchanged, what is left of the output before goes out and the
      // next row tile is looked up while the last PV runs
      float (&sums)[2][128] = sh.red[x];
      sums[part][ln] = l;
      ok = group_all(mine);
      if (!ok) break;
      l = (sums[0][ln] + sums[1][ln]) + (sums[0][ln ^ 64] + sums[1][ln ^ 64]);
      x ^= 1;
      const float inv = l == 0.f ? 0.f : 1.f / l;   // a NaN stays one
      const int slot = sg.slot;
      const int64_t prow = (int64_t)slot * 128 + 64 * rank + row, orow = sg.tok0 + tok;
      if (valid && half == 0 && part == 0) {
        const float lse = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
        if (slot >= 0)
          p.out.part_lse[prow] = lse;
        else if (p.out.lse != nullptr)
          p.out.lse[orow * p.H + head] = lse;
      }
      while (left > 0) store_quarter();
      more = wk.next(p.sched, sg, &g_pair_err);
      const int last = g - 1;
      mine = mine && wait_for(&sh.pv_done[last & 1][3], (last >> 1) & 1, abort);
      tc_fence_after();
      if (slot < 0) {
        // A row tile's 64 KB of output take an SM as long to store as a tile of keys takes.
        // So O only becomes bf16 here, within tensor memory, and a quarter of it is stored behind each
        // of the next tiles
#pragma unroll 1
        for (int r = 0; r < 2; ++r) {
          float v[2][32];
          tmem_ld32(tmem + lane_addr + 128 * part + 64 * r, v[0]);
          tmem_ld32(tmem + lane_addr + 128 * part + 64 * r + 32, v[1]);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int word = 8 * ((k >> 1) & 3) + 4 * i + 2 * (k >> 3) + (k & 1);   // of the 32
              const float* const f = v[word >> 4] + 2 * (word & 15);
              const __nv_bfloat162 h = __floats2bfloat162_rn(f[0] * inv, f[1] * inv);
              w[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
            tmem_st16u(tmem + lane_addr + kTmemOut + 64 * part + 32 * r + 16 * i, w);
          }
        }
        tmem_st_wait();
        left = 4;
        // a lane whose row is not real stores nothing
        to = valid ? static_cast<__nv_bfloat16*>(p.out.o) + orow * p.out.o_s0 + (int64_t)head * p.out.o_s1 + 256 * half +
                         128 * part
                   : nullptr;
      } else {
        // float32, whole lines as above: 16 rows x 32 columns at a time, their columns in the order that
        // tensor memory gives them out in (WindowOut: permuted)
        const unsigned rows = __ballot_sync(0xffffffffu, valid);
        float* const o = p.out.part_o + ((int64_t)slot * 128 + 64 * rank + 32 * (warp & 1)) * 512 + 256 * half + 128 * part +
                         8 * (lane & 3);
        uint32_t w[16];
        tmem_ld_16x32(tmem + lane_addr + 128 * part, w);
#pragma unroll 1
        for (int r = 0; r < 8; ++r) {
          const int h = r & 1, c = r >> 1;
          uint32_t y[2][8];
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float by = __shfl_sync(0xffffffffu, inv, 16 * h + 8 * i + (lane >> 2));
#pragma unroll
            for (int k = 0; k < 8; ++k)
              y[i][k] = __float_as_uint(__uint_as_float(w[4 * (k >> 1) + 2 * i + (k & 1)]) * by);
          }
          if (r < 7)
            tmem_ld_16x32(tmem + lane_addr + ((16u * ((r + 1) & 1)) << 16) + 128 * part + 32 * ((r + 1) >> 1), w);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int rw = 16 * h + 8 * i + (lane >> 2);
            if ((rows >> rw) & 1u) st_global_32B(o + (int64_t)rw * 512 + 32 * c, y[i]);
          }
          __syncwarp();
        }
      }
    }
    while (left > 0) store_quarter();
    if (!ok || !mine) give_up();
  }
  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    volatile int dummy = 0;
    if (!mbar_wait(&sh.fin, 0, &dummy) || sh.abort_flag) atomicOr(&g_pair_err, kErrTimeout);
  }
  __syncthreads();
  cluster_sync();   // neither CTA frees or leaves while the other's MMAs or copies may touch it
  if (warp == 2) {
    tc_fence_after();
    dealloc_pair(tmem, kTmemCols);
  }
  cluster_sync();
}

template <int kRope, bool kSmall, bool kDirect>
int max_pairs() {
  static std::mutex mu;
  static std::vector<int> cache;
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> g(mu);
  if ((int)cache.size() <= dev) cache.resize(dev + 1, 0);
  if (cache[dev] == 0) {
    using C = PairCfg<kRope>;
    cudaFuncSetAttribute(window_attn_kernel<kRope, kSmall, kDirect>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemAlloc);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * device_sm_count(), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmemAlloc;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, window_attn_kernel<kRope, kSmall, kDirect>, &cfg) != cudaSuccess || n <= 0)
      n = device_sm_count() / 2;
    cudaGetLastError();
    cache[dev] = n;
  }
  return cache[dev];
}

template <int kRope, bool kSmall, bool kDirect>
cudaError_t launch_attn(const PairParams& p, const WindowMaps& maps, int units, cudaStream_t st) {
  using C = PairCfg<kRope>;
  const cudaError_t e = cudaFuncSetAttribute(window_attn_kernel<kRope, kSmall, kDirect>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             C::kSmemAlloc);
  if (e != cudaSuccess) return e;
  return launch_k(window_attn_kernel<kRope, kSmall, kDirect>, dim3(2 * units), dim3(kThreads), C::kSmemAlloc, st, maps.keys, maps.boxes,
                  maps.q, p);
}

template <int kRope, bool kSmall>
cudaError_t launch_page(const PairParams& p, const WindowMaps& maps, int units, cudaStream_t st) {
  return p.sched.direct ? launch_attn<kRope, kSmall, true>(p, maps, units, st)
                        : launch_attn<kRope, kSmall, false>(p, maps, units, st);
}

int pair_units(int num_splits) {
  return num_splits > 0 ? std::min(num_splits, kMaxUnits) : max_pairs<64, false, false>();
}

int pair_tokens(int H) { return H > 64 ? 1 : 2 * (64 / H); }

// Whether a CTA's queries fill its 64 rows, so that one load lays all their column groups out.
bool q_whole(int H) { return H >= 64 || 64 % H == 0; }

// A 4-D TMA map of bf16 (dims innermost first, strides of dims 1 to 3 in bytes), 128-byte swizzled.
bool make_map4d(CUtensorMap* m, const void* base, const uint64_t (&dims)[4], const uint64_t (&strides)[3],
                const uint32_t (&box)[4]) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  if (!encode) return false;
  cuuint64_t d[4], st[3];
  cuuint32_t b[4], step[4] = {1, 1, 1, 1};
  std::copy(dims, dims + 4, d);
  std::copy(strides, strides + 3, st);
  std::copy(box, box + 4, b);
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), d, st, b, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor maps: two column groups of 64 of a block, for pages of 64 rows or more; one group of a block or
// a page; queries.
bool pair_maps(const WindowCall& c, WindowMaps* m) {
  const uint64_t row = (uint64_t)c.cache.s_row * 2, blk = (uint64_t)c.cache.s_blk * 2, page = c.cache.page,
                 blocks = c.cache.num_blocks, groups = (c.L + c.R) / 64, H = c.H, T = c.q.n0;
  const uint32_t rows = page < kBlk ? (uint32_t)page : kBlk, hb = H < 64 ? (uint32_t)H : 64, toks = H > 64 ? 1 : 64 / hb;
  const uint64_t kd[4] = {64, page, 8, blocks}, ks[3] = {row, 128, blk};
  const uint32_t kb[4] = {64, rows, 2, 1};
  const uint64_t qd[4] = {64, H, T, groups}, qs[3] = {(uint64_t)c.q.s1 * 2, (uint64_t)c.q.s0 * 2, 128};
  const uint32_t qb[4] = {64, hb, toks, q_whole(c.H) ? (uint32_t)groups : 1};
  return make_map4d(&m->keys, c.cache.data, kd, ks, kb) &&
         make_map3d(&m->boxes, c.cache.data, 64 * groups, page, blocks, row, blk, 64, rows, 1,
                    CU_TENSOR_MAP_SWIZZLE_128B) &&
         make_map4d(&m->q, c.q.data, qd, qs, qb);
}

}  // namespace

bool window_tc_supported(mla_dtype dt, const WindowCall& c, WindowMaps* maps) {
  if (dt != MLA_BF16 || c.L != 512 || (c.R != 0 && c.R != 64) || c.H > 128 || !(c.scale > 0.f)) return false;
  const int page = c.cache.page;
  if (!(page % 64 == 0 || (64 % page == 0 && page % 8 == 0))) return false;
  auto al16 = [](const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15) == 0; };
  if (!al16(c.cache.data) || c.cache.s_blk % 8 || c.cache.s_row % 8) return false;
  if (!al16(c.q.data) || c.q.s0 % 8 || c.q.s1 % 8) return false;
  if (!al16(c.o.data) || c.o.s0 % 8 || c.o.s1 % 8) return false;
  return pair_maps(c, maps);
}

size_t window_tc_workspace(int64_t T, int64_t B, int H, bool decode, int num_splits) {
  if (H <= 0 || H > 128) return 0;
  return window_workspace(T, B, decode, pair_tokens(H), pair_units(num_splits), 128, 512);
}

cudaError_t launch_window_tc(const WindowCall& c, const WindowMaps& maps, int num_splits, void* ws, cudaStream_t st) {
  const int units = pair_units(num_splits), tpt = pair_tokens(c.H);
  PairParams p{};
  cudaError_t e = launch_window_schedule(c, tpt, 2, units, 128, ws, &p.sched, &p.out, st);
  if (e != cudaSuccess) return e;
  p.H = c.H;
  p.out.permuted = true;
  p.tptc = p.out.tptc = c.H > 64 ? 0 : tpt / 2;
  constexpr int kFar = 0x3fffffff;   // positions stay below this
  p.window = std::min(c.window.window, kFar);
  p.sinks = std::min(c.window.sinks, kFar);
  p.scale_log2 = c.scale * 1.4426950408889634f;
  p.page = c.cache.page;
  p.num_blocks = c.cache.num_blocks;
  p.block_table = c.block_table;
  p.bt_stride = c.bt_stride;
  p.prefetch = p.sched.direct || p.sched.unit_start != nullptr;
  p.q_whole = q_whole(c.H);
  p.o_32B = reinterpret_cast<uintptr_t>(c.o.data) % 32 == 0 && c.o.s0 % 16 == 0 && c.o.s1 % 16 == 0;
  if (p.page < kBlk)
    e = c.R == 64 ? launch_page<64, true>(p, maps, units, st) : launch_page<0, true>(p, maps, units, st);
  else
    e = c.R == 64 ? launch_page<64, false>(p, maps, units, st) : launch_page<0, false>(p, maps, units, st);
  if (e != cudaSuccess) return e;
  return launch_window_merge(MLA_BF16, p.sched, p.out, units, st);
}

cudaError_t attn_pair_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_pair_err);
}

}  // namespace mla
