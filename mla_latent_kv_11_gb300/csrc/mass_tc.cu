// Row masses on the tensor cores (tcgen05 + TMEM + TMA): for every cached row the weights
// e^(scale q.k - lse) of the queries that attend it, summed over queries and heads; bf16.
//
// Mathematics. The log-sum-exps are given, so no row's weights wait for another's: S = K Q^T, one
// exponential a score, a sum along S's rows. The keys are the A operand and the queries B (not the other
// way round as in attention): a row of S is then a lane of tensor memory, its sum stays in one thread, and
// a cache row that holds anything at all (rows behind a sequence's end, NaN) reaches no sum but its own.
//
// Tile. 256 cache rows by a cluster of two CTAs, 128 of them each (cta_group::2, M = 256), against N query
// rows (heads, or tokens' heads), half of which each CTA holds for both. The row width goes by in chunks
// of 64 columns, 16 KB of keys a CTA. One of the operands stays in shared memory (resident) while the
// other streams by through a ring:
//   decode:  a sequence's queries stay (N = its heads, rounded up to 32), its rows stream: each
//            crosses HBM and L2 once;
//   prefill: 256 rows stay, the tokens' queries stream (N = 256): each byte of them loaded by a CTA serves
//            512 x 64 multiplications, so that L2 feeds the tensor pipe at 32 bytes a cycle. (With N = 128 the operands'
//            reads of shared memory bound the products: 910 us for the 4 x 512 prefill below instead of 700.)
// Resident chunks are released one by one by the last tile that reads them, and the next ones loaded under it.
//
// Sums. The tensor cores' additions into an accumulator round toward zero, so that a score's error grows with the
// length of the chain and does not average out over queries: with one accumulator for the 36 steps of a 576-wide
// row, masses came out 1.4e-6 of themselves too small. So the first half of the chunks goes to one accumulator and
// the rest to another, which the epilogue adds: 0.7e-6. A decode's two fit into tensor memory twice, so that
// one tile is summed while the next is computed. A prefill's fill it (2 x 256 columns): there the epilogue's eight warps
// take the first into registers (128 a thread, lent by the other warps) while the second is computed, and the second
// while the next tile's first is: 6% slower than one accumulator in two places (12% at 32 tokens over 16K rows).
//
// Work. Tiles (256 rows x N queries) are numbered through all sequences and dealt out in equal consecutive
// ranges, one a cluster; where a range begins is worked out by each cluster from the lengths. A prefill's
// 256 rows may be cut between ranges: their sums then go to the workspace, in pieces that a second kernel adds
// up in order. A decode's never are.
//
// What bounds it and what it measured (152 SMs, 76 clusters; device times):
//   decode of 64 sequences of 1K to 16K rows, 128 heads: 106 us, 665 MB at 6.3 TB/s, 0.92 of a copy's rate: HBM.
//   prefill of 4 x 512 tokens over 1K to 8K rows, 128 heads: 610 us, 1.76 PFLOP/s, in a short run, the tensor
//     pipe 86% active at 1.7 GHz; 675 us a call under the power cap.
//   32 tokens over 16K rows, 64 heads: 31 us for 34 GFLOP: 7 tiles a cluster (15 us of products) between the start (the
//     ranges, the first keys: 4 us), the last tile's weights and the pieces' sums (6 us).
//   decode of one sequence of 700 rows: 8.5 us: three clusters, one tile each, one latency behind the other.
//
// Every wait is bounded; one that gives up winds both CTAs down and is reported.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <limits>
#include <mutex>
#include <type_traits>
#include <vector>

#include "mass.cuh"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

using namespace ptx;

__device__ unsigned g_mass_tc_err = 0;

constexpr int kRows = 256, kCtaRows = 128;         // cache rows of a tile, and of one CTA of the pair
constexpr int kChunkBytes = kCtaRows * 128;        // 128 rows x 64 bf16 columns, 128-byte swizzle
constexpr int kMaxChunks = 9, kMaxStages = 12;
constexpr int kEpiWarp0 = 4, kEpiBar = 1;
template <bool kPrefill>
constexpr int kEpiThreads = kPrefill ? 256 : 128;
template <bool kPrefill>
constexpr int kThreads = 128 + kEpiThreads<kPrefill> + (kPrefill ? 0 : 64);   // a decode's: two more warps that load
// registers of a thread of a prefill: at launch (what 384 threads may have), of the first four warps, of the others
constexpr int kLaunchRegs = 168, kRoleRegs = 72, kEpiRegs = 216;
static_assert(kRoleRegs * 128 + kEpiRegs * 256 <= kLaunchRegs * 384, "the shares draw on the launch's registers");
constexpr int kMiscBytes = 3 * 1024;
constexpr int kArena = 232448 - kMiscBytes;        // shared memory for operands: 224 KB
constexpr int kMaxUnits = 256;
// tensor memory columns from a tile's first accumulator to its second
template <bool kPrefill>
constexpr uint32_t kSecond = kPrefill ? 256 : 128;
constexpr float kLog2e = 1.4426950408889634f;

// Where a tile lies: inner tile `tile` of outer tile `outer` of sequence seq; base: tiles before the sequence.
struct Place {
  int seq, outer, tile;
  long long base;
};

struct Shared {
  uint64_t ring_full[kMaxStages], ring_empty[kMaxStages];   // full: first CTA, bytes of both
  uint64_t res_full[kMaxChunks], res_empty[kMaxChunks];
  // decode: of even and odd tiles; prefill: of a tile's two accumulators. d_empty: first CTA, epilogue warps of both
  uint64_t d_full[2], d_empty[2];
  uint64_t fin;
  uint32_t tmem_base;
  int abort_flag;
  Place found;
  long long wide[12];
  float neg_lse[2][256];     // -lse * log2(e) of a tile's columns, in turn in two places
  int none[2];               // the tile (of this CTA's, in order) whose columns those are, if one of them is without a query
};
static_assert(sizeof(Shared) <= kMiscBytes, "barrier block overflows its slot");

struct TcArgs {
  MassArgs m;
  int chunks, split;         // of 64 columns; those before `split` are summed apart from the others
  int stages;                // of the ring
  int n, half;               // query rows of a tile, and of one CTA
  int tpc;                   // prefill: tokens of a tile per CTA
  // a prefill's pieces of rows that are cut, of each unit: those that end in its first tiles, and that begin in its
  // last ones
  float* part;               // [unit][2][256]
  int4* piece;               // [unit][2] {sequence (-1: none), tile of 256 rows, whether it is the last piece, rows}
};

// Sum over i < n of (a i + b) / m, rounded down each: the integer points under a line, by the well-known reduction with
// Euclid's steps (whole parts apart, then axes exchanged). a, b >= 0, m > 0; a n + b below 2^31.
__device__ long long points_below(int n, int m, int a, int b) {
  long long sum = 0;
  while (n > 0) {
    sum += (long long)(a / m) * n * (n - 1) / 2 + (long long)(b / m) * n;
    a %= m;
    b %= m;
    const int top = a * n + b;     // m times the height at n
    if (top < m) break;
    n = top / m;
    b = top - n * m;
    const int t = a;
    a = m;
    m = t;
  }
  return sum;
}

// A sequence's tiles. Decode: `outer` counts nothing, inner tiles are those of 256 rows. Prefill: outer
// tiles of 256 rows, inner ones of tpt tokens, from the first that attends one of the rows on.
template <bool kPrefill>
struct Tiles {
  MassSeq s;
  int outer, inner, tpt;
  __device__ void open(const TcArgs& a, int b) {
    s = mass_seq(a.m, b, &g_mass_tc_err);
    tpt = kPrefill ? 2 * a.tpc : 1;
    const int rows = (s.kv + kRows - 1) / kRows;
    outer = s.nq == 0 ? 0 : kPrefill ? rows : 1;
    inner = kPrefill ? (s.nq + tpt - 1) / tpt : rows;
  }
  __device__ int first(int k) const { return kPrefill ? max(0, kRows * k - (s.kv - s.nq)) / tpt : 0; }
  // Tiles of the outer ones before k.
  __device__ long long before(int k) const {
    if (!kPrefill) return k > 0 ? inner : 0;
    const int d = s.kv - s.nq;
    const int z = d < 0 ? 0 : min(k, d / kRows + 1);   // outer tiles that the first token attends
    const int left = k - z;
    return (long long)k * inner - (left > 0 ? points_below(left, tpt, kRows, kRows * z - d) : 0);
  }
  __device__ long long total() const { return outer == 0 ? 0 : before(outer); }
};

// Tiles of the whole call. All threads of the block take part here and in find_tile, and every one gets
// the answer.
template <bool kPrefill>
__device__ long long all_tiles(const TcArgs& a, long long* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long sum = 0;
  for (int b = threadIdx.x; b < a.m.B; b += kThreads<kPrefill>) {
    Tiles<kPrefill> t;
    t.open(a, b);
    sum += t.total();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sh[warp] = sum;
  __syncthreads();
  sum = 0;
#pragma unroll
  for (int w = 0; w < kThreads<kPrefill> / 32; ++w) sum += sh[w];
  __syncthreads();
  return sum;
}

// Tile x's place within the sequence that *found names.
template <bool kPrefill>
__device__ Place place_in(const TcArgs& a, long long x, Place* found) {
  Place p = *found;
  Tiles<kPrefill> t;
  t.open(a, p.seq);
  if constexpr (kPrefill) {
    // the outer tile that holds x: the threads look at one each
    for (int k = threadIdx.x; k < t.outer; k += kThreads<kPrefill>) {
      const long long lo = p.base + t.before(k);
      const int n = t.inner - t.first(k);
      if (lo <= x && x < lo + n) {
        found->outer = k;
        found->tile = t.first(k) + (int)(x - lo);
      }
    }
    __syncthreads();
    p = *found;
  } else {
    p.tile = (int)(x - p.base);
  }
  __syncthreads();
  return p;
}

// Where tile x lies, x below the total.
template <bool kPrefill>
__device__ Place find_tile(const TcArgs& a, long long x, long long* sh, Place* found) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long base = 0;
  for (int b0 = 0; b0 < a.m.B; b0 += kThreads<kPrefill>) {
    const int b = b0 + threadIdx.x;
    Tiles<kPrefill> t;
    long long mine = 0;
    if (b < a.m.B) {
      t.open(a, b);
      mine = t.total();
    }
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) sh[warp] = upto;
    __syncthreads();
    long long all = 0, before = base;
#pragma unroll
    for (int w = 0; w < kThreads<kPrefill> / 32; ++w) {
      if (w == warp) before = base + all;
      all += sh[w];
    }
    const long long at = before + upto - mine;
    if (mine > 0 && at <= x && x < at + mine) *found = Place{b, 0, 0, at};
    __syncthreads();
    base += all;
    if (x < base) break;     // the same for every thread
  }
  return place_in<kPrefill>(a, x, found);
}
// This unit's tiles [x0, x1), and where x0 lies if there are any.
template <bool kPrefill>
__device__ Place my_tiles(const TcArgs& a, int unit, int units, long long& x0, long long& x1, long long* sh, Place* found) {
  if (a.m.B > kThreads<kPrefill>) {
    const long long total = all_tiles<kPrefill>(a, sh);
    x0 = total * unit / units;
    x1 = total * (unit + 1) / units;
    return x0 < x1 ? find_tile<kPrefill>(a, x0, sh, found) : Place{};
  }
  // a thread a sequence: total and place from one sum over them
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = threadIdx.x;
  Tiles<kPrefill> t;
  long long mine = 0;
  if (b < a.m.B) {
    t.open(a, b);
    mine = t.total();
  }
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) sh[warp] = upto;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kThreads<kPrefill> / 32; ++w) {
    if (w == warp) before = total;
    total += sh[w];
  }
  x0 = total * unit / units;
  x1 = total * (unit + 1) / units;
  if (x0 >= x1) return Place{};   // the same for every thread
  const long long at = before + upto - mine;
  if (mine > 0 && at <= x0 && x0 < at + mine) *found = Place{b, 0, 0, at};
  __syncthreads();
  return place_in<kPrefill>(a, x0, found);
}

// The segments of a range of tiles: inner tiles [i0, i1) of an outer one.
struct Seg {                 // (of the walker's sequence b, with its rows and queries t.s)
  int outer, i0, i1;
  bool whole, begins, ends;  // it is all of its outer tile; it holds the outer tile's first, and its last
};
// A prefill's range that begins within an outer tile takes that piece last. The clusters of a sequence then
// begin at its first queries together and stay together (the pieces at the end too: the ranges are equally long, so that
// each lies as far behind), and a query chunk that one of them loads is in L2 for the others. In the order of
// the tiles every cluster was at queries of its own: 4 x 512 tokens read 3.66 GB from HBM instead of 0.83.
template <bool kPrefill>
struct Walker {
  int b, k, i;
  long long left;
  int later_b, later_k, later_i, later;   // the piece that comes last: its place and tiles
  Tiles<kPrefill> t;
  __device__ void init(const TcArgs& a, int seq, int outer, int tile, long long count) {
    b = seq;
    k = outer;
    i = tile;
    left = count;
    later = 0;
    if (left <= 0) return;
    t.open(a, b);
    if (kPrefill && i > t.first(k) && t.inner - i < left) {
      later_b = b;
      later_k = k;
      later_i = i;
      later = t.inner - i;
      left -= later;
      ++k;
      i = k < t.outer ? t.first(k) : 0;
    }
  }
  __device__ bool next(const TcArgs& a, Seg& s) {
    if (left <= 0) {
      if (later == 0) return false;
      b = later_b;
      k = later_k;
      i = later_i;
      left = later;
      later = 0;
      t.open(a, b);
    }
    while (k >= t.outer) {   // the next sequence with tiles: there is one, as tiles are left
      if (++b >= a.m.B) return false;
      t.open(a, b);
      k = 0;
      i = t.outer > 0 ? t.first(0) : 0;
    }
    s.outer = k;
    s.i0 = i;
    s.i1 = (int)min((long long)t.inner, i + left);
    s.begins = i == t.first(k);
    s.ends = s.i1 == t.inner;
    s.whole = s.begins && s.ends;
    left -= s.i1 - s.i0;
    ++k;
    i = k < t.outer ? t.first(k) : 0;
    return true;
  }
};

// The wait behind a first look (in line: registers cannot move between warps around a call); the timer is read only every 256 looks.
__device__ __forceinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort) {
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

__device__ __forceinline__ void alloc_pair(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Four MMAs of the pair (64 columns), issued by the first CTA's converged warp through an elected lane. Both
// operands are K-major with a 128-byte swizzle: the descriptors' low words advance by 32 bytes an MMA, their
// high words (stride 1024) are constant. The first MMA replaces D where `fresh`.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void umma_pair4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool fresh) {
  asm volatile(
      "{\n .reg .pred p, t, e;\n .reg .b32 r, x, y;\n .reg .b64 a, b;\n"
      " elect.sync r|e, 0xffffffff;\n setp.eq.b32 p, %3, 0;\n setp.eq.b32 t, 0, 0;\n"
      " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, p;\n"
      " add.u32 x, %1, 2;\n add.u32 y, %2, 2;\n mov.b64 a, {x, %5};\n mov.b64 b, {y, %5};\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, x, 2;\n add.u32 y, y, 2;\n mov.b64 a, {x, %5};\n mov.b64 b, {y, %5};\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, x, 2;\n add.u32 y, y, 2;\n mov.b64 a, {x, %5};\n mov.b64 b, {y, %5};\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, t;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"((uint32_t)fresh), "r"(idesc), "n"(kDescHi)
      : "memory");
}
// Low word of a descriptor (the leading dimension is not used within one swizzle span: 16 bytes).
__device__ __forceinline__ uint32_t desc_lo(const void* p) { return (smem_u32(p) >> 4) | (1u << 16); }
// Arrive on `bar` of both CTAs once every MMA issued so far is complete.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .b32 r;\n elect.sync r|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// A converged warp's elected lane counts the bytes of a phase, and loads a box whose bytes are counted on
// `bar`, a shared::cluster address (the first CTA's barrier).
__device__ __forceinline__ void expect_bytes(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .b32 r;\n elect.sync r|e, 0xffffffff;\n"
      " @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(smem_u32(bar)),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void load_pair_3d(void* dst, const void* map, uint32_t bar, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .b32 r;\n elect.sync r|e, 0xffffffff;\n"
      " @e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5}], [%2];\n}\n" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// The same by every lane that comes here.
__device__ __forceinline__ void load_pair_3d_lane(void* dst, const void* map, uint32_t bar, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ uint64_t pair_f32(float a, float b) {
  return (uint64_t)__float_as_uint(b) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
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

// A column's -lse log2(e) where its query attended nothing (lse -inf). No other column has it: one of a finite lse is
// cut to the largest float32, whose weight is infinite all the same.
constexpr float kNoQuery = std::numeric_limits<float>::infinity();
__device__ __forceinline__ float neg_lse_of(float lse) {
  const float v = -lse * kLog2e;
  return v > FLT_MAX && lse != -kNoQuery ? FLT_MAX : v;
}

// e^(scale s - lse) summed over columns [lo, hi) of 32 scores. kSome: columns without a query among them. (With their
// choice in the ordinary sum too, a prefill's tiles took 2 to 7% longer.)
template <bool kSome>
__device__ __forceinline__ float sum_weights(const float (&v)[32], const float* neg_lse, float scale_log2, int lo, int hi) {
  const uint64_t by = pair_f32(scale_log2, scale_log2);
  uint64_t sum[2] = {0, 0};
  if (!kSome && __all_sync(0xffffffffu, lo <= 0 && hi >= 32)) {
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      const float4 l = *reinterpret_cast<const float4*>(neg_lse + k);
      const uint64_t x = fma_pair(pair_f32(v[k], v[k + 1]), by, pair_f32(l.x, l.y));
      const uint64_t y = fma_pair(pair_f32(v[k + 2], v[k + 3]), by, pair_f32(l.z, l.w));
      sum[0] = add_pair(sum[0], pair_f32(ex2_approx(low(x)), ex2_approx(high(x))));
      sum[1] = add_pair(sum[1], pair_f32(ex2_approx(low(y)), ex2_approx(high(y))));
    }
  } else {
#pragma unroll
    for (int k = 0; k < 32; k += 2) {   // a column that does not count may hold anything: chosen, not multiplied, away
      const float l0 = neg_lse[k], l1 = neg_lse[k + 1];
      const uint64_t x = fma_pair(pair_f32(v[k], v[k + 1]), by, pair_f32(l0, l1));
      const bool c0 = k >= lo && k < hi && (!kSome || l0 != kNoQuery), c1 = k + 1 >= lo && k + 1 < hi && (!kSome || l1 != kNoQuery);
      sum[(k >> 1) & 1] = add_pair(sum[(k >> 1) & 1], pair_f32(c0 ? ex2_approx(low(x)) : 0.f, c1 ? ex2_approx(high(x)) : 0.f));
    }
  }
  const uint64_t all = add_pair(sum[0], sum[1]);
  return low(all) + high(all);
}
// What tensor memory loads asked for, usable behind a wait: arithmetic on the registers, which to the compiler
// have their values from the load on, stays behind this.
__device__ __forceinline__ void loaded(float (&w)[16]) {
  asm volatile(""
               : "+f"(w[0]), "+f"(w[1]), "+f"(w[2]), "+f"(w[3]), "+f"(w[4]), "+f"(w[5]), "+f"(w[6]), "+f"(w[7]),
                 "+f"(w[8]), "+f"(w[9]), "+f"(w[10]), "+f"(w[11]), "+f"(w[12]), "+f"(w[13]), "+f"(w[14]), "+f"(w[15]));
}
__device__ __forceinline__ void loaded(float (&w)[32]) {
  asm volatile(""
               : "+f"(w[0]), "+f"(w[1]), "+f"(w[2]), "+f"(w[3]), "+f"(w[4]), "+f"(w[5]), "+f"(w[6]), "+f"(w[7]),
                 "+f"(w[8]), "+f"(w[9]), "+f"(w[10]), "+f"(w[11]), "+f"(w[12]), "+f"(w[13]), "+f"(w[14]), "+f"(w[15]),
                 "+f"(w[16]), "+f"(w[17]), "+f"(w[18]), "+f"(w[19]), "+f"(w[20]), "+f"(w[21]), "+f"(w[22]), "+f"(w[23]),
                 "+f"(w[24]), "+f"(w[25]), "+f"(w[26]), "+f"(w[27]), "+f"(w[28]), "+f"(w[29]), "+f"(w[30]), "+f"(w[31]));
}
// The second accumulator's 32 columns added to the first's, in halves: 32 more registers would be spilled. (The prefill spills
// as it is: 664 bytes of stores, 372 of loads.)
__device__ __forceinline__ void add_second(uint32_t taddr, float (&v)[32]) {
#pragma unroll
  for (int h = 0; h < 32; h += 16) {
    float w[16];
    tmem_ld16(taddr + h, w);
    tmem_ld_wait();
    loaded(w);
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const uint64_t x = add_pair(pair_f32(v[h + k], v[h + k + 1]), pair_f32(w[k], w[k + 1]));
      v[h + k] = low(x);
      v[h + k + 1] = high(x);
    }
  }
}

template <bool kPrefill>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads<kPrefill>, 1)
    mass_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap, const TcArgs a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem + kArena);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = blockIdx.x & 1;
  const int unit = blockIdx.x >> 1, units = gridDim.x >> 1;
  // the resident operand's chunks, then the ring's
  const int res_bytes = kPrefill ? kChunkBytes : a.half * 128;
  unsigned char* const ring = smem + a.chunks * res_bytes;

  if (tid == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&sh.ring_full[i], 1);
      mbar_init(&sh.ring_empty[i], 1);
    }
    for (int i = 0; i < a.chunks; ++i) {
      mbar_init(&sh.res_full[i], 1);
      mbar_init(&sh.res_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.d_full[i], 1);
      mbar_init(&sh.d_empty[i], 2 * kEpiThreads<kPrefill> / 32);   // the epilogue warps of both CTAs
    }
    mbar_init(&sh.fin, 1);
    sh.abort_flag = 0;
    sh.none[0] = sh.none[1] = -1;
    fence_mbar_init();
  }
  if (warp == 2) alloc_pair(&sh.tmem_base, 512);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&qmap);
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers initialised, both tensor memories allocated
  tc_fence_after();
  pdl_enter();      // lengths, queries and cache come from the kernels before
  constexpr uint32_t tmem = 0;   // all 512 columns are allocated: they begin at 0
  volatile int* abort = &sh.abort_flag;
  auto give_up = [&]() {   // tell both CTAs
    sh.abort_flag = 1;
    const uint32_t remote = map_to_rank(&sh.abort_flag, rank ^ 1u);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(1) : "memory");
  };

  // this cluster's tiles [x0, x1): both CTAs work out the same
  long long x0, x1;
  const Place from = my_tiles<kPrefill>(a, unit, units, x0, x1, sh.wide, &sh.found);
  Walker<kPrefill> wk;
  wk.init(a, from.seq, from.outer, from.tile, x1 - x0);
  Seg sg;

  // (a prefill's registers move by whole warpgroups: warps 0 to 3 give, 4 to 11 take)
  if (warp >= kEpiWarp0 && (kPrefill || warp < 8)) {
    if constexpr (kPrefill) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    // ------------------------------------------------------------ weights and sums: a thread a cache row (two in a
    // prefill, half of the columns each)
    const int et = tid - kEpiWarp0 * 32, e = et & 127;  // tensor memory lane: the CTA's row
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const float scale_log2 = a.m.scale * kLog2e;
    const bool two = a.chunks > 1;
    const uint32_t d_empty = map_to_rank(&sh.d_empty[0], 0);
    volatile int* const none = sh.none;   // written before a tile's barrier and read behind it, as -lse
    bool ok = true, mine = true;   // ok: the group's decision; mine: this thread's waits so far
    int x = 0, place = 0;
    int4 ending = make_int4(-1, 0, 0, 0), beginning = ending;   // this unit's pieces of rows that are cut
    while (ok && wk.next(a, sg)) {
      const int d = wk.t.s.kv - wk.t.s.nq;
      auto row_of = [&](int k) { return kRows * k + kCtaRows * (int)rank + e; };
      // whether row t counts, and its place; a block id outside the cache is recorded
      auto row_mass = [&](int t) -> float* {
        if (t >= wk.t.s.kv) return nullptr;
        const int id = a.m.block_table[wk.b * a.m.bt_stride + t / a.m.page];
        if (id < 0 || id >= a.m.num_blocks) {
          atomicOr(&g_mass_tc_err, kErrDeviceData);
          return nullptr;
        }
        return a.m.mass + wk.b * a.m.mass_stride + t;
      };
      if (!kPrefill) {
        const float mark = e < a.m.H ? neg_lse_of(a.m.lse[(int64_t)wk.t.s.q0 * a.m.H + e]) : 0.f;
        const int tag = x;
        sh.neg_lse[place][e] = mark;
        if (mark == kNoQuery) none[place] = tag;
        for (int i = sg.i0; i < sg.i1; ++i, ++x) {
          const int buf = x & 1;
          float* const to = row_mass(row_of(i));
          const float old = to != nullptr && a.m.decay != 0.f ? *to : 0.f;
          mine = mine && wait_for(&sh.d_full[buf], (x >> 1) & 1, abort);
          ok = named_bar_and(kEpiBar, kEpiThreads<kPrefill>, mine);
          if (!ok) break;
          tc_fence_after();
          const bool some = none[place] == tag;
          float sum = 0.f;
#pragma unroll 1
          for (int c = 0; c < a.m.H; c += 32) {
            float v[32];
            tmem_ld32(tmem + lane_addr + 256 * buf + c, v);
            tmem_ld_wait();
            loaded(v);
            if (two) add_second(tmem + lane_addr + 256 * buf + kSecond<kPrefill> + c, v);
            const float* const l = &sh.neg_lse[place][c];
            sum += some ? sum_weights<true>(v, l, scale_log2, 0, a.m.H - c) : sum_weights<false>(v, l, scale_log2, 0, a.m.H - c);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_smem_released(d_empty + 8 * buf);
          if (to != nullptr) *to = new_mass(old, sum, a.m.decay);
        }
        place ^= 1;
      } else {
        const int t = row_of(sg.outer), H = a.m.H, half = et >> 7;
        float* const to = half == 0 ? row_mass(t) : nullptr;
        const float old = to != nullptr && sg.whole && a.m.decay != 0.f ? *to : 0.f;
        // the columns of this thread's half: head c % H of token c / H of its CTA's; its own of them is column e
        const int tok = e / H, head = e - tok * H;
        float l;
        auto ask = [&](int i) {
          const int q = (2 * i + half) * a.tpc + tok;
          l = tok < a.tpc && q < wk.t.s.nq ? a.m.lse[(int64_t)(wk.t.s.q0 + q) * H + head] : 0.f;
        };
        ask(sg.i0);
        float sum = 0.f;
        for (int i = sg.i0; i < sg.i1; ++i, ++x, place ^= 1) {
          const float mark = neg_lse_of(l);
          sh.neg_lse[place][et] = mark;
          if (mark == kNoQuery) none[place] = x;
          if (i + 1 < sg.i1) ask(i + 1);   // used a tile later
          mine = mine && wait_for(&sh.d_full[0], x & 1, abort);
          ok = named_bar_and(kEpiBar, kEpiThreads<kPrefill>, mine);
          if (!ok) break;
          tc_fence_after();
          // of the half's columns, tokens [seen, there) count: those at or behind the row's position
          const int q0 = (2 * i + half) * a.tpc;
          const int there = min(max(wk.t.s.nq - q0, 0), a.tpc) * H, seen = min(max(t - d - q0, 0), a.tpc) * H;
          const int last = __reduce_max_sync(0xffffffffu, there), first = __reduce_min_sync(0xffffffffu, seen);
          auto counts = [&](int c) { return 32 * c < last && 32 * c + 32 > first; };   // some of columns 32 c .. may
          float v[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (counts(c)) tmem_ld32(tmem + lane_addr + 128 * half + 32 * c, v[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 4; ++c) loaded(v[c]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_smem_released(d_empty);
          if (two) {
            mine = mine && wait_for(&sh.d_full[1], x & 1, abort);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (counts(c)) add_second(tmem + lane_addr + kSecond<kPrefill> + 128 * half + 32 * c, v[c]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_smem_released(d_empty + 8);
          }
          auto add = [&](auto some) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (counts(c))
                sum += sum_weights<decltype(some)::value>(v[c], &sh.neg_lse[place][128 * half + 32 * c], scale_log2,
                                                          seen - 32 * c, there - 32 * c);
          };
          if (none[place] != x)
            add(std::false_type{});
          else
            add(std::true_type{});
        }
        if (!ok) break;
        // the row's two sums, by way of the place that the next tile's -lse take: its thread there is the one that
        // reads the sum
        if (half == 1) sh.neg_lse[place][e] = sum;
        ok = named_bar_and(kEpiBar, kEpiThreads<kPrefill>, mine);
        if (!ok) break;
        if (half == 1) continue;
        sum += sh.neg_lse[place][e];
        if (sg.whole) {
          if (to != nullptr) *to = new_mass(old, sum, a.m.decay);
        } else {
          a.part[((int64_t)unit * 2 + (sg.begins ? 1 : 0)) * kRows + kCtaRows * rank + e] = sum;
          (sg.begins ? beginning : ending) = make_int4(wk.b, sg.outer, sg.ends, wk.t.s.kv);
        }
      }
    }
    if (kPrefill && rank == 0 && et == 0) {
      a.piece[2 * unit] = ending;
      a.piece[2 * unit + 1] = beginning;
    }
    if (!ok || !mine) give_up();
  } else {
    if constexpr (kPrefill) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
    // a tile's boxes of keys in a CTA. A decode's loaders are warps 0, 2 (free behind the allocation), 8 and 9, as far
    // as there is a box for each: one without would hold up nobody, could fall two rounds of the ring behind and then
    // wait for a phase that is over.
    const int rows_box = min(a.m.page, 64), boxes = kCtaRows / rows_box, loader = warp < 8 ? warp >> 1 : warp - 6;
    if (kPrefill ? warp == 0 || warp == 3 : warp == 3 || (warp != 1 && loader < boxes)) {
      // ------------------------------------------------------------ loads, in both CTAs: warp 0 the ring,
      // warp 3 the resident operand; keys are looked up by lanes, one a box. A warp hands over a box every 50 to 70
      // ns, so up to four warps share a decode's ring (64 sequences of 1K-16K, pages of 16 rows: 134 us with one, 115 with
      // two, 111 with four; of 8 rows 200, 149, 120; of 64 rows 106 to 109 with each).
      const bool ring_role = warp != 3;
      bool ok = true;
      auto wait = [&](uint64_t* bar, int parity) { ok = ok && __all_sync(0xffffffffu, wait_for(bar, parity, abort)); };
      // this lane's box of the CTA's rows of tile k: its block (outside the cache: none, loads zeros) and row
      auto look_up = [&](int k, int& id, int& row) {
        const int t = kRows * k + kCtaRows * (int)rank + lane * rows_box;
        id = a.m.num_blocks;
        row = 0;
        if (lane < boxes && t < wk.t.s.kv) {
          const int page = t / a.m.page, got = a.m.block_table[wk.b * a.m.bt_stride + page];
          if (got >= 0 && got < a.m.num_blocks) {
            id = got;
            row = t - page * a.m.page;
          }
        }
      };
      auto load_keys = [&](unsigned char* dst, uint64_t* bar, int c, int id, int row) {
        // each lane its own: handed to one lane, boxes of 16 rows took 170 us
        if (lane < boxes && (kPrefill || (lane & 3) == loader))
          load_pair_3d_lane(dst + lane * rows_box * 128, &kmap, map_to_rank(bar, 0), 64 * c, row, id);
        __syncwarp();
        if (rank == 0 && (kPrefill || warp == 0)) expect_bytes(bar, 2 * kChunkBytes);
      };
      auto load_queries = [&](unsigned char* dst, uint64_t* bar, int c, int h0, int tok) {
        load_pair_3d(dst, &qmap, map_to_rank(bar, 0), 64 * c, h0, tok);
        const int rows = kPrefill ? a.m.H * a.tpc : a.half;
        if (rank == 0) expect_bytes(bar, 2u * rows * 128);
      };
      if (ring_role) {
        int stage = 0, round = 0;
        auto take = [&](auto&& load) {   // every chunk of a tile through the ring
  #pragma unroll 1
          for (int c = 0; ok && c < a.chunks; ++c) {
            if (round > 0) wait(&sh.ring_empty[stage], (round & 1) ^ 1);
            if (!ok) break;
            load(ring + stage * kChunkBytes, &sh.ring_full[stage], c);
            if (++stage == a.stages) {
              stage = 0;
              ++round;
            }
          }
        };
        while (ok && wk.next(a, sg)) {
          if (kPrefill) {
            for (int i = sg.i0; ok && i < sg.i1; ++i) {
              const int tok = wk.t.s.q0 + (2 * i + (int)rank) * a.tpc;
              take([&](unsigned char* dst, uint64_t* bar, int c) { load_queries(dst, bar, c, 0, tok); });
            }
          } else {
            int id, row;
            look_up(sg.i0, id, row);
            for (int i = sg.i0; ok && i < sg.i1; ++i) {
              int id1 = 0, row1 = 0;   // the next tile's: asked for under this one's loads
              if (i + 1 < sg.i1) look_up(i + 1, id1, row1);
              take([&](unsigned char* dst, uint64_t* bar, int c) { load_keys(dst, bar, c, id, row); });
              id = id1;
              row = row1;
            }
          }
        }
      } else {
        for (int g = 0; ok && wk.next(a, sg); ++g) {
          int id = 0, row = 0;
          if (kPrefill) look_up(sg.outer, id, row);
  #pragma unroll 1
          for (int c = 0; ok && c < a.chunks; ++c) {
            if (g > 0) wait(&sh.res_empty[c], (g & 1) ^ 1);
            if (!ok) break;
            if (kPrefill)
              load_keys(smem + c * res_bytes, &sh.res_full[c], c, id, row);
            else
              load_queries(smem + c * res_bytes, &sh.res_full[c], c, (int)rank * a.half, wk.t.s.q0);
          }
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
      // ------------------------------------------------------------ MMA issuer of the pair
      const uint32_t idesc = __reduce_max_sync(0xffffffffu, idesc_bf16(kRows, 0, false, false) | (uint32_t)(a.n >> 3) << 17);
      const uint32_t res_lo = desc_lo(smem), ring_lo = desc_lo(ring);
      bool ok = true;
      auto wait = [&](uint64_t* bar, int parity) {
        ok = ok && __all_sync(0xffffffffu, wait_for(bar, parity, abort));
        return ok;
      };
      int stage = 0, round = 0, x = 0;
      for (int g = 0; ok && wk.next(a, sg); ++g) {
        const int i0 = __reduce_max_sync(0xffffffffu, sg.i0), i1 = __reduce_max_sync(0xffffffffu, sg.i1);
        for (int i = i0; ok && i < i1; ++i, ++x) {
          // decode: both accumulators of a tile, in turn in two places; prefill: one behind the other
          const int buf = kPrefill ? 0 : x & 1;
          if (kPrefill ? x > 0 && !wait(&sh.d_empty[0], (x & 1) ^ 1) : x > 1 && !wait(&sh.d_empty[buf], ((x >> 1) & 1) ^ 1)) break;
  #pragma unroll 1
          for (int c = 0; c < a.chunks; ++c) {
            if (kPrefill && c == a.split) {
              commit_pair(&sh.d_full[0]);
              if (x > 0 && !wait(&sh.d_empty[1], (x & 1) ^ 1)) break;
            }
            if (i == i0 && !wait(&sh.res_full[c], g & 1)) break;
            if (!wait(&sh.ring_full[stage], round & 1)) break;
            tc_fence_after();
            const uint32_t d = __reduce_max_sync(0xffffffffu, 256u * buf + (c < a.split ? 0u : kSecond<kPrefill>));
            const uint32_t r = __reduce_max_sync(0xffffffffu, res_lo + c * (res_bytes >> 4));
            const uint32_t s = __reduce_max_sync(0xffffffffu, ring_lo + stage * (kChunkBytes >> 4));
            umma_pair4(d, kPrefill ? r : s, kPrefill ? s : r, idesc, c == 0 || c == a.split);
            commit_pair(&sh.ring_empty[stage]);
            if (i + 1 == i1) commit_pair(&sh.res_empty[c]);
            if (++stage == a.stages) {
              stage = 0;
              ++round;
            }
          }
          if (ok) commit_pair(&sh.d_full[kPrefill ? (a.chunks > 1 ? 1 : 0) : buf]);
        }
      }
      if (!ok && lane == 0) give_up();
      __syncwarp();
      commit_pair(&sh.fin);
    }
  }
  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    volatile int dummy = 0;
    if (!mbar_wait(&sh.fin, 0, &dummy) || sh.abort_flag) atomicOr(&g_mass_tc_err, kErrTimeout);
  }
  __syncthreads();
  cluster_sync();   // neither CTA frees or leaves while the other's MMAs or copies may touch it
  if (warp == 2) {
    tc_fence_after();
    dealloc_pair(tmem, 512);
  }
  cluster_sync();
}

// Block u - 1 looks at the rows that end in, or go on through, unit u's first tiles. If they begin in the unit
// before (units without tiles aside), it adds up their pieces in order.
__global__ void __launch_bounds__(kRows) mass_merge_kernel(const TcArgs a, int units) {
  pdl_enter();
  __shared__ int4 piece[kMaxUnits][2];
  const int u = blockIdx.x + 1, e = threadIdx.x;
  for (int i = e; i < 2 * units; i += kRows) piece[i >> 1][i & 1] = a.piece[i];
  __syncthreads();
  const int4 p = piece[u][0];
  if (p.x < 0) return;
  int v = u - 1;
  while (v > 0 && piece[v][0].x < 0 && piece[v][1].x < 0) --v;
  if (piece[v][1].x != p.x || piece[v][1].y != p.y) return;   // an earlier piece of the same rows
  const int row = kRows * p.y + e;
  if (row >= p.w) return;
  const int id = a.m.block_table[p.x * a.m.bt_stride + row / a.m.page];
  float* const to = a.m.mass + p.x * a.m.mass_stride + row;
  const float old = a.m.decay == 0.f ? 0.f : *to;
  float sum = a.part[((int64_t)v * 2 + 1) * kRows + e];
  for (v = u; v < units; ++v) {
    if (piece[v][0].x < 0) continue;                          // without tiles
    sum += a.part[(int64_t)v * 2 * kRows + e];
    if (piece[v][0].z != 0) break;
  }
  if (id < 0 || id >= a.m.num_blocks) return;                 // recorded by the kernel before
  *to = new_mass(old, sum, a.m.decay);
}

template <bool kPrefill>
int max_pairs() {
  static std::mutex mu;
  static std::vector<int> cache;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    dev = 0;
  }
  std::lock_guard<std::mutex> g(mu);
  if ((int)cache.size() <= dev) cache.resize(dev + 1, 0);
  if (cache[dev] == 0) {
    cudaFuncSetAttribute(mass_tc_kernel<kPrefill>, cudaFuncAttributeMaxDynamicSharedMemorySize, kArena + kMiscBytes);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * device_sm_count(), 1, 1);
    cfg.blockDim = dim3(kThreads<kPrefill>, 1, 1);
    cfg.dynamicSmemBytes = kArena + kMiscBytes;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, mass_tc_kernel<kPrefill>, &cfg) != cudaSuccess || n <= 0) n = device_sm_count() / 2;
    cudaGetLastError();
    cache[dev] = std::min(n, kMaxUnits);
  }
  return cache[dev];
}

template <bool kPrefill>
cudaError_t launch(const TcArgs& a, const MassMaps& maps, int units, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(mass_tc_kernel<kPrefill>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kArena + kMiscBytes);
  if (e != cudaSuccess) return e;
  if (kPrefill) {
    // the shares of setmaxnreg draw on what the kernel was compiled for: with less they would wait for ever
    static std::atomic<int> regs{0};
    if (regs.load() == 0) {
      cudaFuncAttributes attr;
      const cudaError_t f = cudaFuncGetAttributes(&attr, mass_tc_kernel<kPrefill>);
      if (f != cudaSuccess) return f;
      regs.store(attr.numRegs);
    }
    if (regs.load() != kLaunchRegs) return cudaErrorInvalidKernelImage;
  }
  return launch_k(mass_tc_kernel<kPrefill>, dim3(2 * units), dim3(kThreads<kPrefill>), kArena + kMiscBytes, st, maps.keys, maps.q, a);
}

int tokens_per_cta(int H) { return std::max(1, kCtaRows / H); }
// Query rows of a decode's tile: the heads in whole groups of 32, as cta_group::2 takes them.
int decode_rows(int H) { return (H + 31) / 32 * 32; }

}  // namespace

bool mass_tc_supported(mla_dtype dt, const MassCall& c, MassMaps* maps) {
  const int E = c.cache.entry, page = c.cache.page;
  if (dt != MLA_BF16 || E % 64 != 0 || E > 64 * kMaxChunks || c.H > 128) return false;
  if (!(page % 64 == 0 || (64 % page == 0 && page % 8 == 0))) return false;
  auto al16 = [](const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15) == 0; };
  if (!al16(c.cache.data) || c.cache.s_blk % 8 || c.cache.s_row % 8 || !al16(c.q.data) || c.q.s0 % 8 || c.q.s1 % 8) return false;
  const uint32_t box_rows = (uint32_t)std::min(page, 64);
  const bool decode = c.cu_q == nullptr;
  const uint32_t heads = decode ? (uint32_t)decode_rows(c.H) / 2 : (uint32_t)c.H, toks = decode ? 1u : (uint32_t)tokens_per_cta(c.H);
  return make_map3d(&maps->keys, c.cache.data, E, page, c.cache.num_blocks, (uint64_t)c.cache.s_row * 2,
                    (uint64_t)c.cache.s_blk * 2, 64, box_rows, 1, CU_TENSOR_MAP_SWIZZLE_128B) &&
         make_map3d(&maps->q, c.q.data, E, c.H, c.T, (uint64_t)c.q.s1 * 2, (uint64_t)c.q.s0 * 2, 64, heads, toks,
                    CU_TENSOR_MAP_SWIZZLE_128B);
}

size_t mass_tc_workspace() { return (size_t)max_pairs<true>() * 2 * (kRows * sizeof(float) + sizeof(int4)); }

cudaError_t launch_mass_tc(const MassCall& c, const MassMaps& maps, void* ws, cudaStream_t st) {
  const bool decode = c.cu_q == nullptr;
  TcArgs a{};
  a.m = mass_args(c);
  a.chunks = c.cache.entry / 64;
  a.split = (a.chunks + 1) / 2;
  a.tpc = tokens_per_cta(c.H);
  a.n = decode ? decode_rows(c.H) : kRows;
  a.half = a.n / 2;
  a.stages = std::min(kMaxStages, (kArena - a.chunks * (decode ? a.half * 128 : kChunkBytes)) / kChunkBytes);
  if (decode) return launch<false>(a, maps, max_pairs<false>(), st);
  const int units = max_pairs<true>();
  a.part = static_cast<float*>(ws);
  a.piece = reinterpret_cast<int4*>(a.part + (int64_t)units * 2 * kRows);
  const cudaError_t e = launch<true>(a, maps, units, st);
  if (e != cudaSuccess || units < 2) return e;
  return launch_k(mass_merge_kernel, dim3(units - 1), dim3(kRows), 0, st, a, units);
}

cudaError_t mass_tc_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_mass_tc_err);
}

}  // namespace mla
