// Eviction of the lightest rows of each sequence of a paged cache: of n > budget rows the first
// `sinks`, the last `recent` and the heaviest of the others stay, `budget` in all, and move together
// in their order.
//
// Selection. A mass becomes a 32-bit key of the same order (-0 counts as 0, NaN as the heaviest). The
// smallest key that stays is found eleven, eleven and ten bits at a time from the top: counts of the keys by
// those bits in shared memory (sums, whatever their order), then the digit where the wanted count is reached;
// fewer passes where it is reached exactly. A block (256 to 1024 threads, by the rows that the table and the masses
// have room for), or for long sequences a cluster of up to eight, holds sixteen keys a thread in registers, and
// reads longer sequences again. A cluster's blocks add the few bins that they fill to every block's sums: reading
// one another's 2048 bins instead took 16K rows 45 us with eight blocks of 256 threads, not 22. Two bits a round
// by counting keys above three limits took 20.8 us for 64 sequences of 1K to 8K rows instead of 14.
// Of the rows with the smallest key that stays the lowest stay.
//
// Moving. Row kept[j] becomes row j <= kept[j], in place: what a step writes, rows j .. , no later step
// reads (their sources lie at or behind their targets), so a block that takes rows in ascending order,
// all loads of a step before its stores, needs no second copy, and may load later steps before it stores
// earlier ones. Columns do not touch one another: a sequence is cut into slices of columns, a block each that
// takes all rows of its slice, or a cluster whose blocks take a step's rows in turn, with its barrier between
// the loads and the stores. Rows pass through shared memory (asynchronous copies, two
// steps in flight, each thread its own words): held in registers, one step at a time, 64 sequences of 1K to 8K
// rows took 58 us to move instead of 38 (5.7 TB/s).
#include <algorithm>
#include <climits>

#include "mla_internal.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

__device__ unsigned g_evict_err = 0;

constexpr int kMaxSelectThreads = 1024;
constexpr int kPer = 16;                             // rows a thread holds
constexpr int kBins = 2048;                          // eleven bits
constexpr int kMoveThreads = 256;
constexpr int kInStep = 4;                           // rows a thread moves a step
constexpr int kWords = 2;                            // words of each: its row's look-up serves both
constexpr int kStages = 2;                           // steps in flight
constexpr int kMaxCluster = 8;                       // blocks of one sequence (selection), of one slice (moving)

struct SelectArgs {
  float* mass;
  int64_t mass_stride;
  const int32_t* seq_lens;
  int32_t cap;                                       // rows that the table and the masses hold
  int32_t budget, sinks, recent;
  float* mass_out;
  int64_t out_stride;
  int32_t out_rows;
  int32_t *seq_lens_out, *kept_out;                  // kept_out: null or [B, budget]
  int32_t* list;                                     // [B, list_stride] rows that stay, in order
  int32_t list_stride;
  int2* moved;                                       // [B] {first row that moves, rows that stay}
};

// Larger masses have larger keys; the smallest is above 0 (a place without a row).
__device__ __forceinline__ uint32_t key_of(float m) {
  if (m != m) return 0xffffffffu;
  const uint32_t u = __float_as_uint(m + 0.f);       // -0 + 0 = 0
  return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);  // at least 0x007fffff (-infinity)
}

using Exchange = int (*)[32];   // a word a warp, in turn in two places

// Sum of v over the threads before this one; total: over all.
__device__ __forceinline__ int block_before(int v, Exchange sh, int& turn, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[turn][warp] = x;
  __syncthreads();
  int s = lane < (int)(blockDim.x >> 5) ? sh[turn][lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  turn ^= 1;
  return (warp > 0 ? before : 0) + x - v;
}

// A barrier of the cluster's blocks.
template <bool kClusters>
__device__ __forceinline__ void together() {
  if constexpr (kClusters)
    ptx::cluster_sync();
  else
    __syncthreads();
}

// v added to rank's copy of *p.
__device__ __forceinline__ void add_rank(int* p, int rank, int v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(ptx::map_to_rank(p, rank)), "r"(v) : "memory");
}

// rank's copy of *p.
__device__ __forceinline__ int ld_rank(const int* p, int rank) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(ptx::map_to_rank(p, rank)) : "memory");
  return v;
}

// One cluster a sequence: which rows stay, their masses, the new length. Each barrier of the cluster parts what its
// blocks wrote for one another from the reads; places written before a barrier are written again two barriers later.
template <bool kClusters>
__global__ void __launch_bounds__(kMaxSelectThreads) evict_select_kernel(const SelectArgs a) {
  pdl_enter();
  __shared__ int sh[2][32], hist[kBins], sums[2][kClusters ? kBins : 1], found[3], counts[2], first[kMaxCluster];
  const int b = blockIdx.y, tid = threadIdx.x, threads = blockDim.x;
  const int blocks = kClusters ? gridDim.x : 1, rank = kClusters ? blockIdx.x : 0;
  const int all_threads = threads * blocks, place = threads * rank + tid;
  float* const mass = a.mass + b * a.mass_stride;
  float* const out = a.mass_out + b * a.out_stride;
  int32_t* const list = a.list + (int64_t)b * a.list_stride;
  int32_t* const kept = a.kept_out == nullptr ? nullptr : a.kept_out + (int64_t)b * a.budget;
  int n = a.seq_lens[b];
  if (n < 0 || n > a.cap) {
    if (tid == 0) atomicOr(&g_evict_err, kErrDeviceData);
    n = n < 0 ? 0 : a.cap;
  }
  const bool cut = n > a.budget;
  const int left = cut ? a.budget : n;
  // rows that may go lie in [lo, hi); `take` of them stay
  const int lo = cut ? a.sinks : 0, hi = cut ? n - a.recent : 0, take = cut ? a.budget - a.sinks - a.recent : 0;
  const bool in_regs = n <= all_threads * kPer;
  const int per = in_regs ? (n + all_threads - 1) / all_threads : kPer;
  uint32_t key[kPer];
  float val[kPer];
  auto load = [&](int c0) {                          // the thread's rows of a chunk
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i >= per) break;
      const int t = c0 + place * per + i;
      val[i] = t < n ? mass[t] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i >= per) break;
      const int t = c0 + place * per + i;
      key[i] = t >= lo && t < hi ? key_of(val[i]) : 0u;
    }
  };
  if constexpr (kClusters) {                         // no block writes to another that is not there yet
    for (int i = tid; i < kBins; i += threads) sums[0][i] = 0;
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  if (in_regs) load(0);
  if constexpr (kClusters) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  int turn = 0;
  uint32_t edge = 0;                                 // the smallest key that stays: its upper bits so far
  int above = 0;                                     // rows with a larger one
  if (take > 0) {
    for (int shift = 21, bits = 11;; shift = bits == 11 && shift == 21 ? 10 : 0) {
      bits = shift == 0 ? 10 : 11;
      const int bins = 1 << bits;
      for (int i = tid; i < bins; i += threads) hist[i] = 0;
      __syncthreads();
      // keys with the bits found so far (0: no row that may go)
      auto count = [&](uint32_t k) {
        if (k != 0 && (shift == 21 || k >> (shift + bits) == edge)) atomicAdd(&hist[k >> shift & (bins - 1)], 1);
      };
      if (in_regs) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (i >= per) break;
          count(key[i]);
        }
      } else {
#pragma unroll 8
        for (int t = lo + place; t < hi; t += all_threads) count(key_of(mass[t]));
      }
      __syncthreads();
      int* const sum = kClusters ? sums[shift == 10] : hist;
      if constexpr (kClusters) {                     // most bins are empty
        for (int i = tid; i < kBins; i += threads) {
          const int v = i < bins ? hist[i] : 0;
          for (int r = 0; v != 0 && r < blocks; ++r) add_rank(sum + i, r, v);
          sums[shift != 10][i] = 0;                  // the next pass's: read a barrier ago
        }
        ptx::cluster_sync();
      }
      // from the top bin down, `mine` of them a thread: the one in which the count is reached
      const int want = take - above, mine = bins / threads, top = bins - 1 - tid * mine;
      int here = 0, total;
      for (int i = 0; i < mine; ++i) here += sum[top - i];
      int before = block_before(here, sh, turn, total);
      if (before < want && before + here >= want) {
        int i = 0;
        while (before + sum[top - i] < want) before += sum[top - i++];
        found[0] = top - i;
        found[1] = before;
        found[2] = sum[top - i];
      }
      __syncthreads();
      edge = edge << bits | (uint32_t)found[0];
      above += found[1];
      const bool all = above + found[2] == take;
      if (all) {               // every key of the bin stays: none below it
        edge = (edge << shift) - 1;
        above = take;
      }
      if (all || shift == 0) break;
    }
  }
  const int even = take - above;                     // rows with the edge's key that stay: the lowest
  // rows of the chunks before: that stay for certain; with the edge's key
  int sure_before = 0, even_before = 0, first_moved = left, chunk = 0;
  for (int c0 = 0; c0 < n; c0 += per * all_threads, chunk ^= 1) {
    if (!in_regs) load(c0);
    uint32_t sure = 0, same = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i >= per) break;
      const int t = c0 + place * per + i;
      if (t >= n) continue;
      const bool s = t < lo || t >= hi || (take > 0 && key[i] > edge);
      sure |= (uint32_t)s << i;
      same |= (uint32_t)(!s && even > 0 && key[i] == edge) << i;
    }
    // both counts in one word: a block's are at most 2^14
    int total;
    const int before = block_before(__popc(sure) | __popc(same) << 16, sh, turn, total);
    int s = sure_before + (before & 0xffff), e = even_before + (before >> 16);
    if constexpr (kClusters) {
      if (tid == 0) counts[chunk] = total;
      ptx::cluster_sync();
      for (int r = 0; r < blocks; ++r) {
        const int v = ld_rank(counts + chunk, r);
        if (r < rank) {
          s += v & 0xffff;
          e += v >> 16;
        }
        sure_before += v & 0xffff;
        even_before += v >> 16;
      }
    } else {
      sure_before += total & 0xffff;
      even_before += total >> 16;
    }
    // every block has read the chunk (a barrier lies behind): stores may follow
    int j = s + min(e, even);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i >= per) break;
      const int t = c0 + place * per + i;
      const bool tie = same >> i & 1u;
      if (!(sure >> i & 1u) && !(tie && e < even)) {
        e += tie;
        continue;
      }
      e += tie;
      if (j < left) {                                // (always: as many stay as counted)
        list[j] = t;
        if (kept != nullptr) kept[j] = t;
        if (j < a.out_rows) out[j] = val[i];
        if (t != j) first_moved = min(first_moved, j);
      }
      ++j;
    }
  }
  // What is left of the sequence's old rows has no mass. (In place: every chunk is read by now, and rows behind
  // `left` are stored here alone.)
  for (int t = left + place; t < n && t < a.out_rows; t += all_threads) out[t] = 0.f;
  if (kept != nullptr)
    for (int t = left + place; t < a.budget; t += all_threads) kept[t] = -1;
  first_moved = __reduce_min_sync(0xffffffffu, first_moved);
  if ((tid & 31) == 0) sh[turn][tid >> 5] = first_moved;
  __syncthreads();
  if (tid < 32) {
    first_moved = __reduce_min_sync(0xffffffffu, tid < threads / 32 ? sh[turn][tid] : left);
    if (tid == 0)
      asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(ptx::map_to_rank(first + rank, 0)), "r"(first_moved) : "memory");
  }
  together<kClusters>();                             // behind it no block reads another's memory
  if (rank == 0 && tid == 0) {
    for (int r = 0; r < blocks; ++r) first_moved = min(first_moved, first[r]);
    a.moved[b] = make_int2(first_moved, left);
    a.seq_lens_out[b] = left;
  }
}

struct MoveArgs {
  void* cache;
  int64_t s_blk, s_row;                              // in words
  int32_t num_blocks, words;                         // words of a row
  int32_t blocks;                                    // of a slice
  PageOf page_of;
  const int32_t *table, *table_out;
  int64_t bt_stride, bto_stride;
  int32_t max_blocks_out;
  const int32_t* list;
  int32_t list_stride;
  const int2* moved;
};

// A word of global memory into this thread's place in shared memory, without waiting (a byte: with).
template <typename W>
__device__ __forceinline__ void copy_in(W* dst, const W* src) {
  if constexpr (sizeof(W) == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
  else if constexpr (sizeof(W) == 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
  else
    *dst = *src;
}

// One cluster a sequence and slice of kWords * 2^kShift words: its words of row list[j] to row j, in ascending order,
// a step's rows dealt over the blocks.
template <typename W, int kShift, bool kClusters>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const MoveArgs a) {
  pdl_enter();
  constexpr int kRows = kMoveThreads >> kShift, kStep = kRows * kInStep;
  extern __shared__ __align__(16) unsigned char smem[];
  W (*const buf)[kInStep][kWords][kMoveThreads] = reinterpret_cast<W (*)[kInStep][kWords][kMoveThreads]>(smem);
  // this thread's words are `word` and, where the row has it, the one 2^kShift behind
  const int blocks = kClusters ? a.blocks : 1, slice = blockIdx.x / blocks, rank = blockIdx.x - slice * blocks;
  const int b = blockIdx.y, tid = threadIdx.x, word = (slice * kWords << kShift) + (tid & ((1 << kShift) - 1));
  const int sub = rank * kStep + (tid >> kShift), step = blocks * kStep;
  const int2 m = a.moved[b];
  const int32_t* const list = a.list + (int64_t)b * a.list_stride;
  const int32_t *const table = a.table + b * a.bt_stride, *const table_out = a.table_out + b * a.bto_stride;
  W* const cache = static_cast<W*>(a.cache) + word;
  const int end = word < a.words ? m.y : 0;          // this thread's rows end here
  int next[kInStep];                                 // rows to be loaded in the next step
  auto ask = [&](int j0) {
#pragma unroll
    for (int u = 0; u < kInStep; ++u) {
      const int j = j0 + sub + u * kRows;
      next[u] = j < end ? list[j] : -1;
    }
  };
  // Loads a step; to[u]: the block its row goes to, -1 where nothing is to be done.
  auto load = [&](int stage, int j0, int (&to)[kInStep]) {
#pragma unroll
    for (int u = 0; u < kInStep; ++u) {
      const int j = j0 + sub + u * kRows, t = next[u];
      to[u] = -1;
      if (t < 0) continue;
      const int pf = a.page_of(t), pt = a.page_of(j), rf = t - pf * a.page_of.page;
      const bool there = pt < a.max_blocks_out;
      const int bf = table[pf], bt = there ? table_out[pt] : -1;
      if (there && bf == bt && rf == j - pt * a.page_of.page) continue;   // it stays where it is, whatever the id
      if (bf < 0 || bf >= a.num_blocks || bt < 0 || bt >= a.num_blocks) {
        atomicOr(&g_evict_err, kErrDeviceData);
        continue;
      }
      to[u] = bt;
      const W* const from = cache + bf * a.s_blk + rf * a.s_row;
#pragma unroll
      for (int k = 0; k < kWords; ++k)
        if (k == 0 || word + (k << kShift) < a.words) copy_in(&buf[stage][u][k][tid], from + (k << kShift));
    }
    ptx::cp_async_commit();
  };
  auto store = [&](int stage, int j0, const int (&to)[kInStep]) {
#pragma unroll
    for (int u = 0; u < kInStep; ++u) {
      if (to[u] < 0) continue;
      const int j = j0 + sub + u * kRows;
      W* const o = cache + to[u] * a.s_blk + (j - a.page_of(j) * a.page_of.page) * a.s_row;
#pragma unroll
      for (int k = 0; k < kWords; ++k)
        if (k == 0 || word + (k << kShift) < a.words) o[k << kShift] = buf[stage][u][k][tid];
    }
  };
  const int start = a.table == a.table_out && a.bt_stride == a.bto_stride ? m.x : 0;
  int to[kStages][kInStep];
  ask(start);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    load(s, start + s * step, to[s]);
    ask(start + (s + 1) * step);
  }
  for (int j0 = start; j0 < m.y;) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
      if (j0 >= m.y) break;
      constexpr int kAhead = kStages - 1;
      load((s + kAhead) % kStages, j0 + kAhead * step, to[(s + kAhead) % kStages]);
      ask(j0 + kStages * step);
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
      together<kClusters>();                         // every load up to this step's is done
      store(s, j0, to[s]);
      j0 += step;
    }
  }
}

template <typename W>
cudaError_t launch_move(MoveArgs a, int64_t row_bytes, int32_t batch, int32_t rows, cudaStream_t st) {
  a.words = (int32_t)(row_bytes / sizeof(W));
  a.s_blk /= (int64_t)sizeof(W);
  a.s_row /= (int64_t)sizeof(W);
  // Slices of 8 words (128 bytes), each row's words read in whole sectors. A slice's steps are dealt over 2, 4 or 8
  // blocks while two blocks an SM hold them and the longest list has two steps for each (1 x 128K of which half
  // stay: 375, 215, 133 us; 64 x 1K-8K, where one block a slice fills the SMs: 52.6 us with one, 60.7 with four).
  // Narrower slices where half of the SMs would stay idle all the same (1 x 128K: 107 us of 4 words, 114 of 2).
  auto slices = [&](int shift) { return (a.words + (kWords << shift) - 1) / (kWords << shift); };
  const int64_t sms = device_sm_count(), wide = (int64_t)slices(2) * batch;
  int blocks = 1;
  while (blocks < kMaxCluster && 2 * blocks * wide <= 2 * sms && blocks * (kMoveThreads >> 2) * kInStep * 2 < rows) blocks *= 2;
  a.blocks = blocks;
  constexpr int kBytes = kStages * kInStep * kWords * kMoveThreads * (int)sizeof(W);
  auto go = [&](auto kernel, int shift) {
    if (kBytes > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
      if (e != cudaSuccess) return e;
    }
    return launch_clusters(kernel, blocks, dim3((unsigned)blocks * slices(shift), batch), kMoveThreads, kBytes, st, a);
  };
  const int shift = 2 * blocks * wide >= sms ? 2 : 2 * blocks * slices(1) * batch >= sms ? 1 : 0;
  if (blocks == 1) {
    if (shift == 2) return go(evict_move_kernel<W, 2, false>, 2);
    if (shift == 1) return go(evict_move_kernel<W, 1, false>, 1);
    return go(evict_move_kernel<W, 0, false>, 0);
  }
  if (shift == 2) return go(evict_move_kernel<W, 2, true>, 2);
  if (shift == 1) return go(evict_move_kernel<W, 1, true>, 1);
  return go(evict_move_kernel<W, 0, true>, 0);
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

size_t evict_workspace(int64_t batch, int64_t rows, int64_t budget) {
  return up256(sizeof(int2) * batch) + up256(sizeof(int32_t) * batch * std::min(rows, budget));
}

cudaError_t launch_evict(const EvictCall& c, void* ws, cudaStream_t st) {
  const int32_t list_stride = std::min(c.mass_rows, c.budget);
  int2* const moved = static_cast<int2*>(ws);
  int32_t* const list = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + up256(sizeof(int2) * c.batch));
  const int64_t cap = std::min<int64_t>({(int64_t)c.max_blocks * c.page, c.mass_rows, INT_MAX / 2});
  // eight rows a thread where that keeps the block below 1024: more warps hide a round's latencies
  const int threads = cap <= 256 * kPer / 2 ? 256 : cap <= 512 * kPer / 2 ? 512 : kMaxSelectThreads;
  const SelectArgs s{c.mass, c.mass_stride, c.seq_lens, (int32_t)cap, c.budget, c.sinks, c.recent, c.mass_out, c.mass_out_stride,
                     c.mass_out_rows, c.seq_lens_out, c.kept_out, list, list_stride, moved};
  // Above eight rows a thread of one block: clusters, up to four rows a thread, while every block has an SM (1 x 16K:
  // 21 us instead of 29 for the call, 8 x 32K: 57 instead of 97; 64 x 8K: 61 instead of 60, and below that
  // a cluster's barriers cost more than they save).
  int blocks = 1;
  if (cap > kMaxSelectThreads * kPer / 2)
    while (blocks < kMaxCluster && 2 * (int64_t)blocks * c.batch <= device_sm_count() && blocks * kMaxSelectThreads * kPer / 4 < cap)
      blocks *= 2;
  const cudaError_t e = launch_clusters(blocks > 1 ? evict_select_kernel<true> : evict_select_kernel<false>, blocks, dim3(blocks, c.batch), threads, 0, st, s);
  if (e != cudaSuccess) return e;
  const MoveArgs m{c.cache, c.s_blk, c.s_row, c.num_blocks, 0, 1, PageOf(c.page), c.block_table, c.block_table_out, c.bt_stride,
                   c.bto_stride, c.max_blocks_out, list, list_stride, moved};
  const int64_t all = (int64_t)reinterpret_cast<uintptr_t>(c.cache) | c.s_blk | c.s_row | c.row_bytes;
  if (all % 16 == 0) return launch_move<uint4>(m, c.row_bytes, c.batch, list_stride, st);
  if (all % 4 == 0) return launch_move<uint32_t>(m, c.row_bytes, c.batch, list_stride, st);
  return launch_move<uint8_t>(m, c.row_bytes, c.batch, list_stride, st);
}

cudaError_t evict_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_evict_err);
}

}  // namespace mla
