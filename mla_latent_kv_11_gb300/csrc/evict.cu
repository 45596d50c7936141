// Eviction of the lightest rows of each sequence of a paged cache: of n > budget rows the first
// `sinks`, the last `recent` and the heaviest of the others stay, `budget` in all, and move together
// in their order.
//
// Selection. A mass becomes a 32-bit key of the same order (-0 counts as 0, NaN as the heaviest). The
// smallest key that stays is found eleven, eleven and ten bits at a time from the top: counts of the keys by
// those bits in shared memory (sums, whatever their order), then the digit where the wanted count is reached;
// fewer passes where it is reached exactly. A block (256 to 1024 threads, by the rows that the table and the masses
// have room for) holds sixteen keys a thread in registers, and reads longer sequences again. Two bits a round
// by counting keys above three limits took 20.8 us for 64 sequences of 1K to 8K rows instead of 14.
// Of the rows with the smallest key that stays the lowest stay.
//
// Moving. Row kept[j] becomes row j <= kept[j], in place: what a step writes, rows j .. , no later step
// reads (their sources lie at or behind their targets), so a block that takes rows in ascending order,
// all loads of a step before its stores, needs no second copy, and may load later steps before it stores
// earlier ones. Columns do not touch one another: a sequence is cut into slices of columns, a block each, and
// every block takes all rows of its slice. Rows pass through shared memory (asynchronous copies, two
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

// One block a sequence: which rows stay, their masses, the new length.
__global__ void __launch_bounds__(kMaxSelectThreads) evict_select_kernel(const SelectArgs a) {
  pdl_enter();
  __shared__ int sh[2][32], hist[kBins], found[3];
  const int b = blockIdx.x, tid = threadIdx.x, threads = blockDim.x;
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
  const bool in_regs = n <= threads * kPer;
  const int per = in_regs ? (n + threads - 1) / threads : kPer;
  uint32_t key[kPer];
  float val[kPer];
  auto load = [&](int first) {                       // the thread's rows of a chunk
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i >= per) break;
      const int t = first + tid * per + i;
      val[i] = t < n ? mass[t] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i >= per) break;
      const int t = first + tid * per + i;
      key[i] = t >= lo && t < hi ? key_of(val[i]) : 0u;
    }
  };
  if (in_regs) load(0);
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
        for (int t = lo + tid; t < hi; t += threads) count(key_of(mass[t]));
      }
      __syncthreads();
      // from the top bin down, `mine` of them a thread: the one in which the count is reached
      const int want = take - above, mine = bins / threads, top = bins - 1 - tid * mine;
      int here = 0, total;
      for (int i = 0; i < mine; ++i) here += hist[top - i];
      int before = block_before(here, sh, turn, total);
      if (before < want && before + here >= want) {
        int i = 0;
        while (before + hist[top - i] < want) before += hist[top - i++];
        found[0] = top - i;
        found[1] = before;
        found[2] = hist[top - i];
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
  int at = 0, seen = 0, first_moved = left;
  for (int c0 = 0; c0 < n; c0 += per * threads) {
    if (!in_regs) load(c0);
    int same = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i >= per) break;
      same += even > 0 && key[i] == edge;
    }
    int total = 0, rank = seen;
    if (even > 0) rank += block_before(same, sh, turn, total);
    seen += total;
    uint32_t stay = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i >= per) break;
      const int t = c0 + tid * per + i;
      if (t >= n) continue;
      bool s = t < lo || t >= hi;
      if (!s && take > 0) s = key[i] > edge || (key[i] == edge && rank++ < even);
      stay |= (uint32_t)s << i;
    }
    int j = at + block_before(__popc(stay), sh, turn, total);   // its barrier: the chunk is read, stores may follow
    at += total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i >= per) break;
      const int t = c0 + tid * per + i;
      if (!((stay >> i) & 1u)) continue;
      if (j < left) {                                // (always: as many stay as counted)
        list[j] = t;
        if (kept != nullptr) kept[j] = t;
        if (j < a.out_rows) out[j] = val[i];
        if (t != j) first_moved = min(first_moved, j);
      }
      ++j;
    }
  }
  // behind every store of a mass: what is left of the sequence's old rows has none. (In place, a chunk's
  // loads come before its stores, and rows behind `left` are stored here alone.)
  __syncthreads();
  for (int t = left + tid; t < n && t < a.out_rows; t += threads) out[t] = 0.f;
  if (kept != nullptr)
    for (int t = left + tid; t < a.budget; t += threads) kept[t] = -1;
  first_moved = __reduce_min_sync(0xffffffffu, first_moved);
  if ((tid & 31) == 0) sh[turn][tid >> 5] = first_moved;
  __syncthreads();
  if (tid < 32) {
    first_moved = __reduce_min_sync(0xffffffffu, tid < threads / 32 ? sh[turn][tid] : left);
    if (tid == 0) {
      a.moved[b] = make_int2(first_moved, left);
      a.seq_lens_out[b] = left;
    }
  }
}

struct MoveArgs {
  void* cache;
  int64_t s_blk, s_row;                              // in words
  int32_t num_blocks, words;                         // words of a row
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

// One block a sequence and slice of kWords * 2^kShift words: its words of row list[j] to row j, in ascending order.
template <typename W, int kShift>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const MoveArgs a) {
  pdl_enter();
  constexpr int kRows = kMoveThreads >> kShift, kStep = kRows * kInStep;
  extern __shared__ __align__(16) unsigned char smem[];
  W (*const buf)[kInStep][kWords][kMoveThreads] = reinterpret_cast<W (*)[kInStep][kWords][kMoveThreads]>(smem);
  // this thread's words are `word` and, where the row has it, the one 2^kShift behind
  const int b = blockIdx.y, tid = threadIdx.x, word = ((int)blockIdx.x * kWords << kShift) + (tid & ((1 << kShift) - 1));
  const int sub = tid >> kShift;
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
      const int pf = a.page_of(t), pt = a.page_of(j);
      const int bf = table[pf], bt = pt < a.max_blocks_out ? table_out[pt] : -1;
      if (bf < 0 || bf >= a.num_blocks || bt < 0 || bt >= a.num_blocks) {
        atomicOr(&g_evict_err, kErrDeviceData);
        continue;
      }
      const int rf = t - pf * a.page_of.page;
      if (bf == bt && rf == j - pt * a.page_of.page) continue;
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
    load(s, start + s * kStep, to[s]);
    ask(start + (s + 1) * kStep);
  }
  for (int j0 = start; j0 < m.y;) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
      if (j0 >= m.y) break;
      constexpr int kAhead = kStages - 1;
      load((s + kAhead) % kStages, j0 + kAhead * kStep, to[(s + kAhead) % kStages]);
      ask(j0 + kStages * kStep);
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
      __syncthreads();                               // every load up to this step's is done
      store(s, j0, to[s]);
      j0 += kStep;
    }
  }
}

template <typename W>
cudaError_t launch_move(MoveArgs a, int64_t row_bytes, int32_t batch, cudaStream_t st) {
  a.words = (int32_t)(row_bytes / sizeof(W));
  a.s_blk /= (int64_t)sizeof(W);
  a.s_row /= (int64_t)sizeof(W);
  // slices of 8 words (128 bytes), narrower while that leaves SMs without two blocks
  auto slices = [&](int shift) { return (a.words + (kWords << shift) - 1) / (kWords << shift); };
  constexpr int kBytes = kStages * kInStep * kWords * kMoveThreads * (int)sizeof(W);
  auto go = [&](auto kernel, int shift) {
    if (kBytes > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
      if (e != cudaSuccess) return e;
    }
    return launch_k(kernel, dim3(slices(shift), batch), kMoveThreads, kBytes, st, a);
  };
  const int64_t enough = 2 * device_sm_count();
  if ((int64_t)slices(2) * batch >= enough) return go(evict_move_kernel<W, 2>, 2);
  if ((int64_t)slices(1) * batch >= enough) return go(evict_move_kernel<W, 1>, 1);
  return go(evict_move_kernel<W, 0>, 0);
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
  const cudaError_t e = launch_k(evict_select_kernel, c.batch, threads, 0, st, s);
  if (e != cudaSuccess) return e;
  const MoveArgs m{c.cache, c.s_blk, c.s_row, c.num_blocks, 0, PageOf(c.page), c.block_table, c.block_table_out, c.bt_stride,
                   c.bto_stride, c.max_blocks_out, list, list_stride, moved};
  const int64_t all = (int64_t)reinterpret_cast<uintptr_t>(c.cache) | c.s_blk | c.s_row | c.row_bytes;
  if (all % 16 == 0) return launch_move<uint4>(m, c.row_bytes, c.batch, st);
  if (all % 4 == 0) return launch_move<uint32_t>(m, c.row_bytes, c.batch, st);
  return launch_move<uint8_t>(m, c.row_bytes, c.batch, st);
}

cudaError_t evict_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_evict_err);
}

}  // namespace mla
