// Eviction of the lightest rows of each sequence of a paged cache: of n > budget rows the first
// `sinks`, the last `recent` and the heaviest of the others stay, `budget` in all, and move together
// in their order.
//
// Selection. A mass becomes a 32-bit key of the same order (-0 counts as 0, NaN as the heaviest). The
// smallest key that stays is found two bits at a time from the top: three counts over the sequence a
// round, sixteen rounds. Up to 16384 rows the keys stay in registers, sixteen a thread, and a round is
// a few compares, warp sums and one barrier: no histogram, whose counters the masses of one binade would
// all fight over, and no atomics. Of the rows with that key the lowest stay.
//
// Moving. Row kept[j] becomes row j <= kept[j], in place: what a step writes, rows j .. , no later step
// reads (their sources lie at or behind their targets), so a block that takes rows in ascending order,
// all loads of a step before its stores, needs no second copy. Columns do not touch one another: a
// sequence is cut into slices of columns, a block each, and every block takes all rows of its slice.
#include <algorithm>
#include <climits>

#include "mla_internal.h"

namespace mla {
namespace {

__device__ unsigned g_evict_err = 0;

constexpr int kSelectThreads = 1024;
constexpr int kPer = 16;                             // rows a thread holds
constexpr int kChunk = kSelectThreads * kPer;        // rows of a block in registers
constexpr int kMoveThreads = 256;
constexpr int kInFlight = 4;                         // rows a thread has in flight

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

// Sums of the block's threads: every thread gets each of them. `sh` is used in turn in two places.
template <int N>
__device__ __forceinline__ void block_sums(int (&v)[N], int (*sh)[N][32], int& turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int s = __reduce_add_sync(0xffffffffu, v[i]);
    if (lane == 0) sh[turn][i][warp] = s;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __reduce_add_sync(0xffffffffu, sh[turn][i][lane]);
  turn ^= 1;
}

// Sum of v over the threads before this one; total: over all.
__device__ __forceinline__ int block_before(int v, int (*sh)[3][32], int& turn, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[turn][0][warp] = x;
  __syncthreads();
  int s = sh[turn][0][lane];
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
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const SelectArgs a) {
  pdl_enter();
  __shared__ int sh[2][3][32];
  const int b = blockIdx.x, tid = threadIdx.x;
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
  const bool in_regs = n <= kChunk;
  const int per = in_regs ? (n + kSelectThreads - 1) / kSelectThreads : kPer;
  uint32_t key[kPer];
  float val[kPer];
  auto load = [&](int first) {                       // the thread's rows of a chunk
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = first + tid * per + i;
      const bool real = i < per && t < n;
      val[i] = real ? mass[t] : 0.f;
      key[i] = real && t >= lo && t < hi ? key_of(val[i]) : 0u;
    }
  };
  if (in_regs) load(0);
  int turn = 0;
  uint32_t edge = 0;                                 // the smallest key that stays
  int above = 0;                                     // rows with a larger one
  if (take > 0) {
    for (int shift = 30; shift >= 0; shift -= 2) {
      // rows at or above edge + 3, 2, 1 << shift; `take` of them or more: the edge lies there
      const uint32_t step = 1u << shift, e1 = edge + step, e2 = e1 + step, e3 = e2 + step;
      int c[3] = {0, 0, 0};
      auto count = [&](uint32_t k) {
        c[0] += k >= e1;
        c[1] += k >= e2;
        c[2] += k >= e3;
      };
      if (in_regs) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (i < per) count(key[i]);
      } else {
#pragma unroll 8
        for (int t = lo + tid; t < hi; t += kSelectThreads) count(key_of(mass[t]));
      }
      block_sums(c, sh, turn);
      if (c[2] >= take) {
        edge = e3;
      } else if (c[1] >= take) {
        edge = e2;
        above = c[2];
      } else if (c[0] >= take) {
        edge = e1;
        above = c[1];
      } else {
        above = c[0];
      }
    }
  }
  const int even = take - above;                     // rows with the edge's key that stay: the lowest
  int at = 0, seen = 0, first_moved = left;
  for (int c0 = 0; c0 < n; c0 += per * kSelectThreads) {
    if (!in_regs) load(c0);
    int same = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) same += take > 0 && key[i] == edge;
    int total;
    int rank = seen + block_before(same, sh, turn, total);
    seen += total;
    uint32_t stay = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = c0 + tid * per + i;
      if (i >= per || t >= n) continue;
      bool s = t < lo || t >= hi;
      if (!s && take > 0) s = key[i] > edge || (key[i] == edge && rank++ < even);
      stay |= (uint32_t)s << i;
    }
    int j = at + block_before(__popc(stay), sh, turn, total);   // its barrier: the chunk is read, stores may follow
    at += total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
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
  for (int t = left + tid; t < n && t < a.out_rows; t += kSelectThreads) out[t] = 0.f;
  if (kept != nullptr)
    for (int t = left + tid; t < a.budget; t += kSelectThreads) kept[t] = -1;
  first_moved = __reduce_min_sync(0xffffffffu, first_moved);
  if ((tid & 31) == 0) sh[turn][0][tid >> 5] = first_moved;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kSelectThreads / 32; ++w) first_moved = min(first_moved, sh[turn][0][w]);
    a.moved[b] = make_int2(first_moved, left);
    a.seq_lens_out[b] = left;
  }
}

struct MoveArgs {
  void* cache;
  int64_t s_blk, s_row;                              // in words
  int32_t num_blocks, page, words;                   // words of a row
  const int32_t *table, *table_out;
  int64_t bt_stride, bto_stride;
  int32_t max_blocks_out;
  const int32_t* list;
  int32_t list_stride;
  const int2* moved;
};

// One block a sequence and slice of 2^kShift words: its words of row list[j] to row j, in ascending order.
template <typename W, int kShift>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const MoveArgs a) {
  pdl_enter();
  constexpr int kRows = kMoveThreads >> kShift, kStep = kRows * kInFlight;
  const int b = blockIdx.y, word = ((int)blockIdx.x << kShift) + (threadIdx.x & ((1 << kShift) - 1));
  const int sub = threadIdx.x >> kShift;
  const int2 m = a.moved[b];
  const int32_t* const list = a.list + (int64_t)b * a.list_stride;
  const int32_t *const table = a.table + b * a.bt_stride, *const table_out = a.table_out + b * a.bto_stride;
  W* const cache = static_cast<W*>(a.cache);
  // row list[j] and row j of the sequence as offsets; equal where nothing is to be done
  auto look = [&](int j, int64_t& from, int64_t& to) {
    from = to = 0;
    if (j >= m.y) return;
    const int t = list[j], pf = t / a.page, pt = j / a.page;
    const int bf = table[pf], bt = pt < a.max_blocks_out ? table_out[pt] : -1;
    if (bf < 0 || bf >= a.num_blocks || bt < 0 || bt >= a.num_blocks) {
      atomicOr(&g_evict_err, kErrDeviceData);
      return;
    }
    from = bf * a.s_blk + (t - pf * a.page) * a.s_row;
    to = bt * a.s_blk + (j - pt * a.page) * a.s_row;
  };
  const int start = a.table == a.table_out && a.bt_stride == a.bto_stride ? m.x : 0;
  int64_t from[kInFlight], to[kInFlight];
#pragma unroll
  for (int u = 0; u < kInFlight; ++u) look(start + sub + u * kRows, from[u], to[u]);
  for (int j0 = start; j0 < m.y; j0 += kStep) {
    W v[kInFlight];
    int64_t dst[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      dst[u] = from[u] != to[u] && word < a.words ? to[u] : -1;
      if (dst[u] >= 0) v[u] = cache[from[u] + word];
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) look(j0 + kStep + sub + u * kRows, from[u], to[u]);
    __syncthreads();                                 // every load of this step is done
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (dst[u] >= 0) cache[dst[u] + word] = v[u];
  }
}

template <typename W>
cudaError_t launch_move(MoveArgs a, int64_t row_bytes, int32_t batch, cudaStream_t st) {
  a.words = (int32_t)(row_bytes / sizeof(W));
  a.s_blk /= (int64_t)sizeof(W);
  a.s_row /= (int64_t)sizeof(W);
  const int slices = (a.words + 7) / 8;
  // slices of 8 words (128 bytes), narrower while that leaves SMs without a block
  const int64_t blocks = (int64_t)slices * batch, sms = device_sm_count();
  if (blocks >= sms || a.words <= 2) return launch_k(evict_move_kernel<W, 3>, dim3(slices, batch), kMoveThreads, 0, st, a);
  if (2 * blocks >= sms) return launch_k(evict_move_kernel<W, 2>, dim3((a.words + 3) / 4, batch), kMoveThreads, 0, st, a);
  return launch_k(evict_move_kernel<W, 1>, dim3((a.words + 1) / 2, batch), kMoveThreads, 0, st, a);
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
  const SelectArgs s{c.mass, c.mass_stride, c.seq_lens, (int32_t)cap, c.budget, c.sinks, c.recent, c.mass_out, c.mass_out_stride,
                     c.mass_out_rows, c.seq_lens_out, c.kept_out, list, list_stride, moved};
  const cudaError_t e = launch_k(evict_select_kernel, c.batch, kSelectThreads, 0, st, s);
  if (e != cudaSuccess) return e;
  const MoveArgs m{c.cache, c.s_blk, c.s_row, c.num_blocks, c.page, 0, c.block_table, c.block_table_out, c.bt_stride,
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
