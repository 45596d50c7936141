// The schedule of the windowed attention kernels, and the merge of row tiles cut across work units.
//
// A prefill's tokens form row tiles of `tpt` tokens, a decode's sequences one each. Few queries over a
// long axis keep every SM busy by being cut:
//   - no more row tiles than work units: each gets units of its own, as many as make the longest piece
//     shortest, but one where cutting gains less than the float32 partials and their merge cost
//     (kCutCost; 64 sequences of 33 tensor-core tiles on 76 units: 82 us cut, 71 whole);
//   - up to kSplitItems row tiles: each unit gets a contiguous range of tiles of equal cost (a row
//     tile costing its tiles plus kItemCost) and holds at most two cut row tiles, the end of one and the
//     head of another;
//   - more row tiles balance by themselves and are dealt out whole.
// A unit has two partial slots. The schedule depends on the lengths and the number of units alone:
// results repeat bit for bit.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>

#include "window_sched.cuh"

namespace mla {
namespace {

__device__ unsigned g_window_err = 0;

// In tiles, of kPer blocks each (a tensor-core tile takes 1.7 us, one on the CUDA cores ten times
// that): what a row tile costs beside its tiles (a prefill of ragged prompts, 1 to 8 tensor-core tiles
// a row tile, took 115 us with 2, 135 with 1), and what cutting adds to a unit's time.
template <int kPer>
constexpr int kItemCost = kPer == 2 ? 2 : 1;
template <int kPer>
constexpr int kCutCost = kPer == 2 ? 5 : 0;
constexpr int kSplitItems = 1024;   // row tiles up to which the schedule cuts them

struct SchedArgs {
  const int32_t* cu_q;     // null: a decode, one token a sequence
  const int32_t* kv_lens;
  int B, T, cap, tpt, window, sinks, units;
  int4* items;
  int32_t* total;
  int2* unit_start;
  int32_t* prefix;         // [B + 1] row tiles before each sequence (many row tiles only)
};

__device__ __forceinline__ int kv_len(const SchedArgs& s, int b) {
  int n = s.kv_lens[b];
  if (n < 0 || n > s.cap) {
    atomicOr(&g_window_err, kErrDeviceData);
    n = n < 0 ? 0 : s.cap;
  }
  return n;
}

// Query tokens of sequence b; -1 (and reported) where cu_q leaves [0, T] or decreases. Nothing is
// computed then: only an ascending cu_q keeps the row tiles within the room for them.
__device__ __forceinline__ int q_len(const SchedArgs& s, int b, int& q0) {
  if (s.cu_q == nullptr) {
    q0 = b;
    return 1;
  }
  q0 = s.cu_q[b];
  const int q1 = s.cu_q[b + 1];
  if (q0 < 0 || q1 > s.T || q1 < q0) {
    atomicOr(&g_window_err, kErrDeviceData);
    return -1;
  }
  return q1 - q0;
}

// Exclusive block scan of one int a thread (blockDim.x a multiple of 32).
__device__ int scan_block(int v, int* warp_tot, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_tot[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) before += warp_tot[w];
    all += warp_tot[w];
  }
  *total = all;
  return before + x - v;
}

// Up to kSplitItems row tiles: their descriptions, and the units' starts. One block; a thread a
// sequence, then a thread a row tile, then a thread a unit.
template <int kPer>
__global__ void __launch_bounds__(1024) window_split_kernel(SchedArgs s) {
  __shared__ int warp_tot[32], first[kSplitItems + 1], q_begin[kSplitItems], q_count[kSplitItems], len[kSplitItems],
      cost[kSplitItems + 1], tiles[kSplitItems], longest[32];
  pdl_enter();
  const int i = threadIdx.x;
  int n = 0, q0 = 0, k = 0, total;
  if (i < s.B) k = q_len(s, i, q0);
  if (__syncthreads_or(k < 0)) k = 0;
  if (i < s.B) {
    n = (k + s.tpt - 1) / s.tpt;
    q_begin[i] = q0;
    q_count[i] = k;
    len[i] = kv_len(s, i);
  }
  const int ex = scan_block(n, warp_tot, &total);
  if (i < s.B) first[i] = ex;
  __syncthreads();
  int nt = 0;
  if (i < total) {
    int lo = 0, hi = s.B - 1;   // the last sequence with first <= i: it has row tiles
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= i) lo = mid; else hi = mid - 1;
    }
    const int t0 = (i - first[lo]) * s.tpt, ntok = min(s.tpt, q_count[lo] - t0);
    const Item it = make_item(q_begin[lo] + t0, ntok, len[lo] - q_count[lo] + t0, lo, s.window, s.sinks);
    store_item(s.items, i, it);
    nt = item_tiles<kPer>(it.b.w);
  }
  int all;
  const int at = scan_block(i < total ? nt + kItemCost<kPer> : 0, warp_tot, &all);
  if (i < total) {
    cost[i] = at;
    tiles[i] = nt;
  }
  if (i == 0) *s.total = total;
  if (i < 32) longest[i] = 0;
  __syncthreads();
  const int top = __reduce_max_sync(0xffffffffu, nt);
  if ((i & 31) == 0) longest[i >> 5] = top;
  __syncthreads();
  if (total <= s.units) {
    // pieces of at most `most` tiles: the least `most` whose pieces the units can take
    int lo = 1, hi = 1, pieces;   // hi: the longest row tile
    for (int w = 0; w < 32; ++w) hi = max(hi, longest[w]);
    const int whole = hi;
    while (lo < hi) {
      const int most = (lo + hi) >> 1;
      scan_block(i < total ? (nt + most - 1) / most : 0, warp_tot, &pieces);
      if (pieces <= s.units) hi = most; else lo = most + 1;
    }
    const int k = i < total ? (lo + kCutCost<kPer> < whole ? (nt + lo - 1) / lo : 1) : 0;
    const int first_unit = scan_block(k, warp_tot, &pieces);
    for (int j = 0; j < k; ++j) s.unit_start[first_unit + j] = make_int2(i, (int)((long long)nt * j / k));
    for (int u = pieces + i; u <= s.units; u += blockDim.x) s.unit_start[u] = make_int2(total, 0);
    return;
  }
  // unit u starts at cost u * all / active: units beyond the tiles there are get nothing
  const int active = max(1, min(s.units, all - kItemCost<kPer> * total));
  for (int u = i; u <= s.units; u += blockDim.x) {
    int2 start = make_int2(total, 0);
    if (u < active && total > 0) {
      const int x = (int)((long long)u * all / active);
      int lo = 0, hi = total - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cost[mid] <= x) lo = mid; else hi = mid - 1;
      }
      const int into = max(0, x - cost[lo] - kItemCost<kPer>);
      start = into >= tiles[lo] ? make_int2(lo + 1, 0) : make_int2(lo, into);
    }
    s.unit_start[u] = start;
  }
}

// More row tiles: how many lie before each sequence (one block), then a thread a row tile.
__global__ void __launch_bounds__(1024) window_prefix_kernel(SchedArgs s) {
  __shared__ int warp_tot[32];
  pdl_enter();
  int carry = 0, q0;
  bool bad = false;
  for (int b = threadIdx.x; b < s.B; b += blockDim.x) {
    bad |= q_len(s, b, q0) < 0;
    kv_len(s, b);   // reports a bad length
  }
  bad = __syncthreads_or(bad);
  for (int base = 0; base < s.B; base += blockDim.x) {
    const int b = base + threadIdx.x;
    int tot;
    const int n = b < s.B && !bad ? (q_len(s, b, q0) + s.tpt - 1) / s.tpt : 0;
    const int ex = scan_block(n, warp_tot, &tot);
    if (b < s.B) s.prefix[b] = carry + ex;
    carry += tot;
  }
  if (threadIdx.x == 0) {
    s.prefix[s.B] = carry;
    *s.total = carry;
  }
}

__global__ void __launch_bounds__(256) window_items_kernel(SchedArgs s) {
  pdl_enter();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= s.prefix[s.B]) return;
  int lo = 0, hi = s.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.prefix[mid] <= i) lo = mid; else hi = mid - 1;
  }
  int q0 = lo, q1 = lo + 1;
  if (s.cu_q != nullptr) {
    q0 = s.cu_q[lo];
    q1 = s.cu_q[lo + 1];
  }
  const int t0 = (i - s.prefix[lo]) * s.tpt;
  const int kv = min(max(s.kv_lens[lo], 0), s.cap);
  store_item(s.items, i, make_item(q0 + t0, min(s.tpt, q1 - q0 - t0), kv - (q1 - q0) + t0, lo, s.window, s.sinks));
}

// ---------------------------------------------------------------------------
__device__ __forceinline__ void store4(float* o, float4 v) { *reinterpret_cast<float4*>(o) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* o, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(o) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store1(float* o, float v) { *o = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* o, float v) { *o = __float2bfloat16_rn(v); }

// Row tiles cut across units: their pieces (normalised output and log-sum-exp) merged. Blocks (u, .)
// handle the row tile that unit u + 1 is the first to start inside of; a warp a row. What bounds it
// is latency: a lane a piece looks up how many there are and their sums at once, and the rows of
// four pieces are in flight together.
constexpr int kMergeWarps = 8;
template <typename T, bool kVec>
__global__ void __launch_bounds__(32 * kMergeWarps) window_merge_kernel(WindowSched s, WindowOut out, int units) {
  // the schedule's words come from two launches back, complete before this kernel can start (the
  // attention kernel between waits for them before it lets dependents launch): read before the wait
  const int u = blockIdx.x + 1, lane = threadIdx.x & 31;
  const int2 at = s.unit_start[u], before = s.unit_start[u - 1];
  // the first block waits for the attention kernel though it have nothing to merge: what follows this
  // kernel waits for it alone
  if (at.x >= *s.total || at.y == 0 || (before.x == at.x && before.y > 0)) {
    if (blockIdx.x == 0 && blockIdx.y == 0) pdl_enter();
    return;
  }
  const int4 d = s.items[2 * at.x];
  // row `row` of a slot: its token and head (a CTA of the pair holds 64 rows: a half of the heads of
  // one token, or whole tokens)
  const int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  const int rank = row >> 6, rr = row & 63;
  const int t = out.tptc ? out.tptc * rank + rr / out.H : 0, h = out.tptc ? rr % out.H : row;
  if (row >= out.rows || (out.tptc && rr >= out.tptc * out.H) || h >= out.H || t >= d.y) return;
  // pieces: the head in unit u - 1 (slot 2 (u - 1) + 1), then units u, u + 1, ... (slots 2 v)
  int n = 1;
  for (int base = u;; base += 32) {
    const int v = base + lane;
    const int2 w = v <= units ? s.unit_start[v] : make_int2(-1, 0);
    const unsigned more = __ballot_sync(0xffffffffu, w.x == at.x && w.y > 0);
    const int k = more == 0xffffffffu ? 32 : __ffs(~more) - 1;
    n += k;
    if (k < 32) break;
  }
  auto slot = [&](int i) { return (int64_t)(i == 0 ? 2 * u - 1 : 2 * (u + i - 1)); };
  pdl_enter();
  float m = -CUDART_INF_F;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, out.part_lse[slot(i) * out.rows + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float tot = 0.f;
  constexpr int kCols = kVec ? 4 : 16;   // float4s, or floats, of a row of up to 512 columns in a lane
  float4 acc[4] = {};
  float one[16] = {};
  for (int base = 0; base < n; base += 32) {
    const float li = base + lane < n ? out.part_lse[slot(base + lane) * out.rows + row] : -CUDART_INF_F;
    const float mine = li == -CUDART_INF_F ? 0.f : __expf(li - m);
    const int k = min(32, n - base);
    for (int i0 = 0; i0 < k; i0 += 4) {
      float4 v[4][4];
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = __shfl_sync(0xffffffffu, mine, (i0 + i) & 31);
        if (i0 + i >= k) w[i] = 0.f;
        const float* src = out.part_o + (slot(base + min(i0 + i, k - 1)) * out.rows + row) * out.L;
        if constexpr (kVec) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int col = 128 * c + 4 * lane;
            v[i][c] = col < out.L ? *reinterpret_cast<const float4*>(src + col) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        } else {
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            const int col = 32 * c + lane;
            if (col < out.L) one[c] = fmaf(w[i], src[col], one[c]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        tot += w[i];
        if constexpr (kVec)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          acc[c].x = fmaf(w[i], v[i][c].x, acc[c].x);
          acc[c].y = fmaf(w[i], v[i][c].y, acc[c].y);
          acc[c].z = fmaf(w[i], v[i][c].z, acc[c].z);
          acc[c].w = fmaf(w[i], v[i][c].w, acc[c].w);
        }
      }
    }
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;   // a NaN stays one
  T* o = static_cast<T*>(out.o) + (int64_t)(d.x + t) * out.o_s0 + (int64_t)h * out.o_s1;
  if constexpr (kVec) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int col = 128 * c + 4 * lane;
      if (col < out.L) store4(o + col, make_float4(acc[c].x * inv, acc[c].y * inv, acc[c].z * inv, acc[c].w * inv));
    }
  } else {
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      const int col = 32 * c + lane;
      if (col < out.L) store1(o + col, one[c] * inv);
    }
  }
  if (lane == 0 && out.lse != nullptr)
    out.lse[(int64_t)(d.x + t) * out.H + h] = tot == 0.f ? -CUDART_INF_F : m + logf(tot);
}

// Row tiles at most: T tokens of B sequences, tpt a tile.
int64_t most_items(int64_t T, int64_t B, int tpt, bool decode) {
  if (decode) return B;
  return tpt == 1 ? T : std::min<int64_t>(T, T / tpt + B);
}

struct WindowWs {
  size_t total, items, starts, prefix, o, lse, bytes;
};
WindowWs window_ws(int64_t items, int64_t B, int64_t units, int64_t rows, int64_t L) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  WindowWs w{};
  w.items = 256;
  w.starts = up(w.items + items * sizeof(Item));
  w.prefix = up(w.starts + (units + 1) * sizeof(int2));
  w.o = up(w.prefix + (B + 1) * sizeof(int32_t));
  // partial slots: two a unit where the schedule cuts row tiles
  const size_t slots = items <= kSplitItems ? 2 * units : 0;
  w.lse = up(w.o + slots * rows * L * sizeof(float));
  w.bytes = up(w.lse + slots * rows * sizeof(float));
  return w;
}

}  // namespace

size_t window_workspace(int64_t T, int64_t B, bool decode, int tpt, int64_t units, int64_t rows, int64_t L) {
  return window_ws(most_items(T, B, tpt, decode), B, units, rows, L).bytes;
}

cudaError_t launch_window_schedule(const WindowCall& c, int tpt, int blocks_per_tile, int units, int rows, void* ws,
                                   WindowSched* sched, WindowOut* out, cudaStream_t st) {
  const bool decode = c.cu_q == nullptr;
  const int64_t items = most_items(c.q.n0, c.B, tpt, decode);
  const WindowWs w = window_ws(items, c.B, units, rows, c.L);
  char* base = static_cast<char*>(ws);
  constexpr int kFar = 0x3fffffff;   // positions stay below this
  const int cap = (int)std::min<int64_t>((int64_t)c.max_blocks * c.cache.page, kFar);
  SchedArgs s{c.cu_q, c.kv_lens, c.B, (int)c.q.n0, cap, tpt, std::min(c.window.window, kFar),
              std::min(c.window.sinks, kFar), units, reinterpret_cast<int4*>(base + w.items),
              reinterpret_cast<int32_t*>(base + w.total), reinterpret_cast<int2*>(base + w.starts),
              reinterpret_cast<int32_t*>(base + w.prefix)};
  // cut row tiles while their tiles can be counted in 32 bits
  const int64_t seen = std::min<int64_t>(cap, (int64_t)s.window + s.sinks) / kBlk + 4;
  const bool split = items <= kSplitItems && c.B <= kSplitItems && items * seen < (int64_t)1 << 30;
  // tiles of a row tile at most; whether any can be cut
  const int64_t tiles = (std::min<int64_t>(cap, (int64_t)s.window + tpt) / kBlk + 2 +
                         std::min<int64_t>(cap, s.sinks) / kBlk + 1 + blocks_per_tile - 1) / blocks_per_tile;
  const int cut_cost = blocks_per_tile == 2 ? kCutCost<2> : kCutCost<1>;
  *sched = WindowSched{s.items, s.total, split ? s.unit_start : nullptr,
                       split && units > 1 && tiles > 1 && (items > units || tiles > 1 + cut_cost)};
  *out = WindowOut{c.o.data, c.o.s0, c.o.s1, c.lse, reinterpret_cast<float*>(base + w.o),
                   reinterpret_cast<float*>(base + w.lse), rows, c.L, c.H, 0};
  if (split) {
    const int64_t need = std::max<int64_t>({items, c.B, std::min(units + 1, 128)});
    const int threads = (int)std::min<int64_t>(1024, (need + 31) / 32 * 32);
    return launch_k(blocks_per_tile == 2 ? window_split_kernel<2> : window_split_kernel<1>, 1, threads, 0, st, s);
  }
  const cudaError_t e = launch_k(window_prefix_kernel, 1, 1024, 0, st, s);
  if (e != cudaSuccess) return e;
  return launch_k(window_items_kernel, (unsigned)((items + 255) / 256), 256, 0, st, s);
}

cudaError_t launch_window_merge(mla_dtype dt, const WindowSched& sched, const WindowOut& out, int units, cudaStream_t st) {
  if (!sched.cut) return cudaSuccess;
  const dim3 grid(units - 1, (out.rows + kMergeWarps - 1) / kMergeWarps);
  const size_t es = dt == MLA_F32 ? 4 : 2;
  const bool vec = out.L % 4 == 0 && out.o_s0 % 4 == 0 && out.o_s1 % 4 == 0 &&
                   reinterpret_cast<uintptr_t>(out.o) % (4 * es) == 0;
  if (dt == MLA_F32)
    return launch_k(vec ? window_merge_kernel<float, true> : window_merge_kernel<float, false>, grid, 32 * kMergeWarps,
                    0, st, sched, out, units);
  return launch_k(vec ? window_merge_kernel<__nv_bfloat16, true> : window_merge_kernel<__nv_bfloat16, false>, grid,
                  32 * kMergeWarps, 0, st, sched, out, units);
}

unsigned window_sched_errors_read_clear() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_window_err, sizeof(v)) != cudaSuccess) return 0;
  cudaMemcpyToSymbol(g_window_err, &zero, sizeof(zero));
  return v;
}

}  // namespace mla
