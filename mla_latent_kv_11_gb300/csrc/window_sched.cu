// The schedule of the windowed attention kernels, and the merge of row tiles cut across work units.
//
// A prefill's tokens form row tiles of `tpt` tokens, a decode's sequences one each. Few queries over a
// long axis keep every SM busy by being cut:
//   - no more row tiles than work units: each gets units of its own, as many as make the longest piece
//     shortest, but one where cutting gains less than the float32 pieces and their merge cost (cut_cost).
//     Ranges of equal cost, as below, took 79 us for 64 sequences of 33 tensor-core tiles on 76 units,
//     64 of them a sequence each 69;
//   - up to kSplitItems row tiles: each unit gets a contiguous range of tiles of equal cost (a row
//     tile costing its tiles plus kItemCost) and holds at most two cut row tiles, the end of one and the
//     head of another;
//   - more row tiles balance by themselves and are dealt out whole;
//   - so are those of a short window, without a schedule (kDirectTiles).
// A unit has two partial slots. The schedule depends on the lengths and the number of units alone:
// results repeat bit for bit.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>

#include "window_sched.cuh"

namespace mla {
namespace {

__device__ unsigned g_window_err = 0;

// In tiles (a tensor-core tile takes 1.7 us, one on the CUDA cores four times that): what a row tile
// costs beside its tiles. A prefill of ragged prompts, 1 to 8 tensor-core tiles a row tile, took 115 us
// with 2, 135 with 1.
template <int kPer>
constexpr int kItemCost = kPer == 2 ? 2 : 1;
// What cutting evenly adds to a unit's time, in tiles: the merge's launch, and the float32 pieces written
// and read, 4 KB a row (128 heads: 24 sequences of 6 tiles 20.8 us cut, 17.5 whole; of 16 tiles 27.7 cut,
// 31.9 whole). On the CUDA cores a tile takes longer than that.
constexpr int kMergeCost = 2, kRowsPerTile = 2048;
// Tiles of a row tile up to which no more of them than units go without a schedule, whole. One sequence
// of 3 tiles takes 9.7 us so, 12.8 scheduled and cut; of 5 tiles 13 either way, with one launch instead
// of three. Where cutting would make three pieces of each at most, up to 8 (48 sequences of 6 tiles: 16.3
// us, 19.8 with a schedule that cuts none; 24 of 5: 13.9, 17.4).
constexpr int kDirectTiles = 5, kDirectTilesOfMany = 8;
template <int kPer>
__device__ __forceinline__ int cut_cost(int pieces, int rows) {
  return kPer == 2 ? kMergeCost + pieces * rows / kRowsPerTile : 0;
}
constexpr int kSplitItems = 1024;   // row tiles up to which the schedule cuts them

struct SchedArgs {
  const int32_t* cu_q;     // null: a decode, one token a sequence
  const int32_t* kv_lens;
  int B, T, cap, tpt, window, sinks, units;
  int rows;                // of a full row tile
  int4* items;
  int32_t* total;
  int2* unit_start;
  int32_t* prefix;         // [B + 1] row tiles before each sequence (many row tiles only)
};

__device__ __forceinline__ int kv_len(const SchedArgs& s, int b) { return mla::kv_len(s.kv_lens, s.cap, b, &g_window_err); }

__device__ __forceinline__ int q_len(const SchedArgs& s, int b, int& q0) {
  if (s.cu_q != nullptr) return mla::q_len(s.cu_q, s.T, b, q0, &g_window_err);
  q0 = b;
  return 1;
}

// Exclusive block scan of one int a thread (blockDim.x a multiple of 32).
__device__ __noinline__ int scan_block(int v, int* warp_tot, int* total) {
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

// The last i < n with v[i] <= x.
__device__ __noinline__ int last_at_most(const int* v, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// What bounds it is the fetching of its instructions, none of which are cached when it starts: a
// straight run of them takes 2 us for every 300. So a decode skips what it does not need, scans and
// searches are functions, and pieces start at multiples of their length.
//
// Up to kSplitItems row tiles: their descriptions, and the units' starts. One block; a thread a
// sequence, then a thread a row tile, then a thread a unit.
template <int kPer>
__global__ void __launch_bounds__(1024) window_split_kernel(SchedArgs s) {
  __shared__ int warp_tot[32], first[kSplitItems + 1], q_begin[kSplitItems], q_count[kSplitItems], len[kSplitItems],
      cost[kSplitItems + 1], tiles[kSplitItems], longest[32];
  pdl_enter();
  const int i = threadIdx.x;
  int nt = 0, total;
  Item it;
  if (s.cu_q == nullptr) {
    total = s.B;
    if (i < total) it = make_item(i, 1, kv_len(s, i) - 1, i, s.window, s.sinks);
  } else {
    int n = 0, q0 = 0, k = 0;
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
    if (i < total) {
      const int b = last_at_most(first, s.B, i);   // it has row tiles
      const int t0 = (i - first[b]) * s.tpt;
      it = make_item(q_begin[b] + t0, min(s.tpt, q_count[b] - t0), len[b] - q_count[b] + t0, b, s.window, s.sinks);
    }
  }
  if (i < total) {
    store_item(s.items, i, it);
    nt = item_tiles<kPer>(it.b.w);
  }
  int all;   // the tiles of all, and kItemCost each
  const int at = scan_block(i < total ? nt + kItemCost<kPer> : 0, warp_tot, &all);
  const int sum = all - kItemCost<kPer> * total;
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
    const int lane = i & 31, warp = i >> 5, warps = blockDim.x >> 5;
    const int whole = __reduce_max_sync(0xffffffffu, longest[lane]);   // the longest row tile
    int first_unit = i, pieces = total, piece = 0;
    if (whole > 1 + cut_cost<kPer>(0, 0)) {
      // pieces of at most `lo` tiles: the least `lo` whose pieces the units can take, between sum / units
      // and sum / (units - total). Every warp tries one, evenly between the bounds
      int lo = min(whole, (sum + s.units - 1) / s.units), hi = whole;
      if (s.units > total) hi = max(lo, min(hi, (sum + s.units - total - 1) / (s.units - total)));
      while (lo < hi) {
        const int step = max(1, (hi - lo) / warps), most = min(hi, lo + warp * step);
        int k = 0;
        for (int t = lane; t < total; t += 32) k += (tiles[t] + most - 1) / most;
        k = __reduce_add_sync(0xffffffffu, k);
        if (lane == 0) warp_tot[warp] = k <= s.units;
        __syncthreads();
        int fit = 0;   // the first warp whose pieces fit
        while (fit < warps && !warp_tot[fit]) ++fit;
        __syncthreads();
        if (fit < warps) hi = min(hi, lo + fit * step);
        if (fit > 0) lo = min(hi, lo + (fit - 1) * step + 1);
      }
      piece = lo;
      first_unit = scan_block(i < total ? (nt + lo - 1) / lo : 0, warp_tot, &pieces);
      if (lo + cut_cost<kPer>(pieces, s.rows) >= whole) {
        first_unit = i;
        pieces = total;
      }
    }
    if (i < total) cost[i] = first_unit;
    __syncthreads();
    for (int u = i; u <= s.units; u += blockDim.x) {
      int2 start = make_int2(total, 0);
      if (u < pieces) {
        start.x = last_at_most(cost, total, u);
        start.y = (u - cost[start.x]) * piece;
      }
      s.unit_start[u] = start;
    }
    return;
  }
  // unit u starts at cost u * all / active: units beyond the tiles there are get nothing
  const int active = max(1, min(s.units, sum));
  for (int u = i; u <= s.units; u += blockDim.x) {
    int2 start = make_int2(total, 0);
    if (u < active && total > 0) {
      const int x = (int)((long long)u * all / active);
      const int lo = last_at_most(cost, total, x);
      const int into = max(0, x - cost[lo] - kItemCost<kPer>);
      start = make_int2(lo, into);   // x lies below the next row tile's cost, so into below its tiles
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
__device__ __forceinline__ void store2(float* o, float a, float b) { *reinterpret_cast<float2*>(o) = make_float2(a, b); }
__device__ __forceinline__ void store2(__nv_bfloat16* o, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void store1(float* o, float v) { *o = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* o, float v) { *o = __float2bfloat16_rn(v); }

// Row tiles cut across units: their pieces (normalised output and log-sum-exp) merged. Blocks (i, .)
// handle row tile i, or, with fewer units than row tiles, the one that unit i + 1 is the first to start
// inside of; a warp 128 kC columns of a row. What bounds it is latency: the pieces are looked up 128 at
// once, and sixteen loads of their values are in flight together, of as many pieces (kC 1: few row
// tiles, each of many pieces) or of four (kC 4: enough rows to keep every SM busy). One row tile of 63
// pieces: 23 us with the attention; 43 when a warp took a whole row and looked up its pieces first.
constexpr int kMergeWarps = 8;
template <typename T, bool kVec, int kC>
__global__ void __launch_bounds__(32 * kMergeWarps) window_merge_kernel(WindowSched s, WindowOut out, int units,
                                                                        bool by_item) {
  // the schedule's words come from two launches back, complete before this kernel can start (the
  // attention kernel between waits for them before it lets dependents launch): read before the wait
  const int lane = threadIdx.x & 31;
  int u = blockIdx.x + 1, item = blockIdx.x, n = 1;   // the first unit that starts inside, the row tile, its pieces
  bool found = false;
  if (!by_item) {
    const int2 at = s.unit_start[u], before = s.unit_start[u - 1];
    item = at.x;
    found = at.y > 0 && !(before.x == at.x && before.y > 0);
  }
  if (by_item || found) {
    for (int base = u = found ? u : 1; base < units; base += 128) {
      int2 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = base + 32 * i + lane;
        w[i] = v < units ? s.unit_start[v] : make_int2(-1, 0);
      }
      unsigned in = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        in = __ballot_sync(0xffffffffu, w[i].x == item && w[i].y > 0);
        if (in != 0 && !found) {
          u = base + 32 * i + __ffs(in) - 1;
          found = true;
        }
        n += __popc(in);
      }
      if (found && !(in >> 31)) break;   // the units inside a row tile follow one another
    }
  }
  // the first block waits for the attention kernel though it have nothing to merge: what follows this
  // kernel waits for it alone
  if (n == 1 || item >= *s.total) {
    if (blockIdx.x == 0 && blockIdx.y == 0) pdl_enter();
    return;
  }
  const int4 d = s.items[2 * item];
  const int tok0 = d.x, ntok = d.y;
  // row `row` of a slot: its token and head (a CTA of the pair holds 64 rows: a half of the heads of
  // one token, or whole tokens)
  constexpr int kCols = 128 * kC;
  const int cols = (out.L + kCols - 1) / kCols, job = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  const int row = job / cols, c0 = (job - row * cols) * kCols;
  const int rank = row >> 6, rr = row & 63;
  const int t = out.tptc ? out.tptc * rank + rr / out.H : 0, h = out.tptc ? rr % out.H : row;
  if (row >= out.rows || (out.tptc && rr >= out.tptc * out.H) || h >= out.H || t >= ntok) return;
  // pieces: the head in unit u - 1 (slot 2 (u - 1) + 1), then units u, u + 1, ... (slots 2 v)
  auto slot = [&](int i) { return (int64_t)(i == 0 ? 2 * u - 1 : 2 * (u + i - 1)); };
  pdl_enter();
  constexpr int kPieces = 16 / kC;   // in flight
  float m = -CUDART_INF_F, tot = 0.f;
  float4 acc[kC] = {};
  for (int base = 0; base < n; base += kPieces) {
    const float li = lane < kPieces && base + lane < n ? out.part_lse[slot(base + lane) * out.rows + row] : -CUDART_INF_F;
    float4 v[kPieces][kC];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const float* src = out.part_o + (slot(min(base + i, n - 1)) * out.rows + row) * out.L;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int a = c0 + 128 * c;
        v[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (base + i >= n) continue;
        if constexpr (kVec) {
          if (a + 4 * lane < out.L) v[i][c] = *reinterpret_cast<const float4*>(src + a + 4 * lane);
        } else {
          if (a + lane < out.L) v[i][c].x = src[a + lane];
          if (a + 32 + lane < out.L) v[i][c].y = src[a + 32 + lane];
          if (a + 64 + lane < out.L) v[i][c].z = src[a + 64 + lane];
          if (a + 96 + lane < out.L) v[i][c].w = src[a + 96 + lane];
        }
      }
    }
    float top = li;
#pragma unroll
    for (int o = kPieces / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(m, __shfl_sync(0xffffffffu, top, 0));
    const float by = m == -CUDART_INF_F ? 0.f : __expf(m - top);
    const float mine = li == -CUDART_INF_F ? 0.f : __expf(li - top);
    m = top;
    tot *= by;
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = make_float4(acc[c].x * by, acc[c].y * by, acc[c].z * by, acc[c].w * by);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const float w = __shfl_sync(0xffffffffu, mine, i);
      tot += w;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        acc[c].x = fmaf(w, v[i][c].x, acc[c].x);
        acc[c].y = fmaf(w, v[i][c].y, acc[c].y);
        acc[c].z = fmaf(w, v[i][c].z, acc[c].z);
        acc[c].w = fmaf(w, v[i][c].w, acc[c].w);
      }
    }
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;   // a NaN stays one
  T* o = static_cast<T*>(out.o) + (int64_t)(tok0 + t) * out.o_s0 + (int64_t)h * out.o_s1;
  // a lane's four columns of 128: two pairs at b0 and b1 (kVec; the partial's places 4 lane ..), or lane,
  // 32 + lane, ..
  const int l8 = lane & 7;
  const int b0 = out.permuted ? 32 * (lane >> 3) + 16 * (l8 & 1) + 2 * (l8 >> 1) : 4 * lane;
  const int b1 = b0 + (out.permuted ? 8 : 2);
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int a = c0 + 128 * c;
    if constexpr (kVec) {
      if (a + 4 * lane < out.L) {
        store2(o + a + b0, acc[c].x * inv, acc[c].y * inv);
        store2(o + a + b1, acc[c].z * inv, acc[c].w * inv);
      }
    } else {
      if (a + lane < out.L) store1(o + a + lane, acc[c].x * inv);
      if (a + 32 + lane < out.L) store1(o + a + 32 + lane, acc[c].y * inv);
      if (a + 64 + lane < out.L) store1(o + a + 64 + lane, acc[c].z * inv);
      if (a + 96 + lane < out.L) store1(o + a + 96 + lane, acc[c].w * inv);
    }
  }
  if (c0 == 0 && lane == 0 && out.lse != nullptr)
    out.lse[(int64_t)(tok0 + t) * out.H + h] = tot == 0.f ? -CUDART_INF_F : m + logf(tot);
}

template <typename T>
cudaError_t launch_merge(const WindowSched& sched, const WindowOut& out, int units, cudaStream_t st) {
  const bool vec = out.L % 4 == 0 && out.o_s0 % 4 == 0 && out.o_s1 % 4 == 0 &&
                   reinterpret_cast<uintptr_t>(out.o) % (4 * sizeof(T)) == 0;
  const bool by_item = sched.most < units;
  const int64_t tiles = by_item ? sched.most : units - 1;
  // whole rows a warp where that gives every SM eight warps (24 row tiles of 16 tiles: 31 us, 34 with
  // quarters; one of 63: quarters)
  const bool wide = out.L > 128 && tiles * out.rows >= 8 * (int64_t)device_sm_count();
  const int cols = wide ? (out.L + 511) / 512 : (out.L + 127) / 128;
  const dim3 grid((unsigned)tiles, (out.rows * cols + kMergeWarps - 1) / kMergeWarps);
  auto kernel = wide ? (vec ? window_merge_kernel<T, true, 4> : window_merge_kernel<T, false, 4>)
                     : (vec ? window_merge_kernel<T, true, 1> : window_merge_kernel<T, false, 1>);
  return launch_k(kernel, grid, 32 * kMergeWarps, 0, st, sched, out, units, by_item);
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
              std::min(c.window.sinks, kFar), units, c.H * tpt, reinterpret_cast<int4*>(base + w.items),
              reinterpret_cast<int32_t*>(base + w.total), reinterpret_cast<int2*>(base + w.starts),
              reinterpret_cast<int32_t*>(base + w.prefix)};
  // cut row tiles while their tiles can be counted in 32 bits
  const int64_t seen = std::min<int64_t>(cap, (int64_t)s.window + s.sinks) / (kBlk / 2) + 8;
  const bool split = items <= kSplitItems && c.B <= kSplitItems && items * seen < (int64_t)1 << 30;
  // tiles of a row tile at most; whether any can be cut, or the call needs no schedule (a decode of more
  // sequences than units only where none would be cut)
  const int64_t blocks = std::min<int64_t>((cap + (int64_t)kBlk - 1) / kBlk,
                                           ((int64_t)s.window + tpt + kBlk - 3) / kBlk + 1 + (s.sinks + (int64_t)kBlk - 1) / kBlk);
  const int64_t tiles = blocks_per_tile == 1 ? 2 * blocks : (blocks + blocks_per_tile - 1) / blocks_per_tile, least = 1 + (blocks_per_tile == 2 ? kMergeCost : 0);
  const bool direct = blocks_per_tile == 2 && (decode || c.B <= 32) &&
                      tiles <= (items > units ? (decode ? least : 0) : 4 * items > units ? kDirectTilesOfMany : kDirectTiles);
  *sched = WindowSched{items, s.items, s.total, split ? s.unit_start : nullptr,
                       split && !direct && units > 1 && tiles > 1 && (items > units || tiles > least), direct, c.cu_q,
                       c.kv_lens, c.B, s.T, cap, tpt, s.window, s.sinks};
  *out = WindowOut{c.o.data, c.o.s0, c.o.s1, c.lse, reinterpret_cast<float*>(base + w.o),
                   reinterpret_cast<float*>(base + w.lse), rows, c.L, c.H, 0, false};
  if (direct) return cudaSuccess;
  if (split) {
    const int64_t need = std::max<int64_t>({items, c.B, 128});
    const int threads = (int)std::min<int64_t>(1024, (need + 31) / 32 * 32);
    return launch_k(blocks_per_tile == 2 ? window_split_kernel<2> : window_split_kernel<1>, 1, threads, 0, st, s);
  }
  const cudaError_t e = launch_k(window_prefix_kernel, 1, 1024, 0, st, s);
  if (e != cudaSuccess) return e;
  return launch_k(window_items_kernel, (unsigned)((items + 255) / 256), 256, 0, st, s);
}

cudaError_t launch_window_merge(mla_dtype dt, const WindowSched& sched, const WindowOut& out, int units, cudaStream_t st) {
  if (!sched.cut) return cudaSuccess;
  return dt == MLA_F32 ? launch_merge<float>(sched, out, units, st) : launch_merge<__nv_bfloat16>(sched, out, units, st);
}

cudaError_t window_sched_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_window_err);
}

}  // namespace mla
