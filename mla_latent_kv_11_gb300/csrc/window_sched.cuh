// The work of the windowed attention kernels: row tiles, their visible blocks, and the walk of a work
// unit over its part of them. The schedule itself is made in window_sched.cu.
#pragma once

#include "mla_internal.h"

namespace mla {

constexpr int kBlk = 64;          // cache rows per block
constexpr int kMaxUnits = 4096;   // work units at most, whatever a caller asks for

// A row tile ("item") as the schedule describes it: {first token's row, tokens, its position, sequence}
// and {first window row, sink blocks, first window block behind them, blocks in all}. Its tokens sit
// at pos0 .. pos0 + ntok - 1; the rows they attend lie in the blocks of the sinks and those of the
// window, listed one behind the other and taken `per` at a time (a tile).
struct Item {
  int4 a, b;
};

__device__ __forceinline__ Item make_item(int tok0, int ntok, int pos0, int seq, int window, int sinks) {
  const int hi = pos0 + ntok - 1, lo = max(0, pos0 - window + 1);
  int nsb = 0, wb = 0, nblk = 0;
  if (hi >= 0) {
    nsb = (min(sinks, hi + 1) + kBlk - 1) / kBlk;
    wb = max(lo / kBlk, nsb);
    nblk = nsb + max(0, hi / kBlk + 1 - wb);
  }
  return Item{make_int4(tok0, ntok, pos0, seq), make_int4(lo, nsb, wb, nblk)};
}
__device__ __forceinline__ Item load_item(const int4* items, int i) { return Item{items[2 * i], items[2 * i + 1]}; }
__device__ __forceinline__ void store_item(int4* items, int i, const Item& it) {
  items[2 * i] = it.a;
  items[2 * i + 1] = it.b;
}

// Tiles of a row tile, of kPer blocks each or (kPer 1, the CUDA cores) half a block: one, with nothing
// attended, where there are no blocks, so that its rows are written all the same.
template <int kPer>
__device__ __forceinline__ int item_tiles(int nblk) {
  return nblk > 0 ? (kPer == 1 ? 2 * nblk : (nblk + kPer - 1) / kPer) : 1;
}

// Rows of sequence b in the cache; a length beyond the table is cut to it (and reported in *err).
__device__ __forceinline__ int kv_len(const int32_t* lens, int cap, int b, unsigned* err) {
  int n = lens[b];
  if (n < 0 || n > cap) {
    atomicOr(err, kErrDeviceData);
    n = n < 0 ? 0 : cap;
  }
  return n;
}

// Query tokens of sequence b of a prefill, from q0 on; -1 (and reported) where cu leaves [0, T] or
// decreases. Nothing is computed then: only ascending bounds keep the row tiles within the room for them.
__device__ __forceinline__ int q_len(const int32_t* cu, int T, int b, int& q0, unsigned* err) {
  q0 = cu[b];
  const int q1 = cu[b + 1];
  if (q0 < 0 || q1 > T || q1 < q0) {
    atomicOr(err, kErrDeviceData);
    return -1;
  }
  return q1 - q0;
}

// A part of a row tile: tiles [t0, t1).
struct Seg {
  int tok0, ntok, pos0, b;   // first token's row, tokens, its position, sequence
  int lo, hi;                // first window row and last row any token attends
  int nsb, wb, nblk;         // sink blocks, first window block behind them, blocks in all
  int t0, t1, slot;          // tile range; partial slot or -1
};

// First row of block j of a segment's list; -1 behind its end.
__device__ __forceinline__ int block_row(const Seg& s, int j) {
  return j >= s.nblk ? -1 : kBlk * (j < s.nsb ? j : s.wb + (j - s.nsb));
}

// The segments of one work unit, in tiles of kPer blocks. kDirect: the schedule is (an instance of the
// kernels of its own: the more code in the roles' loops, the slower they fetch it).
template <int kPer, bool kDirect>
struct Walker {
  int unit, item, step, end_item, end_tile, tile;
  Item ahead;   // the next row tile, loaded while the one before it runs
  int q0, count, len, first, tiles;   // kDirect: of lane b's sequence b, its tokens, cache rows and row tiles

  // A direct schedule is worked out by whole warps, a lane a sequence: a prefill has at most 32.

  __device__ Item load(const WindowSched& s, int i, unsigned* err) const {
    if constexpr (kDirect) {
      if (s.cu_q == nullptr) return make_item(i, 1, kv_len(s.kv_lens, s.cap, i, err) - 1, i, s.window, s.sinks);
      const int b = 31 - __clz(__ballot_sync(0xffffffffu, tiles > 0 && first <= i));
      const int t0 = (i - __shfl_sync(0xffffffffu, first, b)) * s.tpt, k = __shfl_sync(0xffffffffu, count, b);
      const int pos0 = __shfl_sync(0xffffffffu, len, b) - k + t0, tok0 = __shfl_sync(0xffffffffu, q0, b) + t0;
      return make_item(tok0, min(s.tpt, k - t0), pos0, b, s.window, s.sinks);
    }
    return load_item(s.items, i);
  }
  __device__ void init(const WindowSched& s, int unit_, int units, unsigned* err) {
    unit = unit_;
    if constexpr (kDirect) {
      item = unit;
      tile = 0;
      end_item = s.B;
      end_tile = 0;
      step = units;
      if (s.cu_q != nullptr) {
        const int b = threadIdx.x & 31;
        q0 = count = len = 0;
        if (b < s.B) {
          count = q_len(s.cu_q, s.T, b, q0, err);
          len = kv_len(s.kv_lens, s.cap, b, err);
        }
        tiles = __any_sync(0xffffffffu, count < 0) ? 0 : (count + s.tpt - 1) / s.tpt;
        int x = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (b >= o) x += y;
        }
        first = x - tiles;
        end_item = __shfl_sync(0xffffffffu, x, 31);
      }
    } else if (s.unit_start != nullptr) {
      const int2 a = s.unit_start[unit], e = s.unit_start[unit + 1];
      item = a.x;
      tile = a.y;
      end_item = e.x;
      end_tile = e.y;
      step = 1;
    } else {   // whole row tiles dealt out, the longest (latest) first
      item = *s.total - 1 - unit;
      tile = 0;
      step = -units;
      end_item = -1;
      end_tile = 0;
    }
    if (more()) ahead = load(s, item, err);
  }
  __device__ bool more() const {
    return step > 0 ? (item < end_item || (item == end_item && tile < end_tile)) : item >= 0;
  }
  __device__ bool next(const WindowSched& sched, Seg& s, unsigned* err) {
    if (!more()) return false;
    s.tok0 = ahead.a.x;
    s.ntok = ahead.a.y;
    s.pos0 = ahead.a.z;
    s.b = ahead.a.w;
    s.lo = ahead.b.x;
    s.hi = s.pos0 + s.ntok - 1;
    s.nsb = ahead.b.y;
    s.wb = ahead.b.z;
    s.nblk = ahead.b.w;
    const int nt = item_tiles<kPer>(s.nblk);
    s.t0 = tile;
    s.t1 = step > 0 && item == end_item ? min(nt, end_tile) : nt;
    s.slot = s.t0 == 0 && s.t1 == nt ? -1 : 2 * unit + (s.t0 == 0 ? 1 : 0);
    item += step;
    tile = 0;
    if (more()) ahead = load(sched, item, err);
    return true;
  }
};

}  // namespace mla
