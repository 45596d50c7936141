// What the two kernels of the row masses share: a call's arguments as the device sees them, and a
// sequence's rows and queries.
#pragma once

#include "mla_internal.h"

namespace mla {

struct MassArgs {
  float* mass;               // row t of sequence b at mass[b * mass_stride + t]
  int64_t mass_stride;
  const float* lse;          // [T, H]
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t *cu_q, *kv_lens;   // cu_q null: a decode, one token a sequence
  int32_t B, T, H, E;
  int32_t cap;               // rows that the table and the masses hold
  int32_t page, num_blocks;
  float scale, decay;
};

inline MassArgs mass_args(const MassCall& c) {
  int64_t cap = (int64_t)c.max_blocks * c.cache.page;
  if (cap > c.mass_rows) cap = c.mass_rows;
  if (cap > 0x3fffffff) cap = 0x3fffffff;   // positions stay below this
  return MassArgs{c.mass, c.mass_stride, c.lse, c.block_table, c.bt_stride, c.cu_q, c.kv_lens, c.B, c.T, c.H, c.cache.entry,
                  (int32_t)cap, c.cache.page, c.cache.num_blocks, c.scale, c.decay};
}

// Sequence b's rows kv and its queries, tokens q0 .. q0 + nq - 1; nq 0: nothing to do (its masses are
// left as they were). Query i sits at position kv - nq + i and attends the rows up to its own.
struct MassSeq {
  int kv, q0, nq;
};

// A length beyond `cap` counts as cap; query bounds that decrease or leave [0, T] as no queries; both
// are reported in *err.
__device__ __forceinline__ MassSeq mass_seq(const MassArgs& a, int b, unsigned* err) {
  MassSeq s;
  s.kv = a.kv_lens[b];
  if (s.kv < 0 || s.kv > a.cap) {
    atomicOr(err, kErrDeviceData);
    s.kv = s.kv < 0 ? 0 : a.cap;
  }
  s.q0 = b;
  s.nq = 1;
  if (a.cu_q != nullptr) {
    s.q0 = a.cu_q[b];
    const int q1 = a.cu_q[b + 1];
    s.nq = q1 - s.q0;
    if (s.q0 < 0 || q1 > a.T || q1 < s.q0) {
      atomicOr(err, kErrDeviceData);
      s.nq = 0;
    }
  }
  if (s.kv == 0) s.nq = 0;
  return s;
}

// A row's mass after the call; `old` is not used where decay is 0.
__device__ __forceinline__ float new_mass(float old, float got, float decay) {
  return decay == 0.f ? got : fmaf(decay, old, got);
}

}  // namespace mla
