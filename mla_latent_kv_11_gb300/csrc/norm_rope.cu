// Norms of query heads and of new latents, with the position rotation in the same pass: what stands
// between a layer's projections and its absorbed attention.
//
// Mathematics. A head's RMS norm is y = x * w / sqrt(mean(x^2) + eps), over its nope and rope columns
// together; a latent's over its L columns. The rotation turns each pair (a, b) of rope columns by its
// token's angle, (a c - b s, b c + a s), pairs side by side or a half apart. Sums, norms and rotations
// are float32; a value is rounded once, as it is stored (or quantised).
//
// Both parts are bound by HBM: every value crosses it once. A row stays in registers between its sum
// and its stores, in 16-byte words: a query head in 8, 16 or 32 lanes of up to four words each (24
// words of a 192-wide bf16 head are three a lane of eight, so that no lane idles), a cache row in one
// warp or half of one. A block takes heads of one token, several a warp one behind the other, so that the token's angles and the
// addresses are worked out once (a head a warp alone issued three times the instructions: 4096 tokens of 128
// heads 113 us). No lane has more than one word of the rope; its partner half a rope away comes from its lane. Both
// parts share one launch: a decode step has 5 to 500 blocks of work in all.
//
// What it measured (device times): 4096 tokens of 128 normed heads of 192 and their rows, bf16: 73 us for 413 MB,
// 5.6 TB/s, 0.83 of a copy's rate (halves rotated 79 us: a word's partner through eight exchanges, and registers spilled for
// them); the same with queries without a norm 38 us for 145 MB, 0.55 of it: a lane has one word of a head in flight and the next
// one, behind its token's position (loads waited for 8 times an issue, DRAM at 34%). One head a token leaves most of a block
// idle: 20000 heads of 512 bf16 columns 44 us for 41 MB. 20011 float32 rows into ds_mla entries 14 us, 4.6 TB/s; 40000 bf16
// rows plain 24 us, e4m3 29 (pairs side by side 21 and 23). A step of 64 tokens 3.5 us, of one 2.1.
#include <algorithm>

#include "e4m3_codes.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

__device__ unsigned g_norm_err = 0;

enum Format { kPlain, kE4m3 };

// A 16-byte word's values.
template <typename T>
struct Word {
  static constexpr int kN = 16 / sizeof(T);
  static __device__ __forceinline__ void open(const uint4& w, float (&x)[kN]) {
    if constexpr (sizeof(T) == 4) {
      x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
      x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
    } else {
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
      }
    }
  }
  static __device__ __forceinline__ uint4 close(const float (&x)[kN]) {
    uint4 w;
    if constexpr (sizeof(T) == 4) {
      w = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    } else {
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    }
    return w;
  }
  // x times by, and times the values of w.
  static __device__ __forceinline__ void scale(float (&x)[kN], float by, const uint4& w) {
    float y[kN];
    open(w, y);
    const uint64_t b = pair(by, by);
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
      uint64_t v = pair(x[i], x[i + 1]);
      asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(v), "l"(b));
      asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(v), "l"(pair(y[i], y[i + 1])));
      x[i] = __uint_as_float((uint32_t)v);
      x[i + 1] = __uint_as_float((uint32_t)(v >> 32));
    }
  }
  static __device__ __forceinline__ float squares(const uint4& w) {
    float x[kN];
    open(w, x);
    uint64_t sum = 0;
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
      const uint64_t v = pair(x[i], x[i + 1]);
      asm("fma.rn.f32x2 %0, %1, %1, %0;" : "+l"(sum) : "l"(v));
    }
    return __uint_as_float((uint32_t)sum) + __uint_as_float((uint32_t)(sum >> 32));
  }
  static __device__ __forceinline__ uint4 load(const T* p) { return *reinterpret_cast<const uint4*>(p); }
};

// Positions and the table of their cosines and sines, [count, R] float32: R / 2 cosines, then R / 2 sines.
struct Angles {
  const int64_t* positions;
  const float* table;
  int64_t stride, count;
  int32_t R, interleaved, words;

  // A position's row of angles; null where it lies outside the table (recorded).
  __device__ __forceinline__ const float* row(int64_t p, int lane) const {
    if (R == 0) return table;   // nothing to rotate
    if (p < 0 || p >= count) {
      if (lane == 0) atomicOr(&g_norm_err, kErrDeviceData);
      return nullptr;
    }
    return table + p * stride;
  }
  // The same of token t.
  __device__ __forceinline__ const float* of(int64_t t) const {
    return R == 0 ? table : row(positions[t], (int)threadIdx.x & 31);
  }
};

// The angles of one word of a rope: columns d .. d + kN - 1. (The rotations are written in fused
// multiply-adds, the same in every kernel, so that which one a call takes does not change a rotation's bits.)
template <int kN, bool kInter>
struct Turn {
  static constexpr int kHas = kInter ? kN / 2 : kN;
  float c[kHas], s[kHas];   // half a rope apart: the first half's sines negative, as its columns are the a's

  static __device__ __forceinline__ void load(const float* p, bool words, float (&x)[kHas]) {
    if (!words) {
#pragma unroll
      for (int k = 0; k < kHas; ++k) x[k] = p[k];
    } else if constexpr (kHas % 4 == 0) {
#pragma unroll
      for (int k = 0; k < kHas; k += 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + k);
        x[k] = v.x; x[k + 1] = v.y; x[k + 2] = v.z; x[k + 3] = v.w;
      }
    } else if constexpr (kHas == 2) {
      const float2 v = *reinterpret_cast<const float2*>(p);
      x[0] = v.x; x[1] = v.y;
    }
  }
  // cs: the token's row of the table.
  __device__ __forceinline__ void open(const float* cs, int d, int half, bool words) {
    const int i = kInter ? d >> 1 : d < half ? d : d - half;
    load(cs + i, words, c);
    load(cs + half + i, words, s);
    if (!kInter && d < half) {
#pragma unroll
      for (int k = 0; k < kHas; ++k) s[k] = -s[k];
    }
  }
  // with: the partners half a rope away (kInter: not used).
  __device__ __forceinline__ void turn(float (&x)[kN], const float (&with)[kN]) const {
    if constexpr (kInter) {
#pragma unroll
      for (int k = 0; k < kN; k += 2) {
        const float a = x[k], b = x[k + 1];
        x[k] = fmaf(a, c[k >> 1], -(b * s[k >> 1]));
        x[k + 1] = fmaf(b, c[k >> 1], a * s[k >> 1]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kN; ++k) x[k] = fmaf(x[k], c[k], with[k] * s[k]);
    }
  }
};

// The lane, modulo the lanes of a row, that holds the word half a rope away from the one at `rope`.
template <int kN>
__device__ __forceinline__ int partner_lane(int rope, int half, int lane) {
  return rope < half ? lane + half / kN : lane - half / kN;
}

struct QueryPart {
  const void* q;
  int64_t q_s0, q_s1;
  void* nope;
  int64_t n_s0, n_s1;
  void* pe;
  int64_t p_s0, p_s1;
  const void* weight;   // null: no norm
  int64_t w_s0;
  int32_t H, P, W;      // heads, columns before the rope, columns
  int32_t first;        // columns before it stay as they are (in place, without a norm)
  int32_t tokens;       // 0: no queries
  int32_t parts;        // blocks of a token: block i takes heads from i * (H / parts, rounded up to whole passes) on
};

struct RowPart {
  const void* kv;
  int64_t k_s0;
  const void* weight;
  void* cache;
  int64_t c_blk, c_row, num_rows;
  PageOf page_of;
  int32_t L, E;
  const int64_t* slots;
  int64_t tokens;
  const float* scale;   // kE4m3
  int32_t eights;       // kE4m3: rows are eight bytes aligned
};

// Offset of slot s in the cache; -1: padding, or outside the view (recorded).
__device__ __forceinline__ int64_t row_offset(const RowPart& p, int64_t s, int lane) {
  if (s < 0) return -1;
  if (s >= p.num_rows) {
    if (lane == 0) atomicOr(&g_norm_err, kErrDeviceData);
    return -1;
  }
  // (a division of 64 bits takes as long as half of a row's arithmetic)
  const int64_t blk = p.num_rows <= INT32_MAX ? p.page_of((int)s) : s / p.page_of.page;
  return blk * p.c_blk + (s - blk * p.page_of.page) * p.c_row;
}

// 1 / sqrt(sum / n + eps), inv = 1 / n: a quotient and a root each mended by a step with its remainder (a division,
// a root and another division took a head a fifth of its instructions). It enters every value of the row, and a
// quantised value next to the middle of two codes tells its last bit. A sum beyond float32 is infinite, and its factor 0:
// it leaves no remainder to mend the quotient with (infinity minus infinity).
__device__ __forceinline__ float norm_factor(float sum, float n, float inv, float eps) {
  float v = sum * inv;
  if (v <= FLT_MAX) v = fmaf(fmaf(-v, n, sum), inv, v);
  v += eps;
  const float y = rsqrtf(v);
  const float p = v * y, low = fmaf(v, y, -p);               // v y = p + low
  const float t = fmaf(-low, y, fmaf(-p, y, 1.f));           // 1 - v y^2
  return t == t && y <= FLT_MAX ? fmaf(0.5f * y, t, y) : y;  // (v infinite, zero or NaN: as it is)
}

// Heads of queries, in words: kG lanes a head, kW words a lane, kPass heads a pass of the block. A block
// takes `per` heads (whole passes) of one token.
constexpr int kThreads = 256;
constexpr int kRowBlocks = 3, kHalfBlocks = 2, kHeadBlocks = 4;   // blocks an SM holds: of rows alone (of half a warp), of heads (and rows)
template <int kG>
constexpr int kPass = kThreads / kG;

template <typename T, int kG, int kW, bool kInter>
__device__ __forceinline__ void query_rows(const QueryPart& p, const Angles& ang, float eps, int block) {
  using V = Word<T>;
  const int l = threadIdx.x & (kG - 1);
  const int t = block / p.parts, part = block - t * p.parts;
  const int per = ((p.H + p.parts - 1) / p.parts + kPass<kG> - 1) / kPass<kG> * kPass<kG>;
  const int h_end = min(p.H, (part + 1) * per);
  int h = part * per + threadIdx.x / kG;
  const float* cs = ang.of(t);
  if (ang.R != 0 && cs == nullptr) return;   // the whole block's token
  const int half = ang.R >> 1;
  // this lane's word of the rope, if it has one
  int rope = -1;
#pragma unroll
  for (int j = 0; j < kW; ++j) {
    const int c = p.first + (l + kG * j) * V::kN;
    if (c >= p.P && c < p.W) rope = c - p.P;
  }
  const int partner = partner_lane<V::kN>(rope, half, l) & (kG - 1);
  Turn<V::kN, kInter> turn;
  if (rope >= 0) turn.open(cs, rope, half, ang.words);
  const T* src = static_cast<const T*>(p.q) + t * p.q_s0 + h * p.q_s1 + p.first + l * V::kN;
  T* nope = static_cast<T*>(p.nope) + t * p.n_s0 + h * p.n_s1 + p.first + l * V::kN;
  T* pe = static_cast<T*>(p.pe) + t * p.p_s0 + h * p.p_s1 + rope;
  const bool norm = p.weight != nullptr;
  const float inv = 1.f / (float)p.W;
  const T* wgt = static_cast<const T*>(p.weight) + h * p.w_s0 + p.first + l * V::kN;
  const int left = p.W - p.first - l * V::kN;      // columns from this lane's first on
  uint4 own[kW];
  auto ask = [&](bool live, uint4 (&w)[kW]) {
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      w[j] = make_uint4(0u, 0u, 0u, 0u);
      if (live && kG * j * V::kN < left) w[j] = V::load(src + kG * j * V::kN);
    }
  };
  ask(h < h_end, own);
  for (; __any_sync(0xffffffffu, h < h_end); h += kPass<kG>) {
    const bool live = h < h_end;
    // the next head is on its way while this one is worked on
    uint4 next[kW];
    src += kPass<kG> * p.q_s1;
    ask(h + kPass<kG> < h_end, next);
    float by = 1.f;
    if (norm) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < kW; ++j) sum += V::squares(own[j]);
#pragma unroll
      for (int m = 1; m < kG; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      by = norm_factor(sum, (float)p.W, inv, eps);
    }
    __syncwarp();   // the outputs may be q's own columns: every load of a head comes before any store
    float r[V::kN] = {}, y[V::kN] = {};
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      if (!live || kG * j * V::kN >= left) continue;
      float x[V::kN];
      V::open(own[j], x);
      if (norm) V::scale(x, by, V::load(wgt + kG * j * V::kN));
      if (p.first + (l + kG * j) * V::kN < p.P) {
        *reinterpret_cast<uint4*>(nope + kG * j * V::kN) = V::close(x);
      } else {
#pragma unroll
        for (int k = 0; k < V::kN; ++k) r[k] = x[k];
      }
    }
    if (!kInter) {
#pragma unroll
      for (int k = 0; k < V::kN; ++k) y[k] = __shfl_sync(0xffffffffu, r[k], partner, kG);
    }
    if (live && rope >= 0) {
      turn.turn(r, y);
      *reinterpret_cast<uint4*>(pe) = V::close(r);
    }
#pragma unroll
    for (int j = 0; j < kW; ++j) own[j] = next[j];
    nope += kPass<kG> * p.n_s1;
    pe += kPass<kG> * p.p_s1;
    wgt += kPass<kG> * p.w_s0;
  }
}

// Codes of x / scale, the quotient first rounded to the nearest float32. For scales of ordinary size by Markstein's
// steps (divide2 with a last step to the nearest), two at a time: quotients beyond 1024 saturate, so
// larger values are cut there, where no step overflows; what underflows in them has the code 0.
struct Quotients {
  float scale, most;
  uint64_t ns, r;
  bool plain;     // a scale so small or large that the steps could leave the range of normal numbers
  __device__ __forceinline__ explicit Quotients(float s) : scale(s), most(1024.f * fabsf(s)), plain(!(fabsf(s) > 0x1p-60f && fabsf(s) < 0x1p60f)) {
    const float inv = __frcp_rn(plain ? 1.f : s);
    ns = pair(-s, -s);
    r = pair(inv, inv);
  }
  __device__ __forceinline__ uint32_t codes(float x0, float x1) const {
    if (plain) return codes2(__fdiv_rn(x0, scale), __fdiv_rn(x1, scale));
    // the smaller magnitude, with x's sign
    asm("min.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(x0) : "f"(most));
    asm("min.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(x1) : "f"(most));
    const uint64_t x = pair(x0, x1);
    uint64_t q, rem;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(r));
    asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(rem) : "l"(q), "l"(ns), "l"(x));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(rem), "l"(r), "l"(q));
    asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(rem) : "l"(q), "l"(ns), "l"(x));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(rem), "l"(r), "l"(q));
    return codes2(__uint_as_float((uint32_t)q), __uint_as_float((uint32_t)(q >> 32)));
  }
};

// New cache rows, plain or e4m3, in words: kG lanes a row, up to kW words a lane. kLoop: rows from `first` on, every
// `step`th, each asked for, with its slot and position, while the one before is worked on; else one row (beside
// query heads, whose registers the second row would take).
template <typename T, int kFmt, int kG, int kW, bool kInter, bool kLoop>
__device__ __forceinline__ void cache_rows(const RowPart& p, const Angles& ang, float eps, int64_t first, int64_t step) {
  using V = Word<T>;
  const int lane = threadIdx.x & (kG - 1), left = p.E - lane * V::kN, half = ang.R >> 1;
  int rope = -1;
#pragma unroll
  for (int j = 0; j < kW; ++j)
    if (kG * j * V::kN < left && (lane + kG * j) * V::kN >= p.L) rope = (lane + kG * j) * V::kN - p.L;
  const int partner = partner_lane<V::kN>(rope, half, lane) & (kG - 1);
  struct Row {
    uint4 own[kW];
    int64_t slot, pos;
  };
  auto ask = [&](int64_t t, Row& r) {
    const T* const src = static_cast<const T*>(p.kv) + t * p.k_s0 + lane * V::kN;
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      r.own[j] = make_uint4(0u, 0u, 0u, 0u);
      if (t < p.tokens && kG * j * V::kN < left) r.own[j] = V::load(src + kG * j * V::kN);
    }
    r.slot = t < p.tokens ? p.slots[t] : -1;
    r.pos = t < p.tokens && ang.R != 0 ? ang.positions[t] : 0;
  };
  Row row;
  ask(first, row);
  const T* const wgt = static_cast<const T*>(p.weight) + lane * V::kN;
  const Quotients quotients(kFmt == kE4m3 ? *p.scale : 1.f);
  const float inv = 1.f / (float)p.L;
  for (int64_t t = first; kG == 32 ? t < p.tokens : __any_sync(0xffffffffu, t < p.tokens); t += step) {
    Row next;
    if (kLoop) ask(t + step, next);
    const int64_t off = row_offset(p, row.slot, lane);
    const float* cs = off < 0 ? nullptr : ang.row(row.pos, lane);
    const bool live = off >= 0 && (ang.R == 0 || cs != nullptr);   // the same for all lanes of a row
    Turn<V::kN, kInter> turn;
    if (rope >= 0 && live) turn.open(cs, rope, half, ang.words);
    if (kG < 32 || live) {                           // (of half a warp the other row may be live)
      const bool mine = kG == 32 || live;
      // the sums that 32 lanes would have, added in their order: a row's bits do not depend on the call's other rows
      constexpr int kSums = 32 / kG;
      float sum[kSums] = {};
#pragma unroll
      for (int j = 0; j < kW; ++j) {
        const float s = V::squares(row.own[j]);
        if ((lane + kG * j) * V::kN < p.L) sum[j % kSums] += s;
      }
#pragma unroll
      for (int m = 1; m < kG; m <<= 1) {
#pragma unroll
        for (int i = 0; i < kSums; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], m);
      }
      const float by = norm_factor(kSums == 1 ? sum[0] : sum[0] + sum[kSums - 1], (float)p.L, inv, eps);
      auto put = [&](int c, const float (&x)[V::kN]) {
        if constexpr (kFmt == kPlain) {
          *reinterpret_cast<uint4*>(static_cast<T*>(p.cache) + off + c) = V::close(x);
        } else {
          uint32_t w[V::kN / 4] = {};
#pragma unroll
          for (int k = 0; k < V::kN; k += 2) w[k >> 2] |= quotients.codes(x[k], x[k + 1]) << (8 * (k & 2));
          uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.cache) + off + c);
          if constexpr (V::kN == 8) {
            if (p.eights) {
              *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
              return;
            }
          }
#pragma unroll
          for (int k = 0; k < V::kN / 4; ++k) o[k] = w[k];
        }
      };
      uint4 turned = make_uint4(0u, 0u, 0u, 0u);     // the lane's word of the rope, as read
#pragma unroll
      for (int j = 0; j < kW; ++j) {
        const int c = (lane + kG * j) * V::kN;
        if (c >= p.E || !mine) continue;
        if (c < p.L) {
          float x[V::kN];
          V::open(row.own[j], x);
          V::scale(x, by, V::load(wgt + kG * j * V::kN));
          put(c, x);
        } else {
          turned = row.own[j];
        }
      }
      uint4 with = turned;
      if (!kInter) {
        with.x = __shfl_sync(0xffffffffu, turned.x, partner, kG);
        with.y = __shfl_sync(0xffffffffu, turned.y, partner, kG);
        with.z = __shfl_sync(0xffffffffu, turned.z, partner, kG);
        with.w = __shfl_sync(0xffffffffu, turned.w, partner, kG);
      }
      if (rope >= 0 && mine) {
        float x[V::kN], y[V::kN];
        V::open(turned, x);
        V::open(with, y);
        turn.turn(x, y);
        put(p.L + rope, x);
      }
    }
    if (!kLoop) break;
    row = next;
  }
}

// New rows as ds_mla entries: a warp a row, sixteen latents and two rope columns a lane, so that a group of 128
// is eight lanes and its scale worked out once a lane (with a 16-byte word a lane, four groups a lane of four
// float32 values each: 25 us for 20011 rows; 17 with one row a warp, 15 with the next row on its way). vec: aligned
// 16-byte words; wide: 32-byte aligned rows.
template <typename T, bool kInter>
__device__ __forceinline__ void ds_mla_rows(const RowPart& p, const Angles& ang, float eps, int64_t first, int64_t step,
                                            bool vec, bool wide) {
  const int lane = threadIdx.x & 31;
  constexpr int kRaw = 16 * sizeof(T) / 4;           // 32-bit words of sixteen values
  struct Row {
    uint32_t x[kRaw];
    float2 pe;
    int64_t slot, pos;
  };
  auto ask = [&](int64_t t, Row& r) {
    r.slot = r.pos = -1;
    if (t >= p.tokens) return;
    const T* const src = static_cast<const T*>(p.kv) + t * p.k_s0 + 16 * lane;
    const T* const rope = static_cast<const T*>(p.kv) + t * p.k_s0 + kDsMlaLatent + 2 * lane;
    if (vec) {
#pragma unroll
      for (int k = 0; k < kRaw; k += 8) load_words(src + k * (int)(4 / sizeof(T)), reinterpret_cast<uint32_t (&)[8]>(r.x[k]), wide);
      r.pe = load2(rope);
    } else {
      T* const x = reinterpret_cast<T*>(r.x);
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = src[k];
      r.pe = make_float2(to_f(rope[0]), to_f(rope[1]));
    }
    r.slot = p.slots[t];
    r.pos = ang.positions[t];
  };
  Row row;
  ask(first, row);
  float w[16];
  {
    const T* const wgt = static_cast<const T*>(p.weight) + 16 * lane;
    if (vec) {
      load16(wgt, w, false);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) w[k] = to_f(wgt[k]);
    }
  }
  for (int64_t t = first; t < p.tokens; t += step) {
    Row next;
    ask(t + step, next);
    const int64_t off = row_offset(p, row.slot, lane);
    const float* cs = off < 0 ? nullptr : ang.row(row.pos, lane);
    if (cs != nullptr) {                             // the same for the whole warp
      Turn<2, kInter> turn;
      turn.open(cs, 2 * lane, kDsMlaRope / 2, false);
      float x[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        if constexpr (sizeof(T) == 4)
          x[k] = __uint_as_float(row.x[k]);
        else
          x[k] = __uint_as_float(k & 1 ? row.x[k >> 1] & 0xffff0000u : row.x[k >> 1] << 16);
      }
      uint64_t sum2 = 0;
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        const uint64_t v = pair(x[k], x[k + 1]);
        asm("fma.rn.f32x2 %0, %1, %1, %0;" : "+l"(sum2) : "l"(v));
      }
      float sum = __uint_as_float((uint32_t)sum2) + __uint_as_float((uint32_t)(sum2 >> 32));
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      const float by = norm_factor(sum, kDsMlaLatent, 1.f / kDsMlaLatent, eps);
      const uint64_t by2 = pair(by, by);
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        uint64_t v = pair(x[k], x[k + 1]);
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(v), "l"(by2));
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(v), "l"(pair(w[k], w[k + 1])));
        x[k] = __uint_as_float((uint32_t)v);
        x[k + 1] = __uint_as_float((uint32_t)(v >> 32));
      }
      uint32_t codes[4];
      const float scale = quantise_group(x, codes);
      uint8_t* const o = static_cast<uint8_t*>(p.cache) + off;
      *reinterpret_cast<uint4*>(o + 16 * lane) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
      if ((lane & 7) == 0) *reinterpret_cast<float*>(o + kDsMlaLatent + 4 * (lane >> 3)) = scale;
      float y[2] = {row.pe.x, row.pe.y}, z[2] = {};
      if (!kInter) {                                 // columns 2 lane and 2 lane + 1: their partners 32 columns on or back
        z[0] = __shfl_xor_sync(0xffffffffu, y[0], 16);
        z[1] = __shfl_xor_sync(0xffffffffu, y[1], 16);
      }
      turn.turn(y, z);
      reinterpret_cast<__nv_bfloat162*>(o + kDsMlaRopeByte)[lane] = __floats2bfloat162_rn(y[0], y[1]);
    }
    row = next;
  }
}

// Blocks [0, q_blocks) take query heads, the others cache rows.
template <typename T, int kFmt, int kG, int kW, bool kInter>
__global__ void __launch_bounds__(kThreads, kW == 0 ? (kG == 16 ? kHalfBlocks : kRowBlocks) : kHeadBlocks) norm_rope_kernel(const QueryPart q, const RowPart r, const Angles ang, float eps,
                                                                int q_blocks) {
  pdl_enter();
  if constexpr (kW > 0) {
    if ((int)blockIdx.x < q_blocks) {
      query_rows<T, kG, kW, kInter>(q, ang, eps, blockIdx.x);
      return;
    }
  }
  // rows alone: kG lanes a row; beside heads a warp
  constexpr int kLanes = kW == 0 ? kG : 32, kRows = kThreads / kLanes;
  const int64_t first = (int64_t)(blockIdx.x - q_blocks) * kRows + threadIdx.x / kLanes;
  cache_rows<T, kFmt, kLanes, kLanes == 16 || sizeof(T) == 4 ? 5 : 3, kInter, kW == 0>(   // 640 or 768 columns
      r, ang, eps, first, (int64_t)(gridDim.x - q_blocks) * kRows);
}

template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreads, kRowBlocks) norm_rope_ds_mla_kernel(const RowPart r, const Angles ang, float eps, int vec,
                                                                       int wide) {
  pdl_enter();
  const int64_t first = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  ds_mla_rows<T, kInter>(r, ang, eps, first, (int64_t)gridDim.x * (kThreads / 32), vec, wide);
}

// ---------------------------------------------------------------------------
// Any widths, strides and alignment (plain and e4m3 rows), a warp a row, value by value; the row is read
// a second time for its stores, from L1. A lane that stores a pair of rope columns has read both, so the
// outputs of the queries may be q's own columns here too.
template <typename T>
__device__ __forceinline__ float row_sum(const T* x, int n, int lane) {
  float sum = 0.f;
  for (int c = lane; c < n; c += 32) {
    const float v = to_f(x[c]);
    sum += v * v;
  }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  return sum;
}

// Columns [0, P) of a row times by * wgt (wgt null: as they are) and the rotated pairs behind them, each
// given to put(column, value); the norm goes over the first `normed` columns.
template <typename T, typename F>
__device__ __forceinline__ void each_column(const T* src, const T* wgt, int normed, int first, int P, const Angles& ang,
                                            const float* cs, float by, int lane, F&& put) {
  auto value = [&](int c) { return wgt != nullptr && c < normed ? to_f(src[c]) * by * to_f(wgt[c]) : to_f(src[c]); };
  for (int c = first + lane; c < P; c += 32) put(c, value(c));
  const int half = ang.R >> 1;
  for (int i = lane; i < half; i += 32) {
    const int ca = P + (ang.interleaved ? 2 * i : i), cb = ang.interleaved ? ca + 1 : ca + half;
    const float a = value(ca), b = value(cb), c = cs[i], s = cs[half + i];
    put(ca, fmaf(a, c, -(b * s)));
    put(cb, fmaf(b, c, a * s));
  }
}

template <typename T, int kFmt>
__global__ void __launch_bounds__(256) norm_rope_any_kernel(const QueryPart q, const RowPart r, const Angles ang, float eps,
                                                            int q_blocks) {
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if ((int)blockIdx.x < q_blocks) {
    const int64_t row = (int64_t)blockIdx.x * 8 + warp;
    if (row >= (int64_t)q.tokens * q.H) return;
    const int t = (int)(row / q.H), h = (int)(row - (int64_t)t * q.H);
    const float* cs = ang.of(t);
    if (ang.R != 0 && cs == nullptr) return;
    const T* src = static_cast<const T*>(q.q) + t * q.q_s0 + h * q.q_s1;
    const T* wgt = q.weight == nullptr ? nullptr : static_cast<const T*>(q.weight) + h * q.w_s0;
    const float by = wgt != nullptr ? norm_factor(row_sum(src, q.W, lane), (float)q.W, 1.f / (float)q.W, eps) : 1.f;
    T* nope = static_cast<T*>(q.nope) + t * q.n_s0 + h * q.n_s1;
    T* pe = static_cast<T*>(q.pe) + t * q.p_s0 + h * q.p_s1;
    __syncwarp();   // sums are done with columns that the stores may overwrite
    each_column(src, wgt, q.W, q.first, q.P, ang, cs, by, lane, [&](int c, float v) {
      if (c < q.P)
        from_f(nope + c, v);
      else
        from_f(pe + (c - q.P), v);
    });
    return;
  }
  const int64_t t = (int64_t)(blockIdx.x - q_blocks) * 8 + warp;
  if (t >= r.tokens) return;
  const int64_t off = row_offset(r, r.slots[t], lane);
  if (off < 0) return;
  const float* cs = ang.of(t);
  if (ang.R != 0 && cs == nullptr) return;
  const T* src = static_cast<const T*>(r.kv) + t * r.k_s0;
  const float by = norm_factor(row_sum(src, r.L, lane), (float)r.L, 1.f / (float)r.L, eps);
  const float scale = kFmt == kE4m3 ? *r.scale : 1.f;
  each_column(src, static_cast<const T*>(r.weight), r.L, 0, r.L, ang, cs, by, lane, [&](int c, float v) {
    if constexpr (kFmt == kPlain)
      from_f(static_cast<T*>(r.cache) + off + c, v);
    else
      static_cast<uint8_t*>(r.cache)[off + c] =
          static_cast<uint8_t>(__nv_cvt_float_to_fp8(__fdiv_rn(v, scale), __NV_SATFINITE, __NV_E4M3));
  });
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether both parts move whole 16-byte words (a part with nothing to do does not matter).
template <typename T>
bool in_words(const QueryPart& q, const RowPart& r, int fmt, const Angles& a) {
  constexpr int per = Word<T>::kN;
  if (a.R % (2 * per) != 0) return false;   // halves of whole words
  if (q.tokens > 0) {
    if (q.P % per || !aligned16(q.q) || !aligned16(q.nope) || !aligned16(q.pe) || q.q_s0 % per || q.q_s1 % per ||
        q.n_s0 % per || q.n_s1 % per || q.p_s0 % per || q.p_s1 % per)
      return false;
    if (q.weight != nullptr && (!aligned16(q.weight) || q.w_s0 % per)) return false;
    if ((q.W - q.first) / per > 32 * 4 || a.R / per > 32) return false;   // four words a lane, one of them the rope's
  }
  if (r.tokens > 0) {
    if (r.L % per || a.R / per > 32 || r.E > (sizeof(T) == 4 ? 5 : 3) * 32 * per || !aligned16(r.kv) || r.k_s0 % per || !aligned16(r.weight))
      return false;
    const int unit = fmt == kPlain ? per : 4;   // an e4m3 row is stored four codes at a time
    if (fmt == kPlain ? !aligned16(r.cache) : reinterpret_cast<uintptr_t>(r.cache) % 4 != 0) return false;
    if (r.c_blk % unit || r.c_row % unit) return false;
  }
  return true;
}

// Blocks for `tokens` rows, `rows` at a time in each: no more than run at once.
unsigned row_blocks(int64_t tokens, int rows, int per_sm) {
  return (unsigned)std::min<int64_t>((tokens + rows - 1) / rows, (int64_t)per_sm * device_sm_count());
}

template <typename T, int kFmt, bool kInter>
cudaError_t launch_words(QueryPart q, const RowPart& r, const Angles& ang, float eps, cudaStream_t st) {
  constexpr int per = Word<T>::kN;
  if (q.tokens == 0) {
    // Half a warp a row where five words a lane hold it and there are more rows than half warps: a row's sum, factor
    // and places are worked out for two at once, and no third of the lanes idles (bf16, us: 40000 rows
    // e4m3 33.6 with a warp a row, 28.6 with half; plain 28.4, 24.1; 2500 rows e4m3 3.8, 3.9, plain 3.0, 3.3).
    if constexpr (per == 8) {
      if (r.E <= 5 * 16 * per && ang.R <= 16 * per && r.tokens > 16 * kHalfBlocks * device_sm_count())
        return launch_k(norm_rope_kernel<T, kFmt, 16, 0, kInter>, row_blocks(r.tokens, 16, kHalfBlocks), kThreads, 0, st, q, r, ang, eps, 0);
    }
    return launch_k(norm_rope_kernel<T, kFmt, 32, 0, kInter>, row_blocks(r.tokens, 8, kRowBlocks), kThreads, 0, st, q, r, ang, eps, 0);
  }
  const unsigned r_blocks = (unsigned)((r.tokens + 7) / 8);
  if constexpr (kFmt == kPlain) {
    // the fewest lanes that hold a head in four words each, the rope in one; and no more words than it takes
    const int words = (q.W - q.first) / per, rope = ang.R / per;
    const int lanes = words <= 32 && rope <= 8 ? 8 : words <= 64 && rope <= 16 ? 16 : 32, w = (words + lanes - 1) / lanes;
    // a token's heads in one block, or in several while that leaves an SM without four
    const int pass = kThreads / lanes, passes = (q.H + pass - 1) / pass;
    q.parts = (int)std::min<int64_t>(passes, (4LL * device_sm_count() + q.tokens - 1) / q.tokens);
    const int64_t q_blocks = (int64_t)q.tokens * q.parts;
    if (q_blocks + r_blocks > INT32_MAX) return cudaErrorInvalidValue;
    auto go = [&](auto kernel) {
      return launch_k(kernel, (unsigned)(q_blocks + r_blocks), kThreads, 0, st, q, r, ang, eps, (int)q_blocks);
    };
    if (lanes == 8) {
      if (w <= 1) return go(norm_rope_kernel<T, kFmt, 8, 1, kInter>);
      return w <= 3 ? go(norm_rope_kernel<T, kFmt, 8, 3, kInter>) : go(norm_rope_kernel<T, kFmt, 8, 4, kInter>);
    }
    if (lanes == 16) return w <= 3 ? go(norm_rope_kernel<T, kFmt, 16, 3, kInter>) : go(norm_rope_kernel<T, kFmt, 16, 4, kInter>);
    return go(norm_rope_kernel<T, kFmt, 32, 4, kInter>);
  }
  return cudaErrorInvalidValue;   // queries go with plain rows alone
}

template <typename T, int kFmt>
cudaError_t launch(const QueryPart& q, const RowPart& r, const Angles& ang, float eps, cudaStream_t st) {
  if (in_words<T>(q, r, kFmt, ang))
    return ang.interleaved ? launch_words<T, kFmt, true>(q, r, ang, eps, st) : launch_words<T, kFmt, false>(q, r, ang, eps, st);
  const unsigned q_blocks = (unsigned)(((int64_t)q.tokens * q.H + 7) / 8);
  return launch_k(norm_rope_any_kernel<T, kFmt>, q_blocks + (unsigned)((r.tokens + 7) / 8), kThreads, 0, st, q, r, ang, eps,
                  (int)q_blocks);
}

template <typename T>
cudaError_t launch_ds_mla(const RowPart& r, const Angles& ang, float eps, cudaStream_t st) {
  constexpr int per = Word<T>::kN;
  const int vec = aligned16(r.kv) && r.k_s0 % per == 0 && aligned16(r.weight);
  const int wide = reinterpret_cast<uintptr_t>(r.kv) % 32 == 0 && r.k_s0 % (2 * per) == 0;
  return launch_k(ang.interleaved ? norm_rope_ds_mla_kernel<T, true> : norm_rope_ds_mla_kernel<T, false>,
                  row_blocks(r.tokens, 8, kRowBlocks), kThreads, 0, st, r, ang, eps, vec, wide);
}

}  // namespace

cudaError_t launch_norm_rope(mla_dtype dt, const NormRopeCall& c, cudaStream_t st) {
  QueryPart q{};
  RowPart r{nullptr, 0, nullptr, nullptr, 0, 0, 0, PageOf(1), 0, 0, nullptr, 0, nullptr, 0};
  Angles ang{c.positions, c.cos_sin, c.cos_sin_stride, c.num_positions, c.R, c.interleaved,
             aligned16(c.cos_sin) && c.cos_sin_stride % 4 == 0 && c.R % 8 == 0};
  if (c.tokens > 0 && c.H > 0) {
    q = QueryPart{c.q.data, c.q.s0, c.q.s1, c.q_nope.data, c.q_nope.s0, c.q_nope.s1, c.q_pe.data, c.q_pe.s0, c.q_pe.s1,
                  c.q_weight, c.q_weight_s0, c.H, c.P, c.P + c.R, 0, (int32_t)c.tokens, 1};
    if (c.q_weight == nullptr && c.q_nope.data == c.q.data && c.q_nope.s0 == c.q.s0 && c.q_nope.s1 == c.q.s1) q.first = c.P;
    // empty outputs: any aligned place serves
    if (c.P == 0) q.nope = const_cast<void*>(q.q), q.n_s0 = q.n_s1 = 0;
    if (c.R == 0) q.pe = const_cast<void*>(q.q), q.p_s0 = q.p_s1 = 0;
    if (q.first == q.W) q.tokens = 0;
  }
  if (c.rows) {
    r = RowPart{c.kv.data, c.kv.s0, c.kv_weight, c.cache.data, c.cache.s0, c.cache.s1, c.cache.n0 * c.cache.n1,
                PageOf((int32_t)c.cache.n1), c.L, c.L + c.R, c.slots, c.tokens, c.scale, 0};
    r.eights = (reinterpret_cast<uintptr_t>(r.cache) | r.c_blk | r.c_row) % 8 == 0;
  }
  if (q.tokens == 0 && r.tokens == 0) return cudaSuccess;
  const bool f32 = dt == MLA_F32;
  if (c.scale != nullptr) return f32 ? launch<float, kE4m3>(q, r, ang, c.eps, st) : launch<__nv_bfloat16, kE4m3>(q, r, ang, c.eps, st);
  if (c.ds_mla) return f32 ? launch_ds_mla<float>(r, ang, c.eps, st) : launch_ds_mla<__nv_bfloat16>(r, ang, c.eps, st);
  return f32 ? launch<float, kPlain>(q, r, ang, c.eps, st) : launch<__nv_bfloat16, kPlain>(q, r, ang, c.eps, st);
}

cudaError_t norm_rope_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_norm_err);
}

}  // namespace mla
