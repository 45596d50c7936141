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
// warp. A word's partner half a rope away is loaded by the lane that needs it (the line is in L1
// already) instead of being exchanged. Both parts share one launch: a decode step has 5 to 500 blocks
// of work in all.
#include <cfloat>

#include "e4m3_codes.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

__device__ unsigned g_norm_err = 0;

enum Format { kPlain, kE4m3, kDsMla };

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
  // The word at p, which need not be aligned where !vec.
  static __device__ __forceinline__ uint4 load(const T* p, bool vec) {
    if (vec) return *reinterpret_cast<const uint4*>(p);
    float x[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] = to_f(p[i]);
    return close(x);   // exact: the values are T's
  }
};

// Positions and the table of their cosines and sines, [count, R] float32: R / 2 cosines, then R / 2 sines.
struct Angles {
  const int64_t* positions;
  const float* table;
  int64_t stride, count;
  int32_t R, interleaved, words;

  // Row of token t's angles; null where its position lies outside the table (recorded).
  __device__ __forceinline__ const float* of(int64_t t) const {
    if (R == 0) return table;   // nothing to rotate
    const int64_t p = positions[t];
    if (p < 0 || p >= count) {
      atomicOr(&g_norm_err, kErrDeviceData);
      return nullptr;
    }
    return table + p * stride;
  }
  // N consecutive cosines or sines, 16 or 8 bytes a load where the table allows (`words`).
  template <int N>
  __device__ __forceinline__ void load(const float* p, float (&x)[N]) const {
    if (!words) {
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = p[k];
    } else if constexpr (N % 4 == 0) {
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + k);
        x[k] = v.x; x[k + 1] = v.y; x[k + 2] = v.z; x[k + 3] = v.w;
      }
    } else {
      const float2 v = *reinterpret_cast<const float2*>(p);
      x[0] = v.x; x[1] = v.y;
    }
  }
  // (The rotations are written in fused multiply-adds, the same in every kernel, so that which one a call
  // takes does not change a rotation's bits.)
  // The rope columns d .. d + N - 1, with their partners half a rope away in `with` (interleaved: unused).
  template <int N>
  __device__ __forceinline__ void turn(float (&x)[N], const float (&with)[N], const float* cs, int d) const {
    const int half = R >> 1;
    if (interleaved) {
      float c[N / 2], s[N / 2];
      load(cs + (d >> 1), c);
      load(cs + half + (d >> 1), s);
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        const float a = x[k], b = x[k + 1];
        x[k] = fmaf(a, c[k >> 1], -(b * s[k >> 1]));
        x[k + 1] = fmaf(b, c[k >> 1], a * s[k >> 1]);
      }
    } else {
      const int i = d < half ? d : d - half;
      const float sign = d < half ? -1.f : 1.f;
      float c[N], s[N];
      load(cs + i, c);
      load(cs + half + i, s);
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = fmaf(x[k], c[k], sign * (with[k] * s[k]));
    }
  }
};

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
  int32_t rows;         // tokens * H
};

struct RowPart {
  const void* kv;
  int64_t k_s0;
  const void* weight;
  void* cache;
  int64_t c_blk, c_row, num_rows;
  int32_t page, L, E;
  const int64_t* slots;
  int64_t tokens;
  const float* scale;   // kE4m3
};

// Offset of token t's row in the cache; -1: padding, or outside the view (recorded).
__device__ __forceinline__ int64_t row_offset(const RowPart& p, int64_t t, int lane) {
  const int64_t s = p.slots[t];
  if (s < 0) return -1;
  if (s >= p.num_rows) {
    if (lane == 0) atomicOr(&g_norm_err, kErrDeviceData);
    return -1;
  }
  const int64_t blk = s / p.page;
  return blk * p.c_blk + (s - blk * p.page) * p.c_row;
}

// 1 / sqrt(sum / n + eps), one Newton step behind the two roundings of a root and a division: it enters every
// value of the row, and a quantised value next to the middle of two codes tells its last bit.
__device__ __forceinline__ float norm_factor(float sum, int n, float eps) {
  const float v = sum / (float)n + eps, y = 1.f / sqrtf(v);
  const float p = v * y, low = fmaf(v, y, -p);               // v y = p + low
  const float t = fmaf(-low, y, fmaf(-p, y, 1.f));           // 1 - v y^2
  return t == t && y <= FLT_MAX ? fmaf(0.5f * y, t, y) : y;  // (v infinite or zero: as it is)
}

// Heads of queries, in words: kG lanes a row, kW words a lane.
template <typename T, int kG, int kW>
__device__ __forceinline__ void query_rows(const QueryPart& p, const Angles& ang, float eps, int block) {
  using V = Word<T>;
  const int lane = threadIdx.x & 31, l = lane & (kG - 1);
  const int64_t row = ((int64_t)block * (blockDim.x >> 5) + (threadIdx.x >> 5)) * (32 / kG) + lane / kG;
  bool live = row < p.rows;
  const int t = live ? (int)row / p.H : 0, h = live ? (int)row - t * p.H : 0;
  const float* cs = live ? ang.of(t) : nullptr;
  live = live && (ang.R == 0 || cs != nullptr);
  const T* src = static_cast<const T*>(p.q) + t * p.q_s0 + h * p.q_s1;
  const T* wgt = p.weight == nullptr ? nullptr : static_cast<const T*>(p.weight) + h * p.w_s0;
  const int half = ang.R >> 1;
  uint4 own[kW], with[kW];
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < kW; ++j) {
    const int c = p.first + (l + kG * j) * V::kN;
    own[j] = with[j] = make_uint4(0u, 0u, 0u, 0u);
    if (!live || c >= p.W) continue;
    own[j] = V::load(src + c, true);
    if (c >= p.P && !ang.interleaved) with[j] = V::load(src + (c < p.P + half ? c + half : c - half), true);
  }
  if (wgt != nullptr) {
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      float x[V::kN];
      V::open(own[j], x);
#pragma unroll
      for (int k = 0; k < V::kN; ++k) sum += x[k] * x[k];
    }
#pragma unroll
    for (int m = 1; m < kG; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  }
  __syncwarp();   // the outputs may be q's own columns: every load comes before any store
  if (!live) return;
  const float by = wgt != nullptr ? norm_factor(sum, p.W, eps) : 1.f;
#pragma unroll
  for (int j = 0; j < kW; ++j) {
    const int c = p.first + (l + kG * j) * V::kN;
    if (c >= p.W) continue;
    float x[V::kN];
    V::open(own[j], x);
    if (wgt != nullptr) {
      float w[V::kN];
      V::open(V::load(wgt + c, true), w);
#pragma unroll
      for (int k = 0; k < V::kN; ++k) x[k] = x[k] * by * w[k];
    }
    if (c < p.P) {
      *reinterpret_cast<uint4*>(static_cast<T*>(p.nope) + t * p.n_s0 + h * p.n_s1 + c) = V::close(x);
      continue;
    }
    float y[V::kN];
    V::open(with[j], y);
    if (wgt != nullptr && !ang.interleaved) {
      float w[V::kN];
      V::open(V::load(wgt + (c < p.P + half ? c + half : c - half), true), w);
#pragma unroll
      for (int k = 0; k < V::kN; ++k) y[k] = y[k] * by * w[k];
    }
    ang.turn(x, y, cs, c - p.P);
    *reinterpret_cast<uint4*>(static_cast<T*>(p.pe) + t * p.p_s0 + h * p.p_s1 + (c - p.P)) = V::close(x);
  }
}

// A group of 128 latents of a ds_mla entry, a word of it in each of its kLanes lanes: the codes of this
// lane's word, and the scale. The quantisation is that of the ds_mla cache write.
template <int kN, int kLanes>
__device__ __forceinline__ float quantise_group(float (&x)[kN], uint32_t (&w)[kN / 4]) {
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < kN; ++k) top = fmaxf(top, fabsf(x[k]));   // fmaxf passes a NaN over
  const bool finite = top <= FLT_MAX;
  top = fminf(top, FLT_MAX);
#pragma unroll
  for (int m = 1; m < kLanes; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
  const float scale = fmaxf(__fdiv_rn(top, kE4m3Max), FLT_MIN);
  float by = scale;
  if (by < 0x1p-80f) {           // the same quotients, out of the way of underflow
    by *= 0x1p64f;
#pragma unroll
    for (int k = 0; k < kN; ++k) x[k] *= 0x1p64f;
  }
  if (!finite) {                 // the scale is FLT_MAX / 448 then: a code of +-448
#pragma unroll
    for (int k = 0; k < kN; ++k) x[k] = fabsf(x[k]) > FLT_MAX ? copysignf(FLT_MAX, x[k]) : x[k];
  }
  const float inv = __frcp_rn(by);
  const uint64_t r = pair(inv, inv), ns = pair(-by, -by);
#pragma unroll
  for (int k = 0; k < kN / 4; ++k) w[k] = 0;
#pragma unroll
  for (int k = 0; k < kN; k += 2) {
    float a, b;
    divide2(x[k], x[k + 1], ns, r, a, b);
    w[k >> 2] |= codes2(a, b) << (8 * (k & 2));
  }
  return scale;
}

// New cache rows, in words: a warp a row, up to kW words a lane. vec: the sources are aligned words.
template <typename T, int kFmt, int kW>
__device__ __forceinline__ void cache_rows(const RowPart& p, const Angles& ang, float eps, int block, bool vec) {
  using V = Word<T>;
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)block * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.tokens) return;
  const int64_t off = row_offset(p, t, lane);
  if (off < 0) return;
  const float* cs = ang.of(t);
  if (ang.R != 0 && cs == nullptr) return;
  const T* src = static_cast<const T*>(p.kv) + t * p.k_s0;
  const T* wgt = static_cast<const T*>(p.weight);
  const int half = ang.R >> 1;
  uint4 own[kW], with[kW];
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < kW; ++j) {
    const int c = (lane + 32 * j) * V::kN;
    own[j] = with[j] = make_uint4(0u, 0u, 0u, 0u);
    if (c >= p.E) continue;
    own[j] = V::load(src + c, vec);
    if (c >= p.L && !ang.interleaved) with[j] = V::load(src + (c < p.L + half ? c + half : c - half), vec);
  }
#pragma unroll
  for (int j = 0; j < kW; ++j) {
    float x[V::kN];
    V::open(own[j], x);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < V::kN; ++k) s += x[k] * x[k];
    if ((lane + 32 * j) * V::kN < p.L) sum += s;
  }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  const float by = norm_factor(sum, p.L, eps);
  const float scale = kFmt == kE4m3 ? *p.scale : 1.f;
#pragma unroll
  for (int j = 0; j < kW; ++j) {
    const int c = (lane + 32 * j) * V::kN;
    if (kFmt != kDsMla && c >= p.E) continue;   // a group's lanes stay together below
    float x[V::kN];
    V::open(own[j], x);
    if (c < p.L) {
      float w[V::kN];
      V::open(V::load(wgt + c, vec), w);
#pragma unroll
      for (int k = 0; k < V::kN; ++k) x[k] = x[k] * by * w[k];
    } else if (c < p.E) {
      float y[V::kN];
      V::open(with[j], y);
      ang.turn(x, y, cs, c - p.L);
    }
    if constexpr (kFmt == kPlain) {
      *reinterpret_cast<uint4*>(static_cast<T*>(p.cache) + off + c) = V::close(x);
    } else if constexpr (kFmt == kE4m3) {
      uint32_t w[V::kN / 4] = {};
#pragma unroll
      for (int k = 0; k < V::kN; k += 2) w[k >> 2] |= codes2(__fdiv_rn(x[k], scale), __fdiv_rn(x[k + 1], scale)) << (8 * (k & 2));
      uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.cache) + off + c);
#pragma unroll
      for (int k = 0; k < V::kN / 4; ++k) o[k] = w[k];
    } else {
      uint8_t* o = static_cast<uint8_t*>(p.cache) + off;
      constexpr int kLanes = kDsMlaGroup / V::kN;
      if ((32 * j) * V::kN < kDsMlaLatent) {     // the word lies in a group: so do all of the warp's
        uint32_t w[V::kN / 4];
        const float s = quantise_group<V::kN, kLanes>(x, w);
        uint32_t* d = reinterpret_cast<uint32_t*>(o + c);
        if constexpr (V::kN == 8)
          *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
        else
          *d = w[0];
        if ((lane & (kLanes - 1)) == 0) *reinterpret_cast<float*>(o + kDsMlaLatent + 4 * (c / kDsMlaGroup)) = s;
      } else if (c < p.E) {
        __nv_bfloat162* d = reinterpret_cast<__nv_bfloat162*>(o + kDsMlaRopeByte + 2 * (c - kDsMlaLatent));
#pragma unroll
        for (int k = 0; k < V::kN; k += 2) d[k >> 1] = __floats2bfloat162_rn(x[k], x[k + 1]);
      }
    }
  }
}

// Blocks [0, q_blocks) take query heads, the others cache rows.
template <typename T, int kFmt, int kG, int kW>
__global__ void __launch_bounds__(256) norm_rope_kernel(const QueryPart q, const RowPart r, const Angles ang, float eps,
                                                        int q_blocks, int vec) {
  pdl_enter();
  if constexpr (kW > 0) {
    if ((int)blockIdx.x < q_blocks) {
      query_rows<T, kG, kW>(q, ang, eps, blockIdx.x);
      return;
    }
  }
  cache_rows<T, kFmt, sizeof(T) == 4 ? 5 : 3>(r, ang, eps, blockIdx.x - q_blocks, vec);   // 640 or 768 columns
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
    if (row >= q.rows) return;
    const int t = (int)row / q.H, h = (int)row - t * q.H;
    const float* cs = ang.of(t);
    if (ang.R != 0 && cs == nullptr) return;
    const T* src = static_cast<const T*>(q.q) + t * q.q_s0 + h * q.q_s1;
    const T* wgt = q.weight == nullptr ? nullptr : static_cast<const T*>(q.weight) + h * q.w_s0;
    const float by = wgt != nullptr ? norm_factor(row_sum(src, q.W, lane), q.W, eps) : 1.f;
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
  const int64_t off = row_offset(r, t, lane);
  if (off < 0) return;
  const float* cs = ang.of(t);
  if (ang.R != 0 && cs == nullptr) return;
  const T* src = static_cast<const T*>(r.kv) + t * r.k_s0;
  const float by = norm_factor(row_sum(src, r.L, lane), r.L, eps);
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
  if (q.rows > 0) {
    if (q.P % per || !aligned16(q.q) || !aligned16(q.nope) || !aligned16(q.pe) || q.q_s0 % per || q.q_s1 % per ||
        q.n_s0 % per || q.n_s1 % per || q.p_s0 % per || q.p_s1 % per)
      return false;
    if (q.weight != nullptr && (!aligned16(q.weight) || q.w_s0 % per)) return false;
    if ((q.W - q.first) / per > 32 * 4) return false;
  }
  if (r.tokens > 0 && fmt != kDsMla) {
    if (r.L % per || r.E > (sizeof(T) == 4 ? 5 : 3) * 32 * per || !aligned16(r.kv) || r.k_s0 % per || !aligned16(r.weight))
      return false;
    const int unit = fmt == kPlain ? per : 4;   // an e4m3 row is stored four codes at a time
    if (fmt == kPlain ? !aligned16(r.cache) : reinterpret_cast<uintptr_t>(r.cache) % 4 != 0) return false;
    if (r.c_blk % unit || r.c_row % unit) return false;
  }
  return true;
}

template <typename T, int kFmt>
cudaError_t launch(const QueryPart& q, const RowPart& r, const Angles& ang, float eps, cudaStream_t st) {
  const unsigned r_blocks = (unsigned)((r.tokens + 7) / 8);
  if (!in_words<T>(q, r, kFmt, ang)) {
    if constexpr (kFmt == kDsMla) {
      return cudaErrorInvalidValue;   // its widths and cache are words by definition
    } else {
      const unsigned q_blocks = (unsigned)(((int64_t)q.rows + 7) / 8);
      return launch_k(norm_rope_any_kernel<T, kFmt>, q_blocks + r_blocks, 256, 0, st, q, r, ang, eps, (int)q_blocks);
    }
  }
  constexpr int per = Word<T>::kN;
  const int vec = kFmt != kDsMla || (aligned16(r.kv) && r.k_s0 % per == 0 && aligned16(r.weight));
  if (q.rows == 0) return launch_k(norm_rope_kernel<T, kFmt, 32, 0>, r_blocks, 256, 0, st, q, r, ang, eps, 0, vec);
  if constexpr (kFmt == kPlain) {
    // the fewest lanes that hold a row in four words each, and no more words than it takes
    const int words = (q.W - q.first) / per, lanes = words <= 32 ? 8 : words <= 64 ? 16 : 32, w = (words + lanes - 1) / lanes;
    const unsigned q_blocks = (unsigned)(((int64_t)q.rows * lanes + 255) / 256), grid = q_blocks + r_blocks;
    auto go = [&](auto kernel) { return launch_k(kernel, grid, 256, 0, st, q, r, ang, eps, (int)q_blocks, vec); };
    if (lanes == 8) {
      if (w <= 1) return go(norm_rope_kernel<T, kFmt, 8, 1>);
      return w <= 3 ? go(norm_rope_kernel<T, kFmt, 8, 3>) : go(norm_rope_kernel<T, kFmt, 8, 4>);
    }
    if (lanes == 16) return w <= 3 ? go(norm_rope_kernel<T, kFmt, 16, 3>) : go(norm_rope_kernel<T, kFmt, 16, 4>);
    return go(norm_rope_kernel<T, kFmt, 32, 4>);
  }
  return cudaErrorInvalidValue;   // queries go with plain rows alone
}

}  // namespace

cudaError_t launch_norm_rope(mla_dtype dt, const NormRopeCall& c, cudaStream_t st) {
  QueryPart q{};
  RowPart r{};
  Angles ang{c.positions, c.cos_sin, c.cos_sin_stride, c.num_positions, c.R, c.interleaved,
             aligned16(c.cos_sin) && c.cos_sin_stride % 4 == 0 && c.R % 8 == 0};
  if (c.tokens > 0 && c.H > 0) {
    q = QueryPart{c.q.data, c.q.s0, c.q.s1, c.q_nope.data, c.q_nope.s0, c.q_nope.s1, c.q_pe.data, c.q_pe.s0, c.q_pe.s1,
                  c.q_weight, c.q_weight_s0, c.H, c.P, c.P + c.R, 0, (int32_t)(c.tokens * c.H)};
    if (c.q_weight == nullptr && c.q_nope.data == c.q.data && c.q_nope.s0 == c.q.s0 && c.q_nope.s1 == c.q.s1) q.first = c.P;
    // empty outputs: any aligned place serves
    if (c.P == 0) q.nope = const_cast<void*>(q.q), q.n_s0 = q.n_s1 = 0;
    if (c.R == 0) q.pe = const_cast<void*>(q.q), q.p_s0 = q.p_s1 = 0;
    if (q.first == q.W) q.rows = 0;
  }
  if (c.rows) {
    r = RowPart{c.kv.data, c.kv.s0, c.kv_weight, c.cache.data, c.cache.s0, c.cache.s1, c.cache.n0 * c.cache.n1,
                (int32_t)c.cache.n1, c.L, c.L + c.R, c.slots, c.tokens, c.scale};
  }
  if (q.rows == 0 && r.tokens == 0) return cudaSuccess;
  const bool f32 = dt == MLA_F32;
  if (c.scale != nullptr) return f32 ? launch<float, kE4m3>(q, r, ang, c.eps, st) : launch<__nv_bfloat16, kE4m3>(q, r, ang, c.eps, st);
  if (c.ds_mla) return f32 ? launch<float, kDsMla>(q, r, ang, c.eps, st) : launch<__nv_bfloat16, kDsMla>(q, r, ang, c.eps, st);
  return f32 ? launch<float, kPlain>(q, r, ang, c.eps, st) : launch<__nv_bfloat16, kPlain>(q, r, ang, c.eps, st);
}

cudaError_t norm_rope_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_norm_err);
}

}  // namespace mla
