// Rows into and out of a quantised paged cache: the write of 656-byte fp8 ds_mla
// entries, and the read-back of plain, e4m3 and ds_mla rows into contiguous rows.
//
// Both are bound by HBM: every byte of a row crosses it once. A warp takes four consecutive
// rows (one where there are few, so that every SM has some): a lane each looks up where they
// lie, at once, and the warp then has all four in flight (eight or more rows a warp, taken
// four by four, left too few warps at the end: 10 to 30% slower at 40000 rows). In the write a lane
// holds 16 consecutive latent values of a row, so a 512-wide latent part is one pass of the
// warp; a 128-column scale group is eight lanes, and its maximum three exchanges.
#include <cfloat>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>
#include <type_traits>

#include "mla_internal.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

__device__ unsigned g_io_err = 0;

constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

constexpr int kInFlight = 4;   // rows a warp takes, at most

// Sixteen consecutive values as floats: 32 bytes a load where `wide` (32-byte aligned), else 16.
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[8], bool wide) {
  if (wide) {
    ptx::ld_global_32B(p, w);
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&x)[16], bool wide) {
  uint32_t w[8];
  load_words(p, w, wide);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load16(const float* p, float (&x)[16], bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    load_words(p + 8 * h, w, wide);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[8 * h + i] = __uint_as_float(w[i]);
  }
}
// Two consecutive values.
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}
__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }

// N consecutive values, each rounded once to T, 16 bytes a store.
template <int N>
__device__ __forceinline__ void store_n(__nv_bfloat16* p, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    uint4 w;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(x[i + 2 * k], x[i + 2 * k + 1]);
    *reinterpret_cast<uint4*>(p + i) = w;
  }
}
template <int N>
__device__ __forceinline__ void store_n(float* p, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}

// Two consecutive values from bf16.
__device__ __forceinline__ void store2(__nv_bfloat16* p, __nv_bfloat162 v) { *reinterpret_cast<__nv_bfloat162*>(p) = v; }
__device__ __forceinline__ void store2(float* p, __nv_bfloat162 v) { *reinterpret_cast<float2*>(p) = __bfloat1622float2(v); }

// Four codes of a 32-bit word as floats (exact: every e4m3 value is a half value).
__device__ __forceinline__ void e4m3x4(uint32_t w, float* x) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>((w >> (16 * k)) & 0xFFFFu), __NV_E4M3);
    x[2 * k] = __half2float(__ushort_as_half(h.x));
    x[2 * k + 1] = __half2float(__ushort_as_half(h.y));
  }
}
__device__ __forceinline__ float e4m3(uint8_t c) {
  __nv_fp8_e4m3 v;
  v.__x = c;
  return static_cast<float>(v);
}

// x / s as a float32 that rounds to the same code as the quotient itself: rounded toward zero, with
// the last bit set where that lost something. (Rounded to nearest it could land on the middle of two
// codes, which a quotient beside it then rounds as: with bf16 values that is not rare, a 448 / top
// times a short value being off a middle only by the rounding of the scale.) r is 1 / s correctly
// rounded, and the steps Markstein's (IBM J. Res. Dev. 34, 1990): x * r is within two units in the
// last place; the remainder of a quotient that near is exact in one fused multiply-add, a step with
// it makes a neighbour of the quotient, and the neighbour's remainder says on which side that lies.
// No remainder of a quotient near a middle (2^-10 and up) may underflow: s is at least 2^-80 here, x
// finite or NaN. (An exact remainder needs no more: a code's middle has 5 bits, so a quotient that is
// none is 2^-29 of itself away from it at least.)
// The remainders are rounded down. That changes none that is exact, but makes a remainder of zero -0: for
// x = -0 each later sum then adds two zeros of its sign and the quotient is -0; for x = +0 it adds zeros of
// different signs, which to nearest and toward zero is +0. (Rounded to nearest, -0 came out as +0.) Where
// a remainder underflows, |x| is below 2^-125 and the quotient below 2^-45, whose code is a zero of x's
// sign: the last step, with a remainder near x where the steps before cancelled, still gives that sign.
// Two quotients at a time, in paired instructions: ns and r hold -s and 1 / s twice.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  return (uint64_t)__float_as_uint(b) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ float odd(uint32_t bits, uint32_t rem) {
  asm("{\n\t.reg .pred p;\n\tsetp.neu.f32 p, %1, 0f00000000;\n\t@p or.b32 %0, %0, 1;\n\t}"
      : "+r"(bits) : "f"(__uint_as_float(rem)));
  return __uint_as_float(bits);
}
__device__ __forceinline__ void divide2(float x0, float x1, uint64_t ns, uint64_t r, float& y0, float& y1) {
  const uint64_t x = pair(x0, x1);
  uint64_t q, a, rem, t;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(r));
  asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(a) : "l"(q), "l"(ns), "l"(x));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(a) : "l"(a), "l"(r), "l"(q));
  asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(rem) : "l"(a), "l"(ns), "l"(x));
  asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(t) : "l"(rem), "l"(r), "l"(a));
  y0 = odd((uint32_t)t, (uint32_t)rem);
  y1 = odd((uint32_t)(t >> 32), (uint32_t)(rem >> 32));
}

// The codes of two quotients: to nearest even, saturating.
__device__ __forceinline__ uint32_t codes2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// ---------------------------------------------------------------------------
// cache[s/page, s%page] = the ds_mla entry of [kv_c[i] | k_pe[i]] for every token i with slot
// s >= 0. A group's scale is its largest magnitude / 448 (an infinity counts as the largest
// float32, a NaN not at all), at least 2^-126 so that the division stays among normal numbers;
// its codes are e4m3(x / scale), rounded once: a value is off by at most half an e4m3 step of its own size, 2^-4 of it, or 2^-10 of the group's scale below the
// smallest normal code. vec: 16-byte aligned source rows; wide: 32-byte aligned latent rows.
// It wants warps more than rows in flight: 40961 bf16 rows from HBM took 17 us with one row's values a warp
// (48 registers, 40 warps an SM), 21 with two rows' (24 warps); 16.4 with the divisions paired, 4.5 TB/s
// (13.1 where the rows lie in L2; float32 rows 20.7 us, 5.8 TB/s, and 19.7).
template <typename T>
__global__ void __launch_bounds__(256, 5) write_ds_mla_kernel(
    uint8_t* __restrict__ cache, int64_t c_blk, int64_t c_row, int64_t num_rows, int32_t page,
    const T* __restrict__ kv_c, int64_t k_s0, const T* __restrict__ k_pe, int64_t p_s0,
    const int64_t* __restrict__ slots, int64_t tokens, int per_warp, int vec, int wide) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t first = ((blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5) * per_warp;
  if (first >= tokens) return;
  const int n = (int)min((int64_t)per_warp, tokens - first);
  // lane i: where token first + i goes (-1: padding, or outside the view: recorded)
  int64_t off = -1;
  if (lane < n) {
    const int64_t s = slots[first + lane];
    if (s >= num_rows) {
      atomicOr(&g_io_err, kErrDeviceData);
    } else if (s >= 0) {
      const int64_t blk = s / page;
      off = blk * c_blk + (s - blk * page) * c_row;
    }
  }
  __syncwarp();
  for (int i = 0; i < n; ++i) {
    const int64_t to = __shfl_sync(0xffffffffu, off, i);
    if (to < 0) continue;
    const int64_t tok = first + i;
    const T* src = kv_c + tok * k_s0 + lane * 16;
    const T* rope = k_pe + tok * p_s0 + lane * 2;
    float x[16];
    float2 pe;
    if (vec) {
      load16(src, x, wide);
      pe = load2(rope);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = to_f(src[k]);
      pe = make_float2(to_f(rope[0]), to_f(rope[1]));
    }
    uint8_t* o = cache + to;
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(x[k]));   // fmaxf passes a NaN over
    const bool finite = top <= FLT_MAX;
    top = fminf(top, FLT_MAX);
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    const float scale = fmaxf(__fdiv_rn(top, kE4m3Max), FLT_MIN);
    float by = scale;
    if (by < 0x1p-80f) {           // the same quotients, out of the way of underflow
      by *= 0x1p64f;
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] *= 0x1p64f;
    }
    if (!finite) {                 // the scale is FLT_MAX / 448 then: a code of +-448
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = fabsf(x[k]) > FLT_MAX ? copysignf(FLT_MAX, x[k]) : x[k];
    }
    uint32_t w[4] = {};
    const float inv = __frcp_rn(by);
    const uint64_t r = pair(inv, inv), ns = pair(-by, -by);
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      float a, b;
      divide2(x[k], x[k + 1], ns, r, a, b);
      w[k >> 2] |= codes2(a, b) << (8 * (k & 2));
    }
    *reinterpret_cast<uint4*>(o + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    if ((lane & 7) == 0) *reinterpret_cast<float*>(o + kDsMlaLatent + 4 * (lane >> 3)) = scale;
    reinterpret_cast<__nv_bfloat162*>(o + kDsMlaRopeByte)[lane] = __floats2bfloat162_rn(pe.x, pe.y);
  }
}

// ---------------------------------------------------------------------------
// Where a row of the read-back comes from: out row i belongs to the sequence b with
// cu[b] <= i < cu[b + 1] and holds its cache row start[b] + i - cu[b].
struct ReadRows {
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t max_blocks;
  const int32_t* cu;
  const int32_t* starts;   // null: every sequence from its first row
  int32_t batch;
  int64_t s_blk, s_row;    // cache strides, in its elements
  int32_t num_blocks, page;

  // Element offset of out row i's cache row; -1: the row belongs to no sequence, or its block id
  // or position lies outside the table or the cache (recorded, the out row left as it was).
  __device__ int64_t offset(int64_t i) const {
    int lo = 0, hi = batch - 1;   // the last b with cu[b] <= i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cu[mid] <= i) lo = mid; else hi = mid - 1;
    }
    const int64_t c0 = cu[lo];
    if (i < c0 || i >= cu[lo + 1]) return -1;
    const int64_t p = (starts != nullptr ? starts[lo] : 0) + (i - c0);
    const int64_t pb = p / page;
    if (p >= 0 && pb < max_blocks) {
      const int32_t blk = block_table[lo * bt_stride + pb];
      if (blk >= 0 && blk < num_blocks) return blk * s_blk + (p - pb * page) * s_row;
    }
    atomicOr(&g_io_err, kErrDeviceData);
    return -1;
  }

  // Calls row(u, out row, offset, load) for the rows of this warp: first with load = true for each of
  // them, then with load = false.
  template <typename F>
  __device__ __forceinline__ void each(int64_t total, int per_warp, F&& row) const {
    const int lane = threadIdx.x & 31;
    const int64_t first = ((blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5) * per_warp;
    if (first >= total) return;
    const int n = (int)min((int64_t)per_warp, total - first);
    const int64_t mine = lane < n ? offset(first + lane) : -1;
    int64_t off[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) off[u] = __shfl_sync(0xffffffffu, mine, u);
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (off[u] >= 0) row(u, first + u, off[u], true);
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (off[u] >= 0) row(u, first + u, off[u], false);
  }
};

// A plain row: E words, bits unchanged; kWords words of each row in a lane at a time.
template <typename W, int kWords>
__global__ void __launch_bounds__(256) read_plain_kernel(W* __restrict__ out, int64_t o_s0, const W* __restrict__ cache,
                                                         ReadRows rows, int64_t total, int per_warp, int32_t E) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  for (int c0 = lane; c0 - lane < E; c0 += 32 * kWords) {
    W v[kInFlight][kWords];
    rows.each(total, per_warp, [&](int u, int64_t i, int64_t off, bool load) {
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        const int c = c0 + 32 * k;
        if (c >= E) continue;
        if (load)
          v[u][k] = cache[off + c];
        else
          out[i * o_s0 + c] = v[u][k];
      }
    });
  }
}

// Sixteen bytes of output: kN = 4 float32 or 8 bf16 values from as many codes, so that a warp's
// stores cover whole lines (sixteen codes a lane, 32 or 64 bytes of output in steps of 16, wrote every
// sector in parts: 29 us instead of 21 for 28K float32 rows).
template <typename T>
struct Chunk {
  static constexpr int kN = 16 / sizeof(T);
  using Codes = typename std::conditional<sizeof(T) == 4, uint32_t, uint2>::type;
  static __device__ __forceinline__ void store(T* o, Codes c, float scale) {
    float x[kN];
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&c);
#pragma unroll
    for (int i = 0; i < kN; i += 4) e4m3x4(w[i / 4], x + i);
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] *= scale;
    store_n(o, x);
  }
};

// A row of E e4m3 codes, each times *scale. vec: E and the strides multiples of 8 codes, 8-byte
// aligned codes, 16-byte aligned output rows; kChunks chunks of each row in a lane at a time.
template <typename T>
__global__ void __launch_bounds__(256) read_fp8_kernel(T* __restrict__ out, int64_t o_s0, const uint8_t* __restrict__ cache,
                                                       ReadRows rows, int64_t total, int per_warp, int32_t E,
                                                       const float* __restrict__ scale_p, int vec) {
  pdl_enter();
  using C = Chunk<T>;
  constexpr int kChunks = sizeof(T) == 4 ? 5 : 3;   // 640 values and 768: a row of 576 in one round
  const float scale = *scale_p;
  const int lane = threadIdx.x & 31;
  if (vec) {
    for (int c0 = 0; c0 < E; c0 += 32 * kChunks * C::kN) {
      typename C::Codes v[kInFlight][kChunks];
      rows.each(total, per_warp, [&](int u, int64_t i, int64_t off, bool load) {
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          const int c = c0 + (32 * k + lane) * C::kN;
          if (c >= E) continue;
          if (load)
            v[u][k] = *reinterpret_cast<const typename C::Codes*>(cache + off + c);
          else
            C::store(out + i * o_s0 + c, v[u][k], scale);
        }
      });
    }
  } else {
    rows.each(total, per_warp, [&](int, int64_t i, int64_t off, bool load) {
      if (load) return;
      for (int c = lane; c < E; c += 32) from_f(out + i * o_s0 + c, e4m3(cache[off + c]) * scale);
    });
  }
}

// A ds_mla entry: 512 codes times their group's scale, then the bf16 rope values. vec: 16-byte
// aligned output rows.
template <typename T>
__global__ void __launch_bounds__(256) read_ds_mla_kernel(T* __restrict__ out, int64_t o_s0,
                                                          const uint8_t* __restrict__ cache, ReadRows rows,
                                                          int64_t total, int per_warp, int vec) {
  pdl_enter();
  using C = Chunk<T>;
  constexpr int kChunks = kDsMlaLatent / (32 * C::kN);
  const int lane = threadIdx.x & 31;
  typename C::Codes codes[kInFlight][kChunks];
  float scale[kInFlight][kChunks];
  __nv_bfloat162 pe[kInFlight];
  rows.each(total, per_warp, [&](int u, int64_t i, int64_t off, bool load) {
    const uint8_t* e = cache + off;
    T* o = out + i * o_s0;
    if (load) {
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const int c = (32 * k + lane) * C::kN;
        codes[u][k] = *reinterpret_cast<const typename C::Codes*>(e + c);
        scale[u][k] = *reinterpret_cast<const float*>(e + kDsMlaLatent + 4 * (c / kDsMlaGroup));
      }
      pe[u] = reinterpret_cast<const __nv_bfloat162*>(e + kDsMlaRopeByte)[lane];
    } else if (vec) {
#pragma unroll
      for (int k = 0; k < kChunks; ++k) C::store(o + (32 * k + lane) * C::kN, codes[u][k], scale[u][k]);
      store2(o + kDsMlaLatent + 2 * lane, pe[u]);
    } else {
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const int c = (32 * k + lane) * C::kN;
        for (int m = 0; m < C::kN; ++m)
          from_f(o + c + m, e4m3(reinterpret_cast<const uint8_t*>(&codes[u][k])[m]) * scale[u][k]);
      }
      const float2 f = __bfloat1622float2(pe[u]);
      from_f(o + kDsMlaLatent + 2 * lane, f.x);
      from_f(o + kDsMlaLatent + 2 * lane + 1, f.y);
    }
  });
}

inline bool aligned(const void* p, int a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Rows a warp takes: four where that still gives each SM eight warps.
int rows_per_warp(int64_t rows) { return rows >= (int64_t)device_sm_count() * 32 ? kInFlight : 1; }
unsigned row_grid(int64_t rows, int per_warp) { return (unsigned)((rows + 8 * per_warp - 1) / (8 * per_warp)); }

ReadRows read_rows(const CacheRead& r) {
  return ReadRows{r.block_table, r.bt_stride, r.max_blocks, r.cu_seqlens, r.seq_starts, r.batch,
                  r.cache.s_blk, r.cache.s_row, r.cache.num_blocks, r.cache.page};
}

template <typename W, int kWords>
cudaError_t launch_plain(const CacheRead& r, int64_t per, cudaStream_t st) {
  ReadRows rows = read_rows(r);
  rows.s_blk /= per;
  rows.s_row /= per;
  const int pw = rows_per_warp(r.rows);
  return launch_k(read_plain_kernel<W, kWords>, row_grid(r.rows, pw), 256, 0, st, (W*)r.out, r.out_s0 / per,
                  (const W*)r.cache.data, rows, r.rows, pw, (int32_t)(r.cache.entry / per));
}

}  // namespace

cudaError_t launch_cache_write_ds_mla(mla_dtype src_dt, const View3& cache, const View3& kv_c, const View3& k_pe,
                                      const int64_t* slots, int64_t tokens, cudaStream_t st) {
  const int64_t per = src_dt == MLA_F32 ? 4 : 8, rows = cache.n0 * cache.n1;
  const int vec = aligned(kv_c.data, 16) && aligned(k_pe.data, 16) && kv_c.s0 % per == 0 && k_pe.s0 % per == 0;
  const int wide = aligned(kv_c.data, 32) && kv_c.s0 % (2 * per) == 0;
  const int pw = rows_per_warp(tokens);
  if (src_dt == MLA_F32)
    return launch_k(write_ds_mla_kernel<float>, row_grid(tokens, pw), 256, 0, st, (uint8_t*)cache.data, cache.s0, cache.s1,
                    rows, (int32_t)cache.n1, (const float*)kv_c.data, kv_c.s0, (const float*)k_pe.data, k_pe.s0, slots,
                    tokens, pw, vec, wide);
  return launch_k(write_ds_mla_kernel<__nv_bfloat16>, row_grid(tokens, pw), 256, 0, st, (uint8_t*)cache.data, cache.s0,
                  cache.s1, rows, (int32_t)cache.n1, (const __nv_bfloat16*)kv_c.data, kv_c.s0,
                  (const __nv_bfloat16*)k_pe.data, k_pe.s0, slots, tokens, pw, vec, wide);
}

cudaError_t launch_cache_read(mla_dtype dt, const CacheRead& r, cudaStream_t st) {
  const int64_t es = dt == MLA_F32 ? 4 : 2, per = 16 / es;
  if (aligned(r.out, 16) && aligned(r.cache.data, 16) && r.out_s0 % per == 0 && r.cache.s_blk % per == 0 &&
      r.cache.s_row % per == 0 && r.cache.entry % per == 0)
    // 96 words hold a bf16 row of 576 values, 160 an fp32 one
    return r.cache.entry / per <= 96 ? launch_plain<uint4, 3>(r, per, st) : launch_plain<uint4, 5>(r, per, st);
  return dt == MLA_F32 ? launch_plain<uint32_t, 5>(r, 1, st) : launch_plain<uint16_t, 5>(r, 1, st);
}

cudaError_t launch_cache_read_fp8(mla_dtype dst_dt, const CacheRead& r, const float* scale, cudaStream_t st) {
  const int64_t per = dst_dt == MLA_F32 ? 4 : 8;
  const int vec = aligned(r.out, 16) && r.out_s0 % per == 0 && aligned(r.cache.data, 8) && r.cache.s_blk % 8 == 0 &&
                  r.cache.s_row % 8 == 0 && r.cache.entry % 8 == 0;
  const ReadRows rows = read_rows(r);
  const int pw = rows_per_warp(r.rows);
  if (dst_dt == MLA_F32)
    return launch_k(read_fp8_kernel<float>, row_grid(r.rows, pw), 256, 0, st, (float*)r.out, r.out_s0,
                    (const uint8_t*)r.cache.data, rows, r.rows, pw, r.cache.entry, scale, vec);
  return launch_k(read_fp8_kernel<__nv_bfloat16>, row_grid(r.rows, pw), 256, 0, st, (__nv_bfloat16*)r.out, r.out_s0,
                  (const uint8_t*)r.cache.data, rows, r.rows, pw, r.cache.entry, scale, vec);
}

cudaError_t launch_cache_read_ds_mla(mla_dtype dst_dt, const CacheRead& r, cudaStream_t st) {
  const int64_t per = dst_dt == MLA_F32 ? 4 : 8;
  const int vec = aligned(r.out, 16) && r.out_s0 % per == 0;
  const ReadRows rows = read_rows(r);
  const int pw = rows_per_warp(r.rows);
  if (dst_dt == MLA_F32)
    return launch_k(read_ds_mla_kernel<float>, row_grid(r.rows, pw), 256, 0, st, (float*)r.out, r.out_s0,
                    (const uint8_t*)r.cache.data, rows, r.rows, pw, vec);
  return launch_k(read_ds_mla_kernel<__nv_bfloat16>, row_grid(r.rows, pw), 256, 0, st, (__nv_bfloat16*)r.out, r.out_s0,
                  (const uint8_t*)r.cache.data, rows, r.rows, pw, vec);
}

cudaError_t cache_io_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_io_err);
}

}  // namespace mla
