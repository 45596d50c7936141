// Rows into and out of a quantised paged cache: the write of 656-byte fp8 ds_mla
// entries, and the read-back of plain, e4m3 and ds_mla rows into contiguous rows.
//
// Both are bound by HBM: every byte of a row crosses it once. One warp owns one
// row at a time, a lane 16 consecutive latent values, so a 512-wide latent part
// is one pass of the warp; a 128-column scale group is eight lanes, and its
// maximum three exchanges.
#include <cfloat>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "mla_internal.h"

namespace mla {
namespace {

__device__ unsigned g_io_err = 0;

constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// N consecutive values as floats, 16 bytes a load.
template <int N>
__device__ __forceinline__ void load_n(const __nv_bfloat16* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    const uint4 w = *reinterpret_cast<const uint4*>(p + i);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __bfloat1622float2(h[k]);
      x[i + 2 * k] = f.x;
      x[i + 2 * k + 1] = f.y;
    }
  }
}
template <int N>
__device__ __forceinline__ void load_n(const float* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 w = *reinterpret_cast<const float4*>(p + i);
    x[i] = w.x;
    x[i + 1] = w.y;
    x[i + 2] = w.z;
    x[i + 3] = w.w;
  }
}

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

// Four codes of a 32-bit word as floats (exact: every e4m3 value is a half value).
__device__ __forceinline__ void e4m3x4(uint32_t w, float* x) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>((w >> (16 * k)) & 0xFFFFu), __NV_E4M3);
    x[2 * k] = __half2float(__ushort_as_half(h.x));
    x[2 * k + 1] = __half2float(__ushort_as_half(h.y));
  }
}
__device__ __forceinline__ void e4m3x16(const uint4 w, float (&x)[16]) {
  e4m3x4(w.x, x);
  e4m3x4(w.y, x + 4);
  e4m3x4(w.z, x + 8);
  e4m3x4(w.w, x + 12);
}
__device__ __forceinline__ float e4m3(uint8_t c) {
  __nv_fp8_e4m3 v;
  v.__x = c;
  return static_cast<float>(v);
}

// ---------------------------------------------------------------------------
// cache[s/page, s%page] = the ds_mla entry of [kv_c[i] | k_pe[i]] for every token i with slot
// s >= 0. A group's scale is its largest magnitude / 448 (an infinity counts as the largest
// float32, a NaN not at all), at least 2^-126 so that the division stays among normal numbers;
// its codes are e4m3(x / scale), the division correctly rounded in float32 and the code rounded
// to nearest even: a value is off by at most half an e4m3 step of its own size, 2^-4 of it, or
// 2^-10 of the group's scale below the smallest normal code. vec: 16-byte aligned source rows.
template <typename T>
__global__ void __launch_bounds__(256) write_ds_mla_kernel(
    uint8_t* __restrict__ cache, int64_t c_blk, int64_t c_row, int64_t num_rows, int32_t page,
    const T* __restrict__ kv_c, int64_t k_s0, const T* __restrict__ k_pe, int64_t p_s0,
    const int64_t* __restrict__ slots, int64_t tokens, int vec) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t step = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t tok = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; tok < tokens; tok += step) {
    const int64_t s = slots[tok];
    if (s < 0) continue;   // padding
    if (s >= num_rows) {   // would land outside the view: skip and record
      if (lane == 0) atomicOr(&g_io_err, kErrDeviceData);
      continue;
    }
    const int64_t blk = s / page;
    uint8_t* o = cache + blk * c_blk + (s - blk * page) * c_row;
    const T* src = kv_c + tok * k_s0 + lane * 16;
    float x[16], r[8] = {};
    if (vec) {
      load_n(src, x);
      if (lane < 8) load_n(k_pe + tok * p_s0 + lane * 8, r);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = to_f(src[i]);
      if (lane < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = to_f(k_pe[tok * p_s0 + lane * 8 + i]);
      }
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));   // fmaxf passes a NaN over
    top = fminf(top, FLT_MAX);
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    const float scale = fmaxf(__fdiv_rn(top, kE4m3Max), FLT_MIN);
    uint32_t w[4] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      w[i >> 2] |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(x[i], scale), __NV_SATFINITE, __NV_E4M3) << (8 * (i & 3));
    *reinterpret_cast<uint4*>(o + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    if ((lane & 7) == 0) *reinterpret_cast<float*>(o + kDsMlaLatent + 4 * (lane >> 3)) = scale;
    if (lane < 8) store_n(reinterpret_cast<__nv_bfloat16*>(o + kDsMlaRopeByte) + lane * 8, r);
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
  __device__ int64_t offset(int64_t i, int lane) const {
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
    if (lane == 0) atomicOr(&g_io_err, kErrDeviceData);
    return -1;
  }
};

// A plain row: E words, bits unchanged.
template <typename W>
__global__ void __launch_bounds__(256) read_plain_kernel(W* __restrict__ out, int64_t o_s0, const W* __restrict__ cache,
                                                         ReadRows rows, int64_t total, int32_t E) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t step = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; i < total; i += step) {
    const int64_t off = rows.offset(i, lane);
    if (off < 0) continue;
    for (int c = lane; c < E; c += 32) out[i * o_s0 + c] = cache[off + c];
  }
}

// A row of E e4m3 codes, each times *scale. vec: E and the strides multiples of 16 codes, 16-byte
// aligned views.
template <typename T>
__global__ void __launch_bounds__(256) read_fp8_kernel(T* __restrict__ out, int64_t o_s0, const uint8_t* __restrict__ cache,
                                                       ReadRows rows, int64_t total, int32_t E,
                                                       const float* __restrict__ scale_p, int vec) {
  pdl_enter();
  const float scale = *scale_p;
  const int lane = threadIdx.x & 31;
  const int64_t step = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; i < total; i += step) {
    const int64_t off = rows.offset(i, lane);
    if (off < 0) continue;
    T* o = out + i * o_s0;
    if (vec) {
      for (int c = lane * 16; c < E; c += 512) {
        float x[16];
        e4m3x16(*reinterpret_cast<const uint4*>(cache + off + c), x);
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] *= scale;
        store_n(o + c, x);
      }
    } else {
      for (int c = lane; c < E; c += 32) from_f(o + c, e4m3(cache[off + c]) * scale);
    }
  }
}

// A ds_mla entry: 512 codes times their group's scale, then the bf16 rope values. vec: 16-byte
// aligned output rows.
template <typename T>
__global__ void __launch_bounds__(256) read_ds_mla_kernel(T* __restrict__ out, int64_t o_s0,
                                                          const uint8_t* __restrict__ cache, ReadRows rows,
                                                          int64_t total, int vec) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t step = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; i < total; i += step) {
    const int64_t off = rows.offset(i, lane);
    if (off < 0) continue;
    const uint8_t* e = cache + off;
    T* o = out + i * o_s0;
    const uint4 codes = *reinterpret_cast<const uint4*>(e + lane * 16);
    const float scale = *reinterpret_cast<const float*>(e + kDsMlaLatent + 4 * (lane >> 3));
    float x[16], r[8] = {};
    if (lane < 8) load_n(reinterpret_cast<const __nv_bfloat16*>(e + kDsMlaRopeByte) + lane * 8, r);
    e4m3x16(codes, x);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] *= scale;
    if (vec) {
      store_n(o + lane * 16, x);
      if (lane < 8) store_n(o + kDsMlaLatent + lane * 8, r);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) from_f(o + lane * 16 + k, x[k]);
      if (lane < 8) {
#pragma unroll
        for (int k = 0; k < 8; ++k) from_f(o + kDsMlaLatent + lane * 8 + k, r[k]);
      }
    }
  }
}

inline bool aligned(const void* p, int a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// One warp a row, eight rows a block, at most 16 blocks an SM (the kernels stride over the rest).
int row_grid(int64_t rows) {
  const int64_t want = (rows + 7) / 8, cap = (int64_t)device_sm_count() * 16;
  return (int)(want < cap ? want : cap);
}

ReadRows read_rows(const CacheRead& r) {
  return ReadRows{r.block_table, r.bt_stride, r.max_blocks, r.cu_seqlens, r.seq_starts, r.batch,
                  r.cache.s_blk, r.cache.s_row, r.cache.num_blocks, r.cache.page};
}

template <typename W>
cudaError_t launch_plain(const CacheRead& r, int64_t per, cudaStream_t st) {
  ReadRows rows = read_rows(r);
  rows.s_blk /= per;
  rows.s_row /= per;
  return launch_k(read_plain_kernel<W>, row_grid(r.rows), 256, 0, st, (W*)r.out, r.out_s0 / per, (const W*)r.cache.data,
                  rows, r.rows, (int32_t)(r.cache.entry / per));
}

}  // namespace

cudaError_t launch_cache_write_ds_mla(mla_dtype src_dt, const View3& cache, const View3& kv_c, const View3& k_pe,
                                      const int64_t* slots, int64_t tokens, cudaStream_t st) {
  const int64_t per = src_dt == MLA_F32 ? 4 : 8, rows = cache.n0 * cache.n1;
  const int vec = aligned(kv_c.data, 16) && aligned(k_pe.data, 16) && kv_c.s0 % per == 0 && k_pe.s0 % per == 0;
  if (src_dt == MLA_F32)
    return launch_k(write_ds_mla_kernel<float>, row_grid(tokens), 256, 0, st, (uint8_t*)cache.data, cache.s0, cache.s1,
                    rows, (int32_t)cache.n1, (const float*)kv_c.data, kv_c.s0, (const float*)k_pe.data, k_pe.s0, slots,
                    tokens, vec);
  return launch_k(write_ds_mla_kernel<__nv_bfloat16>, row_grid(tokens), 256, 0, st, (uint8_t*)cache.data, cache.s0,
                  cache.s1, rows, (int32_t)cache.n1, (const __nv_bfloat16*)kv_c.data, kv_c.s0,
                  (const __nv_bfloat16*)k_pe.data, k_pe.s0, slots, tokens, vec);
}

cudaError_t launch_cache_read(mla_dtype dt, const CacheRead& r, cudaStream_t st) {
  const int64_t es = dt == MLA_F32 ? 4 : 2, per = 16 / es;
  if (aligned(r.out, 16) && aligned(r.cache.data, 16) && r.out_s0 % per == 0 && r.cache.s_blk % per == 0 &&
      r.cache.s_row % per == 0 && r.cache.entry % per == 0)
    return launch_plain<uint4>(r, per, st);
  return dt == MLA_F32 ? launch_plain<uint32_t>(r, 1, st) : launch_plain<uint16_t>(r, 1, st);
}

cudaError_t launch_cache_read_fp8(mla_dtype dst_dt, const CacheRead& r, const float* scale, cudaStream_t st) {
  const int64_t per = dst_dt == MLA_F32 ? 4 : 8;
  const int vec = aligned(r.out, 16) && r.out_s0 % per == 0 && aligned(r.cache.data, 16) && r.cache.s_blk % 16 == 0 &&
                  r.cache.s_row % 16 == 0 && r.cache.entry % 16 == 0;
  const ReadRows rows = read_rows(r);
  if (dst_dt == MLA_F32)
    return launch_k(read_fp8_kernel<float>, row_grid(r.rows), 256, 0, st, (float*)r.out, r.out_s0,
                    (const uint8_t*)r.cache.data, rows, r.rows, r.cache.entry, scale, vec);
  return launch_k(read_fp8_kernel<__nv_bfloat16>, row_grid(r.rows), 256, 0, st, (__nv_bfloat16*)r.out, r.out_s0,
                  (const uint8_t*)r.cache.data, rows, r.rows, r.cache.entry, scale, vec);
}

cudaError_t launch_cache_read_ds_mla(mla_dtype dst_dt, const CacheRead& r, cudaStream_t st) {
  const int64_t per = dst_dt == MLA_F32 ? 4 : 8;
  const int vec = aligned(r.out, 16) && r.out_s0 % per == 0;
  const ReadRows rows = read_rows(r);
  if (dst_dt == MLA_F32)
    return launch_k(read_ds_mla_kernel<float>, row_grid(r.rows), 256, 0, st, (float*)r.out, r.out_s0,
                    (const uint8_t*)r.cache.data, rows, r.rows, vec);
  return launch_k(read_ds_mla_kernel<__nv_bfloat16>, row_grid(r.rows), 256, 0, st, (__nv_bfloat16*)r.out, r.out_s0,
                  (const uint8_t*)r.cache.data, rows, r.rows, vec);
}

unsigned cache_io_errors_read_clear() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_io_err, sizeof(v)) != cudaSuccess) return 0;
  cudaMemcpyToSymbol(g_io_err, &zero, sizeof(zero));
  return v;
}

}  // namespace mla
