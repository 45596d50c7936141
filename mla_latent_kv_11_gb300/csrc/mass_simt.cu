// Row masses on the CUDA cores: every type and shape that the tensor cores do not take.
//
// A block owns 64 rows of a sequence and goes over the query rows (tokens x heads) that attend any of
// them, 64 at a time: their scores as a 64 x 64 float32 tile, four rows by four queries a thread, in
// steps of 32 columns through shared memory; then the weights e^(s - lse), added to the thread's four
// rows. At the end the sixteen threads of a row add up in a fixed order, so a result does not change
// from run to run.
#include <math_constants.h>

#include <cuda_bf16.h>

#include "mass.cuh"

namespace mla {
namespace {

__device__ unsigned g_mass_simt_err = 0;

constexpr int kTileRows = 64, kTileQ = 64, kStep = 32, kMassThreads = 256;

__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ float value(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__global__ void __launch_bounds__(kMassThreads) mass_simt_kernel(const MassArgs a, const T* __restrict__ q, int64_t q_s0,
                                                                 int64_t q_s1, const T* __restrict__ cache, int64_t c_blk,
                                                                 int64_t c_row) {
  pdl_enter();
  __shared__ float sk[kStep][kTileRows + 4], sq[kStep][kTileQ + 4];
  __shared__ int64_t row_at[kTileRows], q_at[kTileQ];
  __shared__ float q_lse[kTileQ];
  __shared__ int q_pos[kTileQ];
  const int b = blockIdx.y, tid = threadIdx.x;
  const MassSeq s = mass_seq(a, b, &g_mass_simt_err);
  const int t0 = blockIdx.x * kTileRows;
  if (s.nq == 0 || t0 >= s.kv) return;
  if (tid < kTileRows) {
    const int t = t0 + tid;
    row_at[tid] = -1;
    if (t < s.kv) {
      const int pb = t / a.page, blk = a.block_table[b * a.bt_stride + pb];
      if (blk >= 0 && blk < a.num_blocks)
        row_at[tid] = blk * c_blk + (t - pb * a.page) * c_row;
      else
        atomicOr(&g_mass_simt_err, kErrDeviceData);
    }
  }
  const int d = s.kv - s.nq;                          // position of the first query
  const int tx = tid & 15, ty = tid >> 4;             // queries 4 tx .., rows 4 ty ..
  float acc[4] = {};
  // 64-bit: tokens times heads may pass 32 bits
  const int64_t end = (int64_t)s.nq * a.H;
  for (int64_t r0 = (int64_t)max(0, t0 - d) * a.H; r0 < end; r0 += kTileQ) {
    __syncthreads();
    if (tid < kTileQ) {
      const int64_t r = r0 + tid;
      q_at[tid] = -1;
      q_lse[tid] = CUDART_INF_F;
      q_pos[tid] = -1;                                // attends nothing
      if (r < end) {
        const int i = (int)(r / a.H), h = (int)(r - (int64_t)i * a.H);
        q_at[tid] = (int64_t)(s.q0 + i) * q_s0 + h * q_s1;
        const float l = a.lse[(int64_t)(s.q0 + i) * a.H + h];
        q_lse[tid] = l;
        if (l != -CUDART_INF_F) q_pos[tid] = d + i;   // a query that attended nothing gives nothing
      }
    }
    __syncthreads();
    float c[4][4] = {};
    for (int e0 = 0; e0 < a.E; e0 += kStep) {
#pragma unroll
      for (int k = 0; k < kTileRows * kStep / kMassThreads; ++k) {
        const int i = tid + k * kMassThreads, e = i & (kStep - 1), r = i / kStep;
        const bool in = e0 + e < a.E;
        sk[e][r] = in && row_at[r] >= 0 ? value(cache[row_at[r] + e0 + e]) : 0.f;
        sq[e][r] = in && q_at[r] >= 0 ? value(q[q_at[r] + e0 + e]) : 0.f;
      }
      __syncthreads();
#pragma unroll 8
      for (int e = 0; e < kStep; ++e) {
        const float4 x = *reinterpret_cast<const float4*>(&sk[e][4 * ty]), y = *reinterpret_cast<const float4*>(&sq[e][4 * tx]);
        const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) c[i][j] = fmaf(xs[i], ys[j], c[i][j]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float l = q_lse[4 * tx + j];
      const int p = q_pos[4 * tx + j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t0 + 4 * ty + i <= p) acc[i] += expf(fmaf(c[i][j], a.scale, -l));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], m);
    const int t = t0 + 4 * ty + i;
    if (tx == 0 && t < s.kv && row_at[4 * ty + i] >= 0) {
      float* const m = a.mass + b * a.mass_stride + t;
      *m = new_mass(a.decay == 0.f ? 0.f : *m, acc[i], a.decay);
    }
  }
}

}  // namespace

cudaError_t launch_mass_simt(mla_dtype dt, const MassCall& c, cudaStream_t st) {
  const MassArgs a = mass_args(c);
  const dim3 grid((unsigned)((a.cap + kTileRows - 1) / kTileRows), (unsigned)c.B);
  if (dt == MLA_F32)
    return launch_k(mass_simt_kernel<float>, grid, kMassThreads, 0, st, a, (const float*)c.q.data, c.q.s0, c.q.s1,
                    (const float*)c.cache.data, c.cache.s_blk, c.cache.s_row);
  return launch_k(mass_simt_kernel<__nv_bfloat16>, grid, kMassThreads, 0, st, a, (const __nv_bfloat16*)c.q.data, c.q.s0,
                  c.q.s1, (const __nv_bfloat16*)c.cache.data, c.cache.s_blk, c.cache.s_row);
}

cudaError_t mass_simt_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_mass_simt_err);
}

}  // namespace mla
