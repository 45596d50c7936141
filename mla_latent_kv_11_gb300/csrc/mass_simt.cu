// Row masses on the CUDA cores: every type and shape that the tensor cores do not take.
//
// A block owns kTile rows of a sequence and goes over the query rows (tokens x heads) that attend any of
// them, kTile at a time: their scores as a float32 tile, kTile / 16 rows by as many queries a thread, in
// steps of columns through shared memory, the next step's values on their way in registers; then the weights
// e^(s - lse), added to the thread's rows. At the end the sixteen threads of a row add up in a fixed order, so a
// result does not change from run to run. Tiles of 64 compute most (1 load of shared memory for 2 products);
// with few query rows a sequence (a decode of up to 32 heads) tiles of 16, as more blocks share the rows and
// fewer queries are padding: 5 sequences of up to 256 float32 rows, 16 heads: 61 us with tiles of 64, 12 with 16.
#include <math_constants.h>

#include <cuda_bf16.h>

#include <algorithm>

#include "mass.cuh"

namespace mla {
namespace {

__device__ unsigned g_mass_simt_err = 0;

constexpr int kMassThreads = 256;

__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ float value(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T, int kTile>
__global__ void __launch_bounds__(kMassThreads) mass_simt_kernel(const MassArgs a, const T* __restrict__ q, int64_t q_s0,
                                                                 int64_t q_s1, const T* __restrict__ cache, int64_t c_blk,
                                                                 int64_t c_row) {
  pdl_enter();
  constexpr int kStep = kTile == 64 ? 32 : 64, kMine = kTile / 16, kLoads = kTile * kStep / kMassThreads;
  __shared__ float sk[kStep][kTile + 4], sq[kStep][kTile + 4];
  __shared__ int64_t row_at[kTile], q_at[kTile];
  __shared__ float q_lse[kTile];
  __shared__ int q_pos[kTile];
  const int b = blockIdx.y, tid = threadIdx.x;
  const MassSeq s = mass_seq(a, b, &g_mass_simt_err);
  if (s.nq == 0) return;
  const int d = s.kv - s.nq;                          // position of the first query
  const int tx = tid & 15, ty = tid >> 4;             // queries kMine tx .., rows kMine ty ..
  const int le = tid % kStep, lr = tid / kStep;       // this thread's column and first row of a step's loads
  constexpr int kLoadRows = kMassThreads / kStep;
  // 64-bit: tokens times heads may pass 32 bits
  const int64_t end = (int64_t)s.nq * a.H;
  for (int t0 = blockIdx.x * kTile; t0 < s.kv; t0 += gridDim.x * kTile) {
    __syncthreads();   // the tile before is done with row_at
    if (tid < kTile) {
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
    float acc[kMine] = {};
    for (int64_t r0 = (int64_t)max(0, t0 - d) * a.H; r0 < end; r0 += kTile) {
      __syncthreads();
      if (tid < kTile) {
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
      float c[kMine][kMine] = {}, nk[kLoads], nq[kLoads];
      auto ask = [&](int e) {
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int r = lr + k * kLoadRows;
          nk[k] = e < a.E && row_at[r] >= 0 ? value(cache[row_at[r] + e]) : 0.f;
          nq[k] = e < a.E && q_at[r] >= 0 ? value(q[q_at[r] + e]) : 0.f;
        }
      };
      ask(le);
      for (int e0 = 0; e0 < a.E; e0 += kStep) {
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          sk[le][lr + k * kLoadRows] = nk[k];
          sq[le][lr + k * kLoadRows] = nq[k];
        }
        __syncthreads();
        if (e0 + kStep < a.E) ask(e0 + kStep + le);
#pragma unroll 8
        for (int e = 0; e < kStep; ++e) {
          float xs[kMine], ys[kMine];
          if constexpr (kMine == 4) {
            const float4 x = *reinterpret_cast<const float4*>(&sk[e][4 * ty]), y = *reinterpret_cast<const float4*>(&sq[e][4 * tx]);
            xs[0] = x.x; xs[1] = x.y; xs[2] = x.z; xs[3] = x.w;
            ys[0] = y.x; ys[1] = y.y; ys[2] = y.z; ys[3] = y.w;
          } else {
            xs[0] = sk[e][ty];
            ys[0] = sq[e][tx];
          }
#pragma unroll
          for (int i = 0; i < kMine; ++i)
#pragma unroll
            for (int j = 0; j < kMine; ++j) c[i][j] = fmaf(xs[i], ys[j], c[i][j]);
        }
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const float l = q_lse[kMine * tx + j];
        const int p = q_pos[kMine * tx + j];
#pragma unroll
        for (int i = 0; i < kMine; ++i)
          if (t0 + kMine * ty + i <= p) acc[i] += expf(fmaf(c[i][j], a.scale, -l));
      }
    }
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
#pragma unroll
      for (int m = 1; m < 16; m <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], m);
      const int t = t0 + kMine * ty + i;
      if (tx == 0 && t < s.kv && row_at[kMine * ty + i] >= 0) {
        float* const m = a.mass + b * a.mass_stride + t;
        *m = new_mass(a.decay == 0.f ? 0.f : *m, acc[i], a.decay);
      }
    }
  }
}

template <typename T, int kTile>
cudaError_t launch(const MassCall& c, const MassArgs& a, cudaStream_t st) {
  // tables are often far longer than their sequences: no more blocks a sequence than fill the SMs a few times
  const int most = std::max(1, 16 * device_sm_count() / c.B);
  const dim3 grid((unsigned)std::min((a.cap + kTile - 1) / kTile, most), (unsigned)c.B);
  return launch_k(mass_simt_kernel<T, kTile>, grid, kMassThreads, 0, st, a, (const T*)c.q.data, c.q.s0, c.q.s1,
                  (const T*)c.cache.data, c.cache.s_blk, c.cache.s_row);
}

}  // namespace

cudaError_t launch_mass_simt(mla_dtype dt, const MassCall& c, cudaStream_t st) {
  const MassArgs a = mass_args(c);
  const bool few = (int64_t)c.T * c.H <= 32 * (int64_t)c.B;   // query rows a sequence, on average
  if (dt == MLA_F32) return few ? launch<float, 16>(c, a, st) : launch<float, 64>(c, a, st);
  return few ? launch<__nv_bfloat16, 16>(c, a, st) : launch<__nv_bfloat16, 64>(c, a, st);
}

cudaError_t mass_simt_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_mass_simt_err);
}

}  // namespace mla
