// Windowed attention on the CUDA cores: any head count, any entry width, any page, fp32 or bf16
// (what the tensor-core kernel of attn_pair_tc.cu does not take).
//
// A block of 256 threads holds the queries of up to kHeads heads of one token in shared memory and
// streams the attended rows in sub-tiles of 32, as fp32. Each step is laid out for latency, which bounds
// small cases: a warp loads whole rows, consecutive lanes on consecutive values, all its loads in
// flight at once; for the scores a warp takes four heads and a part of a row's width, a lane a key, four
// values a load; for the output a thread owns two latent columns of every head. One pass with the
// running maximum and sum of a softmax, all in fp32.
//
// Eight heads a block balance the loads of rows (again for every block of heads) against the products;
// with fewer blocks than the SMs can hold, four are faster. Measured, with 16, 8 and 4 heads (fp32, 16
// heads): 5 sequences of up to 104 attended rows 36, 29 and 23 us; 64 of 512 rows 143, 114 and 180. The
// schedule cuts rows to sub-tiles and no finer than the blocks that the SMs hold at once: the 5 sequences
// 16 us, 23 with pieces of two sub-tiles; 64 of 1024 rows and 128 heads 1.32 ms, 1.52 with a unit an SM.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>

#include "window_sched.cuh"

namespace mla {
namespace {

__device__ unsigned g_window_simt_err = 0;

constexpr int kKeys = 32, kThreads = 256;

__device__ __forceinline__ float ld(const float* p) { return *p; }
__device__ __forceinline__ float ld(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st(float* p, float v) { *p = v; }
__device__ __forceinline__ void st(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

struct SimtArgs {
  WindowSched sched;
  WindowOut out;
  const void* q;
  int64_t q_s0, q_s1;
  CacheView cv;
  const int32_t* block_table;
  int64_t bt_stride;
  int R, window, sinks;
  float scale;
};

// Pitch of a staged row: its width rounded up to four, plus four (lanes reading 16 bytes of
// consecutive rows then hit different banks).
__host__ __device__ inline int row_pitch(int E) { return (E + 3) / 4 * 4 + 4; }
// Parts of a row's width that different warps take, for the scores.
__host__ __device__ constexpr int parts(int heads) { return kThreads / 32 / (heads / 4); }
template <int kHeads>
size_t simt_bytes(int E) {
  constexpr int kParts = parts(kHeads);
  return sizeof(float) * ((size_t)(kHeads + kKeys) * row_pitch(E) + (kParts + 1) * kHeads * kKeys + 3 * kHeads);
}

// A row of E values into shared memory by one warp (zeros up to the pitch; all zeros without a source).
template <typename T>
__device__ __forceinline__ void stage_row(float* dst, const T* src, int E, int P, int lane) {
#pragma unroll 6
  for (int e = lane; e < P; e += 32) dst[e] = src != nullptr && e < E ? ld(src + e) : 0.f;
}

template <typename T, int kHeads>
__global__ void __launch_bounds__(kThreads) window_simt_kernel(SimtArgs a) {
  constexpr int kParts = parts(kHeads);
  extern __shared__ __align__(16) float sm[];
  pdl_enter();
  const int L = a.out.L, E = L + a.R, P = row_pitch(E), H = a.out.H;
  float* const q = sm;
  float* const k = q + kHeads * P;
  float(*const part)[kHeads][kKeys] = reinterpret_cast<float(*)[kHeads][kKeys]>(k + kKeys * P);
  float(*const w)[kKeys] = part[kParts];
  float* const m = reinterpret_cast<float*>(part + kParts + 1);
  float* const l = m + kHeads;
  float* const alpha = l + kHeads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h0 = blockIdx.y * kHeads, hn = min(kHeads, H - h0);
  Walker<1, false> wk;
  wk.init(a.sched, blockIdx.x, gridDim.x, &g_window_simt_err);
  Seg sg;
  while (wk.next(a.sched, sg, &g_window_simt_err)) {
    __syncthreads();   // the last segment's sums are read
    for (int h = warp; h < kHeads; h += kThreads / 32)
      stage_row(q + h * P,
                h < hn ? static_cast<const T*>(a.q) + (int64_t)sg.tok0 * a.q_s0 + (int64_t)(h0 + h) * a.q_s1 : nullptr, E, P,
                lane);
    if (tid < kHeads) {
      m[tid] = -CUDART_INF_F;
      l[tid] = 0.f;
    }
    float acc[kHeads][2];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) acc[h][0] = acc[h][1] = 0.f;
    const int pos = sg.pos0;
    for (int j = sg.t0; j < sg.t1; ++j) {   // halves of blocks
      // lane i: cache row i of the half, attended or not, and where it lies (-1: nowhere)
      const int base = block_row(sg, j >> 1), t = base + kKeys * (j & 1) + lane;
      const bool seen = base >= 0 && t <= pos && (t < a.sinks || t > pos - a.window);
      if (!__any_sync(0xffffffffu, seen)) continue;   // the same in every warp
      int64_t off = -1;
      if (seen) {
        const int blk = a.block_table[(int64_t)sg.b * a.bt_stride + t / a.cv.page];
        if (blk >= 0 && blk < a.cv.num_blocks)
          off = (int64_t)blk * a.cv.s_blk + (int64_t)(t % a.cv.page) * a.cv.s_row;
        else
          atomicOr(&g_window_simt_err, kErrDeviceData);
      }
      __syncthreads();   // the last sub-tile is done with k and w
#pragma unroll
      for (int i = 0; i < kKeys / 8; ++i) {
        const int r = warp + 8 * i;
        const int64_t o = __shfl_sync(0xffffffffu, off, r);
        stage_row(k + r * P, o >= 0 ? static_cast<const T*>(a.cv.data) + o : nullptr, E, P, lane);
      }
      __syncthreads();
      {
        // scores: heads hq .. hq + 3, part w of the row, key `lane`
        const int hq = 4 * (warp % (kHeads / 4)), w = warp / (kHeads / 4), n4 = P / 4 - 1, e0 = w * n4 / kParts,
                  e1 = (w + 1) * n4 / kParts;
        const float4* kr = reinterpret_cast<const float4*>(k + lane * P);
        const float4* qr = reinterpret_cast<const float4*>(q + hq * P);
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int e = e0; e < e1; ++e) {
          const float4 x = kr[e];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const float4 y = qr[h * (P / 4) + e];
            s[h] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s[h]))));
          }
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) part[w][hq + h][lane] = s[h];
      }
      __syncthreads();
#pragma unroll
      for (int h = warp; h < kHeads; h += kThreads / 32) {   // softmax, key `lane`
        float s = part[0][h][lane];
#pragma unroll
        for (int i = 1; i < kParts; ++i) s += part[i][h][lane];
        s = off >= 0 ? s * a.scale : -CUDART_INF_F;
        float top = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float m_old = m[h], m_new = fmaxf(m_old, top);
        const float p = s == -CUDART_INF_F ? 0.f : __expf(s - m_new);
        float sum = p;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        w[h][lane] = p;
        __syncwarp();
        if (lane == 0) {
          const float f = m_old == -CUDART_INF_F ? 0.f : __expf(m_old - m_new);
          alpha[h] = f;
          l[h] = l[h] * f + sum;
          m[h] = m_new;
        }
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = tid + c * kThreads;
        if (col >= L) continue;
#pragma unroll
        for (int h = 0; h < kHeads; ++h) acc[h][c] *= alpha[h];
#pragma unroll 2
        for (int i = 0; i < kKeys; i += 4) {
          const float v0 = k[i * P + col], v1 = k[(i + 1) * P + col], v2 = k[(i + 2) * P + col], v3 = k[(i + 3) * P + col];
#pragma unroll
          for (int h = 0; h < kHeads; ++h) {
            const float4 p = *reinterpret_cast<const float4*>(&w[h][i]);
            acc[h][c] = fmaf(p.x, v0, fmaf(p.y, v1, fmaf(p.z, v2, fmaf(p.w, v3, acc[h][c]))));
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      if (h >= hn) continue;
      const float sum = l[h], inv = sum == 0.f ? 0.f : 1.f / sum;   // a NaN stays one
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = tid + c * kThreads;
        if (col >= L) continue;
        if (sg.slot < 0)
          st(static_cast<T*>(a.out.o) + (int64_t)sg.tok0 * a.out.o_s0 + (int64_t)(h0 + h) * a.out.o_s1 + col, acc[h][c] * inv);
        else
          a.out.part_o[((int64_t)sg.slot * H + h0 + h) * L + col] = acc[h][c] * inv;
      }
      if (tid == 0) {
        const float lse = sum == 0.f ? -CUDART_INF_F : m[h] + logf(sum);
        if (sg.slot >= 0)
          a.out.part_lse[(int64_t)sg.slot * H + h0 + h] = lse;
        else if (a.out.lse != nullptr)
          a.out.lse[(int64_t)sg.tok0 * H + h0 + h] = lse;
      }
    }
  }
}

template <typename T, int kHeads>
cudaError_t launch_simt(const SimtArgs& a, int units, cudaStream_t st) {
  const size_t bytes = simt_bytes<kHeads>(a.out.L + a.R);
  const cudaError_t e = cudaFuncSetAttribute(window_simt_kernel<T, kHeads>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  return launch_k(window_simt_kernel<T, kHeads>, dim3(units, (a.out.H + kHeads - 1) / kHeads), kThreads, bytes, st, a);
}

// Blocks that the SMs hold at once: two each.
int resident() { return 2 * device_sm_count(); }
// Work units: one of `heads` heads a block each, as many as run at once.
int simt_units(int num_splits, int64_t H, int heads) {
  if (num_splits > 0) return std::min(num_splits, kMaxUnits);
  return (int)std::max<int64_t>(1, resident() / std::max<int64_t>(1, (H + heads - 1) / heads));
}

}  // namespace

size_t window_simt_workspace(int64_t T, int64_t B, int64_t H, int64_t L, bool decode, int num_splits) {
  return window_workspace(T, B, decode, 1, simt_units(num_splits, H, 8), H, L);   // the larger number of units
}

cudaError_t launch_window_simt(mla_dtype dt, const WindowCall& c, int num_splits, void* ws, cudaStream_t st) {
  // four heads a block where the SMs hold at once all the blocks that have work, at most
  const int64_t rows = std::min<int64_t>((int64_t)c.max_blocks * c.cache.page, (int64_t)c.window.window + c.window.sinks);
  const int64_t items = c.cu_q == nullptr ? c.B : c.q.n0, tiles = 2 * (rows / kBlk + 3);
  const bool few = items * tiles * ((c.H + 3) / 4) <= resident();
  const int units = simt_units(num_splits, c.H, few ? 4 : 8);
  SimtArgs a{};
  cudaError_t e = launch_window_schedule(c, 1, 1, units, c.H, ws, &a.sched, &a.out, st);
  if (e != cudaSuccess) return e;
  a.q = c.q.data;
  a.q_s0 = c.q.s0;
  a.q_s1 = c.q.s1;
  a.cv = c.cache;
  a.block_table = c.block_table;
  a.bt_stride = c.bt_stride;
  a.R = c.R;
  a.window = c.window.window < 0x3fffffff ? c.window.window : 0x3fffffff;
  a.sinks = c.window.sinks;
  a.scale = c.scale;
  if (dt == MLA_F32)
    e = few ? launch_simt<float, 4>(a, units, st) : launch_simt<float, 8>(a, units, st);
  else
    e = few ? launch_simt<__nv_bfloat16, 4>(a, units, st) : launch_simt<__nv_bfloat16, 8>(a, units, st);
  if (e != cudaSuccess) return e;
  return launch_window_merge(dt, a.sched, a.out, units, st);
}

cudaError_t window_simt_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_window_simt_err);
}

}  // namespace mla
