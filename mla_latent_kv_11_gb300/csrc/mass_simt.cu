// Row masses on the CUDA cores: every type and shape that the tensor cores do not take.
//
// A block owns a tile of rows of a sequence and goes over the query rows (tokens x heads) that attend any of
// them, a tile at a time: their scores as float32, eight rows by up to eight queries a thread, in steps of columns
// through shared memory (asynchronous copies, up to three steps ahead); then the weights e^(s - lse), added to the
// thread's rows. What bounds it is shared memory: a load of 16 bytes by a warp takes four cycles whatever its lanes
// share, so that eight by eight scores a thread (16 loads for 256 products) balance loads and products, and smaller
// ones wait for loads. Where a tile has fewer queries, groups of the block's threads therefore share the columns, not
// the scores, and add up at the end (16 heads over 32 x 4K float32 rows: 110 us; 139 with eight scores a thread, 374
// with one). 32 x 4K rows of 128 heads take 450 us, 43 TFLOP/s. Sums go in a fixed order, so a result does not change
// from run to run. A prefill's few tiles of rows deal their queries over the blocks of a cluster (2 x 256 tokens of 128
// heads over 2K float32 rows: 4.0 ms instead of 20.5 for one block a tile, of 64 rows).
#include <math_constants.h>

#include <cuda_bf16.h>

#include <algorithm>

#include "mass.cuh"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

__device__ unsigned g_mass_simt_err = 0;

constexpr int kMassThreads = 256;
constexpr int kMaxBlocks = 8;                        // blocks of a cluster

// Four or two values of shared memory.
__device__ __forceinline__ void take(const float* p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void take(const float* p, float (&x)[2]) {
  const float2 v = *reinterpret_cast<const float2*>(p);
  x[0] = v.x; x[1] = v.y;
}
__device__ __forceinline__ void take(const __nv_bfloat16* p, float (&x)[2]) {
  const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
  x[0] = __uint_as_float(v << 16); x[1] = __uint_as_float(v & 0xffff0000u);
}
__device__ __forceinline__ void take(const __nv_bfloat16* p, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
}

// A tile of kRows rows and kQueries queries: eight rows, kTY apart, by kQ queries, kTX apart, a thread; where that is
// fewer threads than the block has, kSplit groups of them share the columns. A step of columns is kRowBytes of every row,
// its place in shared memory kPitch: an odd number of 16-byte words, so that rows side by side lie in other banks.
template <int kRowsOf, int kQueriesOf, int kQ>
struct Tile {
  static constexpr int kR = 8, kRows = kRowsOf, kQueries = kQueriesOf, kTY = kRows / kR, kTX = kQueries / kQ;
  static constexpr int kGroup = kTY * kTX, kSplit = kMassThreads / kGroup, kMine = kR / kSplit;   // rows a thread adds up
  static constexpr int kRowBytes = kRows == 16 ? 256 : 128, kPitch = kRowBytes + 16, kWords = kRowBytes / 16;
  static constexpr int kStages = kQueries == 16 ? 4 : kQueries <= 64 ? 3 : 2;   // steps in shared memory, two blocks an SM
  static constexpr int kCols = kQ == 8 ? 2 : 4;      // columns at a time: sixty-four scores leave registers for two
  static constexpr int kStage = (kRows + kQueries) * kPitch, kBytes = kStages * kStage;
  static_assert(kGroup % 32 == 0 && kMassThreads % kGroup == 0 && kR % kSplit == 0 && kTX <= 16);
  static_assert(kSplit == 1 || kSplit * kRows * kQueries * 4 <= kBytes);   // the groups' scores take the steps' place
  static_assert(kRowBytes / (kCols * 4) % kSplit == 0);
};

// clusters: a tile's queries are dealt over the `blocks` blocks of one. vec: rows of whole aligned 16-byte words, but
// for their ends.
template <typename T, int kRowsOf, int kQueriesOf, int kQ>
__global__ void __launch_bounds__(kMassThreads, 2) mass_simt_kernel(const MassArgs a, const T* __restrict__ q, int64_t q_s0,
                                                                    int64_t q_s1, const T* __restrict__ cache, int64_t c_blk,
                                                                    int64_t c_row, int blocks, int vec) {
  pdl_enter();
  using G = Tile<kRowsOf, kQueriesOf, kQ>;
  constexpr int kR = G::kR, kRows = G::kRows, kQueries = G::kQueries, kPer = 16 / sizeof(T), kStep = G::kRowBytes / sizeof(T);
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int64_t row_at[kRows], q_at[kQueries];
  __shared__ float q_lse[kQueries], part[kMaxBlocks][kRows];
  __shared__ int q_pos[kQueries];
  const int b = blockIdx.y, tid = threadIdx.x, rank = blockIdx.x % blocks;
  const MassSeq s = mass_seq(a, b, &g_mass_simt_err);
  if (s.nq == 0) return;
  if (blocks > 1) ptx::cluster_sync();                // no block writes to another that is not there yet
  const int d = s.kv - s.nq;                          // position of the first query
  const int group = tid / G::kGroup, in_group = tid % G::kGroup, tx = in_group % G::kTX, ty = in_group / G::kTX;
  const int first = ty + G::kTY * G::kMine * group;   // this thread adds up rows first + kTY * i
  const int steps = (a.E + kStep - 1) / kStep;
  // 64-bit: tokens times heads may pass 32 bits
  const int64_t end = (int64_t)s.nq * a.H;
  // a step's columns of the tile's rows and queries, zeros where there are none
  auto ask = [&](int step) {
    if (step < steps) {
      unsigned char* const stage = smem + step % G::kStages * G::kStage;
      for (int w = tid; w < (kRows + kQueries) * G::kWords; w += kMassThreads) {
        const int r = w / G::kWords, e = step * kStep + w % G::kWords * kPer;
        const int64_t at = r < kRows ? row_at[r] : q_at[r - kRows];
        const T* const src = (r < kRows ? cache : q) + (at < 0 ? 0 : at + e);
        const int there = at < 0 ? 0 : min(max(a.E - e, 0), kPer);
        unsigned char* const dst = stage + r * G::kPitch + w % G::kWords * 16;
        if (vec) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)), "l"(there > 0 ? src : cache),
                       "r"(there * (int)sizeof(T)) : "memory");
        } else {
#pragma unroll
          for (int i = 0; i < kPer; ++i) reinterpret_cast<T*>(dst)[i] = i < there ? src[i] : T(0.f);
        }
      }
    }
    ptx::cp_async_commit();
  };
  for (int t0 = blockIdx.x / blocks * kRows; t0 < s.kv; t0 += gridDim.x / blocks * kRows) {
    __syncthreads();   // the tile before is done with row_at
    if (tid < kRows) {
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
    float acc[G::kMine] = {};
    for (int64_t r0 = (int64_t)max(0, t0 - d) * a.H + rank * kQueries; r0 < end; r0 += blocks * kQueries) {
      __syncthreads();
      if (tid < kQueries) {
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
      float c[kR][kQ] = {};
#pragma unroll
      for (int i = 0; i < G::kStages - 1; ++i) ask(i);
      for (int step = 0; step < steps; ++step) {
        asm volatile("cp.async.wait_group %0;" ::"n"(G::kStages - 2) : "memory");
        __syncthreads();                                // the step is there, and the one before is done with
        ask(step + G::kStages - 1);
        const unsigned char* const stage = smem + step % G::kStages * G::kStage;
        const unsigned char *const k0 = stage + ty * G::kPitch, *const q0 = stage + (kRows + tx) * G::kPitch;
#pragma unroll 2
        for (int e = group * G::kCols; e < kStep; e += G::kSplit * G::kCols) {
          float xs[kR][G::kCols];
#pragma unroll
          for (int i = 0; i < kR; ++i) take(reinterpret_cast<const T*>(k0 + G::kTY * i * G::kPitch) + e, xs[i]);
#pragma unroll
          for (int j = 0; j < kQ; ++j) {
            float ys[G::kCols];
            take(reinterpret_cast<const T*>(q0 + G::kTX * j * G::kPitch) + e, ys);
#pragma unroll
            for (int k = 0; k < G::kCols; ++k)
#pragma unroll
              for (int i = 0; i < kR; ++i) c[i][j] = fmaf(xs[i][k], ys[k], c[i][j]);
          }
        }
      }
      if constexpr (G::kSplit > 1) {                    // the groups' sums of a score
        float* const sums = reinterpret_cast<float*>(smem) + in_group;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
          for (int j = 0; j < kQ; ++j) sums[((group * kR + i) * kQ + j) * G::kGroup] = c[i][j];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < G::kMine; ++i)
#pragma unroll
          for (int j = 0; j < kQ; ++j) {
            float v = 0.f;
#pragma unroll
            for (int g = 0; g < G::kSplit; ++g) v += sums[((g * kR + G::kMine * group + i) * kQ + j) * G::kGroup];
            c[i][j] = v;
          }
      }
#pragma unroll
      for (int j = 0; j < kQ; ++j) {
        const float l = q_lse[tx + G::kTX * j];
        const int p = q_pos[tx + G::kTX * j];
#pragma unroll
        for (int i = 0; i < G::kMine; ++i)
          if (t0 + first + G::kTY * i <= p) acc[i] += expf(fmaf(c[i][j], a.scale, -l));
      }
    }
#pragma unroll
    for (int i = 0; i < G::kMine; ++i) {
#pragma unroll
      for (int m = 1; m < G::kTX; m <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], m);
    }
    if (blocks > 1) {                                  // the cluster's sums, in its first block
      if (rank > 0 && tx == 0) {
#pragma unroll
        for (int i = 0; i < G::kMine; ++i)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(ptx::map_to_rank(&part[rank][first + G::kTY * i], 0)), "f"(acc[i]) : "memory");
      }
      ptx::cluster_sync();
      if (rank == 0 && tx == 0) {
#pragma unroll
        for (int i = 0; i < G::kMine; ++i)
          for (int r = 1; r < blocks; ++r) acc[i] += part[r][first + G::kTY * i];
      }
    }
    if (rank == 0 && tx == 0) {
#pragma unroll
      for (int i = 0; i < G::kMine; ++i) {
        const int t = t0 + first + G::kTY * i;
        if (t < s.kv && row_at[first + G::kTY * i] >= 0) {
          float* const m = a.mass + b * a.mass_stride + t;
          *m = new_mass(a.decay == 0.f ? 0.f : *m, acc[i], a.decay);
        }
      }
    }
    if (blocks > 1) ptx::cluster_sync();               // the sums are read: the next tile's may come
  }
}

template <typename T, int kRows, int kQueries, int kQ>
cudaError_t launch(const MassCall& c, const MassArgs& a, cudaStream_t st) {
  constexpr int kBytes = Tile<kRows, kQueries, kQ>::kBytes;
  const auto kernel = mass_simt_kernel<T, kRows, kQueries, kQ>;
  if (kBytes > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
  }
  const uintptr_t all = reinterpret_cast<uintptr_t>(c.q.data) | reinterpret_cast<uintptr_t>(c.cache.data) |
                        sizeof(T) * (uintptr_t)(c.q.s0 | c.q.s1 | c.cache.s_blk | c.cache.s_row);
  const int vec = all % 16 == 0;
  const int64_t sms = device_sm_count();
  const int64_t tiles = (a.cap + kRows - 1) / kRows, rows = (int64_t)c.T * c.H / c.B;   // query rows a sequence, on average
  int blocks = 1;                                     // of a cluster, while twice the SMs' blocks are not reached
  while (blocks < kMaxBlocks && blocks * kQueries < rows && 2 * blocks * tiles * c.B <= 4 * sms) blocks *= 2;
  // tables are often far longer than their sequences: no more blocks a sequence than fill the SMs a few times
  const int64_t most = std::max<int64_t>(1, 16 * sms / (c.B * blocks));
  return launch_clusters(kernel, blocks, dim3((unsigned)(std::min(tiles, most) * blocks), (unsigned)c.B),
                         kMassThreads, kBytes, st, a, (const T*)c.q.data, c.q.s0, c.q.s1, (const T*)c.cache.data, c.cache.s_blk,
                         c.cache.s_row, blocks, vec);
}

template <typename T>
cudaError_t launch_t(const MassCall& c, cudaStream_t st) {
  const MassArgs a = mass_args(c);
  const int64_t rows = (int64_t)c.T * c.H / c.B, tiles = (int64_t)c.B * ((a.cap + 127) / 128);
  // Tiles of 16 rows while those of 128 would leave half of the SMs idle (float32, 16 heads, us: 4K rows 9.2 and 20.7, 12K
  // 24.4 and 22.0), then as many queries a tile as there are, up to 128 (32 x 4K: 16 heads 110 in tiles of 16, 167 of
  // 32; 20 heads 212 and 167; 64 heads 327 of 32, 279 of 64, 447 of 128; 128 heads 547 of 64, 450 of 128).
  if (rows <= 64 && 2 * tiles < device_sm_count()) return launch<T, 16, 16, 1>(c, a, st);
  if (rows <= 16) return launch<T, 128, 16, 8>(c, a, st);
  if (rows <= 32) return launch<T, 128, 32, 8>(c, a, st);
  if (rows <= 64) return launch<T, 128, 64, 8>(c, a, st);
  return launch<T, 128, 128, 8>(c, a, st);
}

}  // namespace

cudaError_t launch_mass_simt(mla_dtype dt, const MassCall& c, cudaStream_t st) {
  return dt == MLA_F32 ? launch_t<float>(c, st) : launch_t<__nv_bfloat16>(c, st);
}

cudaError_t mass_simt_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_mass_simt_err);
}

}  // namespace mla
