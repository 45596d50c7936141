// Internal declarations shared by the translation units of libmla.so.
// Nothing here is part of the C ABI (include/mla.h is).
#pragma once

#include <utility>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "mla.h"

namespace mla {

// Bits of the per-module device error words.
constexpr unsigned kErrDeviceData = 1u;  // slot / block id / length out of range
constexpr unsigned kErrTimeout = 2u;     // a bounded wait gave up

// Keys per schedule tile of the split-KV decode (one page of 64 rows at page 64).
constexpr int kTile = 64;

// The fp8 ds_mla cache entry: e4m3 latent codes, then float32 scales (one per group of
// latent columns), then bf16 rope values.
constexpr int kDsMlaLatent = 512;
constexpr int kDsMlaGroup = 128;
constexpr int kDsMlaRope = 64;
constexpr int kDsMlaRopeByte = kDsMlaLatent + 4 * (kDsMlaLatent / kDsMlaGroup);   // 528
constexpr int kDsMlaEntry = kDsMlaRopeByte + 2 * kDsMlaRope;                       // 656
static_assert(kDsMlaEntry == MLA_DS_MLA_ENTRY_BYTES, "ds_mla entry layout");

// A ds_mla cache view: entry (blk, row) at data + blk*s_blk + row*s_row bytes.
struct DsMlaCache {
  const void* data;
  int64_t s_blk, s_row;
  int32_t num_blocks, page;
};

// A rank-3 strided view in ELEMENTS (data already includes the storage offset).
struct View3 {
  void* data;
  int64_t n0, n1, n2;
  int64_t s0, s1, s2;
};

// Programmatic dependent launch. Every kernel of the library is launched with programmatic
// stream serialization, so its launch and prologue overlap the end of the kernel before it in
// the stream. Each kernel calls pdl_enter() before it touches memory an earlier kernel may
// write: griddepcontrol.wait returns once the preceding grid has completed and its writes are
// visible (at once if the preceding stream work was not a programmatic launch), and
// launch_dependents then lets the next kernel start launching.
#ifdef __CUDACC__
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_allow_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_enter() {
  pdl_wait();
  pdl_allow_dependents();
}
#endif

template <typename... KArgs, typename... Args>
inline cudaError_t launch_k(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                            Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// launch_k in clusters of `blocks` blocks along x.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_clusters(void (*kernel)(KArgs...), int blocks, dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                            Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

inline View3 view3(const mla_tensor& t) {
  return View3{t.data, t.shape[0], t.shape[1], t.shape[2], t.stride[0], t.stride[1], t.stride[2]};
}

// Division of rows (below 2^31) by the page: (t * factor) >> shift with factor = 2^shift / page rounded up,
// shift = 31 + log2(page) rounded up; factor is at most 2^32, the error below 2^31 / 2^shift < 1 / page.
struct PageOf {
  uint64_t factor;
  int shift, page;
  explicit PageOf(int p) : shift(31), page(p) {
    while ((1ll << (shift - 31)) < p) ++shift;
    // shift is 62 at most, and 2^62 fits
    factor = ((1ull << shift) + (uint64_t)p - 1) / (uint64_t)p;
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int operator()(int t) const { return (int)(((uint64_t)(uint32_t)t * factor) >> shift); }
#endif
};

// The paged cache as the kernels see it.
struct CacheView {
  const void* data;  // element (blk, row, e) at data + blk*s_blk + row*s_row + e
  int64_t s_blk, s_row;
  int32_t num_blocks, page, entry;
};

// Decode schedule kept in the caller's workspace (all device pointers).
struct DecodeSched {
  int32_t* tile_prefix;  // [B+1] prefix sum of ceil(len_b / kTile)
  int32_t* first_unit;   // [B]   work unit holding the first tile of b
  int32_t* npieces;      // [B]   work units touching b (0 for an empty sequence)
  int32_t* piece_base;   // [B]   first partial slot of b (if npieces[b] > 1)
  int32_t* unit_tile;    // [units+1] first global tile of each work unit (the last entry: total)
  int32_t* unit_seq;     // [units]   first sequence of each unit's range (B for an empty unit)
  int4* seqinfo;         // [B] {tile_prefix[b], clamped length, npieces[b], piece_base[b] - first_unit[b]}
  float* part_o;         // [max_pieces, H, L] normalised partial outputs
  float* part_lse;       // [max_pieces, H]    their natural-log LSE
  int32_t units;         // number of work units W
  int32_t max_pieces;    // B + W
};

// Workspace layout of mla_decode for (B, H, L, units).
struct DecodeWsLayout {
  size_t off_prefix, off_first, off_np, off_base, off_unit, off_useq, off_seqinfo, off_part_o, off_part_lse,
      total;
};
DecodeWsLayout decode_ws_layout(int64_t B, int64_t H, int64_t L, int64_t units);
DecodeSched decode_sched_from_ws(void* ws, const DecodeWsLayout& lay, int32_t B, int32_t units);

// Number of SMs of the current device (cached per device).
int device_sm_count();

// A 3-D TMA map (dims innermost first, strides of dims 1 and 2 in bytes, box b0 x b1 x b2) of
// bf16 elements, or of another element type.
bool make_map3d(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1_bytes,
                uint64_t s2_bytes, uint32_t b0, uint32_t b1, uint32_t b2, CUtensorMapSwizzle swz,
                CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
// True once the driver's tensor-map encoder has been found.
bool tensor_maps_available();

// ---- launchers (return cudaSuccess or the launch error) -------------------
cudaError_t launch_concat_q(mla_dtype dt, const View3& out, const View3& nope, const View3& rope,
                            cudaStream_t st);
cudaError_t launch_cache_write(mla_dtype dt, const View3& cache, const View3& kv_c,
                               const View3& k_pe, int64_t L, int64_t R, const int64_t* slots,
                               int64_t T, cudaStream_t st);
cudaError_t launch_bmm_simt(mla_dtype dt, const View3& out, const View3& a, const View3& b,
                            cudaStream_t st);
// Tensor-core bmm (bmm_tc.cu): bf16, K % 64 == 0, N % 128 == 0, 16-byte aligned views.
bool bmm_tc_supported(mla_dtype dt, const View3& out, const View3& a, const View3& b);
cudaError_t launch_bmm_tc(const View3& out, const View3& a, const View3& b, cudaStream_t st);

// Row tiles per prefill sequence, prefix-summed into out[0..B] (one block).
cudaError_t launch_prefill_items(const int32_t* cu_q, int32_t B, int32_t tpt, int32_t* out, cudaStream_t st);
cudaError_t launch_decode_schedule(const int32_t* seq_lens, int32_t B, int32_t max_blocks,
                                   int32_t page, const DecodeSched& s, cudaStream_t st);
// fp8_cache: the cache holds e4m3 codes (one byte each), read as value * (*descale_k) with the
// query scaled by *descale_q (null pointers read as 1).
cudaError_t launch_decode_simt(mla_dtype dt, const View3& o_lat, float* lse, const View3& q,
                               const CacheView& cache, const int32_t* block_table,
                               int64_t bt_stride, int32_t max_blocks, const int32_t* seq_lens, int32_t B, int32_t H,
                               int32_t L, int32_t R, float scale, const DecodeSched& s,
                               cudaStream_t st, bool fp8_cache = false, const float* descale_q = nullptr,
                               const float* descale_k = nullptr);
// Sparse top-k decode over a ds_mla cache (split kernel only: schedule and combine as above,
// the schedule run with null lengths and cap = topk).
cudaError_t launch_decode_sparse_simt(mla_dtype dt, const View3& o_lat, float* lse, const View3& q,
                                      const DsMlaCache& cache, const int32_t* indices, int64_t idx_stride,
                                      int32_t topk, int32_t B, int32_t H, float scale, const DecodeSched& s,
                                      cudaStream_t st);
// The LSE combine and the W_UV un-projection in one kernel (combine_vup.cu): bf16, L = 512,
// V a multiple of 128, v-contiguous out and W_UV views, W_UV 16-byte aligned.
bool combine_vup_supported(mla_dtype dt, int L, int V, const View3& out, const View3& w_uv);
// out[b, h, :] = combine(o_lat rows / partials of (b, h)) @ w_uv[h], o_lat rounded to bf16 first.
cudaError_t launch_combine_vup(const View3& out, const View3& o_lat, float* lse, const View3& w_uv, int32_t B,
                               int32_t H, int32_t V, const DecodeSched& s, cudaStream_t st);
// The valid slots of each sparse query in listed order ([B, topk], compacted) and their counts.
cudaError_t launch_sparse_compact(const int32_t* indices, int64_t idx_stride, int32_t topk, int32_t B,
                                  int64_t num_rows, int32_t* out, int32_t* counts, cudaStream_t st);
// Tensor-core decode over gathered e4m3 rows (attn_tc.cu): bf16 queries, 64 or 128 heads, a
// 16-byte aligned cache with 16-byte strides, 16-byte aligned query and output views.
bool tc_gather_supported(mla_dtype dt, int H, const void* cache, int64_t s_blk_bytes, int64_t s_row_bytes,
                         const View3& q, const View3& o);
// An e4m3 paged cache (rope 0 or 64, L = 512).
cudaError_t launch_decode_tc_fp8(const View3& o_lat, float* lse, const View3& q, const CacheView& cache,
                                 const int32_t* block_table, int64_t bt_stride, int32_t max_blocks,
                                 int32_t B, int32_t H, int32_t R, float scale, const float* descale_q,
                                 const float* descale_k, const DecodeSched& s, cudaStream_t st);
// A ds_mla cache at compacted slots (the schedule ran on their counts, cap topk).
cudaError_t launch_decode_tc_dsmla(const View3& o_lat, float* lse, const View3& q, const DsMlaCache& cache,
                                   const int32_t* slots, int64_t slot_stride, int32_t topk, int32_t B, int32_t H,
                                   float scale, const DecodeSched& s, cudaStream_t st);
// e4m3 cache write: codes of x / (*scale) (float32, correctly rounded), round to nearest even,
// saturating; src_dt is kv_c's and k_pe's element type.
cudaError_t launch_cache_write_fp8(mla_dtype src_dt, const View3& cache, const View3& kv_c, const View3& k_pe,
                                   int64_t L, int64_t R, const int64_t* slots, int64_t T, const float* scale,
                                   cudaStream_t st);
// ds_mla cache write (cache_io.cu): kv_c [T, 512] and k_pe [T, 64] of src_dt into 656-byte
// entries of a 16-byte aligned cache view (strides in bytes).
cudaError_t launch_cache_write_ds_mla(mla_dtype src_dt, const View3& cache, const View3& kv_c, const View3& k_pe,
                                      const int64_t* slots, int64_t tokens, cudaStream_t st);
// A read-back of cache rows (cache_io.cu): out row i, cu_seqlens[b] <= i < cu_seqlens[b + 1], is
// row seq_starts[b] + i - cu_seqlens[b] of sequence b (null starts: 0). The cache's strides and
// entry count its own elements.
struct CacheRead {
  void* out;
  int64_t out_s0, rows;
  CacheView cache;
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t max_blocks;
  const int32_t *cu_seqlens, *seq_starts;
  int32_t batch;
};
cudaError_t launch_cache_read(mla_dtype dt, const CacheRead& r, cudaStream_t st);
cudaError_t launch_cache_read_fp8(mla_dtype dst_dt, const CacheRead& r, const float* scale, cudaStream_t st);
cudaError_t launch_cache_read_ds_mla(mla_dtype dst_dt, const CacheRead& r, cudaStream_t st);

// Norms and rotations of new queries and cache rows (norm_rope.cu) after validation. H 0: no queries;
// rows false: no cache rows; scale: e4m3 rows; ds_mla: ds_mla entries; else rows of the call's dtype.
struct NormRopeCall {
  int64_t tokens;
  int32_t H, P, R, L, interleaved;
  float eps;
  const int64_t* positions;
  const float* cos_sin;
  int64_t cos_sin_stride, num_positions;
  View3 q, q_nope, q_pe;
  const void* q_weight;      // null: no norm
  int64_t q_weight_s0;
  bool rows, ds_mla;
  View3 cache, kv;
  const void* kv_weight;
  const int64_t* slots;
  const float* scale;
};
cudaError_t launch_norm_rope(mla_dtype dt, const NormRopeCall& c, cudaStream_t st);

// Eviction of the lightest rows (evict.cu) after validation; strides of the cache in bytes.
struct EvictCall {
  void* cache;
  int64_t s_blk, s_row, row_bytes;
  int32_t num_blocks, page;
  float* mass;
  int64_t mass_stride;
  int32_t mass_rows;
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t max_blocks;
  const int32_t* seq_lens;
  int32_t batch, budget, sinks, recent;
  const int32_t* block_table_out;
  int64_t bto_stride;
  int32_t max_blocks_out;
  float* mass_out;
  int64_t mass_out_stride;
  int32_t mass_out_rows;
  int32_t *seq_lens_out, *kept_out;
};
size_t evict_workspace(int64_t batch, int64_t rows, int64_t budget);
cudaError_t launch_evict(const EvictCall& c, void* ws, cudaStream_t st);

// Row masses after validation: what the queries of a prefill (cu_q [B + 1]) or, with cu_q null, of a
// decode give each row.
struct MassCall {
  float* mass;
  int64_t mass_stride;
  int32_t mass_rows;
  View3 q;                 // [T, H, E]
  CacheView cache;
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t max_blocks;
  const int32_t *cu_q, *kv_lens;
  const float* lse;
  int32_t B, T, H;
  float scale, decay;
};
// On the tensor cores (mass_tc.cu): bf16, rows of up to 576 values in whole groups of 64, up to 128 heads,
// pages of whole 64-row blocks or blocks of whole pages of 8 rows or more, 16-byte aligned views. Fills the
// call's tensor maps where it is so.
struct MassMaps {
  CUtensorMap keys, q;
};
bool mass_tc_supported(mla_dtype dt, const MassCall& c, MassMaps* maps);
size_t mass_tc_workspace();   // of a prefill
cudaError_t launch_mass_tc(const MassCall& c, const MassMaps& maps, void* ws, cudaStream_t st);
// On the CUDA cores (mass_simt.cu): everything else.
cudaError_t launch_mass_simt(mla_dtype dt, const MassCall& c, cudaStream_t st);

// Attention limited to a window and sinks. A query at position p of a sequence attends rows t <= p with
// t < sinks or t > p - window.
struct WindowArgs {
  int32_t window, sinks;
};
// A windowed call after validation: a prefill's queries (cu_q [B + 1]) or, with cu_q null, a
// decode's, one token a sequence.
struct WindowCall {
  View3 o, q;
  float* lse;
  CacheView cache;
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t max_blocks;
  const int32_t *cu_q, *kv_lens;
  int32_t B, H, L, R;
  float scale;
  WindowArgs window;
};
// The schedule in the workspace (window_sched.cu): the row tiles' descriptions, how many there are and,
// where row tiles may be cut, {row tile, tile} of each unit's first (null: whole row tiles dealt out);
// most: row tiles at most; cut: some may be cut, so their pieces have to be merged; direct: on the tensor
// cores and without a schedule, units take every units-th row tile and describe it themselves.
struct WindowSched {
  int64_t most;
  int4* items;
  int32_t* total;
  int2* unit_start;
  bool cut, direct;
  const int32_t *cu_q, *kv_lens;   // cu_q null: a decode, one token a sequence
  int32_t B, T, cap, tpt, window, sinks;
};
// Where results go: rows of the output, and the partial slots [2 * units][rows][L] of cut row tiles
// with their log-sum-exps [2 * units][rows]. tptc 0: a slot's row is a head; else rows 64 r .. of a slot
// are tptc tokens' heads each. permuted: of each 32 columns of a partial row, place 8 b + 2 k + i holds
// column 8 k + 2 b + i (b, k < 4, i < 2).
struct WindowOut {
  void* o;
  int64_t o_s0, o_s1;
  float *lse, *part_o, *part_lse;
  int32_t rows, L, H, tptc;
  bool permuted;
};
// Row tiles of tpt tokens over `units` work units, tiles of blocks_per_tile 64-row blocks, slots of
// `rows` rows.
size_t window_workspace(int64_t T, int64_t B, bool decode, int tpt, int64_t units, int64_t rows, int64_t L);
cudaError_t launch_window_schedule(const WindowCall& c, int tpt, int blocks_per_tile, int units, int rows, void* ws,
                                   WindowSched* sched, WindowOut* out, cudaStream_t st);
cudaError_t launch_window_merge(mla_dtype dt, const WindowSched& sched, const WindowOut& out, int units, cudaStream_t st);
// On the tensor cores (attn_pair_tc.cu): bf16, L = 512, R in {0, 64}, up to 128 heads, a positive
// scale, pages of whole 64-row blocks or blocks of whole pages of 8 rows or more, 16-byte aligned
// views. Fills the call's tensor maps where it is so.
struct WindowMaps {
  CUtensorMap keys, boxes, q;
};
bool window_tc_supported(mla_dtype dt, const WindowCall& c, WindowMaps* maps);
// Bytes of workspace for T query tokens of B sequences (0: H is not taken).
size_t window_tc_workspace(int64_t T, int64_t B, int H, bool decode, int num_splits);
cudaError_t launch_window_tc(const WindowCall& c, const WindowMaps& maps, int num_splits, void* ws, cudaStream_t st);
// On the CUDA cores (window_simt.cu): everything else.
size_t window_simt_workspace(int64_t T, int64_t B, int64_t H, int64_t L, bool decode, int num_splits);
cudaError_t launch_window_simt(mla_dtype dt, const WindowCall& c, int num_splits, void* ws, cudaStream_t st);

cudaError_t launch_decode_combine(mla_dtype dt, const View3& o_lat, float* lse,
                                  const int32_t* seq_lens, int32_t B, int32_t H, int32_t L,
                                  const DecodeSched& s, cudaStream_t st);
cudaError_t launch_prefill_simt(mla_dtype dt, const View3& o_lat, float* lse, const View3& q,
                                const CacheView& cache, const int32_t* block_table,
                                int64_t bt_stride, int32_t max_blocks, const int32_t* cu_q,
                                const int32_t* kv_lens, int32_t B, int32_t T, int32_t H,
                                int32_t L, int32_t R, float scale, cudaStream_t st);

// Tensor-core attention (attn_tc.cu): bf16, L = 512, R in {0, 64}, H in {64, 128}, 16-byte
// aligned views.
bool tc_attention_supported(mla_dtype dt, int H, int L, int R, bool decode, const CacheView& cv,
                            const View3& q, const View3& o);
int tc_decode_units(int num_splits);
cudaError_t launch_decode_tc(const View3& o_lat, float* lse, const View3& q, const CacheView& cache,
                             const int32_t* block_table, int64_t bt_stride, int32_t max_blocks,
                             const int32_t* seq_lens, int32_t B, int32_t H, int32_t L, int32_t R,
                             float scale, const DecodeSched& s, cudaStream_t st);
cudaError_t launch_prefill_tc(const View3& o_lat, float* lse, const View3& q, const CacheView& cache,
                              const int32_t* block_table, int64_t bt_stride, int32_t max_blocks,
                              const int32_t* cu_q, const int32_t* kv_lens, int32_t B, int32_t H,
                              int32_t L, int32_t R, float scale, int32_t* item_prefix,
                              cudaStream_t st);

// Validated views of a q concat and of a cache write (mla_api.cu).
struct ConcatPlan {
  bool empty = true;
  View3 out{}, nope{}, rope{};
};
struct WritePlan {
  bool empty = true;
  int64_t L = 0, R = 0;
  View3 cache{}, kv_c{}, k_pe{};
};
mla_status plan_concat(mla_dtype dtype, const mla_tensor& q_cat_out, const mla_tensor& nope,
                       const mla_tensor& rope, ConcatPlan* out);
mla_status plan_cache_write(mla_dtype dtype, const mla_tensor& cache, const mla_tensor& kv_c,
                            const mla_tensor& k_pe, const int64_t* slot_mapping, int64_t num_tokens,
                            WritePlan* out);
// The q concat and the cache write in one launch when both take 16-byte words, else two.
// `alongside`: the launch directly follows a kernel of the same call that writes none of this
// one's inputs or outputs and waits for its own predecessors before it lets dependents launch
// (the absorb into q_cat's latent columns); the copies then run alongside it and wait for it
// only before this kernel ends, so whatever follows still sees both complete.
cudaError_t launch_concat_cache(mla_dtype dt, const View3& out, const View3& nope, const View3& rope,
                                const View3& cache, const View3& kv_c, const View3& k_pe, int64_t L, int64_t R,
                                const int64_t* slots, int64_t T, cudaStream_t st,
                                bool alongside = false);

// Work units of the general (CUDA-core) split-KV decode: num_splits, or two per SM.
int32_t decode_units(int32_t num_splits);

// A decode call after validation: the views the kernels take, the path and its work units.
struct DecodeCall {
  int64_t B = 0, H = 0, L = 0, R = 0;
  bool empty = true;   // nothing to do (B or H is 0)
  CacheView cv{};
  View3 qv{}, ov{};
  bool tc = false;     // tensor-core path
  int32_t units = 0;
};
// The argument checks of mla_decode (every decode entry point uses them, so they report the same
// codes and messages); fills *out on MLA_OK.
mla_status check_decode_args(mla_dtype dtype, const mla_tensor& o_lat_out, const mla_tensor& q_cat,
                             const mla_tensor& cache, const int32_t* block_table, int64_t block_table_stride,
                             int32_t max_blocks, const int32_t* seq_lens, int32_t kv_lora_rank, int32_t rope_dim,
                             float softmax_scale, int32_t num_splits, DecodeCall* out);
// Schedule, split kernel and combine of a validated decode, with its scratch laid out by `lay`.
// fp8_cache: the cache holds e4m3 codes read as value * (*descale_k), the query scaled by *descale_q.
mla_status run_decode(mla_dtype dtype, const DecodeCall& dc, float* lse_out, const int32_t* block_table,
                      int64_t block_table_stride, int32_t max_blocks, const int32_t* seq_lens, float softmax_scale,
                      void* scratch, const DecodeWsLayout& lay, cudaStream_t st, bool fp8_cache = false,
                      const float* descale_q = nullptr, const float* descale_k = nullptr, bool combine = true);

// Set (or clear, with MLA_OK) the calling thread's mla_last_error() message.
mla_status report_status(mla_status st, const char* fmt, ...);

// Per-module error words. Reading one is a blocking copy of 6 us and clearing it another, so most modules
// give the word's address on the current device, and one kernel moves their errors into the copy module's
// word, which is then read (mla_device_error 119 us with a copy and a clearing of each of nine words).
struct ErrorWords {
  static constexpr int kCount = 9;
  unsigned* word[kCount];
};
cudaError_t cache_io_error_word(unsigned** word);
cudaError_t attn_pair_error_word(unsigned** word);
cudaError_t window_sched_error_word(unsigned** word);
cudaError_t window_simt_error_word(unsigned** word);
cudaError_t bmm_tc_error_word(unsigned** word);
cudaError_t norm_rope_error_word(unsigned** word);
cudaError_t evict_error_word(unsigned** word);
cudaError_t mass_simt_error_word(unsigned** word);
cudaError_t mass_tc_error_word(unsigned** word);
cudaError_t launch_gather_errors(const ErrorWords& words, cudaStream_t st);
// Read and clear (after the stream was synchronised).
unsigned copy_errors_read_clear();
unsigned attn_simt_errors_read_clear();
unsigned attn_tc_errors_read_clear();
unsigned combine_vup_errors_read_clear();
cudaError_t launch_wait_check(uint32_t limit_us, cudaStream_t st);

}  // namespace mla
