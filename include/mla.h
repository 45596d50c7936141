/*
 * mla.h - C ABI of the weight-absorbed Multi-head Latent Attention (MLA) hot
 * path over a paged latent KV cache, for NVIDIA GB300 (sm_103a).
 *
 * One decode step is five calls, all asynchronous on the caller's stream:
 *
 *   mla_absorb_q    q_lat[h,b,:] = q_nope[h,b,:] @ W_UK[h]        (step 1)
 *   mla_concat_q    q_cat[t,h,:] = [q_lat[t,h,:] | q_pe[t,h,:]]    (step 2)
 *   mla_cache_write cache[slot]  = [kv_c | k_pe]                   (step 3)
 *   mla_decode      o_lat = softmax(scale * q_cat . cache) c_kv    (step 4)
 *   mla_v_up        out[h,b,:]   = o_lat[h,b,:] @ W_UV[h]          (step 5)
 *
 * and mla_prefill is step 4 for many causal queries per sequence. Fused forms:
 * mla_concat_q_cache_write (steps 2 and 3 in one launch), mla_absorb_concat_cache_write
 * (steps 1 to 3 in one call, the copies alongside the absorb) and mla_decode_v_up (step 4
 * with step 5 in its combine). mla_decode_window and mla_prefill_window are step 4 limited to
 * a sliding window and attention sinks; mla_cache_write_ds_mla is step 3 into quantised
 * entries, and mla_cache_read, _fp8 and _ds_mla read cache rows back. mla_norm_rope_q and the
 * mla_norm_rope_cache_write calls make the queries and rows of steps 1 to 3 from a layer's
 * projections; mla_decode_mass and mla_prefill_mass weigh the cached rows by the attention they
 * receive, and mla_cache_evict keeps the heaviest.
 *
 * Sources of the operations (web pages):
 *   [vt]    vllm.cpp, tests/vt/test_ops_mla_absorb.cpp (BatchedMatmul and
 *           ConcatMlaNopeRope test cases; strided views Contig/View3).
 *   [memra] memra-engine 0.124.1, tests/mla_gpu_forward.rs (absorbed and naive
 *           oracles; cache rows [c_kv | k_pe]; causal prefill and stepwise decode).
 *   [vllm]  vLLM, tests/kernels/attention/test_mla_cross_layer_kernel_equivalence.py
 *           (concat_and_cache_mla into a unified-slot layer view; paged dense
 *           decode with a block table and cache_seqlens).
 *
 * Conventions shared by every call
 *   - Ownership: the caller allocates and owns every buffer. Unless a call says
 *     otherwise the library allocates no device memory; it keeps a host-side
 *     cache of TMA tensor maps and a few bytes of static device state (an
 *     error word per kernel module).
 *   - Pointers: every data pointer is a DEVICE pointer of the current CUDA
 *     device. `stream` is a cudaStream_t (NULL = the legacy default stream).
 *   - Execution: asynchronous; no call synchronises the stream or the device.
 *   - Views: an mla_tensor is {data, rank, shape, stride}; strides count
 *     ELEMENTS and `data` already includes any storage offset ([vt] View3).
 *     The innermost stride must be 1 on every tensor ([vt] "rejects malformed
 *     shapes/strides rather than mis-computing").
 *   - Validation: shapes, strides, dtypes, null pointers and alignment are
 *     checked on the host before any launch. A failed check returns
 *     MLA_ERR_INVALID_ARG (malformed) or MLA_ERR_UNSUPPORTED (well formed but
 *     outside what the kernels handle) and launches nothing.
 *   - Device-resident values (slots, block ids, sequence lengths) cannot be
 *     checked on the host. The kernels check them: an access that would leave
 *     the cache view is skipped and recorded; mla_device_error() reports it.
 *   - Empty work (zero tokens, zero sequences) returns MLA_OK and launches
 *     nothing ([memra]: "never a zero-extent launch").
 *   - Errors: mla_last_error() returns a message for the calling thread's
 *     last failed call. Launch failures return MLA_ERR_CUDA.
 */
#ifndef MLA_H_
#define MLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_ABI_VERSION 1

typedef enum {
  MLA_OK = 0,
  MLA_ERR_INVALID_ARG = 1,  /* malformed shape, stride, dtype or pointer   */
  MLA_ERR_UNSUPPORTED = 2,  /* well formed, but not handled by the kernels  */
  MLA_ERR_CUDA = 3,         /* a CUDA runtime or driver call failed         */
  MLA_ERR_TIMEOUT = 4,      /* a bounded device-side wait gave up           */
  MLA_ERR_DEVICE_DATA = 5   /* a device-resident index was out of range     */
} mla_status;

typedef enum {
  MLA_F32 = 0,   /* IEEE binary32 */
  MLA_BF16 = 1   /* bfloat16; results rounded to nearest even */
} mla_dtype;

/* A strided view: element (i0,..,i_{rank-1}) lives at
 * data + sum_k i_k * stride[k] elements. rank <= 4; unused entries ignored. */
typedef struct {
  void* data;
  int32_t rank;
  int64_t shape[4];
  int64_t stride[4];
} mla_tensor;

/* ABI version of the loaded library (MLA_ABI_VERSION at build time). */
int mla_abi_version(void);

/* Message for the calling thread's last failed call ("" if none). The string
 * stays valid until the thread's next call into the library. */
const char* mla_last_error(void);

/* Static name of a status code. */
const char* mla_status_string(mla_status status);

/* Step 1 - W_UK absorption ([vt] BatchedMatmul, q-side fold: a (B,N,P) -> (N,B,P)
 * transposed view times W_UK_T [N,P,L]; [memra] mla_absorb_q).
 *   q_lat_out [H,B,L] (written), q_nope [H,B,P], w_uk [H,P,L]; any strides with
 *   innermost 1 (q_nope is usually the transpose of a [B,H,P] buffer and
 *   q_lat_out the transpose of a [B,H,L] buffer).
 *   q_lat[h,b,l] = sum_p q_nope[h,b,p] * w_uk[h,p,l], accumulated in fp32 and
 *   stored in `dtype`. All three tensors have `dtype`. */
mla_status mla_absorb_q(mla_dtype dtype, mla_tensor q_lat_out, mla_tensor q_nope,
                        mla_tensor w_uk, void* stream);

/* Step 2 - q concat ([vt] ConcatMlaNopeRope: a pure copy, bit for bit, that must
 * follow the strides of a transposed nope operand; a rope operand with one head
 * is broadcast to every head, as for _concat_k_nope_k_pe).
 *   q_cat_out [T,H,L+R] (written), nope [T,H,L], rope [T,H,R] or [T,1,R]
 *   (a rope stride(1) of 0 also broadcasts). Bits are copied unchanged,
 *   including NaN payloads and signed zeros. R may be 0.
 *   nope may be q_cat_out's own first L columns (the same data pointer and
 *   strides: mla_absorb_q can write q_lat straight into q_cat_out); then only
 *   the rope columns are copied. Any other overlap of q_cat_out with an input
 *   is undefined. */
mla_status mla_concat_q(mla_dtype dtype, mla_tensor q_cat_out, mla_tensor nope,
                        mla_tensor rope, void* stream);

/* Step 3 - paged latent cache write ([vllm] concat_and_cache_mla with kv_cache_dtype
 * "auto"; [memra] mla_append_latent).
 *   cache [num_blocks, page, L+R] view (written): any stride(0) and storage
 *   offset, e.g. one layer of a block-major unified slot; kv_c [T,L], k_pe [T,R];
 *   slot_mapping: device int64 [num_tokens].
 *   For token i with s = slot_mapping[i] >= 0:
 *     cache[s / page, s % page, 0:L]   = kv_c[i]
 *     cache[s / page, s % page, L:L+R] = k_pe[i]
 *   bit for bit. Negative slots are padding and write nothing. Slots at or beyond
 *   num_blocks*page write nothing and set MLA_ERR_DEVICE_DATA in mla_device_error.
 *   No element outside the addressed rows is written. Duplicate slots: the
 *   surviving row is unspecified. */
mla_status mla_cache_write(mla_dtype dtype, mla_tensor cache, mla_tensor kv_c, mla_tensor k_pe,
                           const int64_t* slot_mapping, int64_t num_tokens, void* stream);

/* Step 4 - paged split-KV decode ([vllm] flash_mla_with_kvcache / FlashInfer MLA
 * decode over a strided cache view; [memra] mla_attn_absorbed with t_q = 1).
 *   o_lat_out [B,H,L] (written; `dtype`), lse_out: device float [B,H] contiguous
 *   or NULL; q_cat [B,H,L+R]; cache as in mla_cache_write;
 *   block_table: device int32 [B, max_blocks] with row stride block_table_stride;
 *   seq_lens: device int32 [B].
 *   For every sequence b and head h, over rows t < seq_lens[b] of the cache
 *   (row t at block block_table[b, t / page], offset t % page):
 *     s_t = softmax_scale * (q_cat[b,h,0:L] . c_kv_t + q_cat[b,h,L:] . k_pe_t)
 *     o_lat[b,h,:] = sum_t softmax(s)_t * c_kv_t,  lse[b,h] = ln sum_t e^{s_t}
 *   with fp32 softmax and accumulation. seq_lens[b] == 0 gives o = 0 and
 *   lse = -inf. The context is cut into chunks processed in parallel and merged
 *   by their LSE; num_splits > 0 sets the number of chunks processed in
 *   parallel over the whole batch (0 = chosen from the SM count). For fixed
 *   (seq_lens, num_splits, device) the result is bit-identical from run to run
 *   and does not depend on the cache strides.
 *   workspace: device scratch of at least mla_decode_workspace_size(...) bytes,
 *   256-byte aligned, owned by the caller, not used by concurrent calls. */
mla_status mla_decode(mla_dtype dtype, mla_tensor o_lat_out, float* lse_out, mla_tensor q_cat,
                      mla_tensor cache, const int32_t* block_table, int64_t block_table_stride,
                      int32_t max_blocks, const int32_t* seq_lens, int32_t kv_lora_rank,
                      int32_t rope_dim, float softmax_scale, int32_t num_splits,
                      void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace mla_decode needs for `batch` sequences of `num_heads` heads
 * with latent width `kv_lora_rank` and the given num_splits (0 = automatic) on
 * the current device. */
size_t mla_decode_workspace_size(int32_t batch, int32_t num_heads, int32_t kv_lora_rank,
                                 int32_t num_splits);

/* Steps 2 and 3 in one launch - the q concat and the cache write of the same
 * decode step (the fused pre-attention of the vllm.cpp and memra pages' step
 * order: the new rows' [c_kv | k_pe] go into the cache while the query's rope
 * columns join q_cat).
 *   Arguments: those of mla_concat_q followed by those of mla_cache_write (one
 *   dtype for all tensors). Results, errors and the in-place nope case are
 *   exactly theirs; when either part cannot move 16-byte words the two run as
 *   two launches. */
mla_status mla_concat_q_cache_write(mla_dtype dtype, mla_tensor q_cat_out, mla_tensor nope,
                                    mla_tensor rope, mla_tensor cache, mla_tensor kv_c,
                                    mla_tensor k_pe, const int64_t* slot_mapping,
                                    int64_t num_tokens, void* stream);

/* Steps 1, 2 and 3 of a decode step in one call - the absorb straight into q_cat, the
 * rope columns of q_cat and the cache write of the new rows (the fused pre-attention of the
 * vllm.cpp and memra pages' step order, absorb -> q_cat included).
 *   q_cat [T,H,L+R] (written), q_nope [H,T,P] (any strides with innermost 1: usually the
 *   transpose of a [T,H,P] buffer), w_uk [H,P,L], q_pe [T,H,R] or [T,1,R]; cache, kv_c,
 *   k_pe, slot_mapping and num_tokens as for mla_cache_write. One dtype for all tensors.
 *   Results are exactly those of mla_absorb_q(q_cat's first L columns seen as [H,T,L],
 *   q_nope, w_uk) followed by mla_concat_q_cache_write(q_cat, q_cat's own first L columns,
 *   q_pe, cache, kv_c, k_pe, slot_mapping, num_tokens), and so are the errors (a w_uk wider
 *   than q_cat, or shapes that do not match, return MLA_ERR_INVALID_ARG). The copies touch
 *   only q_cat's rope columns and the cache, none of the absorb's operands or output, so on
 *   the GPU they run alongside the absorb instead of after it; the call's work is complete,
 *   as a whole, before anything queued after it on the stream starts reading it. q_cat,
 *   q_nope, w_uk, q_pe, the cache, kv_c and k_pe must not overlap one another. */
mla_status mla_absorb_concat_cache_write(mla_dtype dtype, mla_tensor q_cat, mla_tensor q_nope,
                                         mla_tensor w_uk, mla_tensor q_pe, mla_tensor cache,
                                         mla_tensor kv_c, mla_tensor k_pe,
                                         const int64_t* slot_mapping, int64_t num_tokens,
                                         void* stream);

/* Step 3, fp8 cache - the cache write into an e4m3 cache ([vllm] concat_and_cache_mla
 * with a quantized cache dtype and its scale).
 *   cache [num_blocks, page, L+R] view of e4m3 codes, one byte per element (strides
 *   count bytes), any stride(0) and storage offset; kv_c [T,L] and k_pe [T,R] in
 *   src_dtype (MLA_F32 or MLA_BF16); slot_mapping: device int64 [num_tokens];
 *   scale: device float [1], the cache scale.
 *   For token i with s = slot_mapping[i] >= 0 the row s becomes the e4m3 codes of
 *   float32(x) / scale (the division correctly rounded), rounded to nearest with
 *   ties to even; finite values beyond 448 saturate to +-448, NaN stays NaN.
 *   Padding slots, out-of-range slots and the untouched rows: as mla_cache_write. */
mla_status mla_cache_write_fp8(mla_dtype src_dtype, mla_tensor cache, mla_tensor kv_c,
                               mla_tensor k_pe, const int64_t* slot_mapping, int64_t num_tokens,
                               const float* scale, void* stream);

/* Step 4, fp8 cache - paged split-KV decode over an e4m3 cache ([vllm]
 * flash_mla_with_kvcache_fp8 with descale_q and descale_k).
 *   Arguments as mla_decode, except: cache holds e4m3 codes (one byte per element,
 *   strides in bytes); every cache value is its code's value times *descale_k and
 *   the query is q_cat times *descale_q (device floats [1]; NULL reads as 1).
 *   o_lat_out and q_cat have `dtype`; the workspace is mla_decode's
 *   (mla_decode_workspace_size). Results: as mla_decode over the dequantised
 *   values. */
mla_status mla_decode_fp8(mla_dtype dtype, mla_tensor o_lat_out, float* lse_out, mla_tensor q_cat,
                          mla_tensor cache, const int32_t* block_table, int64_t block_table_stride,
                          int32_t max_blocks, const int32_t* seq_lens, int32_t kv_lora_rank,
                          int32_t rope_dim, float softmax_scale, const float* descale_q,
                          const float* descale_k, int32_t num_splits, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Bytes of one fp8 ds_mla cache entry: 512 e4m3 latent codes, four float32
 * scales (scale g covers latent columns 128g .. 128g+127), 64 bf16 rope values. */
#define MLA_DS_MLA_ENTRY_BYTES 656

/* Step 4, sparse fp8 - top-k decode over an fp8 ds_mla cache ([vllm]
 * flash_mla_with_kvcache with is_fp8_kvcache and indices, the DeepSeek sparse
 * attention path; the indexer that picks the slots is not part of this library).
 *   o_lat_out [B,H,512] (written), lse_out device float [B,H] or NULL,
 *   q_cat [B,H,576] (latent 512 | rope 64), both in `dtype`;
 *   cache [num_blocks, page, 656] byte view (strides in bytes, any stride(0) and
 *   storage offset: one layer of a unified-slot buffer), data and strides 16-byte
 *   aligned; indices: device int32 [B, topk] with row stride indices_stride
 *   (>= topk); slot = block * page + row; negative entries are padding.
 *   Query b attends the rows at its listed slots (each once per listing, in any
 *   order): key [c_kv | k_pe], value c_kv, c_kv[i] = e4m3 value * scale[i / 128]
 *   and k_pe the bf16 rope values; the softmax and outputs as mla_decode. A query
 *   with no valid slot gets o = 0, lse = -inf. A slot past the cache is skipped and
 *   reported by mla_device_error (MLA_ERR_DEVICE_DATA).
 *   num_splits: as mla_decode; workspace: device scratch of at least
 *   mla_decode_sparse_workspace_size(B, H, topk, num_splits) bytes, 256-byte
 *   aligned, caller-owned. */
/* Bytes of workspace mla_decode_sparse_fp8 needs. */
size_t mla_decode_sparse_workspace_size(int32_t batch, int32_t num_heads, int32_t topk, int32_t num_splits);

mla_status mla_decode_sparse_fp8(mla_dtype dtype, mla_tensor o_lat_out, float* lse_out, mla_tensor q_cat,
                                 mla_tensor cache, const int32_t* indices, int64_t indices_stride,
                                 int32_t topk, float softmax_scale, int32_t num_splits, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* Step 4, prefill - causal attention of many queries per sequence over the same
 * paged cache ([memra] gate 1: pure prefill t_q == t_kv and the chunked shape
 * where the queries are a suffix of an already populated cache).
 *   o_lat_out [T,H,L] (written), lse_out device float [T,H] or NULL,
 *   q_cat [T,H,L+R] with the queries of sequence b in rows
 *   cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1 (device int32 [batch+1]);
 *   seq_lens_kv: device int32 [batch], rows of sequence b already in the cache
 *   (including its own queries' rows).
 *   Query i of sequence b sits at position p = seq_lens_kv[b] - q_len_b + i and
 *   attends rows 0..p (bottom-right causal alignment); otherwise as mla_decode.
 *   max_q_len bounds q_len_b. workspace: device scratch of at least
 *   mla_prefill_workspace_size(batch) bytes, 256-byte aligned, caller-owned. */
mla_status mla_prefill(mla_dtype dtype, mla_tensor o_lat_out, float* lse_out, mla_tensor q_cat,
                       mla_tensor cache, const int32_t* block_table, int64_t block_table_stride,
                       int32_t max_blocks, const int32_t* cu_seqlens_q, const int32_t* seq_lens_kv,
                       int32_t batch, int32_t max_q_len, int32_t kv_lora_rank, int32_t rope_dim,
                       float softmax_scale, void* workspace, size_t workspace_bytes,
                       void* stream);

/* Bytes of workspace mla_prefill needs for `batch` sequences. */
size_t mla_prefill_workspace_size(int32_t batch);

/* Step 5 - W_UV un-projection ([vt] BatchedMatmul at the _v_up_proj call site: a
 * (B,N,L) -> (N,B,L) transposed input, output written into a transposed (B,N,V);
 * [memra] mla_decompress_v).
 *   out [H,B,V] (written), o_lat [H,B,L], w_uv [H,L,V].
 *   out[h,b,v] = sum_l o_lat[h,b,l] * w_uv[h,l,v], fp32 accumulation. */
mla_status mla_v_up(mla_dtype dtype, mla_tensor out, mla_tensor o_lat, mla_tensor w_uv,
                    void* stream);

/* Steps 4 and 5 as one call - split-KV paged decode whose output goes straight
 * through the W_UV un-projection ([vt] _v_up_proj at the end of the absorbed
 * decode; [memra] mla_attn_absorbed -> mla_decompress_v): the LSE combine of the
 * split sequences and the un-projection run as one kernel, so o_lat is never
 * written out.
 *   out [B,H,V] (written; any strides with unit v stride), lse_out device float
 *   [B,H] or NULL, q_cat, cache, block table, lengths, kv_lora_rank, rope_dim,
 *   softmax_scale, num_splits: as mla_decode; w_uv [H,L,V] as mla_v_up.
 *   out[b,h,:] = o_lat[b,h,:] @ w_uv[h] with o_lat the decode's output rounded to
 *   `dtype` (as mla_decode followed by mla_v_up computes it).
 *   workspace: device scratch of at least
 *   mla_decode_v_up_workspace_size(B, H, L, num_splits) bytes, 256-byte aligned,
 *   caller-owned (it also holds o_lat). Errors: as mla_decode and mla_v_up. */
mla_status mla_decode_v_up(mla_dtype dtype, mla_tensor out, float* lse_out, mla_tensor q_cat, mla_tensor cache,
                           const int32_t* block_table, int64_t block_table_stride, int32_t max_blocks,
                           const int32_t* seq_lens, int32_t kv_lora_rank, int32_t rope_dim, float softmax_scale,
                           mla_tensor w_uv, int32_t num_splits, void* workspace, size_t workspace_bytes,
                           void* stream);

/* Bytes of workspace mla_decode_v_up needs. */
size_t mla_decode_v_up_workspace_size(int32_t batch, int32_t num_heads, int32_t kv_lora_rank,
                                      int32_t num_splits);

/* Step 3, ds_mla cache - the cache write into the fp8 ds_mla entries that
 * mla_decode_sparse_fp8 reads ([vllm] concat_and_cache_mla into an fp8 ds_mla cache; the
 * page gives the entry's layout, the quantisation rule is this library's).
 *   cache [num_blocks, page, 656] byte view (strides in bytes, any stride(0) and storage
 *   offset), data and strides 16-byte aligned; kv_c [T,512] and k_pe [T,64] in src_dtype,
 *   any row stride; slot_mapping: device int64 [num_tokens].
 *   For token i with s = slot_mapping[i] >= 0, entry s becomes
 *     scale g    = max(max |kv_c[i, 128g .. 128g+127]| / 448, 2^-126)   (float32)
 *     code c     = e4m3(kv_c[i,c] / scale[c / 128])   (the quotient rounded once, to the
 *                  nearest code, ties to even, saturating)
 *     rope       = k_pe[i] (bf16, rounded to nearest even from float32).
 *   An infinity counts as the largest float32 in the maximum and becomes a code of +-448;
 *   a NaN does not count and becomes the NaN code. Padding slots, out-of-range slots and the
 *   untouched entries: as mla_cache_write. Duplicate slots: the entry's bytes are
 *   unspecified (codes of one token may stand beside a scale of another). */
mla_status mla_cache_write_ds_mla(mla_dtype src_dtype, mla_tensor cache, mla_tensor kv_c,
                                  mla_tensor k_pe, const int64_t* slot_mapping, int64_t num_tokens,
                                  void* stream);

/* Read-back - rows of a paged cache gathered into contiguous rows [c_kv | k_pe], the
 * inverse of the cache writes (what a chunk of prefill over a quantised or shared prefix
 * begins with: the rows read back are a cache for mla_prefill and mla_prefill_window). The
 * source pages have no counterpart of these calls.
 *   out [T,W] (written; any row stride), W values a row; cache as in the writes;
 *   block_table: device int32 [batch, max_blocks] with row stride block_table_stride;
 *   cu_seqlens: device int32 [batch+1], ascending; seq_starts: device int32 [batch] or NULL
 *   (all zero).
 *   Row i of out with cu_seqlens[b] <= i < cu_seqlens[b+1] becomes row
 *   seq_starts[b] + i - cu_seqlens[b] of sequence b (block block_table[b, row / page],
 *   offset row % page). Rows of out before cu_seqlens[0], at or behind cu_seqlens[batch]
 *   are left as they were. A row whose position or block id lies outside the table or the
 *   cache is left as it was and reported by mla_device_error (MLA_ERR_DEVICE_DATA). out must
 *   not overlap the cache.
 *   mla_cache_read: a cache of `dtype` [num_blocks, page, W], bits unchanged.
 *   mla_cache_read_fp8: e4m3 codes [num_blocks, page, W] (strides in bytes); a value is its
 *   code's value times *scale (device float [1]) in float32, rounded once to dst_dtype.
 *   mla_cache_read_ds_mla: W = 576; latent values are code * scale[column / 128] in float32,
 *   rounded once to dst_dtype, rope values the stored ones; cache as in
 *   mla_cache_write_ds_mla. */
mla_status mla_cache_read(mla_dtype dtype, mla_tensor out, mla_tensor cache,
                          const int32_t* block_table, int64_t block_table_stride,
                          int32_t max_blocks, const int32_t* cu_seqlens, const int32_t* seq_starts,
                          int32_t batch, void* stream);
mla_status mla_cache_read_fp8(mla_dtype dst_dtype, mla_tensor out, mla_tensor cache,
                              const int32_t* block_table, int64_t block_table_stride,
                              int32_t max_blocks, const int32_t* cu_seqlens,
                              const int32_t* seq_starts, int32_t batch, const float* scale,
                              void* stream);
mla_status mla_cache_read_ds_mla(mla_dtype dst_dtype, mla_tensor out, mla_tensor cache,
                                 const int32_t* block_table, int64_t block_table_stride,
                                 int32_t max_blocks, const int32_t* cu_seqlens,
                                 const int32_t* seq_starts, int32_t batch, void* stream);

/* Step 4, windowed - the decode limited to a sliding window and attention sinks. The source
 * pages have no counterpart of this call.
 *   Arguments, results and errors as mla_decode, except: the query of sequence b, at position
 *   p = seq_lens[b] - 1, attends the rows t <= p with t < sinks or t > p - window (window >= 1
 *   rows ending with its own, and the sequence's first `sinks` >= 0 rows). Rows outside are
 *   never used, whatever they hold, and the block ids of pages without an attended row are not
 *   read: such pages may have been freed. num_splits beyond 4096 counts as 4096.
 *   A query that attends a row whose block id lies outside the cache gets unspecified values,
 *   and mla_device_error reports it; other queries are not affected.
 *   The tensor cores take bf16 with kv_lora_rank 512, rope_dim 64 or 0, up to 128 heads, a
 *   positive softmax_scale, pages of 8, 16 or 32 rows or a multiple of 64, and q_cat, o_lat_out
 *   and cache with 16-byte aligned data and strides that are multiples of 8 elements. Any
 *   other call runs on the CUDA cores, to the same definition and, where there is much to
 *   compute, 20 to 150 times slower.
 *   workspace: at least mla_decode_window_workspace_size(...) bytes, 256-byte aligned,
 *   caller-owned, not used by concurrent calls. */
mla_status mla_decode_window(mla_dtype dtype, mla_tensor o_lat_out, float* lse_out,
                             mla_tensor q_cat, mla_tensor cache, const int32_t* block_table,
                             int64_t block_table_stride, int32_t max_blocks,
                             const int32_t* seq_lens, int32_t kv_lora_rank, int32_t rope_dim,
                             float softmax_scale, int32_t window, int32_t sinks,
                             int32_t num_splits, void* workspace, size_t workspace_bytes,
                             void* stream);
size_t mla_decode_window_workspace_size(int32_t batch, int32_t num_heads, int32_t kv_lora_rank,
                                        int32_t num_splits);

/* Step 4, prefill, windowed - causal attention of a chunk of tokens per sequence over the
 * paged cache, limited to a sliding window and attention sinks. The source pages have no
 * counterpart of this call.
 *   Arguments and results as mla_prefill (without max_q_len), except: a query at position p
 *   attends the rows t <= p with t < sinks or t > p - window. A query at a negative position
 *   (a chunk longer than its cache) attends nothing: o = 0, lse = -inf. Rows of q_cat outside
 *   every sequence (before cu_seqlens_q[0], at or behind cu_seqlens_q[batch]) leave their rows
 *   of o_lat_out and lse_out as they were; so do all rows where cu_seqlens_q decreases or
 *   leaves [0, tokens], which mla_device_error reports (MLA_ERR_DEVICE_DATA). Rows that no
 *   query of the chunk attends are never used, whatever they hold, and the block ids of pages
 *   without an attended row are not read; a row that some query of the chunk attends must hold
 *   finite values. Block ids outside the cache, and what the tensor cores take: as
 *   mla_decode_window.
 *   workspace: at least mla_prefill_window_workspace_size(tokens, ...) bytes (tokens = rows of
 *   q_cat), 256-byte aligned, caller-owned, not used by concurrent calls. */
mla_status mla_prefill_window(mla_dtype dtype, mla_tensor o_lat_out, float* lse_out,
                              mla_tensor q_cat, mla_tensor cache, const int32_t* block_table,
                              int64_t block_table_stride, int32_t max_blocks,
                              const int32_t* cu_seqlens_q, const int32_t* seq_lens_kv,
                              int32_t batch, int32_t kv_lora_rank, int32_t rope_dim,
                              float softmax_scale, int32_t window, int32_t sinks,
                              void* workspace, size_t workspace_bytes, void* stream);
size_t mla_prefill_window_workspace_size(int32_t tokens, int32_t batch, int32_t num_heads,
                                         int32_t kv_lora_rank);

/* Before step 1 - norms and the position rotation of what a layer's projections give: queries
 * as steps 1 and 2 take them, and rows [c_kv | k_pe] as step 3 writes them. The source pages
 * name the rotation but give no formula, and have no counterpart of these calls.
 *   Queries: q [T,H,P+R]; weight [H,P+R] or [1,P+R] (broadcast to every head), or rank 0 for no
 *   norm. With x a head of q, y = x * weight / sqrt(mean(x^2) + eps), the mean over all P+R
 *   columns (no norm: y = x);
 *     q_nope_out [T,H,P] = y[0:P],  q_pe_out [T,H,R] = rot(y[P:P+R])   (both written)
 *   q_pe_out is usually the last R columns of q_cat. Either output may be q's own columns (the
 *   same data pointer and strides); without a norm such a q_nope_out is not touched. Any other
 *   overlap is undefined.
 *   Rows: kv [T,L+R], weight [L]; with c = kv[t,0:L], the row of token t is
 *     [c * weight / sqrt(mean(c^2) + eps) | rot(kv[t,L:L+R])].
 *   rot turns pairs (a, b) of the R columns into (a cos - b sin, b cos + a sin): pair i is columns
 *   2i and 2i+1 where `interleaved` is not 0, else columns i and i + R/2. Its cosine is
 *   cos_sin[p, i], its sine cos_sin[p, R/2 + i], p = positions[t]: cos_sin is a device float32
 *   table [num_positions, R] with row stride cos_sin_stride, positions device int64 [T]. R is even;
 *   with R = 0 both may be NULL.
 *   Sums (of squares among them), norms and rotations are float32; a value is rounded once, as it
 *   is stored. A sum of squares beyond float32 is infinite: its finite columns become 0, infinite
 *   ones NaN. A token whose position lies outside the table leaves its outputs and its row as
 *   they were and is reported by mla_device_error (MLA_ERR_DEVICE_DATA). Slots, padding and
 *   out-of-range slots: as mla_cache_write; a padding token's queries are computed all the same.
 *   Weights have q's and kv's type. Any widths, strides and alignment are taken. The fast kernels
 *   move 16-byte words: of data and strides aligned to them, R and P or L in whole words (R / 2
 *   too), heads of up to 128 words (1024 bf16 or 512 float32 columns), ropes of up to 32, rows of up
 *   to 768 bf16 or 640 float32 columns. Other calls run value by value: 20000 heads of 1536 bf16
 *   columns take 45 us, 2.5 times what their bytes need. */
mla_status mla_norm_rope_q(mla_dtype dtype, mla_tensor q_nope_out, mla_tensor q_pe_out, mla_tensor q,
                           mla_tensor weight, float eps, const int64_t* positions,
                           const float* cos_sin, int64_t cos_sin_stride, int64_t num_positions,
                           int32_t interleaved, void* stream);
/* The rows, into a cache of `dtype` [num_blocks, page, L+R]. */
mla_status mla_norm_rope_cache_write(mla_dtype dtype, mla_tensor cache, mla_tensor kv,
                                     mla_tensor weight, float eps, const int64_t* positions,
                                     const float* cos_sin, int64_t cos_sin_stride,
                                     int64_t num_positions, int32_t interleaved,
                                     const int64_t* slot_mapping, int64_t num_tokens, void* stream);
/* The rows, into an e4m3 cache: the float32 row becomes codes as in mla_cache_write_fp8. */
mla_status mla_norm_rope_cache_write_fp8(mla_dtype src_dtype, mla_tensor cache, mla_tensor kv,
                                         mla_tensor weight, float eps, const int64_t* positions,
                                         const float* cos_sin, int64_t cos_sin_stride,
                                         int64_t num_positions, int32_t interleaved,
                                         const int64_t* slot_mapping, int64_t num_tokens,
                                         const float* scale, void* stream);
/* The rows (L 512, R 64), into ds_mla entries: the float32 row becomes an entry as in
 * mla_cache_write_ds_mla. */
mla_status mla_norm_rope_cache_write_ds_mla(mla_dtype src_dtype, mla_tensor cache, mla_tensor kv,
                                            mla_tensor weight, float eps, const int64_t* positions,
                                            const float* cos_sin, int64_t cos_sin_stride,
                                            int64_t num_positions, int32_t interleaved,
                                            const int64_t* slot_mapping, int64_t num_tokens,
                                            void* stream);
/* mla_norm_rope_q and mla_norm_rope_cache_write in one launch. */
mla_status mla_norm_rope_q_cache_write(mla_dtype dtype, mla_tensor q_nope_out, mla_tensor q_pe_out,
                                       mla_tensor q, mla_tensor q_weight, mla_tensor cache,
                                       mla_tensor kv, mla_tensor kv_weight, float eps,
                                       const int64_t* positions, const float* cos_sin,
                                       int64_t cos_sin_stride, int64_t num_positions,
                                       int32_t interleaved, const int64_t* slot_mapping,
                                       int64_t num_tokens, void* stream);

/* After step 4 - what the queries give each cached row: its attention weight, summed over the
 * queries that attend it and their heads, added to the row's mass (which mla_cache_evict goes by).
 * The source pages have no counterpart of these calls.
 *   mass: device float [batch, mass_rows], row stride mass_stride; q_cat [T,H,E], cache
 *   [num_blocks, page, E], block table and lengths as in mla_decode and mla_prefill (E = L + R);
 *   lse: device float [T,H] contiguous, what that decode or prefill gave for these queries;
 *   softmax_scale the same as there.
 *   For every row t < seq_lens[b] of a sequence with a query in the call
 *     mass[b,t] = decay * mass[b,t] + sum over queries i that attend t, and heads h, of
 *                 e^(softmax_scale * q_cat[i,h] . cache row t - lse[i,h])
 *   (decay 1 sums up; decay 0 never reads what was there). A decode's query attends every row, a
 *   prefill's the rows up to its own position, as in mla_prefill. Sums are float32 and their order
 *   does not change from run to run on a device. (The tensor cores' partial sums lose what lies below
 *   their last place, toward zero: masses of 576-wide random rows come out 0.7e-6 of themselves too
 *   small, of rows and queries whose products all have one sign, with logits of 8, 3.5e-6. The CUDA
 *   cores round to the nearest.) A query whose lse is -inf (it attended
 *   nothing) gives nothing, whatever it holds. Masses behind a sequence's rows, and those of sequences without a query
 *   or without rows, are left as they were; so are masses of rows whose block id lies outside the
 *   cache, and of sequences whose cu_seqlens_q decrease or leave [0, T], which mla_device_error
 *   reports (MLA_ERR_DEVICE_DATA), as it does a length beyond the table or mass_rows (which counts
 *   as the largest that they hold). Rows outside the sequences are never used, whatever they hold.
 *   The tensor cores take bf16 with E a multiple of 64 up to 576, up to 128 heads, pages of 8, 16 or
 *   32 rows or a multiple of 64, and q_cat and cache with 16-byte aligned data and strides that are
 *   multiples of 8 elements; any other call runs on the CUDA cores.
 *   The lse of a windowed call does not fit: it leaves out rows that are weighed here. Quantised
 *   caches are not taken: read their rows back (mla_cache_read_fp8, mla_cache_read_ds_mla).
 *   workspace (prefill): at least mla_prefill_mass_workspace_size() bytes, 256-byte aligned,
 *   caller-owned, not used by concurrent calls. */
mla_status mla_decode_mass(mla_dtype dtype, float* mass, int64_t mass_stride, int32_t mass_rows,
                           mla_tensor q_cat, mla_tensor cache, const int32_t* block_table,
                           int64_t block_table_stride, int32_t max_blocks, const int32_t* seq_lens,
                           const float* lse, float softmax_scale, float decay, void* stream);
mla_status mla_prefill_mass(mla_dtype dtype, float* mass, int64_t mass_stride, int32_t mass_rows,
                            mla_tensor q_cat, mla_tensor cache, const int32_t* block_table,
                            int64_t block_table_stride, int32_t max_blocks,
                            const int32_t* cu_seqlens_q, const int32_t* seq_lens_kv, int32_t batch,
                            const float* lse, float softmax_scale, float decay, void* workspace,
                            size_t workspace_bytes, void* stream);
size_t mla_prefill_mass_workspace_size(void);

/* Eviction - each sequence of a paged cache cut to its `budget` heaviest rows, which move
 * together in their order. The source pages have no counterpart of this call.
 *   cache [num_blocks, page, W] view of elements of element_bytes (1, 2 or 4) bytes: a plain, an
 *   e4m3 or a ds_mla cache; rows move bit for bit. block_table: device int32 [batch, max_blocks],
 *   row stride block_table_stride; seq_lens: device int32 [batch].
 *   mass: device float [batch, mass_rows], row stride mass_stride (mla_decode_mass and
 *   mla_prefill_mass add to it): mass[b, t] is row t's weight in sequence b.
 *   With n = seq_lens[b] <= budget every row stays. Else the rows t < sinks, the rows
 *   t >= n - recent (sinks + recent <= budget) and, of the others, the heaviest up to `budget` rows in
 *   all stay; of equal masses the lowest row stays first, -0 equals 0, a NaN is the heaviest. The
 *   rows that stay, in ascending order t_0 < t_1 < .., become rows 0, 1, ..:
 *     row j of sequence b (block block_table_out[b, j / page], offset j % page) = row t_j
 *     mass_out[b, j] = mass[b, t_j];  mass_out[b, j] = 0 for the j < n behind them
 *     seq_lens_out[b] = their count;  kept_out[b, j] = t_j, and -1 behind them (device int32
 *     [batch, budget], or NULL)
 *   What lies in the cache behind the rows that stay is left as it was, and so is mass_out from
 *   row n on. A mass_out of fewer rows (mass_out_rows) gets the first of these masses; those of the
 *   rows behind it are dropped. Rows keep the position they were rotated for: a row's place in the cache no longer
 *   is its position.
 *   block_table_out NULL: the rows move within their pages. Else each of its blocks is the one that
 *   block_table names in the same place, or one that no row of the call lies in; a page that two
 *   sequences share must not be written (give others). mass_out NULL (or mass, with its strides): in
 *   place; else the two do not overlap. seq_lens_out may be seq_lens.
 *   A row whose block id, old or new, lies outside the cache or the table is not moved and is
 *   reported by mla_device_error (MLA_ERR_DEVICE_DATA); the ids of pages from which and to which no
 *   row moves need not name a block of the cache. A length beyond the table or mass_rows is
 *   reported and counts as the largest that they hold.
 *   workspace: device scratch of at least mla_cache_evict_workspace_size(batch, mass_rows, budget)
 *   bytes, 256-byte aligned, caller-owned, not used by concurrent calls. */
mla_status mla_cache_evict(int32_t element_bytes, mla_tensor cache, float* mass, int64_t mass_stride,
                           int32_t mass_rows, const int32_t* block_table,
                           int64_t block_table_stride, int32_t max_blocks, const int32_t* seq_lens,
                           int32_t batch, int32_t budget, int32_t sinks, int32_t recent,
                           const int32_t* block_table_out, int64_t block_table_out_stride,
                           int32_t max_blocks_out, float* mass_out, int64_t mass_out_stride,
                           int32_t mass_out_rows, int32_t* seq_lens_out, int32_t* kept_out,
                           void* workspace, size_t workspace_bytes, void* stream);
size_t mla_cache_evict_workspace_size(int32_t batch, int32_t rows, int32_t budget);

/* Bytes of the static scratch behind mla_decode_noalloc (40 MiB). */
#define MLA_DECODE_NOALLOC_SCRATCH_BYTES (40u * 1024u * 1024u)

/* mla_decode without a workspace, for callers that cannot allocate device
 * memory: code running inside another framework's memory pool, plugins whose
 * host forbids cudaMalloc on the hot path (it synchronises the device and can
 * fail under memory pressure), runtimes that reserve all device memory up
 * front. The source pages have no counterpart of this call.
 *   Arguments, results and errors are those of mla_decode minus the workspace.
 *   The split-KV scratch lives in a static device array of
 *   MLA_DECODE_NOALLOC_SCRATCH_BYTES that every GPU loading the library holds
 *   until the process exits; a batch whose scratch would not fit (about
 *   (B + work units) * H * L * 4 bytes) returns MLA_ERR_UNSUPPORTED. The call
 *   allocates nothing. Its first call on a device looks up the array's device
 *   address (once per device and context: again after a reset of the device);
 *   make that first call before any stream capture.
 *   All calls share the array: calls whose kernels overlap on the GPU race and
 *   must be serialised by the caller. */
mla_status mla_decode_noalloc(mla_dtype dtype, mla_tensor o_lat_out, float* lse_out,
                              mla_tensor q_cat, mla_tensor cache, const int32_t* block_table,
                              int64_t block_table_stride, int32_t max_blocks,
                              const int32_t* seq_lens, int32_t kv_lora_rank, int32_t rope_dim,
                              float softmax_scale, int32_t num_splits, void* stream);

/* Synchronises `stream`, then reports and clears the device-side error words the
 * kernels set (out-of-range slot, block id or length: MLA_ERR_DEVICE_DATA; a
 * bounded wait that gave up: MLA_ERR_TIMEOUT). MLA_OK if none was set. */
mla_status mla_device_error(void* stream);

/* Self-check of failure detection. Every wait in the library's kernels is
 * bounded in time: a wait that gives up records MLA_ERR_TIMEOUT for
 * mla_device_error and the kernel winds down, so a stuck pipeline never hangs
 * the GPU. This call launches one warp that runs that same bounded wait on an
 * mbarrier nothing ever arrives on, with a limit of limit_us microseconds
 * (1 .. 1000000) instead of the kernels' 2 s; afterwards mla_device_error on
 * the same stream reports MLA_ERR_TIMEOUT (and clears it) while the context
 * stays usable. Returns MLA_ERR_INVALID_ARG for a limit out of range. The
 * source pages have no counterpart of this call. */
mla_status mla_check_bounded_wait(uint32_t limit_us, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_H_ */
