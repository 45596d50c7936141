"""Python binding of libmla.so: weight-absorbed MLA over a paged latent KV cache.

The functions carry the C ABI's names (``include/mla.h``) and only marshal
arguments: a torch tensor becomes an ``mla_tensor`` view (its ``data_ptr()``,
which includes the storage offset, its shape and its element strides), the
stream defaults to torch's current CUDA stream, and a non-OK status raises
:class:`MlaError` with the library's message. Every step of the path runs in
the library's CUDA kernels; there is no other implementation to fall back on,
so a missing ``libmla.so`` raises on first use.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmla.so")

MLA_OK, MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED, MLA_ERR_CUDA, MLA_ERR_TIMEOUT, MLA_ERR_DEVICE_DATA = range(6)
MLA_F32, MLA_BF16 = 0, 1


class MlaError(RuntimeError):
    """A call into libmla.so returned a status other than MLA_OK."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{_status_name(status)}: {message}")
        self.status = status


class MlaTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("rank", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


# an MlaTensor's bytes by rank: packing them costs half of what filling the fields does
_PACKED = [struct.Struct(f"Qi4x{r}q{8 * (4 - r)}x{r}q{8 * (4 - r)}x") for r in range(5)]


_lib_handle: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded libmla.so (raises if it has not been built)."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m mla_latent_kv_11_gb300.build`")
        h = ctypes.CDLL(LIB_PATH)
        P, I32, I64, F32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        T = MlaTensor
        sigs = {
            "mla_abi_version": ([], ctypes.c_int),
            "mla_last_error": ([], ctypes.c_char_p),
            "mla_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "mla_absorb_q": ([ctypes.c_int, T, T, T, P], ctypes.c_int),
            "mla_concat_q": ([ctypes.c_int, T, T, T, P], ctypes.c_int),
            "mla_cache_write": ([ctypes.c_int, T, T, T, P, I64, P], ctypes.c_int),
            "mla_decode": ([ctypes.c_int, T, P, T, T, P, I64, I32, P, I32, I32, F32, I32, P, SZ, P],
                           ctypes.c_int),
            "mla_decode_workspace_size": ([I32, I32, I32, I32], SZ),
            "mla_prefill": ([ctypes.c_int, T, P, T, T, P, I64, I32, P, P, I32, I32, I32, I32, F32, P,
                             SZ, P], ctypes.c_int),
            "mla_prefill_workspace_size": ([I32], SZ),
            "mla_v_up": ([ctypes.c_int, T, T, T, P], ctypes.c_int),
            "mla_decode_noalloc": ([ctypes.c_int, T, P, T, T, P, I64, I32, P, I32, I32, F32, I32, P],
                                   ctypes.c_int),
            "mla_cache_write_fp8": ([ctypes.c_int, T, T, T, P, I64, P, P], ctypes.c_int),
            "mla_concat_q_cache_write": ([ctypes.c_int, T, T, T, T, T, T, P, I64, P], ctypes.c_int),
            "mla_absorb_concat_cache_write": ([ctypes.c_int, T, T, T, T, T, T, T, P, I64, P], ctypes.c_int),
            "mla_decode_fp8": ([ctypes.c_int, T, P, T, T, P, I64, I32, P, I32, I32, F32, P, P, I32, P, SZ, P],
                               ctypes.c_int),
            "mla_decode_sparse_fp8": ([ctypes.c_int, T, P, T, T, P, I64, I32, F32, I32, P, SZ, P], ctypes.c_int),
            "mla_decode_sparse_workspace_size": ([I32, I32, I32, I32], SZ),
            "mla_decode_v_up": ([ctypes.c_int, T, P, T, T, P, I64, I32, P, I32, I32, F32, T, I32, P, SZ, P],
                                ctypes.c_int),
            "mla_decode_v_up_workspace_size": ([I32, I32, I32, I32], SZ),
            "mla_cache_write_ds_mla": ([ctypes.c_int, T, T, T, P, I64, P], ctypes.c_int),
            "mla_cache_read": ([ctypes.c_int, T, T, P, I64, I32, P, P, I32, P], ctypes.c_int),
            "mla_cache_read_fp8": ([ctypes.c_int, T, T, P, I64, I32, P, P, I32, P, P], ctypes.c_int),
            "mla_cache_read_ds_mla": ([ctypes.c_int, T, T, P, I64, I32, P, P, I32, P], ctypes.c_int),
            "mla_decode_window": ([ctypes.c_int, T, P, T, T, P, I64, I32, P, I32, I32, F32, I32, I32, I32, P, SZ, P],
                                  ctypes.c_int),
            "mla_decode_window_workspace_size": ([I32, I32, I32, I32], SZ),
            "mla_prefill_window": ([ctypes.c_int, T, P, T, T, P, I64, I32, P, P, I32, I32, I32, F32, I32, I32, P, SZ,
                                    P], ctypes.c_int),
            "mla_prefill_window_workspace_size": ([I32, I32, I32, I32], SZ),
            "mla_device_error": ([P], ctypes.c_int),
            "mla_check_bounded_wait": ([ctypes.c_uint32, P], ctypes.c_int),
        }
        for name, (args, res) in sigs.items():
            fn = getattr(h, name)
            fn.argtypes = args
            fn.restype = res
        _lib_handle = h
    return _lib_handle


def _status_name(status: int) -> str:
    names = ["MLA_OK", "MLA_ERR_INVALID_ARG", "MLA_ERR_UNSUPPORTED", "MLA_ERR_CUDA",
             "MLA_ERR_TIMEOUT", "MLA_ERR_DEVICE_DATA"]
    return names[status] if 0 <= status < len(names) else f"status {status}"


def _check(status: int) -> None:
    if status != MLA_OK:
        raise MlaError(status, lib().mla_last_error().decode(errors="replace"))


def _dtype_code(*tensors) -> int:
    import torch
    dt = None
    for t in tensors:
        if t is None:
            continue
        if dt is None:
            dt = t.dtype
        elif t.dtype != dt:
            dts = {t.dtype for t in tensors if t is not None}
            raise MlaError(MLA_ERR_INVALID_ARG, f"tensors disagree on dtype: {sorted(map(str, dts))}")
    if dt == torch.float32:
        return MLA_F32
    if dt == torch.bfloat16:
        return MLA_BF16
    raise MlaError(MLA_ERR_INVALID_ARG, f"unsupported dtype {dt}")


def as_mla_tensor(t) -> MlaTensor:
    """Describe a torch tensor (any strides) as an mla_tensor view."""
    shape = t.shape
    rank = len(shape)
    if rank > 4:
        raise MlaError(MLA_ERR_INVALID_ARG, "rank > 4")
    return MlaTensor.from_buffer_copy(_PACKED[rank].pack(t.data_ptr() if t.numel() > 0 else 0, rank, *shape, *t.stride()))


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def mla_absorb_q(q_lat_out, q_nope, w_uk, stream=None) -> None:
    """Step 1: q_lat[h,b,:] = q_nope[h,b,:] @ w_uk[h] (views [H,B,L], [H,B,P], [H,P,L])."""
    _check(lib().mla_absorb_q(_dtype_code(q_lat_out, q_nope, w_uk), as_mla_tensor(q_lat_out),
                              as_mla_tensor(q_nope), as_mla_tensor(w_uk), _stream(stream)))


def mla_concat_q(q_cat_out, nope, rope, stream=None) -> None:
    """Step 2: q_cat[t,h,:] = [nope[t,h,:] | rope[t,h or 0,:]], a bit copy."""
    _check(lib().mla_concat_q(_dtype_code(q_cat_out, nope, rope), as_mla_tensor(q_cat_out),
                              as_mla_tensor(nope), as_mla_tensor(rope), _stream(stream)))


def mla_cache_write(cache, kv_c, k_pe, slot_mapping, stream=None) -> None:
    """Step 3: cache[s // page, s % page, :] = [kv_c[i] | k_pe[i]] for s = slot_mapping[i] >= 0."""
    import torch
    if slot_mapping.dtype != torch.int64:
        raise MlaError(MLA_ERR_INVALID_ARG, "slot_mapping must be int64")
    if slot_mapping.numel() and not slot_mapping.is_contiguous():
        raise MlaError(MLA_ERR_INVALID_ARG, "slot_mapping must be contiguous")
    _check(lib().mla_cache_write(_dtype_code(cache, kv_c, k_pe), as_mla_tensor(cache),
                                 as_mla_tensor(kv_c), as_mla_tensor(k_pe), _ptr(slot_mapping),
                                 slot_mapping.numel(), _stream(stream)))


def _fp8_cache(cache):
    """An e4m3 cache: torch.float8_e4m3fn or uint8 storage of the codes, whose strides count bytes either way."""
    import torch
    if cache.dtype == torch.uint8 or cache.dtype == getattr(torch, "float8_e4m3fn", None):
        return cache
    raise MlaError(MLA_ERR_INVALID_ARG, "an fp8 cache must be float8_e4m3fn or uint8 codes")


def _f32_scalar(t, name):
    import torch
    if t is None:
        return None
    if t.dtype != torch.float32 or t.numel() != 1 or not t.is_cuda:
        raise MlaError(MLA_ERR_INVALID_ARG, f"{name} must be a device float32 tensor of one element")
    return t.data_ptr()


def mla_cache_write_fp8(cache, kv_c, k_pe, slot_mapping, scale, stream=None) -> None:
    """Step 3 into an e4m3 cache: row s = e4m3([kv_c[i] | k_pe[i]] / scale) for s = slot_mapping[i] >= 0."""
    import torch
    if slot_mapping.dtype != torch.int64:
        raise MlaError(MLA_ERR_INVALID_ARG, "slot_mapping must be int64")
    if slot_mapping.numel() and not slot_mapping.is_contiguous():
        raise MlaError(MLA_ERR_INVALID_ARG, "slot_mapping must be contiguous")
    if kv_c.dtype != k_pe.dtype or kv_c.dtype not in (torch.float32, torch.bfloat16):
        raise MlaError(MLA_ERR_INVALID_ARG, "kv_c and k_pe must both be float32 or both bfloat16")
    src = MLA_F32 if kv_c.dtype == torch.float32 else MLA_BF16
    _check(lib().mla_cache_write_fp8(src, as_mla_tensor(_fp8_cache(cache)), as_mla_tensor(kv_c),
                                     as_mla_tensor(k_pe), _ptr(slot_mapping), slot_mapping.numel(),
                                     _f32_scalar(scale, "scale"), _stream(stream)))


def mla_concat_q_cache_write(q_cat_out, nope, rope, cache, kv_c, k_pe, slot_mapping, stream=None) -> None:
    """Steps 2 and 3 in one launch: mla_concat_q(q_cat_out, nope, rope) and
    mla_cache_write(cache, kv_c, k_pe, slot_mapping)."""
    import torch
    if slot_mapping.dtype != torch.int64:
        raise MlaError(MLA_ERR_INVALID_ARG, "slot_mapping must be int64")
    if slot_mapping.numel() and not slot_mapping.is_contiguous():
        raise MlaError(MLA_ERR_INVALID_ARG, "slot_mapping must be contiguous")
    _check(lib().mla_concat_q_cache_write(_dtype_code(q_cat_out, nope, rope, cache, kv_c, k_pe),
                                          as_mla_tensor(q_cat_out), as_mla_tensor(nope), as_mla_tensor(rope),
                                          as_mla_tensor(cache), as_mla_tensor(kv_c), as_mla_tensor(k_pe),
                                          _ptr(slot_mapping), slot_mapping.numel(), _stream(stream)))


def mla_absorb_concat_cache_write(q_cat, q_nope, w_uk, q_pe, cache, kv_c, k_pe, slot_mapping, stream=None) -> None:
    """Steps 1 to 3 in one call: mla_absorb_q into q_cat's first L columns (q_nope [H,T,P],
    w_uk [H,P,L]), then the rope columns of q_cat and the cache write of the new rows, the
    copies running alongside the absorb."""
    import torch
    if slot_mapping.dtype != torch.int64:
        raise MlaError(MLA_ERR_INVALID_ARG, "slot_mapping must be int64")
    if slot_mapping.numel() and not slot_mapping.is_contiguous():
        raise MlaError(MLA_ERR_INVALID_ARG, "slot_mapping must be contiguous")
    _check(lib().mla_absorb_concat_cache_write(_dtype_code(q_cat, q_nope, w_uk, q_pe, cache, kv_c, k_pe),
                                               as_mla_tensor(q_cat), as_mla_tensor(q_nope), as_mla_tensor(w_uk),
                                               as_mla_tensor(q_pe), as_mla_tensor(cache), as_mla_tensor(kv_c),
                                               as_mla_tensor(k_pe), _ptr(slot_mapping), slot_mapping.numel(),
                                               _stream(stream)))


def mla_decode_workspace_size(batch: int, num_heads: int, kv_lora_rank: int, num_splits: int = 0) -> int:
    return int(lib().mla_decode_workspace_size(batch, num_heads, kv_lora_rank, num_splits))


def _check_int32_table(block_table, seq_lens):
    import torch
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise MlaError(MLA_ERR_INVALID_ARG, "block_table and sequence lengths must be int32")
    if block_table.dim() != 2 or block_table.stride(1) != 1:
        raise MlaError(MLA_ERR_INVALID_ARG, "block_table must be [B, max_blocks] with unit column stride")
    if not seq_lens.is_contiguous():
        raise MlaError(MLA_ERR_INVALID_ARG, "sequence lengths must be contiguous")


def mla_decode(o_lat_out, q_cat, cache, block_table, seq_lens, kv_lora_rank: int, rope_dim: int,
               softmax_scale: float, lse_out=None, num_splits: int = 0, workspace=None,
               stream=None) -> None:
    """Step 4: split-KV paged decode; o_lat_out [B,H,L], optional lse_out float32 [B,H]."""
    import torch
    _check_int32_table(block_table, seq_lens)
    if lse_out is not None and (lse_out.dtype != torch.float32 or not lse_out.is_contiguous()):
        raise MlaError(MLA_ERR_INVALID_ARG, "lse_out must be contiguous float32")
    B, H = q_cat.shape[0], q_cat.shape[1]
    need = mla_decode_workspace_size(B, H, kv_lora_rank, num_splits)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q_cat.device)
    _check(lib().mla_decode(_dtype_code(o_lat_out, q_cat, cache), as_mla_tensor(o_lat_out),
                            _ptr(lse_out), as_mla_tensor(q_cat), as_mla_tensor(cache),
                            block_table.data_ptr(), block_table.stride(0), block_table.shape[1],
                            seq_lens.data_ptr(), kv_lora_rank, rope_dim, softmax_scale, num_splits,
                            workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                            _stream(stream)))


def mla_decode_fp8(o_lat_out, q_cat, cache, block_table, seq_lens, kv_lora_rank: int, rope_dim: int,
                   softmax_scale: float, descale_q=None, descale_k=None, lse_out=None, num_splits: int = 0,
                   workspace=None, stream=None) -> None:
    """Step 4 over an e4m3 cache: mla_decode with cache values = code * descale_k and q * descale_q."""
    import torch
    _check_int32_table(block_table, seq_lens)
    if lse_out is not None and (lse_out.dtype != torch.float32 or not lse_out.is_contiguous()):
        raise MlaError(MLA_ERR_INVALID_ARG, "lse_out must be contiguous float32")
    if o_lat_out.dtype != q_cat.dtype:
        raise MlaError(MLA_ERR_INVALID_ARG, "o_lat_out and q_cat must share a dtype")
    code = MLA_F32 if q_cat.dtype == torch.float32 else MLA_BF16
    B, H = q_cat.shape[0], q_cat.shape[1]
    need = mla_decode_workspace_size(B, H, kv_lora_rank, num_splits)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q_cat.device)
    _check(lib().mla_decode_fp8(code, as_mla_tensor(o_lat_out), _ptr(lse_out), as_mla_tensor(q_cat),
                                as_mla_tensor(_fp8_cache(cache)), block_table.data_ptr(), block_table.stride(0),
                                block_table.shape[1], seq_lens.data_ptr(), kv_lora_rank, rope_dim, softmax_scale,
                                _f32_scalar(descale_q, "descale_q"), _f32_scalar(descale_k, "descale_k"),
                                num_splits, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                _stream(stream)))


def mla_decode_sparse_workspace_size(batch: int, num_heads: int, topk: int, num_splits: int = 0) -> int:
    return int(lib().mla_decode_sparse_workspace_size(batch, num_heads, topk, num_splits))


def mla_decode_sparse_fp8(o_lat_out, q_cat, cache, indices, softmax_scale: float, lse_out=None,
                          num_splits: int = 0, workspace=None, stream=None) -> None:
    """Sparse top-k decode over an fp8 ds_mla cache: query b attends the slots indices[b]
    (int32 [B, topk] or [B, 1, topk], -1 = padding) of a uint8 [num_blocks, page, 656]
    (or [num_blocks, page, 1, 656]) cache; o_lat_out [B,H,512], q_cat [B,H,576]."""
    import torch
    if cache.dtype != torch.uint8:
        raise MlaError(MLA_ERR_INVALID_ARG, "a ds_mla cache is uint8 bytes")
    if cache.dim() == 4 and cache.shape[2] == 1:
        cache = cache[:, :, 0]
    if indices.dim() == 3 and indices.shape[1] == 1:
        indices = indices[:, 0]
    if indices.dtype != torch.int32 or indices.dim() != 2 or (indices.numel() and indices.stride(1) != 1):
        raise MlaError(MLA_ERR_INVALID_ARG, "indices must be int32 [B, topk] with unit column stride")
    if lse_out is not None and (lse_out.dtype != torch.float32 or not lse_out.is_contiguous()):
        raise MlaError(MLA_ERR_INVALID_ARG, "lse_out must be contiguous float32")
    B, H = q_cat.shape[0], q_cat.shape[1]
    if workspace is None:
        workspace = torch.empty(mla_decode_sparse_workspace_size(B, H, indices.shape[-1], num_splits),
                                dtype=torch.uint8, device=q_cat.device)
    _check(lib().mla_decode_sparse_fp8(_dtype_code(o_lat_out, q_cat), as_mla_tensor(o_lat_out), _ptr(lse_out),
                                       as_mla_tensor(q_cat), as_mla_tensor(cache), _ptr(indices),
                                       indices.stride(0) if indices.dim() == 2 else 0, indices.shape[-1],
                                       softmax_scale, num_splits, workspace.data_ptr(),
                                       workspace.numel() * workspace.element_size(), _stream(stream)))


def mla_decode_v_up_workspace_size(batch: int, num_heads: int, kv_lora_rank: int, num_splits: int = 0) -> int:
    return int(lib().mla_decode_v_up_workspace_size(batch, num_heads, kv_lora_rank, num_splits))


def mla_decode_v_up(out, q_cat, cache, block_table, seq_lens, kv_lora_rank: int, rope_dim: int,
                    softmax_scale: float, w_uv, lse_out=None, num_splits: int = 0, workspace=None,
                    stream=None) -> None:
    """Steps 4 and 5 as one call: out[b,h,:] = decode(q_cat)[b,h,:] @ w_uv[h]; out [B,H,V], w_uv [H,L,V]."""
    import torch
    _check_int32_table(block_table, seq_lens)
    if lse_out is not None and (lse_out.dtype != torch.float32 or not lse_out.is_contiguous()):
        raise MlaError(MLA_ERR_INVALID_ARG, "lse_out must be contiguous float32")
    B, H = q_cat.shape[0], q_cat.shape[1]
    if workspace is None:
        workspace = torch.empty(mla_decode_v_up_workspace_size(B, H, kv_lora_rank, num_splits), dtype=torch.uint8,
                                device=q_cat.device)
    _check(lib().mla_decode_v_up(_dtype_code(out, q_cat, cache, w_uv), as_mla_tensor(out), _ptr(lse_out),
                                 as_mla_tensor(q_cat), as_mla_tensor(cache), block_table.data_ptr(),
                                 block_table.stride(0), block_table.shape[1], seq_lens.data_ptr(), kv_lora_rank,
                                 rope_dim, softmax_scale, as_mla_tensor(w_uv), num_splits, workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), _stream(stream)))


def mla_prefill_workspace_size(batch: int) -> int:
    return int(lib().mla_prefill_workspace_size(batch))


def mla_prefill(o_lat_out, q_cat, cache, block_table, cu_seqlens_q, seq_lens_kv, max_q_len: int,
                kv_lora_rank: int, rope_dim: int, softmax_scale: float, lse_out=None, workspace=None,
                stream=None) -> None:
    """Step 4 (prefill): causal attention of many queries per sequence over the paged cache."""
    import torch
    _check_int32_table(block_table, seq_lens_kv)
    if cu_seqlens_q.dtype != torch.int32 or not cu_seqlens_q.is_contiguous():
        raise MlaError(MLA_ERR_INVALID_ARG, "cu_seqlens_q must be contiguous int32")
    if lse_out is not None and (lse_out.dtype != torch.float32 or not lse_out.is_contiguous()):
        raise MlaError(MLA_ERR_INVALID_ARG, "lse_out must be contiguous float32")
    if workspace is None:
        workspace = torch.empty(mla_prefill_workspace_size(seq_lens_kv.numel()), dtype=torch.uint8,
                                device=q_cat.device)
    _check(lib().mla_prefill(_dtype_code(o_lat_out, q_cat, cache), as_mla_tensor(o_lat_out),
                             _ptr(lse_out), as_mla_tensor(q_cat), as_mla_tensor(cache),
                             block_table.data_ptr(), block_table.stride(0), block_table.shape[1],
                             cu_seqlens_q.data_ptr(), seq_lens_kv.data_ptr(), seq_lens_kv.numel(),
                             max_q_len, kv_lora_rank, rope_dim, softmax_scale, workspace.data_ptr(),
                             workspace.numel() * workspace.element_size(), _stream(stream)))


def mla_v_up(out, o_lat, w_uv, stream=None) -> None:
    """Step 5: out[h,b,:] = o_lat[h,b,:] @ w_uv[h] (views [H,B,V], [H,B,L], [H,L,V])."""
    _check(lib().mla_v_up(_dtype_code(out, o_lat, w_uv), as_mla_tensor(out), as_mla_tensor(o_lat),
                          as_mla_tensor(w_uv), _stream(stream)))


def mla_decode_noalloc(o_lat_out, q_cat, cache, block_table, seq_lens, kv_lora_rank: int,
                       rope_dim: int, softmax_scale: float, lse_out=None, num_splits: int = 0,
                       stream=None) -> None:
    """mla_decode for callers that cannot allocate device memory: no workspace, the
    scratch is a fixed array inside the library (shared by all calls; do not overlap
    calls on the GPU)."""
    import torch
    _check_int32_table(block_table, seq_lens)
    if lse_out is not None and (lse_out.dtype != torch.float32 or not lse_out.is_contiguous()):
        raise MlaError(MLA_ERR_INVALID_ARG, "lse_out must be contiguous float32")
    _check(lib().mla_decode_noalloc(_dtype_code(o_lat_out, q_cat, cache), as_mla_tensor(o_lat_out),
                                    _ptr(lse_out), as_mla_tensor(q_cat), as_mla_tensor(cache),
                                    block_table.data_ptr(), block_table.stride(0), block_table.shape[1],
                                    seq_lens.data_ptr(), kv_lora_rank, rope_dim, softmax_scale,
                                    num_splits, _stream(stream)))


def _check_device(*tensors) -> int:
    """Every tensor on one CUDA device, and that the current one: the library launches there. Its index."""
    import torch
    device = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != device or device < 0):
            raise MlaError(MLA_ERR_INVALID_ARG, f"tensors must lie on one CUDA device; one is on {t.device}")
    if torch.cuda.current_device() != device:
        raise MlaError(MLA_ERR_INVALID_ARG, f"tensors must lie on the current device, cuda:{torch.cuda.current_device()}; "
                                            f"they are on cuda:{device}")
    return device


def _stream_on(stream, device: int) -> Optional[int]:
    """The stream a call runs on; without one, the device's current stream (asked for directly where torch
    allows it: the stream object costs more than the rest of a small call)."""
    import torch
    if stream is not None:
        return _stream(stream)
    direct = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return direct(device) if direct is not None else torch.cuda.current_stream(device).cuda_stream


def _check_slots(slot_mapping) -> None:
    import torch
    if slot_mapping.dtype != torch.int64 or slot_mapping.dim() != 1:
        raise MlaError(MLA_ERR_INVALID_ARG, "slot_mapping must be int64 [T]")
    if slot_mapping.numel() and not slot_mapping.is_contiguous():
        raise MlaError(MLA_ERR_INVALID_ARG, "slot_mapping must be contiguous")


def _check_counts(t, n: int, name: str) -> None:
    import torch
    if t.dtype != torch.int32 or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise MlaError(MLA_ERR_INVALID_ARG, f"{name} must be contiguous int32 [{n}]")


def _check_table(block_table, batch: int) -> None:
    import torch
    shape = block_table.shape
    if block_table.dtype != torch.int32 or len(shape) != 2 or shape[0] != batch:
        raise MlaError(MLA_ERR_INVALID_ARG, f"block_table must be int32 [{batch}, max_blocks]")
    if block_table.stride(1) != 1 and block_table.numel():
        raise MlaError(MLA_ERR_INVALID_ARG, "block_table must have unit column stride")


def _table_stride(block_table) -> int:
    """Row stride of a block table (a single row's stride is arbitrary in torch: its width serves)."""
    shape = block_table.shape
    return block_table.stride(0) if shape[0] > 1 else shape[1]


def _check_int32(value: int, name: str) -> None:
    """A count that the library takes in 32 bits (ctypes drops the bits above them)."""
    if not -2 ** 31 <= value < 2 ** 31:
        raise MlaError(MLA_ERR_INVALID_ARG, f"{name} must fit 32 bits, got {value}")


def _rows_and_heads(q_cat):
    shape = q_cat.shape
    if len(shape) != 3:
        raise MlaError(MLA_ERR_INVALID_ARG, "q_cat must be [rows, heads, kv_lora_rank + rope_dim]")
    return shape[0], shape[1]


def _check_lse(lse_out, q_cat) -> None:
    import torch
    if lse_out is None:
        return
    shape, rows = lse_out.shape, q_cat.shape
    if (lse_out.dtype != torch.float32 or not lse_out.is_contiguous() or len(shape) != 2 or shape[0] != rows[0] or
            shape[1] != rows[1]):
        raise MlaError(MLA_ERR_INVALID_ARG, "lse_out must be contiguous float32 with q_cat's rows and heads")


def _scratch(need: int, device: int, stream):
    """A workspace allocated on the stream the call runs on, so that its memory is reused only behind
    the call's work."""
    import torch
    if stream is None:
        return torch.empty(need, dtype=torch.uint8, device=f"cuda:{device}")
    with torch.cuda.stream(torch.cuda.ExternalStream(_stream(stream), device=device)):
        return torch.empty(need, dtype=torch.uint8, device=f"cuda:{device}")


def _workspace_args(workspace):
    if not workspace.is_contiguous():
        raise MlaError(MLA_ERR_INVALID_ARG, "workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _ds_mla_cache(cache):
    import torch
    if cache.dtype != torch.uint8:
        raise MlaError(MLA_ERR_INVALID_ARG, "a ds_mla cache is uint8 bytes")
    return cache[:, :, 0] if cache.dim() == 4 and cache.shape[2] == 1 else cache


def mla_cache_write_ds_mla(cache, kv_c, k_pe, slot_mapping, stream=None) -> None:
    """Step 3 into fp8 ds_mla entries: entry s of a uint8 [num_blocks, page, 656] (or
    [num_blocks, page, 1, 656]) cache = kv_c[i] as e4m3 codes with a float32 scale per 128
    columns, and k_pe[i] as bf16, for s = slot_mapping[i] >= 0; kv_c [T,512], k_pe [T,64]."""
    cache = _ds_mla_cache(cache)
    _check_slots(slot_mapping)
    device = _check_device(cache, kv_c, k_pe, slot_mapping)
    _check(lib().mla_cache_write_ds_mla(_dtype_code(kv_c, k_pe), as_mla_tensor(cache), as_mla_tensor(kv_c),
                                        as_mla_tensor(k_pe), _ptr(slot_mapping), slot_mapping.numel(),
                                        _stream_on(stream, device)))


def _read_args(out, cache, block_table, cu_seqlens, seq_starts, scale=None):
    batch = cu_seqlens.numel() - 1
    _check_table(block_table, batch)
    _check_counts(cu_seqlens, batch + 1, "cu_seqlens")
    if seq_starts is not None:
        _check_counts(seq_starts, batch, "seq_starts")
    device = _check_device(out, cache, block_table, cu_seqlens, seq_starts, scale)
    return device, (as_mla_tensor(out), as_mla_tensor(cache), _ptr(block_table), _table_stride(block_table),
                    block_table.shape[1], _ptr(cu_seqlens), _ptr(seq_starts), batch)


def mla_cache_read(out, cache, block_table, cu_seqlens, seq_starts=None, stream=None) -> None:
    """Read-back of a plain cache: out[i] = row seq_starts[b] + i - cu_seqlens[b] of sequence b for
    cu_seqlens[b] <= i < cu_seqlens[b+1]; out [T,W], bits unchanged, other rows left as they were."""
    device, args = _read_args(out, cache, block_table, cu_seqlens, seq_starts)
    _check(lib().mla_cache_read(_dtype_code(out, cache), *args, _stream_on(stream, device)))


def mla_cache_read_fp8(out, cache, block_table, cu_seqlens, scale, seq_starts=None, stream=None) -> None:
    """Read-back of an e4m3 cache: as mla_cache_read, a value = its code's value * scale, in out's dtype."""
    cache = _fp8_cache(cache)
    device, args = _read_args(out, cache, block_table, cu_seqlens, seq_starts, scale)
    _check(lib().mla_cache_read_fp8(_dtype_code(out), *args, _f32_scalar(scale, "scale"), _stream_on(stream, device)))


def mla_cache_read_ds_mla(out, cache, block_table, cu_seqlens, seq_starts=None, stream=None) -> None:
    """Read-back of a ds_mla cache: as mla_cache_read with 576 values a row, [code * scale | rope]."""
    cache = _ds_mla_cache(cache)
    device, args = _read_args(out, cache, block_table, cu_seqlens, seq_starts)
    _check(lib().mla_cache_read_ds_mla(_dtype_code(out), *args, _stream_on(stream, device)))


def mla_decode_window_workspace_size(batch: int, num_heads: int, kv_lora_rank: int, num_splits: int = 0) -> int:
    return int(lib().mla_decode_window_workspace_size(batch, num_heads, kv_lora_rank, num_splits))


def mla_decode_window(o_lat_out, q_cat, cache, block_table, seq_lens, kv_lora_rank: int, rope_dim: int,
                      softmax_scale: float, window: int, sinks: int = 0, lse_out=None, num_splits: int = 0,
                      workspace=None, stream=None) -> None:
    """Step 4, windowed: mla_decode over the last `window` rows of each sequence and its first `sinks` rows."""
    B, H = _rows_and_heads(q_cat)
    _check_int32(window, "window")
    _check_int32(sinks, "sinks")
    _check_int32(num_splits, "num_splits")
    _check_table(block_table, B)
    _check_counts(seq_lens, B, "seq_lens")
    _check_lse(lse_out, q_cat)
    device = _check_device(o_lat_out, q_cat, cache, block_table, seq_lens, lse_out, workspace)
    if workspace is None:
        workspace = _scratch(mla_decode_window_workspace_size(B, H, kv_lora_rank, num_splits), device, stream)
    _check(lib().mla_decode_window(_dtype_code(o_lat_out, q_cat, cache), as_mla_tensor(o_lat_out), _ptr(lse_out),
                                   as_mla_tensor(q_cat), as_mla_tensor(cache), _ptr(block_table),
                                   _table_stride(block_table), block_table.shape[1], _ptr(seq_lens), kv_lora_rank,
                                   rope_dim, softmax_scale, window, sinks, num_splits, *_workspace_args(workspace),
                                   _stream_on(stream, device)))


def mla_prefill_window_workspace_size(tokens: int, batch: int, num_heads: int, kv_lora_rank: int) -> int:
    return int(lib().mla_prefill_window_workspace_size(tokens, batch, num_heads, kv_lora_rank))


def mla_prefill_window(o_lat_out, q_cat, cache, block_table, cu_seqlens_q, seq_lens_kv, kv_lora_rank: int,
                       rope_dim: int, softmax_scale: float, window: int, sinks: int = 0, lse_out=None,
                       workspace=None, stream=None) -> None:
    """Step 4 (prefill), windowed: each query attends the last `window` rows up to its own and its
    sequence's first `sinks` rows."""
    batch, (T, H) = seq_lens_kv.numel(), _rows_and_heads(q_cat)
    _check_int32(window, "window")
    _check_int32(sinks, "sinks")
    _check_table(block_table, batch)
    _check_counts(seq_lens_kv, batch, "seq_lens_kv")
    _check_counts(cu_seqlens_q, batch + 1, "cu_seqlens_q")
    _check_lse(lse_out, q_cat)
    device = _check_device(o_lat_out, q_cat, cache, block_table, cu_seqlens_q, seq_lens_kv, lse_out, workspace)
    if workspace is None:
        workspace = _scratch(mla_prefill_window_workspace_size(T, batch, H, kv_lora_rank), device, stream)
    _check(lib().mla_prefill_window(_dtype_code(o_lat_out, q_cat, cache), as_mla_tensor(o_lat_out), _ptr(lse_out),
                                    as_mla_tensor(q_cat), as_mla_tensor(cache), _ptr(block_table),
                                    _table_stride(block_table), block_table.shape[1], _ptr(cu_seqlens_q),
                                    _ptr(seq_lens_kv), batch, kv_lora_rank, rope_dim, softmax_scale, window, sinks,
                                    *_workspace_args(workspace), _stream_on(stream, device)))


def mla_check_bounded_wait(limit_us: int, stream=None) -> None:
    """Run the kernels' bounded wait on an mbarrier nothing arrives on (see include/mla.h)."""
    _check(lib().mla_check_bounded_wait(limit_us, _stream(stream)))


def mla_device_error(stream=None) -> None:
    """Synchronise the stream and raise if a kernel recorded a device-side error."""
    _check(lib().mla_device_error(_stream(stream)))
