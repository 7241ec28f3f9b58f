"""Python binding of libmla_nvfp4.so (sparse MLA decode over an NVFP4 paged KV cache).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Functions carry the C names from ``include/mla_nvfp4.h`` and take
torch tensors (device memory) plus an optional stream; they raise
``MlaError`` on any non-OK status.  There is no fallback: if the library is
not built, loading fails with an explicit error.
"""
from __future__ import annotations

import ctypes as C
import functools
import os
from typing import Optional

import torch

__all__ = [
    "MlaError", "MLA_KV_NVFP4", "MLA_KV_FP8", "library_path", "load",
    "mla_kv_row_bytes", "mla_status_string", "mla_last_cuda_error", "mla_device_fault",
    "mla_kv_quantize_append", "mla_sparse_decode_workspace_size", "mla_sparse_decode_plan",
    "mla_sparse_decode_plan_fmt", "mla_sparse_decode",
    "mla_sparse_decode_fp8", "mla_sparse_decode_noalloc", "mla_topk_workspace_size", "mla_topk",
    "mla_indexer_topk_workspace_size", "mla_indexer_topk", "mla_index_key_quantize_append",
    "mla_staged_pool_bytes", "mla_stage_rows_fp8", "mla_sparse_decode_staged_workspace_size",
    "mla_sparse_decode_staged", "mla_sparse_decode_mtp_workspace_size", "mla_sparse_decode_mtp",
    "mla_block_table_extend", "mla_qk_norm_rope", "mla_kv_norm_rope_append", "mla_window_decode_workspace_size",
    "mla_window_decode", "mla_prefix_decode_workspace_size", "mla_prefix_decode",
    "mla_prompt_attention_workspace_size", "mla_prompt_attention_plan", "mla_prompt_attention", "mla_add_norm_quant",
    "mla_fp4_matvec",
]

MLA_KV_NVFP4 = 0
MLA_KV_FP8 = 1
_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libmla_nvfp4.so"
_lib = None

_STATUS = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_WORKSPACE_TOO_SMALL",
           4: "MLA_ERR_CUDA"}


class _Heads(C.Structure):
    """mla_heads_t"""
    _fields_ = [("in_", C.c_void_p), ("out", C.c_void_p), ("heads", C.c_int), ("in_token_stride", C.c_int64),
                ("in_head_stride", C.c_int64), ("out_token_stride", C.c_int64), ("out_head_stride", C.c_int64),
                ("weight", C.c_void_p)]


# Every symbol include/mla_nvfp4.h declares, with (restype, argtypes).
_P, _I32, _I64, _SZ, _F32 = C.c_void_p, C.c_int, C.c_int64, C.c_size_t, C.c_float
SIGNATURES = {
    "mla_kv_row_bytes": (_SZ, [_I32]),
    "mla_status_string": (C.c_char_p, [_I32]),
    "mla_last_cuda_error": (_I32, [_P]),
    "mla_device_fault": (_I32, [_P, _I32, _P]),
    "mla_kv_quantize_append": (_I32, [_P, _P, _P, _I64, _P, _I64, _I32, _I64, _I32, _P]),
    "mla_sparse_decode_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "mla_sparse_decode_plan": (_I32, [_I32, _I32, _I32, _P, _P, _P]),
    "mla_sparse_decode_plan_fmt": (_I32, [_I32, _I32, _I32, _I32, _I64, _I64, _P, _P, _P, _P]),
    "mla_sparse_decode": (_I32, [_P, _P, _P, _I64, _I64, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _F32, _P, _P,
                                 _P, _SZ, _P]),
    "mla_sparse_decode_fp8": (_I32, [_P, _P, _P, _I64, _I64, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _F32, _P,
                                     _P, _P, _SZ, _P]),
    "mla_sparse_decode_noalloc": (_I32, [_P, _P, _P, _I64, _I64, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _F32, _P,
                                         _P, _P]),
    "mla_topk_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "mla_topk": (_I32, [_P, _I64, _P, _I32, _I32, _I32, _P, _P, _SZ, _P]),
    "mla_indexer_topk_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "mla_indexer_topk": (_I32, [_P, _P, _P, _I64, _I64, _P, _I32, _P, _I32, _I32, _I32, _I32, _P, _P, _I32, _P,
                                _SZ, _P]),
    "mla_index_key_quantize_append": (_I32, [_P, _P, _I64, _P, _I64, _I32, _I64, _P]),
    "mla_sparse_decode_mtp_workspace_size": (_SZ, [_I32, _I32, _I32, _I32]),
    "mla_sparse_decode_mtp": (_I32, [_P, _P, _P, _I64, _I64, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _I32, _F32,
                                     _I32, _P, _P, _P, _SZ, _P]),
    "mla_staged_pool_bytes": (_SZ, [_I32, _I32]),
    "mla_stage_rows_fp8": (_I32, [_P, _I64, _I64, _P, _I32, _P, _P, _I32, _I32, _I32, _P, _P, _P]),
    "mla_sparse_decode_staged_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "mla_sparse_decode_staged": (_I32, [_P, _P, _P, _I64, _I64, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _F32, _P,
                                        _P, _P, _SZ, _P]),
    "mla_block_table_extend": (_I32, [_P, _P, _I32, _P, _I32, _P, _I64, _P, _I64, _I32, _P, _P, _I64, _P, _P, _P, _P]),
    "mla_qk_norm_rope": (_I32, [_P, _P, _I64, _I32, _I32, _I32, _F32, _P, _P, _P]),
    "mla_kv_norm_rope_append": (_I32, [_P, _I64, _P, _P, _I32, _I32, _I32, _F32, _P, _P, _P, _I64, _P, _I64, _I32,
                                       _I64, _I32, _P]),
    "mla_window_decode_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32]),
    "mla_window_decode": (_I32, [_P, _P, _P, _I64, _I64, _P, _I32, _P, _I32, _I32, _I32, _I32, _I32, _I32, _F32, _I32,
                                 _P, _P, _P, _SZ, _P]),
    "mla_prefix_decode_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32]),
    "mla_prefix_decode": (_I32, [_P, _P, _P, _I64, _I64, _P, _I32, _P, _I32, _P, _I32, _I32, _I32, _I32, _I32, _F32,
                                 _I32, _P, _P, _P, _SZ, _P]),
    "mla_prompt_attention_workspace_size": (_SZ, [_I64, _I64, _I32, _I32, _I32, _I32]),
    "mla_prompt_attention_plan": (_I32, [_I64, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P]),
    "mla_prompt_attention": (_I32, [_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _P, _I32, _I64, _I64, _I32,
                                    _I32, _I32, _I32, _I32, _F32, _P, _I64, _I64, _P, _P, _SZ, _P]),
    "mla_add_norm_quant": (_I32, [_P, _I64, _I32, _P, _I64, _P, _I64, _P, _I64, _I32, _I32, _F32, _P, _P, _P]),
    "mla_fp4_matvec": (_I32, [_P, _I32, _I64, _I64, _P, _I32, _P, _P, _P, _I64, _I32, _I32, _I32, _P, _I32, _I64, _I64,
                              _P]),
}


class MlaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        detail = _STATUS.get(status, str(status))
        if status == 4:
            err = C.c_int(0)
            load().mla_last_cuda_error(C.byref(err))
            detail += f" (cudaError {err.value})"
        super().__init__(f"{fn} failed: {detail}")
        self.status = status


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def load():
    """Load libmla_nvfp4.so (built by __graft_entry__.build() or build.py)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`"
                               " (or sparse_mla_decode_kv_gb300/build.py); there is no CPU fallback")
        lib = C.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return C.c_void_p(t.data_ptr())


def _stream(stream) -> C.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise MlaError(fn, status)


def _contig(t: torch.Tensor, dtype, name: str) -> torch.Tensor:
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _bits(t: torch.Tensor, name: str) -> torch.Tensor:
    """bf16 tensors are passed as their 16-bit patterns."""
    if t.dtype == torch.bfloat16:
        return _contig(t, torch.bfloat16, name)
    return _contig(t, torch.int16, name) if t.dtype == torch.int16 else _contig(t, torch.uint16, name)


# --------------------------------------------------------------------- misc
def mla_kv_row_bytes(fmt: int) -> int:
    return int(load().mla_kv_row_bytes(fmt))


def mla_status_string(status: int) -> str:
    return load().mla_status_string(status).decode()


def mla_last_cuda_error() -> int:
    err = C.c_int(0)
    load().mla_last_cuda_error(C.byref(err))
    return err.value


def mla_device_fault(clear: bool = False, stream=None) -> int:
    word = C.c_uint(0)
    _check("mla_device_fault", load().mla_device_fault(C.byref(word), int(clear), _stream(stream)))
    return word.value


# --------------------------------------------------------------------- quantize-on-write
def mla_kv_quantize_append(latent: torch.Tensor, rope: torch.Tensor, slot_mapping: torch.Tensor,
                           kv_pool: torch.Tensor, num_blocks: int, block_size: int, kv_block_stride: int,
                           fmt: int = MLA_KV_NVFP4, stream=None) -> None:
    latent = _bits(latent, "latent")
    rope = _bits(rope, "rope")
    slot_mapping = _contig(slot_mapping, torch.int64, "slot_mapping")
    n = slot_mapping.numel()
    if latent.numel() != n * 512 or rope.numel() != n * 64:
        raise ValueError("latent must be [n,512] and rope [n,64] for n = len(slot_mapping)")
    if num_blocks > 0 and kv_pool.numel() * kv_pool.element_size() < (num_blocks - 1) * kv_block_stride + \
            block_size * (352 if fmt == MLA_KV_NVFP4 else 576):
        raise ValueError("kv_pool does not reach the last row of block num_blocks - 1")
    _check("mla_kv_quantize_append",
           load().mla_kv_quantize_append(_ptr(latent), _ptr(rope), _ptr(slot_mapping), n, _ptr(kv_pool),
                                         num_blocks, block_size, kv_block_stride, fmt, _stream(stream)))


def mla_index_key_quantize_append(keys: torch.Tensor, slot_mapping: torch.Tensor, idx_key_pool: torch.Tensor,
                                  num_blocks: int, block_size: int, idx_block_stride: int, stream=None) -> None:
    """Indexer keys bf16 [n, 128] -> 128 e4m3 codes + a float scale per token, by slot."""
    keys = _bits(keys, "keys")
    slot_mapping = _contig(slot_mapping, torch.int64, "slot_mapping")
    n = slot_mapping.numel()
    if keys.numel() != n * 128:
        raise ValueError("keys must be [n,128] for n = len(slot_mapping)")
    if num_blocks > 0 and idx_key_pool.numel() * idx_key_pool.element_size() < (num_blocks - 1) * idx_block_stride + \
            block_size * 132:
        raise ValueError("idx_key_pool does not reach the last scale of block num_blocks - 1")
    _check("mla_index_key_quantize_append",
           load().mla_index_key_quantize_append(_ptr(keys), _ptr(slot_mapping), n, _ptr(idx_key_pool), num_blocks,
                                                block_size, idx_block_stride, _stream(stream)))


# --------------------------------------------------------------------- sparse decode
def mla_sparse_decode_workspace_size(batch: int, num_heads: int, topk: int) -> int:
    return int(load().mla_sparse_decode_workspace_size(batch, num_heads, topk))


def mla_sparse_decode_plan(batch: int, num_heads: int, topk: int) -> dict:
    """{"splits", "rows_per_split", "kernels"} of one decode call on the current device."""
    sp, rows, kern = C.c_int(0), C.c_int(0), C.c_int(0)
    _check("mla_sparse_decode_plan",
           load().mla_sparse_decode_plan(batch, num_heads, topk, C.byref(sp), C.byref(rows), C.byref(kern)))
    return {"splits": sp.value, "rows_per_split": rows.value, "kernels": kern.value}


def mla_sparse_decode_plan_fmt(fmt: int, batch: int, num_heads: int, topk: int, kv_block_stride: int,
                               num_blocks: int) -> dict:
    """The division a decode with this cache format and pool geometry uses,
    including whether it runs the tensor-memory kernel."""
    sp, rows, kern, tm = C.c_int(), C.c_int(), C.c_int(), C.c_int()
    _check("mla_sparse_decode_plan_fmt",
           load().mla_sparse_decode_plan_fmt(fmt, batch, num_heads, topk, kv_block_stride, num_blocks, C.byref(sp),
                                             C.byref(rows), C.byref(kern), C.byref(tm)))
    return {"splits": sp.value, "rows_per_split": rows.value, "kernels": kern.value,
            "tensor_memory": bool(tm.value)}

def _decode(cname: str, q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table, context_lens, topk_idx,
            softmax_scale, block_size=64, out=None, lse=None, workspace=None, stream=None,
            ws_size=mla_sparse_decode_workspace_size):
    q_nope = _bits(q_nope, "q_nope")
    q_rope = _bits(q_rope, "q_rope")
    block_table = _contig(block_table, torch.int32, "block_table")
    context_lens = _contig(context_lens, torch.int32, "context_lens")
    topk_idx = _contig(topk_idx, torch.int32, "topk_idx")
    batch, heads = q_nope.shape[0], q_nope.shape[1]
    topk = topk_idx.shape[1]
    if out is None:
        out = torch.empty((batch, heads, 512), dtype=torch.bfloat16, device=q_nope.device)
    need = ws_size(batch, heads, topk)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q_nope.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    fn = getattr(load(), cname)
    _check(cname, fn(_ptr(q_nope), _ptr(q_rope), _ptr(kv_pool), kv_block_stride, num_blocks, _ptr(block_table),
                     block_table.shape[1], _ptr(context_lens), _ptr(topk_idx), batch, heads, block_size, topk,
                     float(softmax_scale), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes, _stream(stream)))
    return out, lse


def mla_sparse_decode(q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table, context_lens, topk_idx,
                      softmax_scale, block_size=64, out=None, lse=None, workspace=None, stream=None):
    """NVFP4 cache.  Returns (out bf16 [B,H,512], lse or None)."""
    return _decode("mla_sparse_decode", q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table,
                   context_lens, topk_idx, softmax_scale, block_size, out, lse, workspace, stream)


def mla_sparse_decode_fp8(q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table, context_lens, topk_idx,
                          softmax_scale, block_size=64, out=None, lse=None, workspace=None, stream=None):
    """FP8 (576-byte) cache.  Returns (out bf16 [B,H,512], lse or None)."""
    return _decode("mla_sparse_decode_fp8", q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table,
                   context_lens, topk_idx, softmax_scale, block_size, out, lse, workspace, stream)


def mla_sparse_decode_staged_workspace_size(batch: int, num_heads: int, topk: int) -> int:
    return int(load().mla_sparse_decode_staged_workspace_size(batch, num_heads, topk))


def mla_sparse_decode_staged(q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table, context_lens,
                             topk_idx, softmax_scale, block_size=64, out=None, lse=None, workspace=None, stream=None):
    """Staged path over the NVFP4 cache (gather to an FP8 copy, then the FP8
    decode).  Returns (out bf16 [B,H,512], lse or None)."""
    return _decode("mla_sparse_decode_staged", q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table,
                   context_lens, topk_idx, softmax_scale, block_size, out, lse, workspace, stream,
                   ws_size=mla_sparse_decode_staged_workspace_size)


def mla_sparse_decode_mtp_workspace_size(batch: int, q_len: int, num_heads: int, topk: int) -> int:
    return int(load().mla_sparse_decode_mtp_workspace_size(batch, q_len, num_heads, topk))


def mla_sparse_decode_mtp(q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table, context_lens, topk_idx,
                          softmax_scale, fmt=MLA_KV_NVFP4, block_size=64, out=None, lse=None, workspace=None,
                          stream=None):
    """Several query tokens per request: q_nope [B,Q,H,512], q_rope [B,Q,H,64],
    topk_idx int32 [B,Q,k].  Returns (out bf16 [B,Q,H,512], lse or None)."""
    q_nope = _bits(q_nope, "q_nope")
    q_rope = _bits(q_rope, "q_rope")
    block_table = _contig(block_table, torch.int32, "block_table")
    context_lens = _contig(context_lens, torch.int32, "context_lens")
    topk_idx = _contig(topk_idx, torch.int32, "topk_idx")
    batch, q_len, heads = q_nope.shape[0], q_nope.shape[1], q_nope.shape[2]
    topk = topk_idx.shape[2]
    if out is None:
        out = torch.empty((batch, q_len, heads, 512), dtype=torch.bfloat16, device=q_nope.device)
    need = mla_sparse_decode_mtp_workspace_size(batch, q_len, heads, topk)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q_nope.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("mla_sparse_decode_mtp",
           load().mla_sparse_decode_mtp(_ptr(q_nope), _ptr(q_rope), _ptr(kv_pool), kv_block_stride, num_blocks,
                                        _ptr(block_table), block_table.shape[1], _ptr(context_lens), _ptr(topk_idx),
                                        batch, q_len, heads, block_size, topk, float(softmax_scale), fmt, _ptr(out),
                                        _ptr(lse), _ptr(workspace), ws_bytes, _stream(stream)))
    return out, lse


def mla_staged_pool_bytes(batch: int, topk: int) -> int:
    return int(load().mla_staged_pool_bytes(batch, topk))


def mla_stage_rows_fp8(kv_pool, kv_block_stride, num_blocks, block_table, context_lens, topk_idx, block_size=64,
                       staged_pool=None, staged_topk=None, stream=None):
    """Gather step of the staged path.  Returns (staged_pool uint8, staged_topk int32 [B, topk])."""
    block_table = _contig(block_table, torch.int32, "block_table")
    context_lens = _contig(context_lens, torch.int32, "context_lens")
    topk_idx = _contig(topk_idx, torch.int32, "topk_idx")
    batch, topk = topk_idx.shape
    dev = topk_idx.device
    if staged_pool is None:
        staged_pool = torch.empty(mla_staged_pool_bytes(batch, topk), dtype=torch.uint8, device=dev)
    if staged_pool.numel() * staged_pool.element_size() < mla_staged_pool_bytes(batch, topk):
        raise ValueError("staged_pool is smaller than mla_staged_pool_bytes(batch, topk)")
    if staged_topk is None:
        staged_topk = torch.empty((batch, topk), dtype=torch.int32, device=dev)
    _check("mla_stage_rows_fp8",
           load().mla_stage_rows_fp8(_ptr(kv_pool), kv_block_stride, num_blocks, _ptr(block_table),
                                     block_table.shape[1], _ptr(context_lens), _ptr(topk_idx), batch, block_size,
                                     topk, _ptr(staged_pool), _ptr(staged_topk), _stream(stream)))
    return staged_pool, staged_topk


def mla_sparse_decode_noalloc(q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table, context_lens,
                              topk_idx, softmax_scale, block_size=64, out=None, lse=None, stream=None):
    """NVFP4 decode whose split-K scratch is the library's own fixed device
    array (for callers that cannot allocate); same results as
    mla_sparse_decode.  Returns (out bf16 [B,H,512], lse or None)."""
    q_nope = _bits(q_nope, "q_nope")
    q_rope = _bits(q_rope, "q_rope")
    block_table = _contig(block_table, torch.int32, "block_table")
    context_lens = _contig(context_lens, torch.int32, "context_lens")
    topk_idx = _contig(topk_idx, torch.int32, "topk_idx")
    batch, heads = q_nope.shape[0], q_nope.shape[1]
    if out is None:
        out = torch.empty((batch, heads, 512), dtype=torch.bfloat16, device=q_nope.device)
    _check("mla_sparse_decode_noalloc",
           load().mla_sparse_decode_noalloc(_ptr(q_nope), _ptr(q_rope), _ptr(kv_pool), kv_block_stride, num_blocks,
                                            _ptr(block_table), block_table.shape[1], _ptr(context_lens),
                                            _ptr(topk_idx), batch, heads, block_size, topk_idx.shape[1],
                                            float(softmax_scale), _ptr(out), _ptr(lse), _stream(stream)))
    return out, lse


# --------------------------------------------------------------------- top-k and indexer
def mla_topk_workspace_size(batch: int, max_context_len: int, topk: int) -> int:
    return int(load().mla_topk_workspace_size(batch, max_context_len, topk))


def mla_topk(scores: torch.Tensor, context_lens: torch.Tensor, topk: int, out=None, workspace=None, stream=None):
    """scores float32 [B, max_context_len] -> int32 [B, topk] (ascending, -1 padded)."""
    scores = _contig(scores, torch.float32, "scores")
    context_lens = _contig(context_lens, torch.int32, "context_lens")
    batch, max_ctx = scores.shape
    if out is None:
        out = torch.empty((batch, topk), dtype=torch.int32, device=scores.device)
    need = mla_topk_workspace_size(batch, max_ctx, topk)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=scores.device)
    ws_bytes = 0 if workspace is None else workspace.numel()
    _check("mla_topk", load().mla_topk(_ptr(scores), max_ctx, _ptr(context_lens), batch, topk, max_ctx, _ptr(out),
                                       _ptr(workspace), ws_bytes, _stream(stream)))
    return out


def mla_indexer_topk_workspace_size(batch: int, max_context_len: int, topk: int) -> int:
    return int(load().mla_indexer_topk_workspace_size(batch, max_context_len, topk))


def mla_indexer_topk(q_idx, head_w, idx_key_pool, idx_block_stride, num_blocks, block_table, context_lens, topk,
                     max_context_len, block_size=64, topk_out=None, scores_out=None, workspace=None, stream=None):
    """Indexer scores + exact top-k.  Returns (topk_out int32 [B,topk], scores_out or None)."""
    q_idx = _bits(q_idx, "q_idx")
    head_w = _contig(head_w, torch.float32, "head_w")
    block_table = _contig(block_table, torch.int32, "block_table")
    context_lens = _contig(context_lens, torch.int32, "context_lens")
    batch, nh = q_idx.shape[0], q_idx.shape[1]
    if topk_out is None:
        topk_out = torch.empty((batch, topk), dtype=torch.int32, device=q_idx.device)
    need = mla_indexer_topk_workspace_size(batch, max_context_len, topk)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q_idx.device)
    ws_bytes = 0 if workspace is None else workspace.numel()
    _check("mla_indexer_topk",
           load().mla_indexer_topk(_ptr(q_idx), _ptr(head_w), _ptr(idx_key_pool), idx_block_stride, num_blocks,
                                   _ptr(block_table), block_table.shape[1], _ptr(context_lens), batch, nh, block_size,
                                   topk, _ptr(topk_out), _ptr(scores_out), max_context_len, _ptr(workspace),
                                   ws_bytes, _stream(stream)))
    return topk_out, scores_out


# --------------------------------------------------------------------- block tables, norms, dense decodes
# These calls are also made for single tokens, where the host's share is most of
# the time: devices are compared as numbers, addresses passed as numbers, and
# the current stream read without a stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_INT_MAX = 2 ** 31 - 1


def _here(*tensors) -> int:
    """The one device of `tensors` (None left out), which has to be the current one."""
    device = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            if not t.is_cuda:
                raise ValueError("expected a CUDA tensor")
            raise ValueError(f"a tensor on {t.device}, but cuda:{device} is the current device")
    return device


def _on(stream, device: int) -> int:
    """The address of `stream`, or of the device's current one."""
    if stream is None:
        return _raw_stream(device) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _new(like, shape, dtype, stream) -> torch.Tensor:
    """Memory on `like`'s device whose reuse is ordered behind the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)  # 1.5 us, like.new_empty 2.4
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _take(t, shape, dtype, name, like, stream) -> torch.Tensor:
    """The caller's output tensor, checked, or a new one."""
    if t is None:
        return _new(like, shape, dtype, stream)
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return _contig(t, dtype, name)


def _at(t):
    return None if t is None else t.data_ptr()


def _c_int(v, name) -> None:
    """Refuses what a C int would keep the low 32 bits of."""
    if not -_INT_MAX <= v <= _INT_MAX:
        raise ValueError(f"{name} {v} does not fit 32 bits")


def _c_ints(**values) -> None:
    for name, v in values.items():
        _c_int(v, name)


def _length(v, name) -> int:
    """A length cut to the longest that a context can have."""
    if v < 0:
        _c_int(v, name)
    return min(v, _INT_MAX)


def _check_pool(kv_pool, num_blocks, block_size, kv_block_stride, fmt) -> None:
    _c_int(block_size, "block_size")
    _c_int(fmt, "fmt")
    if num_blocks > 0 and kv_pool.numel() * kv_pool.element_size() < (num_blocks - 1) * kv_block_stride + \
            block_size * (352 if fmt == MLA_KV_NVFP4 else 576):
        raise ValueError("kv_pool does not reach the last row of block num_blocks - 1")


def mla_block_table_extend(context_lens, new_lens, block_table, free_blocks, free_state, num_blocks, num_slots,
                           block_size=64, slot_mapping=None, positions=None, query_start=None, context_lens_out=None,
                           free_state_out=None, stream=None):
    """Blocks, positions and slots of every request's new tokens.  context_lens,
    new_lens int32 [B]; block_table int32 [B, W], extended in place; free_blocks
    int32 ring with free_state int64 [3] (head, tail, -).  Returns (slot_mapping
    int64 [num_slots], positions int32 [num_slots], query_start int32 [B + 1],
    context_lens_out int32 [B], free_state_out int64 [3])."""
    context_lens = _contig(context_lens, torch.int32, "context_lens")
    new_lens = _contig(new_lens, torch.int32, "new_lens")
    block_table = _contig(block_table, torch.int32, "block_table")
    free_blocks = _contig(free_blocks, torch.int32, "free_blocks")
    free_state = _contig(free_state, torch.int64, "free_state")
    device = _here(context_lens, new_lens, block_table, free_blocks, free_state, slot_mapping, positions, query_start,
                   context_lens_out, free_state_out)
    batch = context_lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != batch or new_lens.numel() != batch or \
            free_state.numel() != 3:
        raise ValueError("new_lens [B], block_table [B, W] and free_state [3] must fit context_lens [B]")
    _c_int(block_size, "block_size")
    slot_mapping = _take(slot_mapping, (num_slots,), torch.int64, "slot_mapping", free_state, stream)
    positions = _take(positions, (num_slots,), torch.int32, "positions", context_lens, stream)
    query_start = _take(query_start, (batch + 1,), torch.int32, "query_start", context_lens, stream)
    context_lens_out = _take(context_lens_out, (batch,), torch.int32, "context_lens_out", context_lens, stream)
    free_state_out = _take(free_state_out, (3,), torch.int64, "free_state_out", free_state, stream)
    _check("mla_block_table_extend",
           load().mla_block_table_extend(_at(context_lens), _at(new_lens), batch, _at(block_table),
                                         block_table.shape[1], _at(free_blocks), free_blocks.numel(), _at(free_state),
                                         num_blocks, block_size, _at(slot_mapping), _at(positions), num_slots,
                                         _at(query_start), _at(context_lens_out), _at(free_state_out),
                                         _on(stream, device)))
    return slot_mapping, positions, query_start, context_lens_out, free_state_out


def _head_strides(x, what):
    """Token and head stride of bf16 heads [n, H, D] whose last axis is contiguous."""
    if x.dtype != torch.bfloat16:
        raise TypeError(f"{what}: expected torch.bfloat16, got {x.dtype}")
    strides = x.stride()
    if len(strides) != 3 or (strides[2] != 1 and x.numel() > 0):
        raise ValueError(f"{what} must be [n, heads, dim] with a contiguous last axis")
    return strides


def _heads(x, weight, out, name, stream):
    """(mla_heads_t, output) of the heads x."""
    in_token, in_head, _ = _head_strides(x, name)
    shape = x.shape
    _, heads, dim = shape
    if weight is not None and _contig(weight, torch.bfloat16, name + "_weight").numel() != dim:
        raise ValueError(f"{name}_weight must have one value for each of {dim} dims")
    if out is None:
        out = _new(x, shape, torch.bfloat16, stream)
        out_token, out_head = heads * dim, dim
    else:
        if out.shape != shape:
            raise ValueError(f"{name}_out must be shaped like {name}")
        out_token, out_head, _ = _head_strides(out, name + "_out")
    return _Heads(x.data_ptr(), out.data_ptr(), heads, in_token, in_head, out_token, out_head,
                  None if weight is None else weight.data_ptr()), out


def _angles(positions, inv_freq, n, rope_offset):
    _c_int(rope_offset, "rope_offset")
    if _contig(positions, torch.int32, "positions").numel() != n:
        raise ValueError(f"positions must have one entry for each of {n} tokens")
    if _contig(inv_freq, torch.float64, "inv_freq").numel() != 32:
        raise ValueError("inv_freq must have 32 entries")


def mla_qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, rope_offset=0,
                     interleaved=True, q_out=None, k_out=None, stream=None):
    """Norm per head (with a weight) and rotation of 64 values from rope_offset
    on.  q bf16 [n, Hq, D], k bf16 [n, Hk, D] or None, any strides over tokens
    and heads; positions int32 [n]; inv_freq float64 [32].  Returns (q_out,
    k_out or None); q_out may be q, k_out may be k."""
    device = _here(q, k, positions, inv_freq, q_weight, k_weight, q_out, k_out)
    hq, q_out = _heads(q, q_weight, q_out, "q", stream)
    n, _, dim = q.shape
    _angles(positions, inv_freq, n, rope_offset)
    hk = None
    if k is not None:
        hk, k_out = _heads(k, k_weight, k_out, "k", stream)
        if k.shape[0] != n or k.shape[2] != dim:
            raise ValueError("q and k must have the same tokens and head dim")
    _check("mla_qk_norm_rope",
           load().mla_qk_norm_rope(C.byref(hq), None if hk is None else C.byref(hk), n, dim, rope_offset,
                                   int(interleaved), float(eps), _at(positions), _at(inv_freq),
                                   _on(stream, device)))
    return q_out, (None if k is None else k_out)


def mla_kv_norm_rope_append(kv, latent_weight, positions, inv_freq, slot_mapping, kv_pool, num_blocks, block_size,
                            kv_block_stride, fmt=MLA_KV_NVFP4, eps=1e-6, interleaved=True, q=None, q_weight=None,
                            rope_offset=0, q_out=None, stream=None):
    """kv bf16 [n, 576] (latent 512 | key 64): norm of the latent, rotation of
    the key, quantise-on-write by slot, and q's norm and rotation (as
    mla_qk_norm_rope) in the same launch.  Returns q_out, or None without q."""
    device = _here(kv, latent_weight, positions, inv_freq, slot_mapping, kv_pool, q,
                   q_weight if q is not None else None, q_out)
    if kv.dtype != torch.bfloat16:
        raise TypeError(f"kv: expected torch.bfloat16, got {kv.dtype}")
    if kv.dim() != 2 or kv.shape[1] != 576 or (kv.numel() > 0 and kv.stride(1) != 1):
        raise ValueError("kv must be [n, 576] with a contiguous last axis")
    n = kv.shape[0]
    if _contig(latent_weight, torch.bfloat16, "latent_weight").numel() != 512:
        raise ValueError("latent_weight must have 512 values")
    if _contig(slot_mapping, torch.int64, "slot_mapping").numel() != n:
        raise ValueError(f"slot_mapping must have one entry for each of {n} tokens")
    _angles(positions, inv_freq, n, rope_offset)
    _check_pool(kv_pool, num_blocks, block_size, kv_block_stride, fmt)
    hq = None
    if q is not None:
        if q.dim() != 3 or q.shape[0] != n:
            raise ValueError("q must be [n, heads, dim] for the tokens of kv")
        hq, q_out = _heads(q, q_weight, q_out, "q", stream)
    _check("mla_kv_norm_rope_append",
           load().mla_kv_norm_rope_append(_at(kv), kv.stride(0), _at(latent_weight),
                                          None if hq is None else C.byref(hq), 0 if q is None else q.shape[2],
                                          rope_offset, int(interleaved), float(eps), _at(positions), _at(inv_freq),
                                          _at(slot_mapping), n, _at(kv_pool), num_blocks, block_size,
                                          kv_block_stride, fmt, _on(stream, device)))
    return None if q is None else q_out


def _dense_tensors(q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table, context_lens, fmt, block_size,
                   out, lse, workspace, stream):
    """Checks what the two dense decodes share; returns (q_nope, q_rope, batch, q_len, heads, out, device)."""
    q_nope = _bits(q_nope, "q_nope")
    q_rope = _bits(q_rope, "q_rope")
    _contig(block_table, torch.int32, "block_table")
    _contig(context_lens, torch.int32, "context_lens")
    device = _here(q_nope, q_rope, kv_pool, block_table, context_lens, out, lse, workspace)
    if q_nope.dim() != 4 or q_nope.shape[3] != 512 or tuple(q_rope.shape) != (*q_nope.shape[:3], 64):
        raise ValueError("q_nope must be [B, Q, H, 512] and q_rope [B, Q, H, 64]")
    batch, q_len, heads = q_nope.shape[:3]
    if block_table.dim() != 2 or block_table.shape[0] != batch or context_lens.numel() != batch:
        raise ValueError("block_table [B, W] and context_lens [B] must fit q_nope [B, Q, H, 512]")
    _check_pool(kv_pool, num_blocks, block_size, kv_block_stride, fmt)
    out = _take(out, (batch, q_len, heads, 512), torch.bfloat16, "out", q_nope, stream)
    if lse is not None:
        _take(lse, (batch, q_len, heads), torch.float32, "lse", q_nope, stream)
    return q_nope, q_rope, batch, q_len, heads, out, device


def mla_window_decode_workspace_size(batch: int, q_len: int, num_heads: int, max_blocks_per_req: int, sinks: int,
                                     window: int) -> int:
    sinks, window = _length(sinks, "sinks"), _length(window, "window")
    return int(load().mla_window_decode_workspace_size(batch, q_len, num_heads, max_blocks_per_req, sinks, window))


def mla_window_decode(q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table, context_lens, softmax_scale,
                      sinks, window, fmt=MLA_KV_NVFP4, block_size=64, out=None, lse=None, workspace=None,
                      stream=None):
    """Every query token sees the first `sinks` positions and the last `window`
    up to its own.  q_nope [B,Q,H,512], q_rope [B,Q,H,64], the Q tokens the last
    positions of context_lens.  Returns (out bf16 [B,Q,H,512], lse or None)."""
    q_nope, q_rope, batch, q_len, heads, out, device = _dense_tensors(
        q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table, context_lens, fmt, block_size, out, lse,
        workspace, stream)
    sinks, window = _length(sinks, "sinks"), _length(window, "window")
    if workspace is None:
        need = mla_window_decode_workspace_size(batch, q_len, heads, block_table.shape[1], sinks, window)
        workspace = _new(kv_pool, (need,), torch.uint8, stream) if need > 0 else None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("mla_window_decode",
           load().mla_window_decode(_at(q_nope), _at(q_rope), _at(kv_pool), kv_block_stride, num_blocks,
                                    _at(block_table), block_table.shape[1], _at(context_lens), batch, q_len, heads,
                                    block_size, sinks, window, float(softmax_scale), fmt, _at(out), _at(lse),
                                    _at(workspace), ws_bytes, _on(stream, device)))
    return out, lse


def mla_prefix_decode_workspace_size(batch: int, q_len: int, num_heads: int, prefix_len: int,
                                     max_blocks_per_req: int, max_context_len: int) -> int:
    max_context_len = _length(max_context_len, "max_context_len")
    _c_int(prefix_len, "prefix_len")
    return int(load().mla_prefix_decode_workspace_size(batch, q_len, num_heads, prefix_len, max_blocks_per_req,
                                                       max_context_len))


def mla_prefix_decode(q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, prefix_table, prefix_len, block_table,
                      context_lens, softmax_scale, max_context_len, fmt=MLA_KV_NVFP4, block_size=64, out=None,
                      lse=None, workspace=None, stream=None):
    """Every query token sees the `prefix_len` rows of prefix_table and its own
    request's rows up to itself.  q_nope [B,Q,H,512], q_rope [B,Q,H,64];
    context_lens counts the tokens after the prefix, at most max_context_len.
    Returns (out bf16 [B,Q,H,512], lse or None)."""
    q_nope, q_rope, batch, q_len, heads, out, device = _dense_tensors(
        q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table, context_lens, fmt, block_size, out, lse,
        workspace, stream)
    max_context_len = _length(max_context_len, "max_context_len")
    _c_int(prefix_len, "prefix_len")
    if prefix_len > 0:
        _here(out, prefix_table)
        if _contig(prefix_table, torch.int32, "prefix_table").numel() * block_size < prefix_len:
            raise ValueError("prefix_table does not reach prefix_len")
    if workspace is None:
        need = mla_prefix_decode_workspace_size(batch, q_len, heads, prefix_len, block_table.shape[1],
                                                max_context_len)
        workspace = _new(kv_pool, (need,), torch.uint8, stream) if need > 0 else None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("mla_prefix_decode",
           load().mla_prefix_decode(_at(q_nope), _at(q_rope), _at(kv_pool), kv_block_stride, num_blocks,
                                    _at(prefix_table), prefix_len, _at(block_table), block_table.shape[1],
                                    _at(context_lens), batch, q_len, heads, block_size, max_context_len,
                                    float(softmax_scale), fmt, _at(out), _at(lse), _at(workspace), ws_bytes,
                                    _on(stream, device)))
    return out, lse


# --------------------------------------------------------------------- prompts, and around the attention of a layer
def mla_prompt_attention_workspace_size(q_tokens: int, kv_tokens: int, batch: int, num_heads: int, num_kv_heads: int,
                                        v_dim: int) -> int:
    _c_ints(batch=batch, num_heads=num_heads, num_kv_heads=num_kv_heads, v_dim=v_dim)
    return int(load().mla_prompt_attention_workspace_size(q_tokens, kv_tokens, batch, num_heads, num_kv_heads, v_dim))


def mla_prompt_attention_plan(q_tokens: int, kv_tokens: int, batch: int, num_heads: int, num_kv_heads: int,
                              v_dim: int) -> dict:
    """{"row_tiles", "slices", "units", "variant"} of a call of these sizes on the current device;
    variant is "plain", "turns" or "pairs"."""
    _c_ints(batch=batch, num_heads=num_heads, num_kv_heads=num_kv_heads, v_dim=v_dim)
    tiles, slices, units, variant = C.c_int(), C.c_int(), C.c_int64(), C.c_int()
    _check("mla_prompt_attention_plan",
           load().mla_prompt_attention_plan(q_tokens, kv_tokens, batch, num_heads, num_kv_heads, v_dim, C.byref(tiles),
                                            C.byref(slices), C.byref(units), C.byref(variant)))
    return {"row_tiles": tiles.value, "slices": slices.value, "units": units.value,
            "variant": ("plain", "turns", "pairs")[variant.value]}


@functools.lru_cache(maxsize=1024)
def _prompt_workspace(device, *sizes) -> int:
    """The size for the current device (its number is part of the key), without a call into the library."""
    return int(load().mla_prompt_attention_workspace_size(*sizes))


def mla_prompt_attention(q, k, v, query_start, kv_start, softmax_scale, causal=True, out=None, lse=None,
                         workspace=None, stream=None):
    """Attention of packed sequences: b's query tokens are query_start[b] ..
    query_start[b + 1] - 1 of q [Tq, H, D], its keys and values kv_start[b] ..
    kv_start[b + 1] - 1 of k [Tk, Hk, D], v [Tk, Hk, Dv], its queries the last of
    those positions.  All bf16 with any strides over tokens and heads, the starts
    int32 [B + 1].  Returns (out bf16 [Tq, H, Dv], lse or None)."""
    device = _here(q, k, v, query_start, kv_start, out, lse, workspace)
    q_token, q_head, _ = _head_strides(q, "q")
    k_token, k_head, _ = _head_strides(k, "k")
    v_token, v_head, _ = _head_strides(v, "v")
    q_tokens, heads, dk = q.shape
    kv_tokens, kv_heads, dv = v.shape
    if k.shape != (kv_tokens, kv_heads, dk):
        raise ValueError("k [Tk, Hk, D] and v [Tk, Hk, Dv] must have the same tokens and heads, and k the dims of q")
    batch = _contig(query_start, torch.int32, "query_start").numel() - 1
    if batch < 0 or _contig(kv_start, torch.int32, "kv_start").numel() != batch + 1:
        raise ValueError("query_start and kv_start must have one entry for each sequence and one more")
    if max(batch, heads, kv_heads, dk, dv) > _INT_MAX:
        _c_ints(batch=batch, heads=heads, kv_heads=kv_heads, dk=dk, dv=dv)
    if out is None:
        out = _new(q, (q_tokens, heads, dv), torch.bfloat16, stream)
        out_token, out_head = heads * dv, dv
    else:
        if out.shape != (q_tokens, heads, dv):
            raise ValueError(f"out: expected shape {(q_tokens, heads, dv)}, got {tuple(out.shape)}")
        out_token, out_head, _ = _head_strides(out, "out")
    if lse is not None:
        _take(lse, (q_tokens, heads), torch.float32, "lse", q, stream)
    if workspace is None:
        ws_bytes = _prompt_workspace(device, q_tokens, kv_tokens, batch, heads, kv_heads, dv)
        workspace = _new(q, (ws_bytes,), torch.uint8, stream) if ws_bytes > 0 else None
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check("mla_prompt_attention",
           load().mla_prompt_attention(q.data_ptr(), q_token, q_head, k.data_ptr(), k_token, k_head, v.data_ptr(),
                                       v_token, v_head, query_start.data_ptr(), kv_start.data_ptr(), batch, q_tokens,
                                       kv_tokens, heads, kv_heads, dk, dv, int(causal), float(softmax_scale),
                                       out.data_ptr(), out_token, out_head, _at(lse), _at(workspace), ws_bytes,
                                       _on(stream, device)))
    return out, lse


def _rows(t, dtype, name):
    """(shape, row stride) of a [n, dim] tensor whose last axis is contiguous."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    shape, strides = t.shape, t.stride()
    if len(strides) != 2 or (strides[1] != 1 and shape[1] > 1 and t.numel() > 0):
        raise ValueError(f"{name} must be [n, dim] with a contiguous last axis")
    return shape, strides[0]


def _bytes(t, name):
    """A contiguous tensor of e4m3 values, as float8_e4m3fn or bytes."""
    if t.dtype is not torch.float8_e4m3fn and t.dtype is not torch.uint8:
        raise TypeError(f"{name}: expected torch.float8_e4m3fn or torch.uint8, got {t.dtype}")
    return _contig(t, t.dtype, name)


def mla_add_norm_quant(x, weight, residual=None, eps=1e-6, group=128, codes=None, scales=None, residual_out=None,
                       stream=None):
    """h = x + residual, its norm times weight, and that in e4m3 with a float
    scale per 128 values (group=128) or per row (group=0).  x bf16 [n, D],
    residual bf16 or float32 [n, D] or None; rows may be strided.  Returns
    (codes float8_e4m3fn [n, D], scales [n, ceil(D / 128) or 1], h in the
    residual's type or None); residual_out may be residual."""
    device = _here(x, weight, residual, codes, scales, None if residual is None else residual_out)
    shape, x_stride = _rows(x, torch.bfloat16, "x")
    n, dim = shape
    if _contig(weight, torch.bfloat16, "weight").numel() != dim:
        raise ValueError(f"weight must have one value for each of {dim} dims")
    _c_int(group, "group")
    _c_int(dim, "dim")
    res_type = res_stride = out_stride = 0
    if residual is not None:
        kind = residual.dtype
        if kind is not torch.bfloat16 and kind is not torch.float32:
            raise TypeError(f"residual: expected torch.bfloat16 or torch.float32, got {kind}")
        res_type = 1 if kind is torch.bfloat16 else 2
        res_shape, res_stride = _rows(residual, kind, "residual")
        if residual_out is None:
            residual_out, out_stride = _new(residual, shape, kind, stream), dim
        else:
            out_shape, out_stride = _rows(residual_out, kind, "residual_out")
            if out_shape != shape:
                raise ValueError("residual_out must be shaped like x")
        if res_shape != shape:
            raise ValueError("residual must be shaped like x")
    if codes is None:
        codes = _new(x, shape, torch.float8_e4m3fn, stream)
    elif _bytes(codes, "codes").shape != shape:
        raise ValueError("codes must be shaped like x")
    scales = _take(scales, (n, -(-dim // group) if group > 0 else 1), torch.float32, "scales", x, stream)
    _check("mla_add_norm_quant",
           load().mla_add_norm_quant(x.data_ptr(), x_stride, res_type, _at(residual), res_stride,
                                     None if residual is None else residual_out.data_ptr(), out_stride,
                                     weight.data_ptr(), n, dim, group, float(eps), codes.data_ptr(), scales.data_ptr(),
                                     _on(stream, device)))
    return codes, scales, None if residual is None else residual_out


def _token_groups(t, what):
    """(token stride, group stride) of [T, K] or [T, G, K] with a contiguous last axis."""
    strides = t.stride()
    if len(strides) not in (2, 3) or (strides[-1] != 1 and t.shape[-1] > 1 and t.numel() > 0):
        raise ValueError(f"{what} must be [T, K] or [T, G, K] with a contiguous last axis")
    return strides[0], strides[1] if len(strides) == 3 else 0


def mla_fp4_matvec(x, codes, scales, weight_scale=None, x_scales=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """Products of T tokens with 4-bit weights.  x [T, K] with codes uint8 [N,
    K / 2] and scales e4m3 [N, K / 16], or x [T, G, K] with a matrix for each
    group: codes [G, N, K / 2], scales [G, N, K / 16].  x bf16, or float8_e4m3fn
    with x_scales float32 [T(, G), ceil(K / 128) or 1]; weight_scale float32, one
    for each matrix, or None.  Returns out [T, N] or [T, G, N], bf16 or float32."""
    device = _here(x, codes, scales, weight_scale, x_scales, out)
    x_token, x_group = _token_groups(x, "x")
    shape, c_shape, kind = x.shape, _contig(codes, torch.uint8, "codes").shape, x.dtype
    tokens, k = shape[0], shape[-1]
    groups = shape[1] if len(shape) == 3 else 1
    if len(c_shape) != len(shape) or c_shape[-1] * 2 != k or k % 16 != 0 or (len(shape) == 3 and c_shape[0] != groups):
        raise ValueError(f"codes {tuple(c_shape)} do not fit x {tuple(shape)}: [N, K / 2] or [G, N, K / 2]")
    n = c_shape[-2]
    if max(n, k, groups) > _INT_MAX:
        _c_ints(n=n, k=k, groups=groups)
    if _bytes(scales, "scales").shape != (*c_shape[:-1], k // 16):
        raise ValueError("scales must have one value for 16 codes")
    if weight_scale is not None and _contig(weight_scale, torch.float32, "weight_scale").numel() != groups:
        raise ValueError(f"weight_scale must have one value for each of {groups} matrices")
    scale_groups = 0
    if kind is torch.float8_e4m3fn:
        if x_scales is None:
            raise ValueError("x in 8 bits needs x_scales")
        s_shape = _contig(x_scales, torch.float32, "x_scales").shape
        scale_groups = s_shape[-1] if len(s_shape) > 0 else 0
        if s_shape[:-1] != shape[:-1] or scale_groups not in (1, -(-k // 128)):
            raise ValueError("x_scales must have one value for 128 of x's, or one for each of its rows")
    elif kind is not torch.bfloat16:
        raise TypeError(f"x: expected torch.bfloat16 or torch.float8_e4m3fn, got {kind}")
    elif x_scales is not None:
        raise ValueError("x_scales belong to x in 8 bits")
    out_shape = (*shape[:-1], n)
    if out is None:
        if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
            raise TypeError(f"out_dtype: expected torch.bfloat16 or torch.float32, got {out_dtype}")
        out = _new(x, out_shape, out_dtype, stream)
        out_token, out_group = groups * n, n
    else:
        out_dtype = out.dtype
        if out.shape != out_shape:
            raise ValueError(f"out: expected shape {out_shape}, got {tuple(out.shape)}")
        if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
            raise TypeError(f"out: expected torch.bfloat16 or torch.float32, got {out_dtype}")
        out_token, out_group = _token_groups(out, "out")
    _check("mla_fp4_matvec",
           load().mla_fp4_matvec(x.data_ptr(), 1 if scale_groups else 0, x_token, x_group, _at(x_scales), scale_groups,
                                 codes.data_ptr(), scales.data_ptr(), _at(weight_scale), tokens, groups, n, k,
                                 out.data_ptr(), 1 if out_dtype is torch.float32 else 0, out_token, out_group,
                                 _on(stream, device)))
    return out
