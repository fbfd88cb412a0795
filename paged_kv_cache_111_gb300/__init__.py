"""Python binding of libpagedkv.so: paged KV-cache attention on one GB300.

Argument marshalling only.  Every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/pkv.h``; this module passes
torch tensors' device pointers, sizes and the current CUDA stream through
ctypes.  There is no fallback: if the library is missing or the tensors are
not on a CUDA device, the calls raise.

Calls (same names as the C ABI without the ``pkv_`` prefix):

* ``kv_write(kv_cache, key, value, slot_mapping, device_status=None)``
* ``paged_attn(out, query, kv_cache, block_tables, seq_lens, query_start_loc,
  max_query_len, max_seq_len, scale, workspace, num_splits=0)``
* ``paged_attn_combine(out, workspace)``
* ``copy_blocks(kv_cache, block_mapping)`` (copy-on-write of shared blocks)
* ``paged_attn_shared_prefix(..., shared_prefix_blocks, workspace)`` (cascade:
  a batch sharing a table prefix reads the shared blocks once)
* ``kv_write_fp8`` / ``paged_attn_fp8`` / ``paged_attn_shared_prefix_fp8`` (E4M3 cache with per-tensor
  K and V scales)
* ``qk_norm_rope_kv_write`` / ``qk_norm_rope_kv_write_fp8`` (norm and rotation of query and key heads with the
  cache write, in one pass)
* ``latent_kv_write`` / ``latent_paged_attn`` / ``latent_gather`` (a cache of one latent row a token, and attention
  over it in the latent space)
* ``latent_attn_expanded`` (attention over the per-head keys and values that gathered latent rows expand to)

plus ``paged_attn_workspace_size(...)`` (the C call's size query) and
``workspace_status(workspace)`` (reads the device status word).
"""

from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

from . import _build

__all__ = [
    "BLOCK_SIZE", "PagedKVError", "load", "kv_write", "paged_attn", "paged_attn_combine",
    "paged_attn_workspace_size", "workspace_status", "STATUS_NAMES", "library_path", "copy_blocks",
    "paged_attn_noalloc", "paged_attn_shared_prefix", "paged_attn_shared_prefix_workspace_size",
    "kv_write_fp8", "paged_attn_fp8", "paged_attn_shared_prefix_fp8", "workspace_schedule",
    "qk_norm_rope_kv_write", "qk_norm_rope_kv_write_fp8", "LATENT_DIM", "LATENT_ROPE_DIM", "latent_kv_write",
    "latent_gather", "latent_paged_attn", "latent_paged_attn_workspace_size", "latent_attn_expanded",
]

BLOCK_SIZE = 16
LATENT_DIM, LATENT_ROPE_DIM = 512, 64        # dims of a latent cache row: latent, then rotated key
STATUS_NAMES = {
    0: "PKV_OK", 1: "PKV_ERR_NULL", 2: "PKV_ERR_SHAPE", 3: "PKV_ERR_UNSUPPORTED", 4: "PKV_ERR_ALIGNMENT",
    5: "PKV_ERR_WORKSPACE", 6: "PKV_ERR_CUDA", 7: "PKV_ERR_DEVICE_INDEX", 8: "PKV_ERR_DEVICE_METADATA",
    9: "PKV_ERR_DEVICE_TIMEOUT", 10: "PKV_ERR_PROTOCOL",
}

_lib = None
_lock = threading.Lock()


class PagedKVError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)}")
        self.code = code


def library_path() -> str:
    return _build.LIB


def load():
    """Load libpagedkv.so (built by ``__graft_entry__.build()`` or ``_build.build()``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_build.LIB):
            raise RuntimeError(
                f"{_build.LIB} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(_build.LIB)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        lib.pkv_kv_write.argtypes = [P, i64, i32, i32, i32, P, i64, P, i64, P, i32, P, P]
        lib.pkv_kv_write.restype = ctypes.c_int
        lib.pkv_paged_attn.argtypes = [P, P, i64, P, i64, P, i32, P, P, i32, i32, i32, i32, i32, i32, i32, i32,
                                       ctypes.c_float, i32, P, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t), P]
        lib.pkv_paged_attn.restype = ctypes.c_int
        lib.pkv_paged_attn_combine.argtypes = [P, P, ctypes.c_size_t, i32, i32, i32, P]
        lib.pkv_paged_attn_combine.restype = ctypes.c_int
        lib.pkv_copy_blocks.argtypes = [P, i64, i32, i32, i32, P, i32, P, P]
        lib.pkv_copy_blocks.restype = ctypes.c_int
        lib.pkv_paged_attn_shared_prefix.argtypes = [P, P, i64, P, i64, P, i32, P, P, i32, i32, i32, i32, i32, i32,
                                                     i32, i32, ctypes.c_float, i32, i32, P, ctypes.c_size_t,
                                                     ctypes.POINTER(ctypes.c_size_t), P]
        lib.pkv_paged_attn_shared_prefix.restype = ctypes.c_int
        lib.pkv_kv_write_fp8.argtypes = [P, i64, i32, i32, i32, P, i64, P, i64, P, i32, ctypes.c_float,
                                         ctypes.c_float, P, P]
        lib.pkv_kv_write_fp8.restype = ctypes.c_int
        lib.pkv_paged_attn_fp8.argtypes = [P, P, i64, P, i64, P, i32, P, P, i32, i32, i32, i32, i32, i32, i32,
                                           i32, ctypes.c_float, ctypes.c_float, ctypes.c_float, i32, P,
                                           ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t), P]
        lib.pkv_paged_attn_fp8.restype = ctypes.c_int
        lib.pkv_paged_attn_shared_prefix_fp8.argtypes = [P, P, i64, P, i64, P, i32, P, P, i32, i32, i32, i32, i32,
                                                         i32, i32, i32, ctypes.c_float, ctypes.c_float,
                                                         ctypes.c_float, i32, i32, P, ctypes.c_size_t,
                                                         ctypes.POINTER(ctypes.c_size_t), P]
        lib.pkv_paged_attn_shared_prefix_fp8.restype = ctypes.c_int
        f32 = ctypes.c_float
        qk = [P, i64, P, i64, i32, i32, i32, i32, P, i64, P, i64, P, i64, P, P, f32, P, i64, i32, i32, P, P, i32]
        lib.pkv_qk_norm_rope_kv_write.argtypes = qk + [P, P]
        lib.pkv_qk_norm_rope_kv_write.restype = ctypes.c_int
        lib.pkv_qk_norm_rope_kv_write_fp8.argtypes = qk + [f32, f32, P, P]
        lib.pkv_qk_norm_rope_kv_write_fp8.restype = ctypes.c_int
        lib.pkv_latent_kv_write.argtypes = [P, i64, i32, P, i64, P, i64, P, f32, P, i64, i32, P, P, i32, P, i64, i64,
                                            P, i64, i64, i32, P, P]
        lib.pkv_latent_kv_write.restype = ctypes.c_int
        lib.pkv_latent_gather.argtypes = [P, i64, P, i64, i32, P, i32, P, P, i32, i32, P, P]
        lib.pkv_latent_gather.restype = ctypes.c_int
        lib.pkv_latent_paged_attn.argtypes = [P, P, i64, P, i64, P, i32, P, P, i32, i32, i32, i32, i32, i32, f32, P,
                                              ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t), P]
        lib.pkv_latent_paged_attn.restype = ctypes.c_int
        lib.pkv_latent_attn_expanded.argtypes = [P, P, i64, P, i64, i64, P, i64, P, i64, i64, P, P, i32, i32, i32, i32,
                                                 i32, i32, f32, P, P]
        lib.pkv_latent_attn_expanded.restype = ctypes.c_int
        _lib = lib
        return lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor, stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return ctypes.c_void_p(handle)


def _need_cuda(*tensors: torch.Tensor) -> None:
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError("paged KV-cache calls take CUDA tensors only")


def _check(rc: int, what: str) -> None:
    if rc != 0:
        raise PagedKVError(rc, what)


def kv_write(kv_cache: torch.Tensor, key: torch.Tensor, value: torch.Tensor, slot_mapping: torch.Tensor,
             device_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Scatter key/value [T, Hkv, d] (bf16) into kv_cache [NB, Hkv, 2, 16, d] through slot_mapping [T] (int64)."""
    _need_cuda(kv_cache, key, value, slot_mapping, device_status)
    nb, hkv, _, bs, d = kv_cache.shape
    T = int(slot_mapping.shape[0])
    if key.dim() != 3 or key.stride(2) != 1 or key.stride(1) != d or value.stride(2) != 1 or value.stride(1) != d:
        raise ValueError("key/value must be [T, Hkv, d] with contiguous heads")
    rc = load().pkv_kv_write(_ptr(kv_cache), nb, hkv, d, bs, _ptr(key), key.stride(0), _ptr(value),
                             value.stride(0), _ptr(slot_mapping), T, _ptr(device_status), _stream(kv_cache, stream))
    _check(rc, "pkv_kv_write")


def copy_blocks(kv_cache: torch.Tensor, block_mapping: torch.Tensor, device_status: Optional[torch.Tensor] = None,
                stream=None) -> None:
    """Copy-on-write: block_mapping int64 [num_pairs, 2] of {source, destination} block ids."""
    _need_cuda(kv_cache, block_mapping, device_status)
    nb, hkv, _, bs, d = kv_cache.shape
    if block_mapping.dim() != 2 or block_mapping.shape[1] != 2 or not block_mapping.is_contiguous():
        raise ValueError("block_mapping must be a contiguous [num_pairs, 2] int64 tensor")
    rc = load().pkv_copy_blocks(_ptr(kv_cache), nb, hkv, d, bs, _ptr(block_mapping), int(block_mapping.shape[0]),
                                _ptr(device_status), _stream(kv_cache, stream))
    _check(rc, "pkv_copy_blocks")


def paged_attn_workspace_size(num_seqs: int, num_tokens: int, max_query_len: int, max_seq_len: int,
                              num_q_heads: int, num_kv_heads: int, head_size: int) -> int:
    """Bytes of workspace pkv_paged_attn needs for these sizes (no GPU work)."""
    need = ctypes.c_size_t(0)
    max_blocks = (max_seq_len + BLOCK_SIZE - 1) // BLOCK_SIZE
    rc = load().pkv_paged_attn(None, None, num_q_heads * head_size, None, 1, None, max_blocks, None, None,
                               num_seqs, num_tokens, max_query_len, max_seq_len, num_q_heads, num_kv_heads,
                               head_size, BLOCK_SIZE, ctypes.c_float(1.0), 0, None, 0, ctypes.byref(need), None)
    if rc not in (0, 1, 5):
        _check(rc, "pkv_paged_attn (size query)")
    return int(need.value)


def paged_attn(out: torch.Tensor, query: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor,
               seq_lens: torch.Tensor, query_start_loc: torch.Tensor, max_query_len: int, max_seq_len: int,
               scale: float, workspace: torch.Tensor, num_splits: int = 0, stream=None) -> None:
    """Causal paged attention; out [T, H, d] bf16.  Follow with paged_attn_combine on the same stream."""
    _need_cuda(out, query, kv_cache, block_tables, seq_lens, query_start_loc, workspace)
    nb, hkv, _, bs, d = kv_cache.shape
    T, H = int(query.shape[0]), int(query.shape[1])
    if query.stride(2) != 1 or query.stride(1) != d:
        raise ValueError("query must be [T, H, d] with contiguous heads")
    if not out.is_contiguous() or tuple(out.shape) != (T, H, d):
        raise ValueError("out must be a contiguous [T, H, d] tensor")
    if block_tables.dim() != 2 or not block_tables.is_contiguous():
        raise ValueError("block_tables must be a contiguous [num_seqs, max_blocks] tensor")
    S = int(seq_lens.shape[0])
    need = ctypes.c_size_t(0)
    rc = load().pkv_paged_attn(_ptr(out), _ptr(query), query.stride(0), _ptr(kv_cache), nb, _ptr(block_tables),
                               int(block_tables.shape[1]), _ptr(seq_lens), _ptr(query_start_loc), S, T,
                               int(max_query_len), int(max_seq_len), H, hkv, d, bs, ctypes.c_float(scale),
                               int(num_splits), _ptr(workspace), workspace.numel() * workspace.element_size(),
                               ctypes.byref(need), _stream(out, stream))
    _check(rc, "pkv_paged_attn")


def paged_attn_shared_prefix_workspace_size(num_seqs: int, num_tokens: int, max_query_len: int, max_seq_len: int,
                                            num_q_heads: int, num_kv_heads: int, head_size: int,
                                            shared_prefix_blocks: int) -> int:
    """Bytes of workspace pkv_paged_attn_shared_prefix needs (no GPU work)."""
    need = ctypes.c_size_t(0)
    max_blocks = max((max_seq_len + BLOCK_SIZE - 1) // BLOCK_SIZE, shared_prefix_blocks)
    rc = load().pkv_paged_attn_shared_prefix(None, None, num_q_heads * head_size, None, 1, None, max_blocks, None,
                                             None, num_seqs, num_tokens, max_query_len, max_seq_len, num_q_heads,
                                             num_kv_heads, head_size, BLOCK_SIZE, ctypes.c_float(1.0), 0,
                                             shared_prefix_blocks, None, 0, ctypes.byref(need), None)
    if rc not in (0, 1, 5):
        _check(rc, "pkv_paged_attn_shared_prefix (size query)")
    return int(need.value)


def paged_attn_shared_prefix(out: torch.Tensor, query: torch.Tensor, kv_cache: torch.Tensor,
                             block_tables: torch.Tensor, seq_lens: torch.Tensor, query_start_loc: torch.Tensor,
                             max_query_len: int, max_seq_len: int, scale: float, shared_prefix_blocks: int,
                             workspace: torch.Tensor, num_splits: int = 0, stream=None) -> None:
    """paged_attn with the first shared_prefix_blocks table entries shared by the batch (cascade)."""
    _need_cuda(out, query, kv_cache, block_tables, seq_lens, query_start_loc, workspace)
    nb, hkv, _, bs, d = kv_cache.shape
    T, H = int(query.shape[0]), int(query.shape[1])
    if query.stride(2) != 1 or query.stride(1) != d:
        raise ValueError("query must be [T, H, d] with contiguous heads")
    if not out.is_contiguous() or tuple(out.shape) != (T, H, d):
        raise ValueError("out must be a contiguous [T, H, d] tensor")
    if block_tables.dim() != 2 or not block_tables.is_contiguous():
        raise ValueError("block_tables must be a contiguous [num_seqs, max_blocks] tensor")
    need = ctypes.c_size_t(0)
    rc = load().pkv_paged_attn_shared_prefix(
        _ptr(out), _ptr(query), query.stride(0), _ptr(kv_cache), nb, _ptr(block_tables), int(block_tables.shape[1]),
        _ptr(seq_lens), _ptr(query_start_loc), int(seq_lens.shape[0]), T, int(max_query_len), int(max_seq_len), H,
        hkv, d, bs, ctypes.c_float(scale), int(num_splits), int(shared_prefix_blocks), _ptr(workspace),
        workspace.numel() * workspace.element_size(), ctypes.byref(need), _stream(out, stream))
    _check(rc, "pkv_paged_attn_shared_prefix")


def kv_write_fp8(kv_cache: torch.Tensor, key: torch.Tensor, value: torch.Tensor, slot_mapping: torch.Tensor,
                 k_scale: float, v_scale: float, device_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """kv_write into an E4M3 cache (uint8 or float8_e4m3fn [NB, Hkv, 2, 16, d]): code = E4M3(x / scale)."""
    _need_cuda(kv_cache, key, value, slot_mapping, device_status)
    if kv_cache.element_size() != 1:
        raise ValueError("an FP8 cache holds one byte per element")
    nb, hkv, _, bs, d = kv_cache.shape
    T = int(slot_mapping.shape[0])
    if key.dim() != 3 or key.stride(2) != 1 or key.stride(1) != d or value.stride(2) != 1 or value.stride(1) != d:
        raise ValueError("key/value must be [T, Hkv, d] with contiguous heads")
    rc = load().pkv_kv_write_fp8(_ptr(kv_cache), nb, hkv, d, bs, _ptr(key), key.stride(0), _ptr(value),
                                 value.stride(0), _ptr(slot_mapping), T, ctypes.c_float(k_scale),
                                 ctypes.c_float(v_scale), _ptr(device_status), _stream(kv_cache, stream))
    _check(rc, "pkv_kv_write_fp8")


def paged_attn_fp8(out: torch.Tensor, query: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor,
                   seq_lens: torch.Tensor, query_start_loc: torch.Tensor, max_query_len: int, max_seq_len: int,
                   scale: float, k_scale: float, v_scale: float, workspace: torch.Tensor, num_splits: int = 0,
                   stream=None) -> None:
    """paged_attn over an E4M3 cache; the workspace is sized as for paged_attn."""
    _need_cuda(out, query, kv_cache, block_tables, seq_lens, query_start_loc, workspace)
    if kv_cache.element_size() != 1:
        raise ValueError("an FP8 cache holds one byte per element")
    nb, hkv, _, bs, d = kv_cache.shape
    T, H = int(query.shape[0]), int(query.shape[1])
    if query.stride(2) != 1 or query.stride(1) != d:
        raise ValueError("query must be [T, H, d] with contiguous heads")
    if not out.is_contiguous() or tuple(out.shape) != (T, H, d):
        raise ValueError("out must be a contiguous [T, H, d] tensor")
    if block_tables.dim() != 2 or not block_tables.is_contiguous():
        raise ValueError("block_tables must be a contiguous [num_seqs, max_blocks] tensor")
    need = ctypes.c_size_t(0)
    rc = load().pkv_paged_attn_fp8(
        _ptr(out), _ptr(query), query.stride(0), _ptr(kv_cache), nb, _ptr(block_tables), int(block_tables.shape[1]),
        _ptr(seq_lens), _ptr(query_start_loc), int(seq_lens.shape[0]), T, int(max_query_len), int(max_seq_len), H,
        hkv, d, bs, ctypes.c_float(scale), ctypes.c_float(k_scale), ctypes.c_float(v_scale), int(num_splits),
        _ptr(workspace), workspace.numel() * workspace.element_size(), ctypes.byref(need), _stream(out, stream))
    _check(rc, "pkv_paged_attn_fp8")


def paged_attn_shared_prefix_fp8(out: torch.Tensor, query: torch.Tensor, kv_cache: torch.Tensor,
                                 block_tables: torch.Tensor, seq_lens: torch.Tensor, query_start_loc: torch.Tensor,
                                 max_query_len: int, max_seq_len: int, scale: float, k_scale: float, v_scale: float,
                                 shared_prefix_blocks: int, workspace: torch.Tensor, num_splits: int = 0,
                                 stream=None) -> None:
    """paged_attn_shared_prefix over an E4M3 cache; the workspace is sized as for paged_attn_shared_prefix."""
    _need_cuda(out, query, kv_cache, block_tables, seq_lens, query_start_loc, workspace)
    if kv_cache.element_size() != 1:
        raise ValueError("an FP8 cache holds one byte per element")
    nb, hkv, _, bs, d = kv_cache.shape
    T, H = int(query.shape[0]), int(query.shape[1])
    if query.stride(2) != 1 or query.stride(1) != d:
        raise ValueError("query must be [T, H, d] with contiguous heads")
    if not out.is_contiguous() or tuple(out.shape) != (T, H, d):
        raise ValueError("out must be a contiguous [T, H, d] tensor")
    if block_tables.dim() != 2 or not block_tables.is_contiguous():
        raise ValueError("block_tables must be a contiguous [num_seqs, max_blocks] tensor")
    need = ctypes.c_size_t(0)
    rc = load().pkv_paged_attn_shared_prefix_fp8(
        _ptr(out), _ptr(query), query.stride(0), _ptr(kv_cache), nb, _ptr(block_tables), int(block_tables.shape[1]),
        _ptr(seq_lens), _ptr(query_start_loc), int(seq_lens.shape[0]), T, int(max_query_len), int(max_seq_len), H,
        hkv, d, bs, ctypes.c_float(scale), ctypes.c_float(k_scale), ctypes.c_float(v_scale), int(num_splits),
        int(shared_prefix_blocks), _ptr(workspace), workspace.numel() * workspace.element_size(),
        ctypes.byref(need), _stream(out, stream))
    _check(rc, "pkv_paged_attn_shared_prefix_fp8")


def paged_attn_combine(out: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """Log-sum-exp merge of the rows pkv_paged_attn split; out as given to paged_attn."""
    _need_cuda(out, workspace)
    T, H, d = out.shape
    rc = load().pkv_paged_attn_combine(_ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                       T, H, d, _stream(out, stream))
    _check(rc, "pkv_paged_attn_combine")


def workspace_status(workspace: torch.Tensor) -> int:
    """The device status word (first int32 of the workspace); synchronises on its read."""
    return int(workspace[:4].view(torch.int32)[0].item())


# per-CTA record of the persistent prefill kernels' dynamic schedule: int32
# [2][1024] right after the workspace's 256-byte header
_SCHEDULE_OFFSET, _SCHEDULE_CTAS = 256, 1024


def workspace_schedule(workspace: torch.Tensor):
    """Work items each CTA of the tensor-core prefill kernel (first list) and of
    the shared-prefix pass (second list) took in the last attention call on
    this workspace, trailing idle CTAs dropped; synchronises on its read."""
    a = workspace[_SCHEDULE_OFFSET:_SCHEDULE_OFFSET + 8 * _SCHEDULE_CTAS].view(torch.int32).cpu().tolist()

    def trim(v):
        while v and v[-1] == 0:
            v.pop()
        return v
    return trim(a[:_SCHEDULE_CTAS]), trim(a[_SCHEDULE_CTAS:])


def paged_attn_noalloc(out: torch.Tensor, query: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor,
                       seq_lens: torch.Tensor, query_start_loc: torch.Tensor, max_query_len: int, max_seq_len: int,
                       scale: float, num_splits: int = 0, device_status: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    """paged_attn + paged_attn_combine without a caller workspace: for callers
    that cannot allocate device memory.  The scratch is the library's own
    fixed device array (see pkv_paged_attn_noalloc in include/pkv.h)."""
    _need_cuda(out, query, kv_cache, block_tables, seq_lens, query_start_loc, device_status)
    lib = load()
    fn = lib.pkv_paged_attn_noalloc
    if fn.argtypes is None:
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        fn.argtypes = [P, P, i64, P, i64, P, i32, P, P, i32, i32, i32, i32, i32, i32, i32, i32,
                       ctypes.c_float, i32, P, P]
        fn.restype = ctypes.c_int
    nb, hkv, _, bs, d = kv_cache.shape
    T, H = int(query.shape[0]), int(query.shape[1])
    if query.stride(2) != 1 or query.stride(1) != d:
        raise ValueError("query must be [T, H, d] with contiguous heads")
    if not out.is_contiguous() or tuple(out.shape) != (T, H, d):
        raise ValueError("out must be a contiguous [T, H, d] tensor")
    rc = fn(_ptr(out), _ptr(query), query.stride(0), _ptr(kv_cache), nb, _ptr(block_tables),
            int(block_tables.shape[1]), _ptr(seq_lens), _ptr(query_start_loc), int(seq_lens.shape[0]), T,
            int(max_query_len), int(max_seq_len), H, hkv, d, bs, ctypes.c_float(scale), int(num_splits),
            _ptr(device_status), _stream(out, stream))
    _check(rc, "pkv_paged_attn_noalloc")


# ---- norm, rotation and the latent cache: calls that check types and devices too -------------------------------

def _expect(what: str, t: Optional[torch.Tensor], dtype, ndim: int, device) -> None:
    """One tensor argument: a CUDA tensor of this type and rank on the call's device."""
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError("paged KV-cache calls take CUDA tensors only")
    if t.dtype != dtype or t.dim() != ndim:
        raise ValueError(f"{what} must be a {ndim}-dimensional {dtype} tensor, not {t.dim()}-dimensional {t.dtype}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, the call's other tensors on {device}")


def _contiguous(what: str, t: Optional[torch.Tensor], shape=None) -> None:
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must be {tuple(shape)}, not {tuple(t.shape)}")


def _step(x: torch.Tensor, dim: int, least: int) -> int:
    """The stride of a dim in elements; of a dim of one entry (where it means nothing), the least that the call takes."""
    return x.stride(dim) if x.shape[dim] > 1 else least


def _call(device, stream, fn, *args) -> None:
    """Enqueue on `stream` (default: the current one of the tensors' device), with that device current."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    handle = ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))
    if torch.cuda.current_device() == device.index:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
    _check(rc, fn.__name__)


def _qk_norm_rope(fp8: bool, query_out, kv_cache, query, key, value, q_weight, k_weight, eps, cos_sin, positions,
                  slot_mapping, scales, interleaved, device_status, stream) -> None:
    dev, bf = kv_cache.device, torch.bfloat16
    if kv_cache.dim() != 5 or kv_cache.element_size() != (1 if fp8 else 2) or (not fp8 and kv_cache.dtype != bf):
        raise ValueError("kv_cache must be [NB, Hkv, 2, 16, d], bf16 (one byte per element for an FP8 cache)")
    _expect("kv_cache", kv_cache, kv_cache.dtype, 5, dev)
    _contiguous("kv_cache", kv_cache)
    nb, hkv, _, bs, d = kv_cache.shape
    for what, x in (("query_out", query_out), ("query", query), ("key", key), ("value", value)):
        _expect(what, x, bf, 3, dev)
        if x.stride(2) != 1 or (x.shape[1] > 1 and x.stride(1) != d) or x.shape[2] != d:
            raise ValueError(f"{what} must be [T, heads, {d}] with contiguous heads")
    T, H = int(query.shape[0]), int(query.shape[1])
    if tuple(query_out.shape) != (T, H, d) or tuple(key.shape) != (T, hkv, d) or tuple(value.shape) != (T, hkv, d):
        raise ValueError("query_out must be [T, H, d], key and value [T, Hkv, d]")
    for what, x in (("q_weight", q_weight), ("k_weight", k_weight)):
        _expect(what, x, bf, 1, dev)
        _contiguous(what, x, (d,))
    _expect("cos_sin", cos_sin, torch.float32, 2, dev)
    _contiguous("cos_sin", cos_sin)
    for what, x in (("positions", positions), ("slot_mapping", slot_mapping)):
        _expect(what, x, torch.int64, 1, dev)
        _contiguous(what, x, (T,))
    _expect("device_status", device_status, torch.int32, 1, dev)
    lib = load()
    _call(dev, stream, lib.pkv_qk_norm_rope_kv_write_fp8 if fp8 else lib.pkv_qk_norm_rope_kv_write,
          _ptr(query_out), _step(query_out, 0, H * d), _ptr(kv_cache), nb, H, hkv, d, bs,
          _ptr(query), _step(query, 0, H * d), _ptr(key), _step(key, 0, hkv * d), _ptr(value),
          _step(value, 0, hkv * d), _ptr(q_weight), _ptr(k_weight),
          float(eps), _ptr(cos_sin), int(cos_sin.shape[0]), int(cos_sin.shape[1]),
          1 if interleaved else 0, _ptr(positions), _ptr(slot_mapping), T, *scales, _ptr(device_status))


def qk_norm_rope_kv_write(query_out: torch.Tensor, kv_cache: torch.Tensor, query: torch.Tensor, key: torch.Tensor,
                          value: torch.Tensor, q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor],
                          eps: float, cos_sin: torch.Tensor, positions: torch.Tensor, slot_mapping: torch.Tensor,
                          interleaved: bool = False, device_status: Optional[torch.Tensor] = None,
                          stream=None) -> None:
    """Norm and rotate query [T, H, d] into query_out and key [T, Hkv, d] into the cache, and write value there.

    Weights are bf16 [d] (None: no norm); cos_sin is fp32 [max_position, rotary_dim] (cosines, then sines);
    positions and slot_mapping are int64 [T].  Takes the place of kv_write; query_out may be query."""
    _qk_norm_rope(False, query_out, kv_cache, query, key, value, q_weight, k_weight, eps, cos_sin, positions,
                  slot_mapping, (), interleaved, device_status, stream)


def qk_norm_rope_kv_write_fp8(query_out: torch.Tensor, kv_cache: torch.Tensor, query: torch.Tensor,
                              key: torch.Tensor, value: torch.Tensor, q_weight: Optional[torch.Tensor],
                              k_weight: Optional[torch.Tensor], eps: float, cos_sin: torch.Tensor,
                              positions: torch.Tensor, slot_mapping: torch.Tensor, k_scale: float, v_scale: float,
                              interleaved: bool = False, device_status: Optional[torch.Tensor] = None,
                              stream=None) -> None:
    """qk_norm_rope_kv_write into an E4M3 cache (uint8 or float8_e4m3fn [NB, Hkv, 2, 16, d])."""
    _qk_norm_rope(True, query_out, kv_cache, query, key, value, q_weight, k_weight, eps, cos_sin, positions,
                  slot_mapping, (float(k_scale), float(v_scale)), interleaved, device_status, stream)


def _latent_cache(latent_cache: torch.Tensor):
    _expect("latent_cache", latent_cache, torch.bfloat16, 3, latent_cache.device)
    _contiguous("latent_cache", latent_cache)
    if latent_cache.shape[2] != LATENT_DIM + LATENT_ROPE_DIM:
        raise ValueError(f"latent_cache must be [NB, 16, {LATENT_DIM + LATENT_ROPE_DIM}]")
    return latent_cache.device, int(latent_cache.shape[0]), int(latent_cache.shape[1])


def latent_kv_write(latent_cache: torch.Tensor, latent: torch.Tensor, key_rope: torch.Tensor,
                    weight: Optional[torch.Tensor], eps: float, cos_sin: torch.Tensor, positions: torch.Tensor,
                    slot_mapping: torch.Tensor, query_rope_out: Optional[torch.Tensor] = None,
                    query_rope: Optional[torch.Tensor] = None, interleaved: bool = False,
                    device_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Norm latent [T, 512], rotate key_rope [T, 64] and store both in latent_cache [NB, 16, 576]; rotate
    query_rope [T, H, 64] into query_rope_out (which may be query_rope, or a view of the attention's query rows).
    weight is bf16 [512] (None: no norm), cos_sin fp32 [max_position, 64]."""
    dev, nb, bs = _latent_cache(latent_cache)
    bf = torch.bfloat16
    T = int(slot_mapping.shape[0])
    for what, x, width in (("latent", latent, LATENT_DIM), ("key_rope", key_rope, LATENT_ROPE_DIM)):
        _expect(what, x, bf, 2, dev)
        if tuple(x.shape) != (T, width) or x.stride(1) != 1:
            raise ValueError(f"{what} must be [{T}, {width}] with contiguous rows")
    _expect("weight", weight, bf, 1, dev)
    _contiguous("weight", weight, (LATENT_DIM,))
    _expect("cos_sin", cos_sin, torch.float32, 2, dev)
    _contiguous("cos_sin", cos_sin, (cos_sin.shape[0], LATENT_ROPE_DIM))
    for what, x in (("positions", positions), ("slot_mapping", slot_mapping)):
        _expect(what, x, torch.int64, 1, dev)
        _contiguous(what, x, (T,))
    _expect("device_status", device_status, torch.int32, 1, dev)
    if (query_rope is None) != (query_rope_out is None):
        raise ValueError("query_rope and query_rope_out go together")
    H = 0
    q = [None, 0, 0, None, 0, 0]
    if query_rope is not None:
        H = int(query_rope.shape[1])
        for what, x in (("query_rope_out", query_rope_out), ("query_rope", query_rope)):
            _expect(what, x, bf, 3, dev)
            if tuple(x.shape) != (T, H, LATENT_ROPE_DIM) or x.stride(2) != 1:
                raise ValueError(f"{what} must be [{T}, H, {LATENT_ROPE_DIM}] with contiguous rows")
        q = []
        for x in (query_rope_out, query_rope):
            head = _step(x, 1, LATENT_ROPE_DIM)
            q += [_ptr(x), _step(x, 0, max(H - 1, 0) * head + LATENT_ROPE_DIM), head]
    _call(dev, stream, load().pkv_latent_kv_write, _ptr(latent_cache), nb, bs, _ptr(latent),
          _step(latent, 0, LATENT_DIM), _ptr(key_rope), _step(key_rope, 0, LATENT_ROPE_DIM), _ptr(weight),
          float(eps), _ptr(cos_sin),
          int(cos_sin.shape[0]), 1 if interleaved else 0, _ptr(positions), _ptr(slot_mapping), T, *q, H,
          _ptr(device_status))


def _tables(dev, block_tables, S, **lists) -> None:
    _expect("block_tables", block_tables, torch.int32, 2, dev)
    _contiguous("block_tables", block_tables)
    if block_tables.shape[0] != S:
        raise ValueError("block_tables must have a row per request")
    for what, x in lists.items():
        _expect(what, x, torch.int32, 1, dev)
        _contiguous(what, x)


def latent_gather(out: torch.Tensor, latent_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                  key_start_loc: torch.Tensor, max_seq_len: int, device_status: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    """Copy the cached rows of request r into out[key_start_loc[r]:][:seq_lens[r]] (bf16 [rows, 576])."""
    dev, nb, bs = _latent_cache(latent_cache)
    S = int(seq_lens.shape[0])
    _tables(dev, block_tables, S, seq_lens=seq_lens, key_start_loc=key_start_loc)
    if key_start_loc.shape[0] < S:
        raise ValueError("key_start_loc must have an entry per request")
    _expect("out", out, torch.bfloat16, 2, dev)
    _contiguous("out", out, (out.shape[0], LATENT_DIM + LATENT_ROPE_DIM))
    _expect("device_status", device_status, torch.int32, 1, dev)
    _call(dev, stream, load().pkv_latent_gather, _ptr(out), int(out.shape[0]), _ptr(latent_cache), nb, bs,
          _ptr(block_tables), int(block_tables.shape[1]), _ptr(seq_lens), _ptr(key_start_loc), S, int(max_seq_len),
          _ptr(device_status))


def latent_paged_attn_workspace_size(num_seqs: int, num_tokens: int, max_query_len: int, max_seq_len: int,
                                     num_heads: int) -> int:
    """Bytes of workspace pkv_latent_paged_attn needs for these sizes (no GPU work)."""
    need = ctypes.c_size_t(0)
    rc = load().pkv_latent_paged_attn(None, None, num_heads * (LATENT_DIM + LATENT_ROPE_DIM), None, 1, None,
                                      (max_seq_len + BLOCK_SIZE - 1) // BLOCK_SIZE, None, None, num_seqs, num_tokens,
                                      max_query_len, max_seq_len, num_heads, BLOCK_SIZE, 1.0, None, 0,
                                      ctypes.byref(need), None)
    if rc not in (0, 5):
        _check(rc, "pkv_latent_paged_attn (size query)")
    return int(need.value)


def latent_paged_attn(out: torch.Tensor, query: torch.Tensor, latent_cache: torch.Tensor, block_tables: torch.Tensor,
                      seq_lens: torch.Tensor, query_start_loc: torch.Tensor, max_query_len: int, max_seq_len: int,
                      scale: float, workspace: torch.Tensor, stream=None) -> None:
    """Causal attention of query [T, H, 576] over the latent cache [NB, 16, 576]; out [T, H, 512] bf16.

    One call (no combine after it); workspace_status(workspace) reads its device status."""
    dev, nb, bs = _latent_cache(latent_cache)
    S = int(seq_lens.shape[0])
    _tables(dev, block_tables, S, seq_lens=seq_lens, query_start_loc=query_start_loc)
    if query_start_loc.shape[0] != S + 1:
        raise ValueError("query_start_loc must have an entry per request and one more")
    _expect("query", query, torch.bfloat16, 3, dev)
    T, H, D = query.shape
    if D != LATENT_DIM + LATENT_ROPE_DIM or query.stride(2) != 1 or (H > 1 and query.stride(1) != D):
        raise ValueError(f"query must be [T, H, {LATENT_DIM + LATENT_ROPE_DIM}] with contiguous heads")
    _expect("out", out, torch.bfloat16, 3, dev)
    _contiguous("out", out, (T, H, LATENT_DIM))
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    _call(dev, stream, load().pkv_latent_paged_attn, _ptr(out), _ptr(query), _step(query, 0, H * D),
          _ptr(latent_cache), nb, _ptr(block_tables), int(block_tables.shape[1]), _ptr(seq_lens),
          _ptr(query_start_loc), S, T, int(max_query_len), int(max_seq_len), H, bs, float(scale), _ptr(workspace),
          workspace.numel() * workspace.element_size(), None)


_NOPE, _VALUE = 128, 128        # plain key dims and value dims of a head in the expanded form


def latent_attn_expanded(out: torch.Tensor, query: torch.Tensor, key: torch.Tensor, key_rope: torch.Tensor,
                         value: torch.Tensor, query_start_loc: torch.Tensor, key_start_loc: torch.Tensor,
                         max_query_len: int, max_key_len: int, scale: float,
                         device_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Causal attention of query [T, H, 192] over key [K, H, 128], key_rope [K, 64] (shared by the heads) and
    value [K, H, 128], requests side by side; out [T, H, 128] bf16."""
    dev, bf = query.device, torch.bfloat16
    _expect("query", query, bf, 3, dev)
    T, H, D = query.shape
    if D != _NOPE + LATENT_ROPE_DIM or query.stride(2) != 1 or (H > 1 and query.stride(1) != D):
        raise ValueError(f"query must be [T, H, {_NOPE + LATENT_ROPE_DIM}] with contiguous heads")
    _expect("key_rope", key_rope, bf, 2, dev)
    K = int(key_rope.shape[0])
    for what, x, width in (("key", key, _NOPE), ("value", value, _VALUE)):
        _expect(what, x, bf, 3, dev)
        if tuple(x.shape) != (K, H, width) or x.stride(2) != 1:
            raise ValueError(f"{what} must be [{K}, {H}, {width}] with contiguous rows")
    if key_rope.shape[1] != LATENT_ROPE_DIM or key_rope.stride(1) != 1:
        raise ValueError(f"key_rope must be [K, {LATENT_ROPE_DIM}] with contiguous rows")
    _expect("out", out, bf, 3, dev)
    _contiguous("out", out, (T, H, _VALUE))
    S = int(query_start_loc.shape[0]) - 1
    for what, x in (("query_start_loc", query_start_loc), ("key_start_loc", key_start_loc)):
        _expect(what, x, torch.int32, 1, dev)
        _contiguous(what, x, (S + 1,))
    _expect("device_status", device_status, torch.int32, 1, dev)
    kh, vh = _step(key, 1, _NOPE), _step(value, 1, _VALUE)
    _call(dev, stream, load().pkv_latent_attn_expanded, _ptr(out), _ptr(query), _step(query, 0, H * D),
          _ptr(key), _step(key, 0, _NOPE), kh, _ptr(key_rope), _step(key_rope, 0, LATENT_ROPE_DIM), _ptr(value),
          _step(value, 0, _VALUE), vh, _ptr(query_start_loc), _ptr(key_start_loc), S, T, K, int(max_query_len),
          int(max_key_len), H, float(scale), _ptr(device_status))
