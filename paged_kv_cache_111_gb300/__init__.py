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
#
# These calls stand in a decode step of some microseconds, so their checks read each property of a tensor once and
# pass plain integers on: the device index (-1 on the CPU, so one comparison also refuses CPU tensors), the type, the
# shape and the strides.

_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
_ROW = LATENT_DIM + LATENT_ROPE_DIM
_NOPE, _VALUE = 128, 128        # plain key dims and value dims of a head in the expanded form
_QK = _NOPE + LATENT_ROPE_DIM


def _refuse(what: str, x: torch.Tensor, dtype, dev: int, form: str) -> None:
    """The reason why a tensor argument does not do."""
    if not x.is_cuda:
        raise ValueError("paged KV-cache calls take CUDA tensors only")
    if x.get_device() != dev:
        raise ValueError(f"{what} is on {x.device}, the call's other tensors on cuda:{dev}")
    if dtype is not None and x.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, not {x.dtype}")
    raise ValueError(f"{what} must be {form}, not {list(x.shape)} with strides {list(x.stride())}")


def _full(what: str, x: Optional[torch.Tensor], dtype, dev: int, shape: tuple, form: str) -> Optional[int]:
    """Pointer of a contiguous tensor of this type and shape (-1: any size), or None."""
    if x is None:
        return None
    if x.get_device() != dev or x.dtype is not dtype or not x.is_contiguous():
        _refuse(what, x, dtype, dev, form)
    have = x.shape
    if have != shape:
        if len(have) != len(shape):
            _refuse(what, x, dtype, dev, form)
        for a, b in zip(have, shape):
            if a != b and b >= 0:
                _refuse(what, x, dtype, dev, form)
    return x.data_ptr()


def _heads(what: str, x: torch.Tensor, dev: int, T: int, H: int, width: int, packed: bool):
    """(pointer, token stride, head stride) of bf16 [T, H, width] with contiguous rows; packed: heads side by side.

    The stride of a dim of one entry, which means nothing, is given as the least that the call takes."""
    if x.get_device() != dev or x.dtype is not _BF16 or x.shape != (T, H, width):
        _refuse(what, x, _BF16, dev, f"[{T}, {H}, {width}]")
    token, head, one = x.stride()
    if H <= 1:
        head = width
    if one != 1 or (packed and head != width):
        _refuse(what, x, _BF16, dev, f"[{T}, {H}, {width}] with contiguous " + ("heads" if packed else "rows"))
    if T <= 1:
        token = max((H - 1) * head + width, 0)
    return x.data_ptr(), token, head


def _tokens(what: str, x: torch.Tensor, dev: int, T: int, width: int):
    """(pointer, token stride) of bf16 [T, width] with contiguous rows."""
    if x.get_device() != dev or x.dtype is not _BF16 or x.shape != (T, width):
        _refuse(what, x, _BF16, dev, f"[{T}, {width}]")
    token, one = x.stride()
    if one != 1:
        _refuse(what, x, _BF16, dev, f"[{T}, {width}] with contiguous rows")
    return x.data_ptr(), (token if T > 1 else width)


def _latent_cache(x: torch.Tensor):
    """(pointer, device, blocks, block size) of a latent cache."""
    dev = x.get_device()
    if dev < 0 or x.dtype is not _BF16 or x.dim() != 3 or not x.is_contiguous() or x.shape[2] != _ROW:
        _refuse("latent_cache", x, _BF16, dev, f"a contiguous [NB, 16, {_ROW}]")
    nb, bs, _ = x.shape
    return x.data_ptr(), dev, nb, bs


def _raw_stream(dev: int, stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _call(dev: int, name: str, fn, *args) -> None:
    """The C call, with the tensors' device current."""
    if torch._C._cuda_getDevice() == dev:
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc != 0:
        raise PagedKVError(rc, name)


def _qk_norm_rope(fp8: bool, query_out, kv_cache, query, key, value, q_weight, k_weight, eps, cos_sin, positions,
                  slot_mapping, scales, interleaved, device_status, stream) -> None:
    dev = kv_cache.get_device()
    if (dev < 0 or kv_cache.dim() != 5 or not kv_cache.is_contiguous()
            or (kv_cache.element_size() != 1 if fp8 else kv_cache.dtype is not _BF16)):
        _refuse("kv_cache", kv_cache, None if fp8 else _BF16, dev, "a contiguous [NB, Hkv, 2, 16, d], "
                + ("one byte per element" if fp8 else "bf16"))
    nb, hkv, two, bs, d = kv_cache.shape
    if two != 2 or query.dim() != 3:
        raise ValueError("kv_cache must be [NB, Hkv, 2, 16, d] and query [T, H, d]")
    T, H, _ = query.shape
    qo, qo_step, _ = _heads("query_out", query_out, dev, T, H, d, True)
    q, q_step, _ = _heads("query", query, dev, T, H, d, True)
    k, k_step, _ = _heads("key", key, dev, T, hkv, d, True)
    v, v_step, _ = _heads("value", value, dev, T, hkv, d, True)
    table = _full("cos_sin", cos_sin, _F32, dev, (-1, -1), "a contiguous [max_position, rotary_dim]")
    max_position, rot = cos_sin.shape
    name = "pkv_qk_norm_rope_kv_write_fp8" if fp8 else "pkv_qk_norm_rope_kv_write"
    _call(dev, name, getattr(_lib or load(), name),
          qo, qo_step, kv_cache.data_ptr(), nb, H, hkv, d, bs, q, q_step, k, k_step, v, v_step,
          _full("q_weight", q_weight, _BF16, dev, (d,), "[d]"), _full("k_weight", k_weight, _BF16, dev, (d,), "[d]"),
          eps, table, max_position, rot, 1 if interleaved else 0,
          _full("positions", positions, _I64, dev, (T,), "a contiguous [T]"),
          _full("slot_mapping", slot_mapping, _I64, dev, (T,), "a contiguous [T]"), T, *scales,
          _full("device_status", device_status, _I32, dev, (-1,), "a contiguous vector"), _raw_stream(dev, stream))


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
                  slot_mapping, (k_scale, v_scale), interleaved, device_status, stream)


def latent_kv_write(latent_cache: torch.Tensor, latent: torch.Tensor, key_rope: torch.Tensor,
                    weight: Optional[torch.Tensor], eps: float, cos_sin: torch.Tensor, positions: torch.Tensor,
                    slot_mapping: torch.Tensor, query_rope_out: Optional[torch.Tensor] = None,
                    query_rope: Optional[torch.Tensor] = None, interleaved: bool = False,
                    device_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Norm latent [T, 512], rotate key_rope [T, 64] and store both in latent_cache [NB, 16, 576]; rotate
    query_rope [T, H, 64] into query_rope_out (which may be query_rope, or a view of the attention's query rows).
    weight is bf16 [512] (None: no norm), cos_sin fp32 [max_position, 64]."""
    cache, dev, nb, bs = _latent_cache(latent_cache)
    T = slot_mapping.numel()
    lat, lat_step = _tokens("latent", latent, dev, T, LATENT_DIM)
    kr, kr_step = _tokens("key_rope", key_rope, dev, T, LATENT_ROPE_DIM)
    if query_rope is None and query_rope_out is None:
        H, q = 0, (None, 0, 0, None, 0, 0)
    elif query_rope is None or query_rope_out is None or query_rope.dim() != 3:
        raise ValueError(f"query_rope and query_rope_out go together, [T, H, {LATENT_ROPE_DIM}] both")
    else:
        H = query_rope.shape[1]
        q = (_heads("query_rope_out", query_rope_out, dev, T, H, LATENT_ROPE_DIM, False)
             + _heads("query_rope", query_rope, dev, T, H, LATENT_ROPE_DIM, False))
    _call(dev, "pkv_latent_kv_write", (_lib or load()).pkv_latent_kv_write, cache, nb, bs, lat, lat_step, kr, kr_step,
          _full("weight", weight, _BF16, dev, (LATENT_DIM,), f"[{LATENT_DIM}]"), eps,
          _full("cos_sin", cos_sin, _F32, dev, (-1, LATENT_ROPE_DIM),
                f"a contiguous [max_position, {LATENT_ROPE_DIM}]"), cos_sin.shape[0],
          1 if interleaved else 0, _full("positions", positions, _I64, dev, (T,), "a contiguous [T]"),
          _full("slot_mapping", slot_mapping, _I64, dev, (T,), "a contiguous [T]"), T, *q, H,
          _full("device_status", device_status, _I32, dev, (-1,), "a contiguous vector"), _raw_stream(dev, stream))


def latent_gather(out: torch.Tensor, latent_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                  key_start_loc: torch.Tensor, max_seq_len: int, device_status: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    """Copy the cached rows of request r into out[key_start_loc[r]:][:seq_lens[r]] (bf16 [rows, 576])."""
    cache, dev, nb, bs = _latent_cache(latent_cache)
    S = seq_lens.numel()
    if key_start_loc.numel() < S:
        raise ValueError("key_start_loc must have an entry per request")
    _call(dev, "pkv_latent_gather", (_lib or load()).pkv_latent_gather,
          _full("out", out, _BF16, dev, (-1, _ROW), f"a contiguous [rows, {_ROW}]"), out.shape[0], cache, nb, bs,
          _full("block_tables", block_tables, _I32, dev, (S, -1), "a contiguous [num_seqs, max_blocks]"),
          block_tables.shape[1], _full("seq_lens", seq_lens, _I32, dev, (S,), "a contiguous [num_seqs]"),
          _full("key_start_loc", key_start_loc, _I32, dev, (-1,), "a contiguous vector"), S, max_seq_len,
          _full("device_status", device_status, _I32, dev, (-1,), "a contiguous vector"), _raw_stream(dev, stream))


def latent_paged_attn_workspace_size(num_seqs: int, num_tokens: int, max_query_len: int, max_seq_len: int,
                                     num_heads: int) -> int:
    """Bytes of workspace pkv_latent_paged_attn needs for these sizes (no GPU work)."""
    need = ctypes.c_size_t(0)
    rc = load().pkv_latent_paged_attn(None, None, num_heads * _ROW, None, 1, None,
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
    cache, dev, nb, bs = _latent_cache(latent_cache)
    S = seq_lens.numel()
    if query.dim() != 3:
        raise ValueError(f"query must be [T, H, {_ROW}]")
    T, H, _ = query.shape
    q, q_step, _ = _heads("query", query, dev, T, H, _ROW, True)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse("workspace", workspace, None, dev, "contiguous")
    _call(dev, "pkv_latent_paged_attn", (_lib or load()).pkv_latent_paged_attn,
          _full("out", out, _BF16, dev, (T, H, LATENT_DIM), f"a contiguous [T, H, {LATENT_DIM}]"), q, q_step, cache, nb,
          _full("block_tables", block_tables, _I32, dev, (S, -1), "a contiguous [num_seqs, max_blocks]"),
          block_tables.shape[1], _full("seq_lens", seq_lens, _I32, dev, (S,), "a contiguous [num_seqs]"),
          _full("query_start_loc", query_start_loc, _I32, dev, (S + 1,), "a contiguous [num_seqs + 1]"), S, T,
          max_query_len, max_seq_len, H, bs, scale, workspace.data_ptr(), workspace.nbytes, None,
          _raw_stream(dev, stream))


def latent_attn_expanded(out: torch.Tensor, query: torch.Tensor, key: torch.Tensor, key_rope: torch.Tensor,
                         value: torch.Tensor, query_start_loc: torch.Tensor, key_start_loc: torch.Tensor,
                         max_query_len: int, max_key_len: int, scale: float,
                         device_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Causal attention of query [T, H, 192] over key [K, H, 128], key_rope [K, 64] (shared by the heads) and
    value [K, H, 128], requests side by side; out [T, H, 128] bf16."""
    dev = query.get_device()
    if dev < 0 or query.dim() != 3:
        _refuse("query", query, _BF16, dev, f"[T, H, {_QK}]")
    T, H, _ = query.shape
    K = key_rope.shape[0]
    S = query_start_loc.numel() - 1
    q, q_step, _ = _heads("query", query, dev, T, H, _QK, True)
    _call(dev, "pkv_latent_attn_expanded", (_lib or load()).pkv_latent_attn_expanded,
          _full("out", out, _BF16, dev, (T, H, _VALUE), f"a contiguous [T, H, {_VALUE}]"), q, q_step,
          *_heads("key", key, dev, K, H, _NOPE, False), *_tokens("key_rope", key_rope, dev, K, LATENT_ROPE_DIM),
          *_heads("value", value, dev, K, H, _VALUE, False),
          _full("query_start_loc", query_start_loc, _I32, dev, (S + 1,), "a contiguous [num_seqs + 1]"),
          _full("key_start_loc", key_start_loc, _I32, dev, (S + 1,), "a contiguous [num_seqs + 1]"), S, T, K,
          max_query_len, max_key_len, H, scale,
          _full("device_status", device_status, _I32, dev, (-1,), "a contiguous vector"), _raw_stream(dev, stream))
