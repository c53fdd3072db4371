"""Torch front ends of the operators that read and thin out paged caches:
``kvcs_paged_attention``, ``kvcs_attention_mass`` and ``kvcs_evict``.

Argument checks and marshalling only, as in ``_binding``.
"""

from __future__ import annotations

import ctypes
from typing import Sequence

import torch

from . import _binding as B

_Q_DTYPES = {torch.bfloat16: B.KVCS_DTYPE_BF16, torch.float16: B.KVCS_DTYPE_FP16}
_KV_DTYPES = dict(_Q_DTYPES)
_KV_DTYPES[torch.float8_e4m3fn] = B.KVCS_DTYPE_FP8_E4M3


def _stream_handle(stream, dev) -> int:
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _total(total_positions, pos_offsets) -> int:
    if total_positions is not None:
        return total_positions
    if not getattr(pos_offsets, "is_cuda", False) or pos_offsets.numel() < 1:
        raise ValueError("pos_offsets must be a CUDA int64 tensor of num_requests + 1")
    return int(pos_offsets[-1].item())


def _requests(pos_offsets, first_position, num_tokens, block_ids):
    return B.kvcs_requests(pos_offsets.numel() - 1, pos_offsets.data_ptr(),
                           first_position.data_ptr(), num_tokens.data_ptr(),
                           block_ids.data_ptr())


def _raise(rc: int, where: str) -> None:
    if rc != B.KVCS_OK:
        raise B.KvcsError(rc, where)


def _workspace(given, n: int, stream, handle: int, dev):
    """The caller's workspace, checked, or one of ``n`` bytes."""
    if given is not None:
        B._check_tensor("workspace", given, (torch.uint8,), n, dev)
        return given
    if stream is None or handle == torch.cuda.current_stream(dev).cuda_stream:
        return torch.empty(n, dtype=torch.uint8, device=dev)
    # freed on return: it has to belong to the stream that uses it
    with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=dev)):
        return torch.empty(n, dtype=torch.uint8, device=dev)


def _queries(cache, q, new_offsets, num_requests, kv_dtype, dev):
    """Checks q and new_offsets; returns a kvcs_attention with their fields."""
    if not (getattr(q, "is_cuda", False) and q.dim() == 3):
        raise ValueError("q must be a CUDA tensor [total_new, q_heads, head_dim]")
    if q.dtype not in _Q_DTYPES:
        raise ValueError("q must be a torch.bfloat16 or torch.float16 tensor")
    if q.device != dev:
        raise ValueError(f"q is on {q.device}, the call runs on {dev}")
    total_new, q_heads, dim = q.shape
    if kv_dtype is None:
        pool = getattr(cache.pool, "dtype", torch.uint8)
        kv_dtype = pool if pool in _KV_DTYPES else q.dtype
    if kv_dtype not in _KV_DTYPES:
        raise ValueError("kv_dtype must be torch.bfloat16, torch.float16 or torch.float8_e4m3fn")
    element = 1 if kv_dtype == torch.float8_e4m3fn else 2
    if dim * element != cache.head_bytes:
        raise ValueError(f"q has heads of {dim} elements, the cache of "
                         f"{cache.head_bytes // element}")
    if total_new > 0 and (q.stride(2) != 1 or (q_heads > 1 and q.stride(1) != dim)
                          or (total_new > 1 and q.stride(0) < q_heads * dim)):
        raise ValueError("q's heads must be packed within a token")
    B._check_tensor("new_offsets", new_offsets, (torch.int64,), num_requests + 1, dev)
    if new_offsets.numel() != num_requests + 1:
        raise ValueError(f"new_offsets must hold num_requests + 1 elements ({num_requests + 1})")
    a = B.kvcs_attention()
    a.q = q.data_ptr()
    a.q_stride = q.stride(0) if total_new > 1 else 0
    a.new_offsets = new_offsets.data_ptr()
    a.total_new = total_new
    a.q_heads = q_heads
    a.q_dtype = _Q_DTYPES[q.dtype]
    a.kv_dtype = _KV_DTYPES[kv_dtype]
    return a


def _scores(a, dim, scale, softcap, window, k_scale, v_scale, max_new) -> None:
    a.scale = dim ** -0.5 if scale is None else scale
    a.softcap = softcap
    a.window = window
    a.k_scale = k_scale
    a.v_scale = v_scale
    a.max_new = min(max_new, a.total_new) if max_new is not None else 0


def attention_workspace_bytes(cache, block_size: int, num_requests: int, total_positions: int, q,
                              *, max_new=None, kv_dtype=None) -> int:
    """Bytes of workspace ``paged_attention`` needs for ``num_requests``
    requests of ``total_positions`` blocks and queries like ``q``
    (``kvcs_attention_workspace``)."""
    dev = B._current_device()
    offsets = torch.empty(num_requests + 1, dtype=torch.int64, device=dev)
    a = _queries(cache, q, offsets, num_requests, kv_dtype, dev)
    _scores(a, q.shape[2], None, 0.0, 0, 1.0, 1.0, max_new)
    n = ctypes.c_int64()
    _raise(B.load_library().kvcs_attention_workspace(
        B.cache_array([cache]), block_size, num_requests, total_positions, ctypes.byref(a), 0,
        ctypes.byref(n)),
        "kvcs_attention_workspace")
    return n.value


def paged_attention(cache, block_size: int, pos_offsets, first_position, num_tokens, block_ids,
                    q, new_offsets, *, out=None, lse=None, scale=None, softcap: float = 0.0,
                    window: int = 0, k_scale: float = 1.0, v_scale: float = 1.0, kv_dtype=None,
                    max_new: int | None = None, workspace=None, status=None, stream=None,
                    total_positions: int | None = None):
    """Torch front end of ``kvcs_paged_attention``: attention of the batch's
    new tokens over one layer's paged cache.

    ``q`` is a bfloat16 or float16 CUDA tensor ``[total_new, q_heads,
    head_dim]`` (rows may be strided, as a slice of a fused projection is);
    ``new_offsets`` (int64, num_requests + 1) gives each request's rows, its
    last tokens.  ``kv_dtype`` is what the pool holds: by default the pool's
    own dtype, or q's for a pool of raw bytes.  ``max_new``, the most new
    tokens of a request, lets a decode step take a single launch.
    ``workspace`` is a CUDA uint8 tensor of ``attention_workspace_bytes``
    (by default allocated from the call's stream).

    Returns ``(out, lse)``: ``out`` like a packed ``q``, ``lse`` float32
    ``[total_new, q_heads]``.
    """
    B._check_pool(cache, block_size)
    total_positions = _total(total_positions, pos_offsets)
    dev = B._check_requests(pos_offsets, first_position, num_tokens, block_ids, total_positions)
    R = pos_offsets.numel() - 1
    a = _queries(cache, q, new_offsets, R, kv_dtype, dev)
    _scores(a, q.shape[2], scale, softcap, window, k_scale, v_scale, max_new)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    else:
        B._check_tensor("out", out, (q.dtype,), q.numel(), dev)
    rows = q.shape[0] * q.shape[1]
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev)
    else:
        B._check_tensor("lse", lse, (torch.float32,), rows, dev)
    B._check_status(status, dev)
    a.out = out.data_ptr()
    a.lse = lse.data_ptr()
    lib = B.load_library()
    arr = B.cache_array([cache])
    n = ctypes.c_int64()
    a_ref = ctypes.byref(a)
    _raise(lib.kvcs_attention_workspace(arr, block_size, R, total_positions, a_ref, 0, ctypes.byref(n)),
           "kvcs_attention_workspace")
    handle = _stream_handle(stream, dev)
    workspace = _workspace(workspace, n.value, stream, handle, dev)
    a.workspace = workspace.data_ptr()
    a.workspace_bytes = workspace.numel()
    reqs = _requests(pos_offsets, first_position, num_tokens, block_ids)
    _raise(lib.kvcs_paged_attention(arr, block_size, ctypes.byref(reqs), total_positions, a_ref,
                                    B._ptr(status), handle), "kvcs_paged_attention")
    return out, lse


def attention_mass(cache, block_size: int, pos_offsets, first_position, num_tokens, block_ids,
                   q, new_offsets, lse, mass, *, observe: int = 0, scale=None,
                   softcap: float = 0.0, window: int = 0, k_scale: float = 1.0, kv_dtype=None,
                   max_new: int | None = None, status=None, stream=None,
                   total_positions: int | None = None):
    """Torch front end of ``kvcs_attention_mass``: adds to ``mass`` (float32
    ``[num_blocks, num_heads, block_size]``) the weights that each cached
    token gets from the last ``observe`` new tokens of its request (0: all).
    ``q``, ``new_offsets`` and the score arguments as in ``paged_attention``,
    ``lse`` as that call returned it.  Returns ``mass``."""
    B._check_pool(cache, block_size)
    total_positions = _total(total_positions, pos_offsets)
    dev = B._check_requests(pos_offsets, first_position, num_tokens, block_ids, total_positions)
    R = pos_offsets.numel() - 1
    a = _queries(cache, q, new_offsets, R, kv_dtype, dev)
    _scores(a, q.shape[2], scale, softcap, window, k_scale, 1.0, max_new)
    a.observe = observe
    B._check_tensor("lse", lse, (torch.float32,), q.shape[0] * q.shape[1], dev)
    B._check_tensor("mass", mass, (torch.float32,),
                    cache.num_blocks * cache.num_heads * block_size, dev)
    B._check_status(status, dev)
    a.lse = lse.data_ptr()
    reqs = _requests(pos_offsets, first_position, num_tokens, block_ids)
    _raise(B.load_library().kvcs_attention_mass(
        B.cache_array([cache]), block_size, ctypes.byref(reqs), total_positions, ctypes.byref(a),
        mass.data_ptr(), B._ptr(status), _stream_handle(stream, dev)), "kvcs_attention_mass")
    return mass


def eviction_workspace_bytes(caches: Sequence, block_size: int, num_requests: int,
                             total_positions: int) -> int:
    """Bytes of workspace ``evict`` needs (``kvcs_eviction_workspace``)."""
    n = ctypes.c_int64()
    _raise(B.load_library().kvcs_eviction_workspace(
        B.cache_array(caches), len(caches), block_size, num_requests, total_positions,
        ctypes.byref(n)), "kvcs_eviction_workspace")
    return n.value


def evict(caches: Sequence, block_size: int, pos_offsets, first_position, num_tokens, block_ids,
          scores: Sequence, keep, *, sinks: int = 0, recent: int = 0, new_block_ids=None,
          block_sums=None, workspace=None, status=None, stream=None,
          total_positions: int | None = None) -> None:
    """Torch front end of ``kvcs_evict``: keeps ``keep[r]`` (int64 CUDA) tokens
    of each request in every cache of ``caches``, chosen per KV head by
    ``scores`` (one float32 tensor ``[num_blocks, num_heads, block_size]`` per
    cache), and moves them to the front of the request's blocks, or of
    ``new_block_ids`` (int32, one per position).  ``block_sums`` (one word per
    block) get the filled blocks' checksums.  ``workspace`` is a CUDA uint8
    tensor of ``eviction_workspace_bytes`` (by default allocated)."""
    if not isinstance(caches, (list, tuple)):
        caches, scores = [caches], [scores]
    if len(scores) != len(caches):
        raise ValueError("scores must hold one tensor per cache")
    for c in caches:
        B._check_pool(c, block_size)
    total_positions = _total(total_positions, pos_offsets)
    dev = B._check_requests(pos_offsets, first_position, num_tokens, block_ids, total_positions)
    for c, t in zip(caches, scores):
        B._check_tensor("scores", t, (torch.float32,), c.num_blocks * c.num_heads * block_size, dev)
    B._check_tensor("keep", keep, (torch.int64,), pos_offsets.numel() - 1, dev)
    if new_block_ids is not None:
        B._check_tensor("new_block_ids", new_block_ids, (torch.int32,), total_positions, dev)
    if block_sums is not None:
        B._check_tensor("block_sums", block_sums, B._words(),
                        min(c.num_blocks for c in caches), dev)
    B._check_status(status, dev)
    ptrs = (ctypes.c_void_p * max(1, len(caches)))(*[t.data_ptr() for t in scores])
    lib, arr, R = B.load_library(), B.cache_array(caches), pos_offsets.numel() - 1
    n = ctypes.c_int64()
    _raise(lib.kvcs_eviction_workspace(arr, len(caches), block_size, R, total_positions,
                                       ctypes.byref(n)), "kvcs_eviction_workspace")
    handle = _stream_handle(stream, dev)
    workspace = _workspace(workspace, n.value, stream, handle, dev)
    ev = B.kvcs_eviction(ptrs, keep.data_ptr(), sinks, recent, B._ptr(new_block_ids),
                         B._ptr(block_sums), workspace.data_ptr(), workspace.numel())
    reqs = _requests(pos_offsets, first_position, num_tokens, block_ids)
    _raise(lib.kvcs_evict(arr, len(caches), block_size, ctypes.byref(reqs), total_positions,
                          ctypes.byref(ev), B._ptr(status), handle), "kvcs_evict")
