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


def _checked(name: str, t, dtype, n: int, index: int):
    """The address of ``t`` after ``_binding._check_tensor``'s checks (made
    here first in the shortest way: a decode step makes a dozen of them)."""
    if type(t) is torch.Tensor and t.is_cuda and t.dtype is dtype and t.numel() >= n and \
            t.is_contiguous() and t.get_device() == index:
        return t.data_ptr()
    B._check_tensor(name, t, (dtype,), n, torch.device("cuda", index))
    return t.data_ptr()


def _tables(pos_offsets, first_position, num_tokens, block_ids, total_positions):
    """The checked request table, its request count and position count, and
    the current device's index."""
    total = _total(total_positions, pos_offsets)
    index = B._current_device().index
    R = pos_offsets.numel() - 1
    if not (type(pos_offsets) is type(num_tokens) is type(first_position) is torch.Tensor
            and num_tokens.numel() == R == first_position.numel() and total >= 0):
        B._check_requests(pos_offsets, first_position, num_tokens, block_ids, total)
    i64 = torch.int64
    reqs = B.kvcs_requests(R, _checked("pos_offsets", pos_offsets, i64, max(R, 0) + 1, index),
                           _checked("first_position", first_position, i64, R, index),
                           _checked("num_tokens", num_tokens, i64, R, index),
                           _checked("block_ids", block_ids, torch.int32, total, index))
    return reqs, R, total, index


def _total(total_positions, pos_offsets) -> int:
    if total_positions is not None:
        return total_positions
    if not getattr(pos_offsets, "is_cuda", False) or pos_offsets.numel() < 1:
        raise ValueError("pos_offsets must be a CUDA int64 tensor of num_requests + 1")
    return int(pos_offsets[-1].item())


def _raise(rc: int, where: str) -> None:
    if rc != B.KVCS_OK:
        raise B.KvcsError(rc, where)


def _empty(shape, dtype, stream, handle: int, dev):
    """A tensor that belongs to the stream the call writes it on."""
    if stream is None or handle == torch.cuda.current_stream(dev).cuda_stream:
        return torch.empty(shape, dtype=dtype, device=dev)
    # (a handle of 0 is no external stream to torch: it would make one of its own)
    owner = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    with torch.cuda.stream(owner):
        return torch.empty(shape, dtype=dtype, device=dev)


def _workspace(given, n: int, stream, handle: int, dev):
    """The caller's workspace, checked, or one of ``n`` bytes (freed on
    return: its memory goes back to the stream that uses it)."""
    if given is None:
        return _empty(n, torch.uint8, stream, handle, dev)
    B._check_tensor("workspace", given, (torch.uint8,), n, dev)
    return given


def _attention_args(cache, q, new_offsets, R, index, kv_dtype, scale, softcap, window, k_scale,
                    v_scale, max_new, out=None, lse=None, observe=0):
    """Checks q and new_offsets and packs a kvcs_attention."""
    if not (getattr(q, "is_cuda", False) and q.dim() == 3):
        raise ValueError("q must be a CUDA tensor [total_new, q_heads, head_dim]")
    q_dtype = _Q_DTYPES.get(q.dtype)
    if q_dtype is None:
        raise ValueError("q must be a torch.bfloat16 or torch.float16 tensor")
    if q.device.index != index:
        raise ValueError(f"q is on {q.device}, the call runs on cuda:{index}")
    total_new, q_heads, dim = q.shape
    if kv_dtype is None:
        pool = getattr(cache.pool, "dtype", torch.uint8)
        kv_dtype = pool if pool in _KV_DTYPES else q.dtype
    kv = _KV_DTYPES.get(kv_dtype)
    if kv is None:
        raise ValueError("kv_dtype must be torch.bfloat16, torch.float16 or torch.float8_e4m3fn")
    element = 1 if kv == B.KVCS_DTYPE_FP8_E4M3 else 2
    if dim * element != cache.head_bytes:
        raise ValueError(f"q has heads of {dim} elements, the cache of "
                         f"{cache.head_bytes // element}")
    row, head, step = q.stride(0), q.stride(1), q.stride(2)
    if total_new > 0 and (step != 1 or (q_heads > 1 and head != dim)
                          or (total_new > 1 and row < q_heads * dim)):
        raise ValueError("q's heads must be packed within a token")
    new = _checked("new_offsets", new_offsets, torch.int64, R + 1, index)
    if new_offsets.numel() != R + 1:
        raise ValueError(f"new_offsets must hold num_requests + 1 elements ({R + 1})")
    return B.kvcs_attention(
        q.data_ptr(), row if total_new > 1 else 0, new, total_new,
        0 if max_new is None else min(max_new, total_new), q_heads, q_dtype, kv,
        dim ** -0.5 if scale is None else scale, softcap, k_scale, v_scale, window, out, lse, None,
        0, observe)


def attention_workspace_bytes(cache, block_size: int, num_requests: int, total_positions: int, q,
                              *, max_new=None, kv_dtype=None) -> int:
    """Bytes of workspace ``paged_attention`` needs for ``num_requests``
    requests of ``total_positions`` blocks and queries like ``q``
    (``kvcs_attention_workspace``)."""
    dev = B._current_device()
    offsets = torch.empty(num_requests + 1, dtype=torch.int64, device=dev)
    a = _attention_args(cache, q, offsets, num_requests, dev.index, kv_dtype, None, 0.0, 0, 1.0, 1.0,
                        max_new)
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
    tokens of a request, lets a decode step take a single kernel.
    ``workspace`` is a CUDA uint8 tensor of ``attention_workspace_bytes``.
    What is not given (``out``, ``lse``, ``workspace``) is allocated on the
    stream that the call runs on.

    Returns ``(out, lse)``: ``out`` like a packed ``q``, ``lse`` float32
    ``[total_new, q_heads]``.
    """
    B._check_pool(cache, block_size)
    reqs, R, total, index = _tables(pos_offsets, first_position, num_tokens, block_ids,
                                    total_positions)
    a = _attention_args(cache, q, new_offsets, R, index, kv_dtype, scale, softcap, window, k_scale,
                        v_scale, max_new)
    dev = q.device
    if out is not None:
        a.out = _checked("out", out, q.dtype, q.numel(), index)
    if lse is not None:
        a.lse = _checked("lse", lse, torch.float32, q.shape[0] * q.shape[1], index)
    B._check_status(status, dev)
    lib = B.load_library()
    arr = B.cache_array((cache,))
    n = ctypes.c_int64()
    a_ref = ctypes.byref(a)
    _raise(lib.kvcs_attention_workspace(arr, block_size, R, total, a_ref, 0, ctypes.byref(n)),
           "kvcs_attention_workspace")
    handle = _stream_handle(stream, dev)
    if out is None:
        out = _empty(q.shape, q.dtype, stream, handle, dev)
        a.out = out.data_ptr()
    if lse is None:
        lse = _empty(q.shape[:2], torch.float32, stream, handle, dev)
        a.lse = lse.data_ptr()
    workspace = _workspace(workspace, n.value, stream, handle, dev)
    a.workspace = workspace.data_ptr()
    a.workspace_bytes = workspace.numel()
    _raise(lib.kvcs_paged_attention(arr, block_size, ctypes.byref(reqs), total, a_ref,
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
    reqs, R, total, index = _tables(pos_offsets, first_position, num_tokens, block_ids,
                                    total_positions)
    a = _attention_args(cache, q, new_offsets, R, index, kv_dtype, scale, softcap, window, k_scale,
                        1.0, max_new, observe=observe)
    a.lse = _checked("lse", lse, torch.float32, q.shape[0] * q.shape[1], index)
    at = _checked("mass", mass, torch.float32, cache.num_blocks * cache.num_heads * block_size, index)
    B._check_status(status, q.device)
    _raise(B.load_library().kvcs_attention_mass(
        B.cache_array((cache,)), block_size, ctypes.byref(reqs), total, ctypes.byref(a), at,
        B._ptr(status), _stream_handle(stream, q.device)), "kvcs_attention_mass")
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
    reqs, R, total, index = _tables(pos_offsets, first_position, num_tokens, block_ids,
                                    total_positions)
    dev = torch.device("cuda", index)
    at = [_checked("scores", t, torch.float32, c.num_blocks * c.num_heads * block_size, index)
          for c, t in zip(caches, scores)]
    ev = B.kvcs_eviction((ctypes.c_void_p * max(1, len(caches)))(*at),
                         _checked("keep", keep, torch.int64, R, index), sinks, recent, None, None,
                         None, 0)
    if new_block_ids is not None:
        ev.new_block_ids = _checked("new_block_ids", new_block_ids, torch.int32, total, index)
    if block_sums is not None:
        B._check_tensor("block_sums", block_sums, B._words(),
                        min(c.num_blocks for c in caches), dev)
        ev.block_sums = block_sums.data_ptr()
    B._check_status(status, dev)
    lib, arr = B.load_library(), B.cache_array(caches)
    n = ctypes.c_int64()
    _raise(lib.kvcs_eviction_workspace(arr, len(caches), block_size, R, total, ctypes.byref(n)),
           "kvcs_eviction_workspace")
    handle = _stream_handle(stream, dev)
    workspace = _workspace(workspace, n.value, stream, handle, dev)
    ev.workspace = workspace.data_ptr()
    ev.workspace_bytes = workspace.numel()
    _raise(lib.kvcs_evict(arr, len(caches), block_size, ctypes.byref(reqs), total, ctypes.byref(ev),
                          B._ptr(status), handle), "kvcs_evict")
