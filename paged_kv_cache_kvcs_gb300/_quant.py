"""Torch front ends of the operators that write 8-bit caches and read cached
tokens back: ``kvcs_write_kv_quantised`` and ``kvcs_read_kv``.

Argument checks and marshalling only, as in ``_binding``.
"""

from __future__ import annotations

import ctypes

import torch

from . import _attention as A
from . import _binding as B


def _rows(name: str, tensors, caches, n: int, element: int, dtype, index: int):
    """Pointers of one tensor per cache, and the elements between their rows
    (0: packed): 16-bit ``[rows >= n, heads, elements]`` of one dtype, rows
    strided alike."""
    ptrs = []
    stride = None
    for c, t in zip(caches, tensors):
        if t is None:
            ptrs.append(None)
            continue
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype):
            raise ValueError(f"{name} must be CUDA tensors of one 16-bit dtype")
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{index}")
        heads, dim = c.num_heads, c.head_bytes // element
        shape, steps = t.shape, t.stride()
        if len(shape) == 2 and heads == 1:
            shape, steps = (shape[0], 1, shape[1]), (steps[0], dim, steps[1])
        if len(shape) != 3 or shape[1] != heads or shape[2] != dim or shape[0] < n:
            raise ValueError(f"{name} must be [{n}, {heads}, {dim}]")
        row = steps[0]
        if n > 0 and (steps[2] != 1 or (heads > 1 and steps[1] != dim)
                      or (n > 1 and row < heads * dim)):
            raise ValueError(f"{name}'s heads must be packed within a token")
        if n <= 1 or row == heads * dim:
            row = 0
        if row != stride:
            if stride is not None:
                raise ValueError(f"{name}'s rows must be strided alike in all caches")
            stride = row
        ptrs.append(t.data_ptr())
    return (ctypes.c_void_p * len(ptrs))(*ptrs), stride or 0


def _quantisation(caches, block_size, kv_dtype, dtype, k_scales, v_scales, k_scale, v_scale, index):
    """A kvcs_quantisation without strides."""
    kv = A._KV_DTYPES.get(kv_dtype)
    if kv is None:
        raise ValueError("kv_dtype must be torch.int8, torch.float8_e4m3fn or a 16-bit dtype")
    if dtype not in A._Q_DTYPES:
        raise ValueError("keys and values must be torch.bfloat16 or torch.float16")
    q = B.kvcs_quantisation(kv, A._Q_DTYPES[dtype], None, None, k_scale, v_scale, 0, 0)
    for name, given in (("k_scales", k_scales), ("v_scales", v_scales)):
        if given is None:
            continue
        setattr(q, name, (ctypes.c_void_p * len(caches))(*[      # (which keeps it)
            None if t is None else A._scales(name, t, c, block_size, index)
            for c, t in zip(caches, given)]))
    return q


def _listed(where: str, caches, *given):
    """The caches as a list, and what goes with them as lists or None."""
    if isinstance(caches, (list, tuple)):
        if not caches:
            raise B.KvcsError(B.KVCS_EINVAL, where)
        for g in given:
            if g is not None and len(g) != len(caches):
                raise ValueError("keys, values and scales must hold one tensor per cache")
        return (caches, *given)
    return ([caches], *(None if g is None else [g] for g in given))


def write_kv_quantised(caches, block_size: int, keys, values, slot_mapping, positions, *, kv_dtype,
                       k_scales=None, v_scales=None, k_scale: float = 1.0, v_scale: float = 1.0,
                       block_sums=None, status=None, stream=None) -> None:
    """Torch front end of ``kvcs_write_kv_quantised`` over one cache or a list
    of caches: ``write_kv`` of bfloat16 or float16 ``keys`` and ``values``
    (``[num_tokens, heads, elements]``, rows may be strided, as slices of a
    fused projection are; ``values`` None for latent caches), stored as
    ``kv_dtype`` (``torch.int8`` or ``torch.float8_e4m3fn``).  ``k_scales`` and
    ``v_scales`` (one float32 tensor ``[num_blocks, num_heads, block_size]``
    per cache) get each token's and head's scale; without them ``k_scale`` and
    ``v_scale`` are the scales of all (float8 only).  ``block_sums`` cover the
    caches' bytes, not the scales."""
    caches, keys, values, k_scales, v_scales = _listed("kvcs_write_kv_quantised", caches, keys, values,
                                                       k_scales, v_scales)
    n = slot_mapping.numel()
    dev = B._current_device()
    index = dev.index
    arr = A._packed(caches, block_size, index)
    if positions.numel() != n:
        raise ValueError("positions and slot_mapping differ in length")
    slots = A._checked("slot_mapping", slot_mapping, torch.int64, n, index)
    pos = A._checked("positions", positions, torch.int64, n, index)
    if keys is None or any(k is None for k in keys):
        raise ValueError("keys must hold one tensor per cache")
    dtype = getattr(keys[0], "dtype", None)
    q = _quantisation(caches, block_size, kv_dtype, dtype, k_scales, v_scales, k_scale, v_scale, index)
    kp, q.key_stride = _rows("keys", keys, caches, n, 1, dtype, index)
    vp = None
    if values is not None:
        vp, q.value_stride = _rows("values", values, caches, n, 1, dtype, index)
    if block_sums is not None:
        B._check_tensor("block_sums", block_sums, B._words(), min(c.num_blocks for c in caches), dev)
    B._check_status(status, dev)
    A._raise(B.load_library().kvcs_write_kv_quantised(
        arr, len(caches), block_size, n, kp, vp, slots if n else None,
        pos if n else None, ctypes.byref(q), B._ptr(block_sums), B._ptr(status),
        A._stream_handle(stream, dev)), "kvcs_write_kv_quantised")


def read_kv(caches, block_size: int, pos_offsets, first_position, num_tokens, block_ids,
            token_offsets, *, keys=None, values=None, dtype=torch.bfloat16, kv_dtype=None,
            k_scales=None, v_scales=None, k_scale: float = 1.0, v_scale: float = 1.0,
            total_tokens: int | None = None, status=None, stream=None,
            total_positions: int | None = None):
    """Torch front end of ``kvcs_read_kv``: reads tokens of one cache or a list
    of caches back into bfloat16 or float16 ``[total_tokens, heads, elements]``
    tensors.  Request r's last ``token_offsets[r+1] - token_offsets[r]`` tokens
    are its rows (``token_offsets``: int64 CUDA, num_requests + 1).
    ``kv_dtype`` (by default the pools' own dtype) and scales as in
    ``write_kv_quantised``; 16-bit caches are read too.  ``keys`` and
    ``values`` (rows may be strided) are allocated, as ``dtype``, on the stream
    that the call runs on if not given.

    Returns ``(keys, values)``: tensors for one cache, lists for a list;
    ``values`` None for latent caches."""
    one = not isinstance(caches, (list, tuple))
    caches, keys, values, k_scales, v_scales = _listed("kvcs_read_kv", caches, keys, values, k_scales,
                                                       v_scales)
    reqs, R, total, index = A._tables(pos_offsets, first_position, num_tokens, block_ids,
                                      total_positions)
    dev = B._current_device()
    arr = A._packed(caches, block_size, index)
    at = A._checked("token_offsets", token_offsets, torch.int64, R + 1, index)
    if token_offsets.numel() != R + 1:
        raise ValueError(f"token_offsets must hold num_requests + 1 elements ({R + 1})")
    if kv_dtype is None:
        kv_dtype = getattr(caches[0].pool, "dtype", None)
    if keys is not None:
        if any(k is None for k in keys):
            raise ValueError("keys must hold one tensor per cache")
        dtype = getattr(keys[0], "dtype", None)
    q = _quantisation(caches, block_size, kv_dtype, dtype, k_scales, v_scales, k_scale, v_scale, index)
    if total_tokens is None:
        total_tokens = keys[0].shape[0] if keys is not None else int(token_offsets[-1].item())
    B._check_status(status, dev)
    element = 1 if q.kv_dtype in (B.KVCS_DTYPE_FP8_E4M3, B.KVCS_DTYPE_INT8) else 2
    handle = A._stream_handle(stream, dev)

    def room(c):
        return A._empty((total_tokens, c.num_heads, c.head_bytes // element), dtype, stream, handle, dev)

    if keys is None:
        keys = [room(c) for c in caches]
    if values is None and any(c.layout != B.KVCS_LAYOUT_LATENT for c in caches):
        values = [None if c.layout == B.KVCS_LAYOUT_LATENT else room(c) for c in caches]
    kp, q.key_stride = _rows("keys", keys, caches, total_tokens, element, dtype, index)
    vp = None
    if values is not None:
        vp, q.value_stride = _rows("values", values, caches, total_tokens, element, dtype, index)
    A._raise(B.load_library().kvcs_read_kv(
        arr, len(caches), block_size, ctypes.byref(reqs), total, at, total_tokens,
        kp, vp, ctypes.byref(q), B._ptr(status), handle), "kvcs_read_kv")
    if one:
        return keys[0], None if values is None else values[0]
    return keys, values
