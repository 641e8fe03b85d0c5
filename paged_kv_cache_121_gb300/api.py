"""Python binding of libpa: one function per C entry point, same names.

Argument marshalling only -- shapes are read off the tensors, pointers and
the current CUDA stream are passed through, and a non-OK status raises
:class:`PAError`. Every computation runs in libpa's kernels (or, for the
block manager and slot map, in its host C++).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import numpy as np
import torch

from . import _lib

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_OUT_OF_BLOCKS = 0, 1, 2, 3
PA_ERR_WORKSPACE, PA_ERR_TIMEOUT, PA_ERR_CUDA, PA_ERR_NOT_FOUND = 4, 5, 6, 7
PA_F32, PA_BF16, PA_F16 = 0, 1, 2
PA_ROPE_HALF, PA_ROPE_INTERLEAVED = 0, 1
PA_ROPE_UNSCALED, PA_ROPE_LINEAR, PA_ROPE_NTK, PA_ROPE_YARN, PA_ROPE_BANDS = 0, 1, 2, 3, 4


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class PAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        text = _lib.load().pa_status_string(status).decode()
        super().__init__(f"{where}: {text} (status {status})")


def _check(status: int, where: str) -> None:
    if status != PA_OK:
        raise PAError(status, where)


_DTYPES = {torch.float32: PA_F32, torch.bfloat16: PA_BF16, torch.float16: PA_F16}


def _dtype(t: torch.Tensor) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libpa must be contiguous")
    return t.data_ptr()   # an int: ctypes converts it through the c_void_p argtype


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:   # the handle without a Stream object around it (0.1 us against 3)
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _cache_dims(k_cache: torch.Tensor) -> Tuple[int, int, int, int]:
    if k_cache.dim() != 4:
        raise ValueError("caches are [num_blocks, block_size, num_kv_heads, head_dim]")
    return tuple(int(x) for x in k_cache.shape)


def pa_reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, stream=None) -> None:
    """Write key[i], value[i] ([T, Hkv, D]) into slot slot_mapping[i] (int64) of the caches."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    T = int(slot_mapping.numel())
    if T and tuple(key.shape) != (T, hkv, d):
        raise ValueError("key must be [num_tokens, num_kv_heads, head_dim]")
    _check(_lib.load().pa_reshape_and_cache(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
                                           _ptr(slot_mapping), T, nb, bs, hkv, d, _dtype(k_cache),
                                           _stream(stream)), "pa_reshape_and_cache")


def _on_current_device(*tensors) -> None:
    """The kernels run on a stream of the current device: every tensor has to live there."""
    dev = torch.cuda.current_device() if tensors[0].is_cuda else 0   # (on the CPU every device id is -1)
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError("tensors must be on the current CUDA device")


def _token_stride(t: torch.Tensor, T: int, h: int, d: int) -> int:
    """Token stride of a [T, h, d] view whose heads and dims are contiguous."""
    st, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError("heads and dims must be contiguous")
    return st if T > 1 else h * d


def _rope_vectors(positions, inv_freq, num_tokens: int) -> int:
    """Check the position and frequency vectors; returns rotary_dim."""
    if positions.dtype != torch.int32 or positions.shape != (num_tokens,):
        raise TypeError("positions must be int32 [num_tokens]")
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1:
        raise TypeError("inv_freq must be float64 [rotary_dim / 2]")
    return 2 * inv_freq.shape[0]


def pa_rope_frequencies(rotary_dim, base, scaling=PA_ROPE_UNSCALED, scale=1.0, original_context=0, low=1.0,
                        high=32.0) -> Tuple[np.ndarray, float]:
    """(inv_freq float64 [rotary_dim / 2], factor) of a rotary scaling kind (host only)."""
    out = np.empty(max(int(rotary_dim) // 2, 1), dtype=np.float64)
    factor = ctypes.c_float(1.0)
    _check(_lib.load().pa_rope_frequencies(out.ctypes.data_as(ctypes.POINTER(ctypes.c_double)),
                                           ctypes.byref(factor), int(rotary_dim), float(base), int(scaling),
                                           float(scale), int(original_context), float(low), float(high)),
           "pa_rope_frequencies")
    return out, factor.value


def pa_rope(out, x, positions, inv_freq, layout=PA_ROPE_HALF, factor=1.0, transpose=False, stream=None) -> None:
    """Rotate the heads of ``x`` [T, H, D] by their token's position into ``out``
    (which may be ``x``): ``positions`` [T] int32, negative for padding (left
    unwritten); ``inv_freq`` float64 [rotary_dim / 2] on the device. The token
    rows of either may be strided (heads and dims contiguous). ``transpose``
    applies the gradient of the rotation."""
    T, h, d = x.shape
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out must have x's shape and dtype")
    rot = _rope_vectors(positions, inv_freq, T)
    so, sx = _token_stride(out, T, h, d), _token_stride(x, T, h, d)
    _on_current_device(out, x, positions, inv_freq)
    _check(_lib.load().pa_rope(out.data_ptr(), so, x.data_ptr(), sx, _ptr(positions), _ptr(inv_freq), T, h, d, rot,
                               layout, factor, bool(transpose), _dtype(x), _stream(stream)), "pa_rope")


def _append_args(query_out, query, key, value, k_cache, v_cache, slot_mapping, positions, inv_freq, *weights):
    """Checks the two appends share; returns (the strided rows' arguments, the sizes)."""
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("caches are [num_blocks, block_size, num_kv_heads, head_dim], both alike")
    nb, bs, hkv, d = k_cache.shape
    T, hq, _ = query.shape
    if slot_mapping.dtype != torch.int64 or slot_mapping.shape != (T,):
        raise TypeError("slot_mapping must be int64 [num_tokens]")
    if query.shape[2] != d or query_out.shape != query.shape:
        raise ValueError("query and query_out must be [num_tokens, num_heads, head_dim]")
    if key.shape != (T, hkv, d) or value.shape != key.shape:
        raise ValueError("key and value must be [num_tokens, num_kv_heads, head_dim]")
    dt = k_cache.dtype
    if not (dt == v_cache.dtype == query.dtype == query_out.dtype == key.dtype == value.dtype):
        raise TypeError("query, key, value and the caches must have one dtype")
    rot = _rope_vectors(positions, inv_freq, T)
    so, sq = _token_stride(query_out, T, hq, d), _token_stride(query, T, hq, d)
    sk, sv = _token_stride(key, T, hkv, d), _token_stride(value, T, hkv, d)
    _on_current_device(query_out, query, key, value, k_cache, v_cache, slot_mapping, positions, inv_freq, *weights)
    return ((query_out.data_ptr(), so, query.data_ptr(), sq, key.data_ptr(), sk, value.data_ptr(), sv),
            (T, hq, nb, bs, hkv, d, rot))


def pa_rope_and_cache(query_out, query, key, value, k_cache, v_cache, slot_mapping, positions, inv_freq,
                      layout=PA_ROPE_HALF, factor=1.0, stream=None) -> None:
    """:func:`pa_rope` on ``query`` [T, Hq, D] into ``query_out`` and on ``key`` [T, Hkv, D] into slot
    slot_mapping[i] (int64) of the caches, ``value`` copied beside it, in one launch."""
    rows, sizes = _append_args(query_out, query, key, value, k_cache, v_cache, slot_mapping, positions, inv_freq)
    _check(_lib.load().pa_rope_and_cache(
        *rows, _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping), _ptr(positions), _ptr(inv_freq), *sizes, layout, factor,
        _dtype(k_cache), _stream(stream)), "pa_rope_and_cache")


def _norm_weight(weight, d: int, dtype) -> None:
    if weight.dtype != dtype or weight.shape != (d,):
        raise TypeError("the norm's weight must be [head_dim], of the heads' dtype")


def pa_norm_rope(out, x, weight, eps, positions, inv_freq, layout=PA_ROPE_HALF, factor=1.0, stream=None) -> None:
    """:func:`pa_rope` on the heads of ``x`` [T, H, D] normed first: each divided by the root of its mean
    square plus ``eps`` and multiplied by ``weight`` [D] (x's dtype). ``out`` may be ``x``."""
    T, h, d = x.shape
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out must have x's shape and dtype")
    _norm_weight(weight, d, x.dtype)
    rot = _rope_vectors(positions, inv_freq, T)
    so, sx = _token_stride(out, T, h, d), _token_stride(x, T, h, d)
    _on_current_device(out, x, weight, positions, inv_freq)
    _check(_lib.load().pa_norm_rope(out.data_ptr(), so, x.data_ptr(), sx, _ptr(weight), eps, _ptr(positions),
                                    _ptr(inv_freq), T, h, d, rot, layout, factor, _dtype(x), _stream(stream)),
           "pa_norm_rope")


def pa_norm_rope_backward_workspace_size(num_tokens, num_heads, head_dim) -> int:
    return int(_lib.load().pa_norm_rope_backward_workspace_size(num_tokens, num_heads, head_dim))


def pa_norm_rope_backward(grad_x, grad_weight, grad_out, x, weight, eps, positions, inv_freq, workspace,
                          layout=PA_ROPE_HALF, factor=1.0, stream=None) -> None:
    """The gradients of :func:`pa_norm_rope`: ``grad_x`` [T, H, D] (may be ``x`` or ``grad_out``) and
    ``grad_weight`` [D] float32, overwritten, from ``grad_out`` and the forward's arguments. The token rows
    of grad_x, grad_out and x may be strided. ``workspace``: a uint8 tensor of at least
    :func:`pa_norm_rope_backward_workspace_size` bytes."""
    T, h, d = x.shape
    if not (grad_x.shape == grad_out.shape == x.shape) or not (grad_x.dtype == grad_out.dtype == x.dtype):
        raise ValueError("grad_x and grad_out must have x's shape and dtype")
    _norm_weight(weight, d, x.dtype)
    if grad_weight.dtype != torch.float32 or grad_weight.shape != (d,):
        raise TypeError("grad_weight must be float32 [head_dim]")
    rot = _rope_vectors(positions, inv_freq, T)
    sg, so, sx = (_token_stride(t, T, h, d) for t in (grad_x, grad_out, x))
    _on_current_device(grad_x, grad_weight, grad_out, x, weight, positions, inv_freq, workspace)
    _check(_lib.load().pa_norm_rope_backward(
        grad_x.data_ptr(), sg, _ptr(grad_weight), grad_out.data_ptr(), so, x.data_ptr(), sx, _ptr(weight), eps,
        _ptr(positions), _ptr(inv_freq), T, h, d, rot, layout, factor, _dtype(x), _ptr(workspace), workspace.nbytes,
        _stream(stream)), "pa_norm_rope_backward")


def pa_norm_rope_and_cache(query_out, query, key, value, query_weight, key_weight, eps, k_cache, v_cache, slot_mapping,
                           positions, inv_freq, layout=PA_ROPE_HALF, factor=1.0, stream=None) -> None:
    """:func:`pa_rope_and_cache` with queries and keys normed on the way (:func:`pa_norm_rope`, by
    ``query_weight`` and ``key_weight`` [D]), in one launch."""
    rows, sizes = _append_args(query_out, query, key, value, k_cache, v_cache, slot_mapping, positions, inv_freq,
                               query_weight, key_weight)
    for w in (query_weight, key_weight):
        _norm_weight(w, sizes[5], k_cache.dtype)
    _check(_lib.load().pa_norm_rope_and_cache(
        *rows, _ptr(query_weight), _ptr(key_weight), eps, _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping),
        _ptr(positions), _ptr(inv_freq), *sizes, layout, factor, _dtype(k_cache), _stream(stream)),
        "pa_norm_rope_and_cache")


def pa_copy_blocks(k_cache, v_cache, block_mapping, stream=None) -> None:
    """For each (src, dst) row of block_mapping ([N, 2] int64), copy block src to dst."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    if block_mapping.dtype != torch.int64:
        raise TypeError("block_mapping must be int64")
    N = int(block_mapping.shape[0]) if block_mapping.numel() else 0
    _check(_lib.load().pa_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(block_mapping), N, nb, bs,
                                     hkv, d, _dtype(k_cache), _stream(stream)), "pa_copy_blocks")


def pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                             max_context_len) -> int:
    return int(_lib.load().pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                                    block_size, max_context_len))


class DecodePlan(ctypes.Structure):
    """pa_decode_plan_t: how pa_decode runs a problem on the current device."""
    _fields_ = [("tensor_cores", ctypes.c_int), ("heads_per_cta", ctypes.c_int),
                ("num_splits", ctypes.c_int), ("partition_tokens", ctypes.c_int),
                ("cluster_merge", ctypes.c_int), ("kernel_launches", ctypes.c_int),
                ("workspace_bytes", ctypes.c_size_t), ("balanced", ctypes.c_int)]

    def as_dict(self) -> dict:
        return {name: int(getattr(self, name)) for name, _ in self._fields_}


def pa_decode_plan(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len,
                   kv_dtype=PA_BF16, with_workspace=True) -> dict:
    """The plan pa_decode uses for this problem (host only; no launch)."""
    plan = DecodePlan()
    _check(_lib.load().pa_decode_plan(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                     max_context_len, int(kv_dtype), int(bool(with_workspace)),
                                     ctypes.byref(plan)), "pa_decode_plan")
    return plan.as_dict()


def pa_decode(out, query, k_cache, v_cache, block_tables, context_lens, max_context_len, scale,
              workspace=None, stream=None) -> None:
    """Paged decode attention into ``out`` [B, Hq, D] (float32, bfloat16 or float16).

    ``workspace`` is a uint8 tensor of at least :func:`pa_decode_workspace_size`
    bytes (its contents need no initialisation; calls sharing it must not
    overlap on the GPU), or None: then the tensor-core kernel merges a split of
    up to 8 partitions inside a thread-block cluster and trims a wider one to
    8, and the CUDA-core kernel does not split."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    B, hq, dq = (int(x) for x in query.shape)
    ws_bytes = int(workspace.numel() * workspace.element_size()) if workspace is not None else 0
    _check(_lib.load().pa_decode(_ptr(out), _dtype(out), _ptr(query), _dtype(query), _ptr(k_cache),
                                _ptr(v_cache), _dtype(k_cache), _ptr(block_tables),
                                _ptr(context_lens), B, hq, hkv, d, bs, int(block_tables.shape[1]),
                                nb, int(max_context_len), float(scale), _ptr(workspace), ws_bytes,
                                _stream(stream)), "pa_decode")


def pa_decode_append(out, query, new_key, new_value, k_cache, v_cache, block_tables, context_lens,
                     max_context_len, scale, workspace=None, stream=None) -> None:
    """One decode step: sequence b's new token (``new_key[b]``, ``new_value[b]``,
    [B, Hkv, D]) is written to position ``context_lens[b] - 1`` through its
    block table, then :func:`pa_decode` runs into ``out``."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    B, hq, _ = (int(x) for x in query.shape)
    if tuple(new_key.shape) != (B, hkv, d) or tuple(new_value.shape) != (B, hkv, d):
        raise ValueError("new_key / new_value must be [num_seqs, num_kv_heads, head_dim]")
    ws_bytes = int(workspace.numel() * workspace.element_size()) if workspace is not None else 0
    _check(_lib.load().pa_decode_append(_ptr(out), _dtype(out), _ptr(query), _dtype(query), _ptr(new_key),
                                       _ptr(new_value), _ptr(k_cache), _ptr(v_cache), _dtype(k_cache),
                                       _ptr(block_tables), _ptr(context_lens), B, hq, hkv, d, bs,
                                       int(block_tables.shape[1]), nb, int(max_context_len), float(scale),
                                       _ptr(workspace), ws_bytes, _stream(stream)), "pa_decode_append")


def pa_prefill_workspace_size(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, block_size, max_query_len,
                              max_context_len, kv_dtype=PA_BF16) -> int:
    return int(_lib.load().pa_prefill_workspace_size(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim,
                                                     block_size, max_query_len, max_context_len, kv_dtype))


def _prefill_args(out, query, k, v, lens, query_start, workspace, tables):
    """Checks pa_prefill and pa_cross_attention share; returns the workspace's bytes."""
    if out.shape != query.shape:
        raise ValueError("out must have query's shape")
    if k.dim() != 4 or v.shape != k.shape or k.shape[3] != query.shape[2]:
        raise ValueError("keys and values are [blocks or sequences, tokens, num_kv_heads, head_dim], both alike")
    if not (query.dtype == k.dtype == v.dtype):
        raise TypeError("query, keys and values must have one dtype")
    if lens.dtype != torch.int32 or query_start.dtype != torch.int32:
        raise TypeError("lengths and query_start must be int32")
    if lens.dim() != 1 or query_start.shape != (lens.shape[0] + 1,):
        raise ValueError("query_start must be [num_seqs + 1]")
    if workspace is None:
        _on_current_device(out, query, k, v, lens, query_start, tables)
        return 0
    _on_current_device(out, query, k, v, lens, query_start, tables, workspace)
    return workspace.nbytes


def pa_prefill(out, query, k_cache, v_cache, block_tables, context_lens, query_start, max_query_len, max_context_len,
               scale, causal=True, workspace=None, stream=None) -> None:
    """Attention of several query tokens a sequence over the paged cache into
    ``out`` [T, Hq, D]: sequence b owns tokens ``query_start[b]`` to
    ``query_start[b + 1]`` of ``query`` [T, Hq, D] (int32 [B + 1]), the last of
    its ``context_lens[b]`` tokens. ``causal``: token i sees the context up to
    itself; else all of it. ``workspace``: a uint8 tensor of at least
    :func:`pa_prefill_workspace_size` bytes, or None (contexts are not split)."""
    if block_tables.dtype != torch.int32 or block_tables.dim() != 2 or block_tables.shape[0] != context_lens.shape[0]:
        raise TypeError("block_tables must be int32 [num_seqs, max_blocks]")
    ws_bytes = _prefill_args(out, query, k_cache, v_cache, context_lens, query_start, workspace, block_tables)
    nb, bs, hkv, d = k_cache.shape
    T, hq, _ = query.shape
    _check(_lib.load().pa_prefill(_ptr(out), _dtype(out), _ptr(query), _dtype(query), _ptr(k_cache), _ptr(v_cache),
                                  _dtype(k_cache), _ptr(block_tables), _ptr(context_lens), _ptr(query_start),
                                  context_lens.shape[0], T, hq, hkv, d, bs, block_tables.shape[1], nb, max_query_len,
                                  max_context_len, scale, bool(causal), _ptr(workspace), ws_bytes, _stream(stream)),
           "pa_prefill")


def _weights_table(t, num_seqs: int, num_kv_heads: int, at_least: int, name: str) -> int:
    """Row stride of a [num_seqs, num_kv_heads, S] fp32 table of weights, S at least `at_least`."""
    if t.dtype != torch.float32 or t.dim() != 3:
        raise TypeError(f"{name} must be float32 [num_seqs, num_kv_heads, tokens]")
    if t.shape[0] != num_seqs or t.shape[1] != num_kv_heads or t.shape[2] < at_least:
        raise ValueError(f"{name} must be [num_seqs, num_kv_heads, tokens], with room for max_context_len")
    return t.shape[2]


def _paged_args(tables, lens, k_cache) -> None:
    if tables.dtype != torch.int32 or tables.dim() != 2 or lens.dtype != torch.int32 or lens.shape != (tables.shape[0],):
        raise TypeError("block_tables must be int32 [num_seqs, max_blocks], lengths int32 [num_seqs]")
    if k_cache.dim() != 4:
        raise ValueError("caches are [num_blocks, block_size, num_kv_heads, head_dim]")


def pa_decode_weights_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len) -> int:
    return int(_lib.load().pa_decode_weights_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                                            max_context_len))


def pa_decode_weights(out, weights, query, k_cache, v_cache, block_tables, context_lens, max_context_len, scale,
                      workspace, decay=1.0, stream=None) -> None:
    """:func:`pa_decode` into ``out`` [B, Hq, D], and the weight its rows gave each cached token: ``weights``
    [B, Hkv, S] float32 (S at least max_context_len; entry t belongs to position t) becomes ``decay`` times
    itself plus the softmax weights summed over the query heads of each KV head; the newest token's entry
    starts from zero. ``workspace``: a uint8 tensor of at least :func:`pa_decode_weights_workspace_size` bytes."""
    _paged_args(block_tables, context_lens, k_cache)
    nb, bs, hkv, d = k_cache.shape
    B, hq, _ = query.shape
    if out.shape != query.shape or query.shape[2] != d or v_cache.shape != k_cache.shape:
        raise ValueError("query and out are [num_seqs, num_heads, head_dim], both caches alike")
    if not (query.dtype == k_cache.dtype == v_cache.dtype):
        raise TypeError("query and caches must have one dtype")
    if block_tables.shape[0] != B:
        raise ValueError("block_tables must have a row for each query")
    stride = _weights_table(weights, B, hkv, max_context_len, "weights")
    _on_current_device(out, weights, query, k_cache, v_cache, block_tables, context_lens, workspace)
    _check(_lib.load().pa_decode_weights(
        _ptr(out), _dtype(out), _ptr(weights), stride, _ptr(query), _dtype(query), _ptr(k_cache), _ptr(v_cache),
        _dtype(k_cache), _ptr(block_tables), _ptr(context_lens), B, hq, hkv, d, bs, block_tables.shape[1], nb,
        max_context_len, scale, decay, _ptr(workspace), workspace.nbytes, _stream(stream)), "pa_decode_weights")


def pa_prefill_weights_workspace_size(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, block_size, max_query_len,
                                      max_context_len, window=0) -> int:
    return int(_lib.load().pa_prefill_weights_workspace_size(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim,
                                                             block_size, max_query_len, max_context_len, window))


def pa_prefill_weights(weights, query, k_cache, block_tables, context_lens, query_start, max_query_len, max_context_len,
                       scale, workspace, decay=0.0, window=0, stream=None) -> None:
    """The weights that several query tokens a sequence give the cached tokens, into ``weights`` [B, Hkv, S] as
    :func:`pa_decode_weights` does: tokens ``query_start[b]`` to ``query_start[b + 1]`` of ``query`` [T, Hq, D]
    are the last of sequence b's ``context_lens[b]`` tokens, each seeing the context up to itself. ``window``: only
    the last so many of each sequence count (0: all). ``workspace``: a uint8 tensor of at least
    :func:`pa_prefill_weights_workspace_size` bytes."""
    _paged_args(block_tables, context_lens, k_cache)
    nb, bs, hkv, d = k_cache.shape
    T, hq, dq = query.shape
    B = context_lens.shape[0]
    if dq != d:
        raise ValueError("query must be [num_tokens, num_heads, head_dim]")
    if query.dtype != k_cache.dtype:
        raise TypeError("query and cache must have one dtype")
    if query_start.dtype != torch.int32 or query_start.shape != (B + 1,):
        raise TypeError("query_start must be int32 [num_seqs + 1]")
    stride = _weights_table(weights, B, hkv, max_context_len, "weights")
    _on_current_device(weights, query, k_cache, block_tables, context_lens, query_start, workspace)
    _check(_lib.load().pa_prefill_weights(
        _ptr(weights), stride, _ptr(query), _dtype(query), _ptr(k_cache), _dtype(k_cache), _ptr(block_tables),
        _ptr(context_lens), _ptr(query_start), B, T, hq, hkv, d, bs, block_tables.shape[1], nb, max_query_len,
        max_context_len, scale, decay, window, _ptr(workspace), workspace.nbytes, _stream(stream)),
        "pa_prefill_weights")


def pa_evict(kept, new_weights, weights, k_cache, v_cache, block_tables, context_lens, new_tables, keep_lens,
             max_context_len, sinks=0, recent=0, stream=None) -> None:
    """Keep ``keep_lens[b]`` (int32 [B], negative: leave the sequence alone) tokens of each sequence and KV head:
    the last ``recent``, the first ``sinks`` and those with the largest ``weights`` [B, Hkv, S]; in the order of
    their positions they move to the blocks that ``new_tables`` [B, max_new_blocks] (int32) lists, blocks that
    nothing else in the call reads or writes. ``kept`` [B, Hkv, K] int32 gets the positions they had,
    ``new_weights`` [B, Hkv, S'] float32 their weights."""
    _paged_args(block_tables, context_lens, k_cache)
    _paged_args(new_tables, keep_lens, k_cache)
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("both caches must be alike")
    nb, bs, hkv, d = k_cache.shape
    B = context_lens.shape[0]
    if new_tables.shape[0] != B:
        raise ValueError("new_tables must have a row for each sequence")
    if kept.dtype != torch.int32 or kept.dim() != 3 or kept.shape[:2] != (B, hkv):
        raise TypeError("kept must be int32 [num_seqs, num_kv_heads, tokens]")
    stride = _weights_table(weights, B, hkv, max_context_len, "weights")
    new_stride = _weights_table(new_weights, B, hkv, 0, "new_weights")
    _on_current_device(kept, new_weights, weights, k_cache, v_cache, block_tables, context_lens, new_tables, keep_lens)
    _check(_lib.load().pa_evict(
        _ptr(kept), kept.shape[2], _ptr(new_weights), new_stride, _ptr(weights), stride, _ptr(k_cache), _ptr(v_cache),
        _dtype(k_cache), _ptr(block_tables), _ptr(context_lens), _ptr(new_tables), _ptr(keep_lens), B, hkv, d, bs,
        block_tables.shape[1], new_tables.shape[1], nb, max_context_len, sinks, recent, _stream(stream)), "pa_evict")


def pa_cross_attention(out, query, k, v, state_lens, query_start, max_query_len, max_state_len, scale, workspace=None,
                       stream=None) -> None:
    """Every query token of sequence b (tokens ``query_start[b]`` to
    ``query_start[b + 1]`` of ``query`` [T, Hq, D]) over the first
    ``state_lens[b]`` of an encoder's states ``k``, ``v`` [B, S, Hkv, D], into
    ``out`` [T, Hq, D]. ``workspace`` as for :func:`pa_prefill`, sized with
    block_size 16."""
    ws_bytes = _prefill_args(out, query, k, v, state_lens, query_start, workspace, query_start)
    if k.shape[0] != state_lens.shape[0]:
        raise ValueError("keys and values are [num_seqs, max_states, num_kv_heads, head_dim]")
    n, states, hkv, d = k.shape
    T, hq, _ = query.shape
    _check(_lib.load().pa_cross_attention(_ptr(out), _dtype(out), _ptr(query), _dtype(query), _ptr(k), _ptr(v),
                                          _dtype(k), _ptr(state_lens), _ptr(query_start), n, T, hq, hkv, d, states,
                                          max_query_len, max_state_len, scale, _ptr(workspace), ws_bytes,
                                          _stream(stream)), "pa_cross_attention")


def pa_swap_blocks(dst_k, dst_v, src_k, src_v, block_mapping, stream=None) -> None:
    """Copy blocks block_mapping[i, 0] of (src_k, src_v) to blocks
    block_mapping[i, 1] of (dst_k, dst_v); either pool may be a pinned host
    tensor, the mapping a device or pinned host int64 tensor [n, 2]."""
    snb, bs, hkv, d = _cache_dims(src_k)
    dnb = int(dst_k.shape[0])
    _check(_lib.load().pa_swap_blocks(_ptr(dst_k), _ptr(dst_v), _ptr(src_k), _ptr(src_v), _ptr(block_mapping),
                                     int(block_mapping.shape[0]), snb, dnb, bs, hkv, d, _dtype(src_k),
                                     _stream(stream)), "pa_swap_blocks")


def pa_decode_shared_prefix_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                           max_context_len, shared_blocks) -> int:
    return int(_lib.load().pa_decode_shared_prefix_workspace_size(
        num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len, shared_blocks))


def pa_decode_shared_prefix(out, query, k_cache, v_cache, block_tables, context_lens, max_context_len,
                            shared_blocks, scale, workspace, stream=None) -> None:
    """Decode attention where the first ``shared_blocks`` entries of every
    block-table row are the same (full) physical blocks: they are read once
    for the whole batch. ``workspace``: a uint8 tensor of at least
    :func:`pa_decode_shared_prefix_workspace_size` bytes."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    B, hq, _ = (int(x) for x in query.shape)
    ws_bytes = int(workspace.numel() * workspace.element_size()) if workspace is not None else 0
    _check(_lib.load().pa_decode_shared_prefix(
        _ptr(out), _dtype(out), _ptr(query), _dtype(query), _ptr(k_cache), _ptr(v_cache), _dtype(k_cache),
        _ptr(block_tables), _ptr(context_lens), B, hq, hkv, d, bs, int(block_tables.shape[1]), nb,
        int(max_context_len), int(shared_blocks), float(scale), _ptr(workspace), ws_bytes, _stream(stream)),
        "pa_decode_shared_prefix")


def pa_decode_contiguous(out, query, k, v, context_lens, max_context_len, scale, workspace=None,
                         stream=None) -> None:
    """Decode attention over a contiguous cache ``k``, ``v`` [B, max_seq_len,
    Hkv, D] (bfloat16 or float16, no block table): the unpaged baseline. ``workspace``
    as for :func:`pa_decode`, sized with block_size 16."""
    B, L, hkv, d = (int(x) for x in k.shape)
    _, hq, _ = (int(x) for x in query.shape)
    ws_bytes = int(workspace.numel() * workspace.element_size()) if workspace is not None else 0
    _check(_lib.load().pa_decode_contiguous(_ptr(out), _dtype(out), _ptr(query), _dtype(query), _ptr(k),
                                           _ptr(v), _dtype(k), _ptr(context_lens), B, hq, hkv, d, L,
                                           int(max_context_len), float(scale), _ptr(workspace), ws_bytes,
                                           _stream(stream)), "pa_decode_contiguous")


def pa_decode_static_scratch(out, query, k_cache, v_cache, block_tables, context_lens, max_context_len,
                             scale, stream=None) -> None:
    """pa_decode without a workspace argument, for callers that cannot
    allocate device memory: a split of up to 8 partitions is merged inside a
    thread-block cluster, a wider one through the library's own fixed
    scratch (calls must not overlap on the GPU)."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    B, hq, _ = (int(x) for x in query.shape)
    _check(_lib.load().pa_decode_static_scratch(
        _ptr(out), _dtype(out), _ptr(query), _dtype(query), _ptr(k_cache), _ptr(v_cache),
        _dtype(k_cache), _ptr(block_tables), _ptr(context_lens), B, hq, hkv, d, bs,
        int(block_tables.shape[1]), nb, int(max_context_len), float(scale), _stream(stream)),
        "pa_decode_static_scratch")


def pa_decode_splitk(tmp_out, max_logits, exp_sums, partition_size, query, k_cache, v_cache,
                     block_tables, context_lens, max_context_len, scale, stream=None) -> None:
    """Per-partition attention: tmp_out [B, Hq, P, D], max_logits / exp_sums [B, Hq, P] (float32)."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    B, hq, _ = (int(x) for x in query.shape)
    _check(_lib.load().pa_decode_splitk(_ptr(tmp_out), _ptr(max_logits), _ptr(exp_sums),
                                       int(partition_size), _ptr(query), _dtype(query),
                                       _ptr(k_cache), _ptr(v_cache), _dtype(k_cache),
                                       _ptr(block_tables), _ptr(context_lens), B, hq, hkv, d, bs,
                                       int(block_tables.shape[1]), nb, int(max_context_len),
                                       float(scale), _stream(stream)), "pa_decode_splitk")


def pa_lse_merge(out, tmp_out, max_logits, exp_sums, context_lens, partition_size, stream=None) -> None:
    """Log-sum-exp merge of pa_decode_splitk's partitions into ``out`` [B, Hq, D]."""
    B, hq, P, d = (int(x) for x in tmp_out.shape)
    _check(_lib.load().pa_lse_merge(_ptr(out), _dtype(out), _ptr(tmp_out), _ptr(max_logits),
                                   _ptr(exp_sums), _ptr(context_lens), B, hq, d, P,
                                   int(partition_size), _stream(stream)), "pa_lse_merge")


def pa_device_status(clear: bool = True, stream=None) -> int:
    """The device status word (0, or PA_ERR_TIMEOUT after a kernel gave up waiting)."""
    v = ctypes.c_int(0)
    _check(_lib.load().pa_device_status(ctypes.byref(v), int(clear), _stream(stream)), "pa_device_status")
    return v.value


def pa_check_wait_timeout(timeout_us: int = 1000, stream=None) -> None:
    """Run the failure-detection check: one CTA's bounded wait on a stage no
    copy fills runs out after ``timeout_us`` and records PA_ERR_TIMEOUT in the
    device status word (read it with :func:`pa_device_status`)."""
    _check(_lib.load().pa_check_wait_timeout(int(timeout_us), _stream(stream)), "pa_check_wait_timeout")


def pa_compute_slot_mapping(block_tables: np.ndarray, seq_index, positions, block_size: int) -> np.ndarray:
    """Host slot map: table[seq][pos // B] * B + pos % B (pos < 0 -> -1)."""
    tables = np.ascontiguousarray(block_tables, dtype=np.int32)
    seq = np.ascontiguousarray(seq_index, dtype=np.int32)
    pos = np.ascontiguousarray(positions, dtype=np.int32)
    out = np.empty(pos.shape[0], dtype=np.int64)
    _check(_lib.load().pa_compute_slot_mapping(
        out.ctypes.data_as(_lib.P_I64), tables.ctypes.data_as(_lib.P_I32), tables.shape[0],
        tables.shape[1], seq.ctypes.data_as(_lib.P_I32), pos.ctypes.data_as(_lib.P_I32),
        pos.shape[0], int(block_size)), "pa_compute_slot_mapping")
    return out


class BlockManager:
    """Handle on the host block manager (pa_bm_*)."""

    def __init__(self, num_blocks: int, block_size: int, reserve_null_block: bool = True,
                 free_order=None):
        self._lib = _lib.load()
        h = ctypes.c_void_p()
        if free_order is None:
            st = self._lib.pa_bm_create(num_blocks, block_size, int(reserve_null_block), ctypes.byref(h))
        else:
            arr = np.ascontiguousarray(free_order, dtype=np.int32)
            st = self._lib.pa_bm_create_with_free_list(num_blocks, block_size,
                                                       arr.ctypes.data_as(_lib.P_I32), arr.size,
                                                       ctypes.byref(h))
        _check(st, "pa_bm_create")
        self._h = h
        self.num_blocks = num_blocks
        self.block_size = block_size

    def close(self) -> None:
        if getattr(self, "_h", None):
            self._lib.pa_bm_destroy(self._h)
            self._h = None

    def __del__(self):
        self.close()

    def allocate(self, seq: int, num_tokens: int) -> None:
        _check(self._lib.pa_bm_allocate(self._h, seq, num_tokens), "pa_bm_allocate")

    def append_slot(self, seq: int) -> Tuple[int, int, int]:
        slot, src, dst = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(self._lib.pa_bm_append_slot(self._h, seq, ctypes.byref(slot), ctypes.byref(src),
                                           ctypes.byref(dst)), "pa_bm_append_slot")
        return slot.value, src.value, dst.value

    def fork(self, parent: int, child: int) -> None:
        _check(self._lib.pa_bm_fork(self._h, parent, child), "pa_bm_fork")

    def compact_group(self, seqs, num_tokens):
        """The blocks of compacted copies of the sequences that one :func:`pa_evict` takes (num_tokens[i] of seqs[i], at
        most what it holds), now their tables; none is an old block of the group, and those are released."""
        ids, counts = np.ascontiguousarray(seqs, dtype=np.int64), np.ascontiguousarray(num_tokens, dtype=np.int32)
        if ids.ndim != 1 or counts.shape != ids.shape:
            raise ValueError("num_tokens must have one entry for each sequence")
        need = [-(-max(int(t), 0) // self.block_size) for t in counts]
        buf, n = (ctypes.c_int32 * max(1, sum(need)))(), ctypes.c_int(0)
        _check(self._lib.pa_bm_compact_group(self._h, ids.ctypes.data_as(_lib.P_I64), ids.size,
                                             counts.ctypes.data_as(_lib.P_INT), buf, sum(need), ctypes.byref(n)),
               "pa_bm_compact_group")
        at = np.concatenate([[0], np.cumsum(need)]).astype(int)
        return [[int(b) for b in buf[lo:hi]] for lo, hi in zip(at, at[1:])]

    def compact(self, seq: int, num_tokens: int):
        """:meth:`compact_group` of one sequence. Not one by one for the sequences of one eviction: the second would be
        handed blocks that the first one's data still lies in."""
        cap = -(-max(num_tokens, 0) // self.block_size)
        buf, n = (ctypes.c_int32 * max(1, cap))(), ctypes.c_int(0)
        _check(self._lib.pa_bm_compact(self._h, seq, num_tokens, buf, cap, ctypes.byref(n)), "pa_bm_compact")
        return [int(buf[i]) for i in range(n.value)]

    def free(self, seq: int) -> None:
        _check(self._lib.pa_bm_free(self._h, seq), "pa_bm_free")

    def _list(self, fn, *args):
        n = ctypes.c_int(0)
        fn(self._h, *args, None, 0, ctypes.byref(n))
        buf = (ctypes.c_int32 * max(1, n.value))()
        _check(fn(self._h, *args, buf, n.value, ctypes.byref(n)), fn.__name__)
        return [int(buf[i]) for i in range(n.value)]

    def block_table(self, seq: int):
        return self._list(self._lib.pa_bm_block_table, seq)

    def free_list(self):
        return self._list(self._lib.pa_bm_free_list)

    def num_tokens(self, seq: int) -> int:
        n = ctypes.c_int()
        _check(self._lib.pa_bm_num_tokens(self._h, seq, ctypes.byref(n)), "pa_bm_num_tokens")
        return n.value

    def refcount(self, block: int) -> int:
        n = ctypes.c_int()
        _check(self._lib.pa_bm_refcount(self._h, block, ctypes.byref(n)), "pa_bm_refcount")
        return n.value

    def stats(self) -> dict:
        s = _lib.PaBmStats()
        _check(self._lib.pa_bm_stats(self._h, ctypes.byref(s)), "pa_bm_stats")
        return {name: int(getattr(s, name)) for name, _ in _lib.PaBmStats._fields_}

    # -- swapping to a CPU pool -------------------------------------------
    def enable_swap(self, num_host_blocks: int) -> None:
        _check(self._lib.pa_bm_enable_swap(self._h, num_host_blocks), "pa_bm_enable_swap")

    def _swap(self, fn, seqs) -> np.ndarray:
        ids = np.ascontiguousarray(seqs, dtype=np.int64)
        cap = int(sum(len(self.block_table(int(s))) for s in ids)) if ids.size else 0
        out = np.zeros((max(cap, 1), 2), dtype=np.int64)
        n = ctypes.c_int(0)
        _check(fn(self._h, ids.ctypes.data_as(_lib.P_I64), ids.size, out.ctypes.data_as(_lib.P_I64), cap,
                  ctypes.byref(n)), fn.__name__)
        return out[: n.value].copy()

    def swap_out(self, seqs) -> np.ndarray:
        """Move a group of sequences to the CPU pool; returns [n, 2] (GPU id, CPU id) pairs."""
        return self._swap(self._lib.pa_bm_swap_out, seqs)

    def swap_in(self, seqs) -> np.ndarray:
        """Bring a swapped-out group back; returns [n, 2] (CPU id, GPU id) pairs."""
        return self._swap(self._lib.pa_bm_swap_in, seqs)

    def is_swapped(self, seq: int) -> bool:
        v = ctypes.c_int(0)
        _check(self._lib.pa_bm_is_swapped(self._h, seq, ctypes.byref(v)), "pa_bm_is_swapped")
        return bool(v.value)

    def swap_stats(self) -> dict:
        a, b, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(self._lib.pa_bm_swap_stats(self._h, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)),
               "pa_bm_swap_stats")
        return {"host_blocks": a.value, "free_host_blocks": b.value, "swapped_seqs": c.value}
