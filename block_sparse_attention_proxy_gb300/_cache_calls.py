"""Python calls of the C entry points of rotary positions and the paged cache (include/msa.h)."""
from __future__ import annotations

import ctypes

from . import _check, _ptr, _stream
from ._abi import MsaCache, MsaPagedParams, MsaRotaryParams, MsaTable, load


def make_rotary_params(total_tokens, hq, hkv, d, frequencies, num_docs=0, interleaved=False,
                       inverse=False, dtype=0, position_bytes=4, amplitude=1.0, q_stride=0,
                       k_stride=0, flags=0) -> MsaRotaryParams:
    """msa_rotary_params; frequencies: turns a position as fractions of 2^64 (RotaryPlan's)."""
    n = len(frequencies)
    freq = (ctypes.c_uint64 * n)(*frequencies) if n else None
    return MsaRotaryParams(total_tokens=int(total_tokens), num_docs=int(num_docs), hq=int(hq),
                           hkv=int(hkv), d=int(d), dims=2 * n, interleaved=int(interleaved),
                           inverse=int(inverse), dtype=int(dtype),
                           position_bytes=int(position_bytes), freq=freq, q_stride=int(q_stride),
                           k_stride=int(k_stride), amplitude=float(amplitude), flags=int(flags))


def make_cache(cache) -> MsaCache:
    """msa_cache of a PagedCache; the tensors must outlive it."""
    k, v, weight, position = cache
    if k.dim() != 4 or k.shape != v.shape or k.stride(3) != 1 or v.stride(3) != 1:
        raise ValueError("k and v must be [pages, page size, Hkv, d], heads contiguous")
    for t in (weight, position):
        if t is not None and tuple(t.shape) != (k.shape[0], k.shape[2], k.shape[1]):
            raise ValueError("weight and position must be [pages, Hkv, page size]")
    return MsaCache(k=k.data_ptr(), v=v.data_ptr(), weight=_ptr(weight), position=_ptr(position),
                    num_pages=k.shape[0], page_size=k.shape[1], hkv=k.shape[2], d=k.shape[3],
                    k_page_stride=k.stride(0), k_slot_stride=k.stride(1), k_head_stride=k.stride(2),
                    v_page_stride=v.stride(0), v_slot_stride=v.stride(1), v_head_stride=v.stride(2))


def make_table(table, lens) -> MsaTable:
    """msa_table of [sequences, pages] and [sequences] int32 tensors, which must outlive it."""
    if table.dim() != 2 or lens.shape != table.shape[:1] or (table.shape[1] > 1
                                                             and table.stride(1) != 1):
        raise ValueError("table [sequences, pages], rows contiguous, and lens [sequences] expected")
    return MsaTable(pages=table.data_ptr(), lens=_ptr(lens), num_seqs=table.shape[0],
                    max_pages=table.shape[1], stride=table.stride(0))


def make_paged_params(hq, softmax_scale=1.0, accumulate=False, q_stride=0,
                      flags=0) -> MsaPagedParams:
    return MsaPagedParams(hq=int(hq), accumulate=int(accumulate), q_stride=int(q_stride),
                          softmax_scale=float(softmax_scale), flags=int(flags))


def _given(t, tokens: int, heads: int, d: int, stride: int):
    """A [tokens, heads, d] tensor whose token stride (0: packed) the call carries."""
    if t is None:
        return None
    if tuple(t.shape) != (tokens, heads, d) or t.stride(2) != 1 or (heads > 1 and t.stride(1) != d):
        raise ValueError("the params say [%d, %d, %d]" % (tokens, heads, d))
    if tokens > 1 and t.stride(0) != (stride or heads * d):
        raise ValueError("the tensor's token stride differs from the given one")
    return t.data_ptr()


def msa_rotary(params, cu_seqlens, positions, q, k, q_out, k_out, stream=None) -> None:
    p = params
    _check(load().msa_rotary(ctypes.byref(p), _ptr(cu_seqlens), _ptr(positions),
                             _given(q, p.total_tokens, p.hq, p.d, p.q_stride),
                             _given(k, p.total_tokens, p.hkv, p.d, p.k_stride), _ptr(q_out),
                             _ptr(k_out), _stream(stream)), "msa_rotary")


def msa_cache_append(cache, table, params, cu_seqlens, positions, q, k, v, q_out, stream=None) -> None:
    """v may be a slice of a wider tensor; q's and k's strides are the params'."""
    p = params
    v_stride = v.stride(0) if p.total_tokens > 1 else 0
    _check(load().msa_cache_append(ctypes.byref(cache), ctypes.byref(table), ctypes.byref(p),
                                   v_stride, _ptr(cu_seqlens), _ptr(positions),
                                   _given(q, p.total_tokens, p.hq, p.d, p.q_stride),
                                   _given(k, p.total_tokens, p.hkv, p.d, p.k_stride),
                                   _given(v, p.total_tokens, p.hkv, p.d, v_stride), _ptr(q_out),
                                   _stream(stream)), "msa_cache_append")


def msa_paged_attention_workspace_size(cache, table, params) -> int:
    return int(load().msa_paged_attention_workspace_size(ctypes.byref(cache), ctypes.byref(table),
                                                         ctypes.byref(params)))


def msa_paged_attention(cache, table, params, q, o, ws, stream=None) -> None:
    _check(load().msa_paged_attention(ctypes.byref(cache), ctypes.byref(table),
                                      ctypes.byref(params),
                                      _given(q, table.num_seqs, params.hq, cache.d, params.q_stride),
                                      _ptr(o), _ptr(ws), ws.numel() * ws.element_size(),
                                      _stream(stream)), "msa_paged_attention")


def msa_cache_evict_workspace_size(cache, table, keep: int) -> int:
    return int(load().msa_cache_evict_workspace_size(ctypes.byref(cache), ctypes.byref(table),
                                                     int(keep)))


def msa_cache_evict(cache, table, keep: int, recent: int, new_lens, ws, stream=None) -> None:
    _check(load().msa_cache_evict(ctypes.byref(cache), ctypes.byref(table), int(keep), int(recent),
                                  _ptr(new_lens), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream)), "msa_cache_evict")
