"""Dense causal attention over packed documents as a torch function.

    o = dense_attention(q, k, v, cu_seqlens)
    o = dense_attention(q, k, v, cu_seqlens, bias=table, bucket_starts=log_buckets(32, 128))

The layers of a model that attend to every earlier key, beside `msa_attention`
for the block-sparse ones: grouped heads, packed documents of any lengths and
an optional learned relative position bias, with gradients of q, k, v and the
bias table.  Nothing is read back to the host, so the calls do not wait for
the GPU and may be captured in a CUDA graph.  This module only moves tensors in
and out of the library; every step runs in its kernels.

Layouts (packed varlen, token-major): q [T, Hq, d], k/v [T, Hkv, d], bias
[Hq, buckets], all bf16; cu_seqlens int32 [num_docs + 1] on the device.  q, k
and v may be slices of a fused projection (any token stride that keeps rows on
16 bytes); other layouts are copied.  Rows behind cu_seqlens[-1] come out zero.
"""
from __future__ import annotations

import functools

import torch

from . import (make_dense_params, msa_dense_bwd, msa_dense_bwd_workspace_size, msa_dense_fwd,
               workspace)


def log_buckets(num_buckets: int, max_distance: int) -> tuple[int, ...]:
    """First distance of each of `num_buckets` buckets: one distance per bucket for
    the first half, then spaced evenly in the logarithm; the last bucket begins
    at `max_distance`.  Needs num_buckets >= 4 and max_distance >= num_buckets."""
    if num_buckets < 4 or max_distance < num_buckets:
        raise ValueError("num_buckets >= 4 and max_distance >= num_buckets expected")
    half = num_buckets // 2
    starts = list(range(half))
    for i in range(num_buckets - half):
        at = round(half * (max_distance / half) ** (i / (num_buckets - half - 1)))
        starts.append(max(at, starts[-1] + 1))
    return tuple(starts)


@functools.lru_cache(maxsize=256)
def _params(*args):
    """The call's parameters and the backward's workspace bytes."""
    prm = make_dense_params(*args)
    return prm, msa_dense_bwd_workspace_size(prm)


def _rows(t: torch.Tensor) -> torch.Tensor:
    """`t` [tokens, heads, d] as the library takes it: heads packed, a token stride that
    is a multiple of 8 elements and rows that do not overlap, on 16 bytes."""
    heads, d = t.shape[1], t.shape[2]
    s = t.stride()
    if (s[2] == 1 and (s[1] == d or heads == 1) and s[0] >= heads * d and s[0] % 8 == 0
            and t.data_ptr() % 16 == 0):
        return t
    # contiguous tensors off a 16-byte boundary are copied too
    return t.clone(memory_format=torch.contiguous_format)


class DenseFunction(torch.autograd.Function):
    """o = softmax(scale q k^T + bias, causal in each document) v."""

    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, bias, softmax_scale: float, starts: tuple):
        o, lse, saved, args = _forward(q, k, v, cu_seqlens, bias, softmax_scale, starts,
                                       any(ctx.needs_input_grad))
        ctx.args = args
        ctx.save_for_backward(*saved, o, lse)
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_o):
        q, k, v, cu, bias, o, lse = ctx.saved_tensors
        with torch.cuda.device(q.device):
            if d_o.dtype != torch.bfloat16:
                d_o = d_o.to(torch.bfloat16)
            d_o = _rows(d_o)
            prm, nbytes = _params(*ctx.args, d_o.stride(0) if d_o.shape[0] > 1 else 0)
            dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device)
                          for t in (q, k, v))
            dbias = torch.empty_like(bias) if bias is not None else None
            # its own workspace per call: calls on other streams, and other graphs, share none
            msa_dense_bwd(prm, cu, q, k, v, bias, o, lse, d_o, dq, dk, dv, dbias,
                          workspace(nbytes, q.device))
        return dq, dk, dv, None, dbias, None, None


def _forward(q, k, v, cu_seqlens, bias, softmax_scale, starts, keep):
    T, hq, d = q.shape
    with torch.cuda.device(q.device):
        q, k, v = _rows(q), _rows(k), _rows(v)
        cu = cu_seqlens
        if cu.dtype != torch.int32 or not cu.is_contiguous():
            cu = cu.to(torch.int32).contiguous()
        if bias is not None:
            bias = bias.contiguous()
        strides = [t.stride(0) if T > 1 else 0 for t in (q, k, v)]  # one token: no stride
        args = (T, cu.numel() - 1, hq, k.shape[1], d, softmax_scale, starts, *strides)
        prm, _ = _params(*args)
        o = torch.empty((T, hq, d), dtype=q.dtype, device=q.device)
        lse = torch.empty((T, hq), dtype=torch.float32, device=q.device) if keep else None
        msa_dense_fwd(prm, cu, q, k, v, bias, o, lse)
    return o, lse, (q, k, v, cu, bias), args


def _check(q, k, v, cu_seqlens, bias, starts):
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError("q, k, v must be bf16 CUDA tensors")
        if t.dim() != 3 or t.device != q.device:
            raise ValueError("q, k, v must be [tokens, heads, d] on one device")
    if k.shape != v.shape or k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
        raise ValueError("q [T, Hq, d] and k, v [T, Hkv, d] expected")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or cu_seqlens.device != q.device:
        raise ValueError("cu_seqlens must be [num_docs + 1] on the device of q")
    if cu_seqlens.dtype not in (torch.int32, torch.int64):
        raise TypeError("cu_seqlens must be integers")
    if (bias is None) != (not starts):
        raise ValueError("bias and bucket_starts go together")
    if bias is not None:
        if bias.dtype != torch.bfloat16 or bias.device != q.device:
            raise TypeError("bias must be a bf16 tensor on the device of q")
        if tuple(bias.shape) != (q.shape[1], len(starts)):
            raise ValueError("bias must be [Hq, number of buckets]")


def dense_attention(q, k, v, cu_seqlens, softmax_scale: float = 1.0, bias=None,
                    bucket_starts=None) -> torch.Tensor:
    """Causal attention inside each document of a packed batch (see module docstring).

    bias: learned table [Hq, buckets]; the score of query i and key j gets the entry of
    the last bucket whose first distance, `bucket_starts[b]`, is at most i - j.
    bucket_starts begins with 0 and increases strictly (`log_buckets` makes one).
    Malformed cu_seqlens are found on the device (`msa_get_device_status`)."""
    starts = tuple(bucket_starts) if bucket_starts is not None else ()
    _check(q, k, v, cu_seqlens, bias, starts)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad
                                    or (bias is not None and bias.requires_grad)):
        return DenseFunction.apply(q, k, v, cu_seqlens, bias, float(softmax_scale), starts)
    return _forward(q, k, v, cu_seqlens, bias, float(softmax_scale), starts, False)[0]
