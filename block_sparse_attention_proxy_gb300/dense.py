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

import contextlib
import ctypes
import functools

import torch

from . import _check as _raise_on
from . import load, make_dense_params, msa_dense_bwd_workspace_size


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


class _Plan:
    """What a call's shapes decide: the library's parameters and buffer sizes."""

    def __init__(self, T, num_docs, hq, hkv, d, scale, starts, strides, do_stride):
        self.params = make_dense_params(T, num_docs, hq, hkv, d, scale, starts, *strides, do_stride)
        self.ref = ctypes.byref(self.params)
        self.workspace = max(msa_dense_bwd_workspace_size(self.params), 256)
        self.o_res_at = (T * hq * 4 + 255) // 256 * 256  # saved for the backward: lse, then o_res
        self.saved = max(self.o_res_at + T * hq * d * 2, 256)
        lib = load()
        self.fwd, self.bwd = lib.msa_dense_fwd, lib.msa_dense_bwd


def _stride_of(shape, stride):
    """Token stride the library takes for a [tokens, heads, d] tensor (0: packed), or None
    where the layout has to be copied: heads not packed, rows that overlap, off 16 bytes."""
    tokens, heads, d = shape
    if tokens <= 1 and stride[2] == 1 and (heads == 1 or stride[1] == d):
        return 0
    if (stride[2] != 1 or (heads > 1 and stride[1] != d) or stride[0] < heads * d
            or stride[0] % 8):
        return None
    return stride[0]


# The checks and the plan depend on shapes, strides, types and devices alone, so they
# are made once for each combination and not once per call.
@functools.lru_cache(maxsize=512)
def _plan(qs, ks, vs, q_st, k_st, v_st, types, devices, cus, biass, scale, starts):
    if types[:3] != (torch.bfloat16,) * 3 or devices[0].type != "cuda":
        raise TypeError("q, k, v must be bf16 CUDA tensors")
    if len(qs) != 3 or len(ks) != 3 or len(vs) != 3 or any(x != devices[0] for x in devices):
        raise ValueError("q, k, v must be [tokens, heads, d], all tensors on one device")
    if ks != vs or ks[0] != qs[0] or ks[2] != qs[2]:
        raise ValueError("q [T, Hq, d] and k, v [T, Hkv, d] expected")
    if len(cus) != 1 or cus[0] < 2:
        raise ValueError("cu_seqlens must be [num_docs + 1]")
    if types[3] not in (torch.int32, torch.int64):
        raise TypeError("cu_seqlens must be integers")
    if (biass is None) != (not starts):
        raise ValueError("bias and bucket_starts go together")
    if biass is not None:
        if types[4] != torch.bfloat16:
            raise TypeError("bias must be bf16")
        if biass != (qs[1], len(starts)):
            raise ValueError("bias must be [Hq, number of buckets]")
    strides = [_stride_of(s, st) for s, st in ((qs, q_st), (ks, k_st), (vs, v_st))]
    copy = tuple(s is None for s in strides)
    args = (qs[0], cus[0] - 1, qs[1], ks[1], qs[2], scale, starts,
            tuple(s or 0 for s in strides))
    return _Plan(*args, 0), copy, args


@functools.lru_cache(maxsize=512)
def _bwd_plan(args, do_stride):
    return _Plan(*args, do_stride)


def _take(t, copy):
    # tensors off a 16-byte boundary are copied too
    if copy or t.data_ptr() % 16:
        return t.clone(memory_format=torch.contiguous_format)
    return t


# The current stream's handle; torch.cuda.current_stream would build an object around it,
# which costs as much host time as a kernel launch.
_stream = torch._C._cuda_getCurrentRawStream


_HERE = contextlib.nullcontext()


def _on(device):
    """Makes `device` current; nothing to do (and no host time) where it is already."""
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _forward(q, k, v, cu, bias, scale, starts, keep):
    devices = (q.device, k.device, v.device, cu.device)
    types = (q.dtype, k.dtype, v.dtype, cu.dtype)
    if bias is not None:
        devices, types = devices + (bias.device,), types + (bias.dtype,)
    plan, copy, args = _plan(q.shape, k.shape, v.shape, q.stride(), k.stride(), v.stride(), types,
                             devices, cu.shape, None if bias is None else bias.shape, scale, starts)
    with _on(devices[0]):
        q, k, v = _take(q, copy[0]), _take(k, copy[1]), _take(v, copy[2])
        if any(copy):  # copies are packed
            args = args[:7] + (tuple(0 if c else s for c, s in zip(copy, args[7])),)
        if cu.dtype != torch.int32:
            cu = cu.to(torch.int32)
        cu = cu.contiguous()
        if bias is not None:
            bias = bias.contiguous()
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = o_res = saved = None
        if keep:
            saved = torch.empty(plan.saved, dtype=torch.uint8, device=q.device)
            lse = saved.data_ptr()
            o_res = lse + plan.o_res_at
        _raise_on(plan.fwd(plan.ref, cu.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                           None if bias is None else bias.data_ptr(), o.data_ptr(), o_res, lse,
                           _stream(devices[0].index)), "msa_dense_fwd")
    return o, saved, (q, k, v, cu, bias), args


class DenseFunction(torch.autograd.Function):
    """o = softmax(scale q k^T + bias, causal in each document) v."""

    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, bias, softmax_scale: float, starts: tuple):
        o, saved, tensors, ctx.args = _forward(q, k, v, cu_seqlens, bias, softmax_scale, starts,
                                               True)
        ctx.save_for_backward(*tensors, o, saved)
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_o):
        q, k, v, cu, bias, o, saved = ctx.saved_tensors
        device = q.device
        with _on(device):
            if d_o.dtype != torch.bfloat16:
                d_o = d_o.to(torch.bfloat16)
            stride = _stride_of(d_o.shape, d_o.stride())
            d_o = _take(d_o, stride is None)
            plan = _bwd_plan(ctx.args, stride or 0)
            dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=device) for t in (q, k, v))
            dbias = torch.empty_like(bias) if bias is not None else None
            # its own workspace per call: calls on other streams, and other graphs, share none
            ws = torch.empty(plan.workspace, dtype=torch.uint8, device=device)
            lse = saved.data_ptr()
            _raise_on(plan.bwd(plan.ref, cu.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                               None if bias is None else bias.data_ptr(), o.data_ptr(),
                               lse + plan.o_res_at, lse, d_o.data_ptr(), dq.data_ptr(),
                               dk.data_ptr(), dv.data_ptr(),
                               None if bias is None else dbias.data_ptr(), ws.data_ptr(),
                               plan.workspace, _stream(device.index)), "msa_dense_bwd")
        return dq, dk, dv, None, dbias, None, None


def dense_attention(q, k, v, cu_seqlens, softmax_scale: float = 1.0, bias=None,
                    bucket_starts=None) -> torch.Tensor:
    """Causal attention inside each document of a packed batch (see module docstring).

    bias: learned table [Hq, buckets]; the score of query i and key j gets the entry of
    the last bucket whose first distance, `bucket_starts[b]`, is at most i - j.
    bucket_starts begins with 0 and increases strictly (`log_buckets` makes one).
    Malformed cu_seqlens are found on the device (`msa_get_device_status`)."""
    starts = () if bucket_starts is None else tuple(bucket_starts)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad
                                    or (bias is not None and bias.requires_grad)):
        return DenseFunction.apply(q, k, v, cu_seqlens, bias, float(softmax_scale), starts)
    return _forward(q, k, v, cu_seqlens, bias, float(softmax_scale), starts, False)[0]
