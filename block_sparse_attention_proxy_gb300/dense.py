"""Dense causal attention over packed documents as a torch function.

    o = dense_attention(q, k, v, cu_seqlens)
    o = dense_attention(q, k, v, cu_seqlens, bias=table, bucket_starts=log_buckets(32, 128))

The layers of a model that attend to every earlier key, beside `msa_attention`
for the block-sparse ones: grouped heads, packed documents of any lengths and
an optional learned relative position bias, with gradients of q, k, v and the
bias table.  Nothing is read back to the host, so the calls do not wait for
the GPU and may be captured in a CUDA graph.  The front end (csrc/dense_torch.cpp)
only moves tensors in and out of the library; every step runs in its kernels.

Layouts (packed varlen, token-major): q [T, Hq, d], k/v [T, Hkv, d], bias
[Hq, buckets], all bf16; cu_seqlens int32 [num_docs + 1] on the device.  q, k
and v may be slices of a fused projection (any token stride that keeps rows on
16 bytes); other layouts are copied.  Rows behind cu_seqlens[-1] come out zero.
"""
from __future__ import annotations

import os

import torch

from ._abi import load
from .build import TORCH_LIB

_call = None


def _load():
    """The front end's extension.  Raises if it has not been built, or does not load: there is
    no fallback."""
    global _call
    load()  # the kernels' library, with its own message where that is missing
    if not os.path.exists(TORCH_LIB):
        raise RuntimeError(f"{TORCH_LIB} is missing: build the library first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    try:
        from ._dense_torch import dense_attention as call
    except ImportError as e:
        raise RuntimeError(f"{TORCH_LIB} does not load: {e}") from e
    _call = call
    return call


def log_buckets(num_buckets: int, max_distance: int) -> tuple[int, ...]:
    """First distance of each of `num_buckets` buckets: one distance per bucket for
    the first half, then spaced evenly in the logarithm; the last bucket begins
    at `max_distance`.  This package's own rule: a table trained with another one, whose
    last bucket may begin earlier, needs that rule's first distances.  Needs num_buckets >= 4 and max_distance >= num_buckets."""
    if num_buckets < 4 or max_distance < num_buckets:
        raise ValueError("num_buckets >= 4 and max_distance >= num_buckets expected")
    half = num_buckets // 2
    starts = list(range(half))
    for i in range(num_buckets - half):
        at = round(half * (max_distance / half) ** (i / (num_buckets - half - 1)))
        starts.append(max(at, starts[-1] + 1))
    return tuple(starts)


def dense_attention(q, k, v, cu_seqlens, softmax_scale: float = 1.0, bias=None,
                    bucket_starts=None) -> torch.Tensor:
    """Causal attention inside each document of a packed batch (see module docstring).

    bias: learned table [Hq, buckets]; the score of query i and key j gets the entry of
    the last bucket whose first distance, `bucket_starts[b]`, is at most i - j.
    bucket_starts begins with 0 and increases strictly (`log_buckets` makes one).
    Differentiable once, in reverse mode; inputs with a forward-mode tangent are refused.
    Finite biases of any size are exact, -inf masks.  Malformed cu_seqlens are found on the
    device (`msa_get_device_status`); the results are undefined then."""
    return (_call or _load())(q, k, v, cu_seqlens, softmax_scale, bias, bucket_starts)
