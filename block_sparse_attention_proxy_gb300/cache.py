"""Rotary positions and a paged key-value cache: for answering with layers of plain causal
attention (no block selection, no position bias), one new token of each sequence at a time.

    plan = rotary_plan(d)                                           # once
    q, k = rotary(q, k, plan, cu_seqlens=cu_seqlens)                # in training, differentiable

    cache = paged_cache(pages, page_size, hkv, d, scores=True)      # once
    q = cache_append(cache, k, v, table, lens, positions=at, plan=plan, q=q)  # a token a sequence
    lens, at = lens + 1, at + 1
    o = paged_attention(q, cache, table, lens, accumulate=True)
    lens = cache_evict(cache, table, lens, keep=4096, recent=128)   # where a budget is set

Entry i of a sequence lies in page table[b, i // page_size], slot i % page_size; which pages a
sequence has is the caller's.  Keys are stored rotated, so the order of the entries carries no
meaning and eviction may move them.  From the first eviction on a sequence has fewer entries than
its text has tokens: a new token's position is then the caller's to count (`at`); where nothing is ever
evicted it may be left out.  Nothing is read back to the host: no call waits for the GPU,
all may be captured in a CUDA graph.  The front end (csrc/cache_torch.cpp) only moves tensors in and
out of the library; every step runs in its kernels.

Layouts: q [T, Hq, d], k/v [T, Hkv, d] (slices of a fused projection are taken as they are),
table [sequences, pages] and lens [sequences] integers on the device (int32 is taken as it is).
"""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

import torch

from . import dense

_front = None

_DIGITS = 10 ** 60


def _arctan(n):  # of 1 / n, times 10^60, rounded down term by term: off by less than 100
    return sum((-1) ** i * _DIGITS // ((2 * i + 1) * n ** (2 * i + 1)) for i in range(45))


_TWO_PI = 32 * _arctan(5) - 8 * _arctan(239)  # times 10^60, right to 56 digits (Machin's formula)


def _load():
    """The front end's extension.  Raises if it has not been built, or does not load."""
    global _front
    dense._load()
    from . import _dense_torch

    _front = _dense_torch
    return _front


def _turns(f: float) -> int:
    """Radians a position as turns a position modulo one, a fraction of 2^64."""
    n, d = f.as_integer_ratio()
    return ((n * _DIGITS << 65) // (d * _TWO_PI) + 1 >> 1) % 2 ** 64


def rotary_plan(dims: int, base: float = 10000.0, interleaved: bool = False, stretch: float = 1.0,
                trained_length: Optional[int] = None, low: float = 1.0, high: float = 32.0,
                amplitude: float = 1.0, frequencies=None):
    """The frequencies of a rotation of the first `dims` elements of a head (a multiple of 16).

    Pair i turns by base ** (-2 i / dims) radians a position; pairs are elements (i, i + dims/2), or
    neighbours where `interleaved` is set.  For texts `stretch` times longer than a model was
    trained on all frequencies are divided by `stretch`; with `trained_length` only as far as a
    pair turns less than `high` times over that length, fully where it turns less than
    `low` times, in between in proportion.  `frequencies`: dims / 2 of the caller's own instead (radians
    a position, after any stretching).  `amplitude` scales the rotated elements."""
    if dims < 0 or dims % 16 or dims > 256:
        raise ValueError("dims must be a multiple of 16 up to 256")
    if not math.isfinite(amplitude):
        raise ValueError("amplitude must be finite")
    if frequencies is None:
        if not (base > 0 and stretch > 0 and math.isfinite(base) and math.isfinite(stretch)):
            raise ValueError("base and stretch must be positive and finite")
        if trained_length is not None and not (trained_length > 0 and 0 <= low < high):
            raise ValueError("trained_length > 0 and 0 <= low < high expected")
        frequencies = []
        for i in range(dims // 2):
            f = float(base) ** (-2 * i / dims)
            part = 0.0
            if trained_length is not None:
                turns = trained_length * f / (2 * math.pi)
                part = min(1.0, max(0.0, (turns - low) / (high - low)))
            frequencies.append(f * (part + (1 - part) / stretch))
    elif stretch != 1.0 or trained_length is not None:
        raise ValueError("frequencies are taken as they are: no stretch")
    frequencies = [float(f) for f in frequencies]
    if len(frequencies) != dims // 2 or not all(map(math.isfinite, frequencies)):
        raise ValueError("dims / 2 finite frequencies expected")
    return (_front or _load()).RotaryPlan([_turns(f) for f in frequencies], bool(interleaved),
                                          float(amplitude))


def rotary(q, k, plan, cu_seqlens=None, positions=None):
    """(q, k) turned by their positions: places in the documents of `cu_seqlens` (rows behind the
    last one come out zero), or `positions` [T].  bf16, fp16 or fp32; k may be None.  Head dims are
    multiples of 16 up to 256.  Differentiable in reverse mode, its gradients too."""
    return (_front or _load()).rotary(q, k, plan, cu_seqlens, positions)


class PagedCache(NamedTuple):
    """Pages of keys and values.  k, v [pages, page size, Hkv, d] bf16, any strides that keep rows on
    16 bytes; weight [pages, Hkv, page size] fp32, attention weight that each entry has received,
    and position [pages, Hkv, page size] int32, its position in its text (None: not kept).  Page
    size 16, 32, 64, 128 or 256, d 64 or 128."""

    k: torch.Tensor
    v: torch.Tensor
    weight: Optional[torch.Tensor] = None
    position: Optional[torch.Tensor] = None


def paged_cache(pages: int, page_size: int, hkv: int, d: int, scores: bool = False,
                device="cuda") -> PagedCache:
    """An empty cache; `scores`: with the weights and positions that eviction goes by."""
    k, v = (torch.zeros(pages, page_size, hkv, d, dtype=torch.bfloat16, device=device)
            for _ in range(2))
    if not scores:
        return PagedCache(k, v)
    return PagedCache(k, v, torch.zeros(pages, hkv, page_size, device=device),
                      torch.zeros(pages, hkv, page_size, dtype=torch.int32, device=device))


def cache_append(cache: PagedCache, k, v, table, lens, cu_seqlens=None, positions=None, plan=None,
                 q=None):
    """Stores new tokens behind the `lens` entries of each sequence, which it does not change: one a
    sequence, or those that `cu_seqlens` [sequences + 1] gives it.  With `plan` k is rotated,
    by `positions` [T] or else the entries' numbers, and q, if given, is returned rotated
    too.  After an eviction those numbers are no positions any more: `positions` has to be given.
    New entries have weight 0.  k, v and q may be rows of the cache, but none that the call
    writes.  Inference only."""
    return (_front or _load()).cache_append(*cache, k, v, table, lens, cu_seqlens, positions, plan,
                                            q)


def paged_attention(q, cache: PagedCache, table, lens, softmax_scale: float = 1.0,
                    accumulate: bool = False) -> torch.Tensor:
    """Attention of one token of each sequence, q [sequences, Hq, d], over its first `lens` entries;
    zero without any.  Hq / Hkv from 1 to 64.  `accumulate` adds the weights that an entry gets
    from the heads of its group to cache.weight; it takes 4 bytes of workspace a query head for every
    entry that `table` can name, so a narrower view of it saves memory.  Inference only."""
    return (_front or _load()).paged_attention(q, *cache, table, lens, softmax_scale, accumulate)


def cache_evict(cache: PagedCache, table, lens, keep: int, recent: int) -> torch.Tensor:
    """Cuts sequences down to `keep` entries and returns the new lengths.  For each KV head by
    itself the entries of the newest `recent` positions stay, and of the others those with the largest
    accumulated weights (equal ones: the lower entry).  What stays moves to the first `keep`
    entries; pages behind them are free.  From then on cache_append needs `positions`.  Weights come
    from paged_attention alone, one token at a time: those of a prompt that no token has attended to are
    0, and of such entries the oldest stay, unless the caller fills cache.weight."""
    return (_front or _load()).cache_evict(*cache, table, lens, keep, recent)
