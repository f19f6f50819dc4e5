"""Rotary positions and the paged cache's operators from their definitions in fp64, with limits for
results of kernels that compute in fp32 from 16-bit operands.

Rotary.  A turn is exact to 2^-32 before it becomes a float in [-1, 1) (2^-25 of half a turn:
less than 2^-23 radians), sine and cosine are off by at most 2^-23 more, the amplitude's product
and the two products' sum by 2^-24 each of |a| + |b|: together 2^-21 amplitude (|a| + |b|),
and the rounding of the result, half a step.  For 16-bit results 2^-20 is allowed (enough for the
hardware's sine and cosine, off by 2^-21.19 between -pi and pi); test_sines_of_16_bit_results has
the kernel's own limit.

Attention.  U = 2^-8, half a bf16 step.  A score is a sum of at most 128 products accumulated in
fp32, each addition off by at most 2^-23 of A = sum |q||k| scale: 2^-16 A; exponentials, sums
over the entries and the parts' joining less than 2^-15.  Twice (numerator and normaliser):
eps = 2 (2^-16 A + 2^-15) relative for a weight.  P enters its product in two bf16 parts, which
drop 2^-17 of it at most, and o is rounded once: (eps + 2^-17) sum_j p |v| + U |o|.  An entry's
weight is a sum of the group's: eps times what it gains, and 2^-22 of its size for the additions.
"""
import torch


def positions_of(lens, tail=0):
    at = [torch.arange(n) for n in lens] + [torch.zeros(tail, dtype=torch.int64)]
    return torch.cat(at)


def rotary_exact(x, positions, frequencies, interleaved=False, amplitude=1.0, inverse=False):
    """(rotated x, limits) in fp64; positions whole numbers of any size, as a list."""
    import math
    from fractions import Fraction

    y, n = x.detach().double().cpu(), len(frequencies)
    two_pi = Fraction(int("6283185307179586476925286766559005768394338798750"), 10 ** 48)
    freq = [Fraction(f) for f in frequencies]
    angle = torch.empty(len(positions), n, dtype=torch.float64)
    for i, p in enumerate(positions):
        for j, f in enumerate(freq):
            t = p * f / two_pi
            angle[i, j] = float((t - math.floor(t)) * two_pi)
    c, s = angle.cos()[:, None] * amplitude, angle.sin()[:, None] * amplitude
    if inverse:
        s = -s
    a, b = ((slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else
            (slice(0, n), slice(n, 2 * n)))
    out, lim = y.clone(), torch.zeros_like(y)
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    size = 2.0 ** (-21 if x.dtype == torch.float32 else -20) * abs(amplitude) * (y[..., a].abs() + y[..., b].abs())
    lim[..., a] = lim[..., b] = size
    turned = torch.zeros(y.shape[-1], dtype=torch.bool)
    turned[:2 * n] = True
    # half a step of the result, or of the type's smallest normal number
    step = torch.finfo(x.dtype).eps / 2 * (out.abs() + torch.finfo(x.dtype).tiny)
    return out, torch.where(turned, lim + step, 0.0)


def gather(x, table, n):
    """The first n entries of one sequence: [n, ...] of a cache tensor [pages, page size, ...]."""
    page = x.shape[1]
    return x[table[:-(-n // page)].long()].flatten(0, 1)[:n]


def attend_exact(q, k, v, table, lens, scale=1.0):
    """(o, limits, [weights of each sequence: [Hkv, n], limits]) in fp64."""
    (b, hq, d), hkv = q.shape, k.shape[2]
    o, lim, weights = torch.zeros(b, hq, d).double(), torch.zeros(b, hq, d).double(), []
    q, k, v, table = (t.detach().cpu() for t in (q, k, v, table))
    for i, n in enumerate(lens):
        gain = torch.zeros(hkv, n).double()
        bound = torch.zeros(hkv, n).double()
        if n:
            kk, vv = gather(k, table[i], n).double(), gather(v, table[i], n).double()
            for h in range(hkv):
                heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                x = q[i, heads].double()
                s = scale * x @ kk[:, h].T
                size = scale * x.abs() @ kk[:, h].abs().T
                p = torch.softmax(s, 1)
                p = torch.where(torch.isneginf(s).all(1, keepdim=True), 0.0, p)
                eps = 2 * (2.0 ** -16 * size.masked_fill(~size.isfinite(), 0).max() + 2.0 ** -15)
                o[i, heads] = p @ vv[:, h]
                lim[i, heads] = (eps + 2.0 ** -17) * (p @ vv[:, h].abs()) * (1 + 2.0 ** -6) + \
                    2.0 ** -8 * o[i, heads].abs()
                gain[h], bound[h] = p.sum(0), eps * p.sum(0) * (1 + 2.0 ** -6)
        weights.append((gain, bound))
    return o, lim, weights


def evict_exact(weight, position, table, lens, keep, recent):
    """For each sequence and KV head the moves [(from, to)], by sorting."""
    moves = {}
    for i, n in enumerate(lens):
        if n <= keep:
            continue
        for h in range(weight.shape[1]):
            w = gather(weight.transpose(1, 2), table[i], n)[:, h].tolist()
            if recent:
                pos = gather(position.transpose(1, 2), table[i], n)[:, h].tolist()
                edge = max(pos) - recent
                w = [float("inf") if p > edge else x for x, p in zip(w, pos)]
                first = [p > edge for p in pos]
            else:
                first = [False] * n
            order = sorted(range(n), key=lambda j: (not first[j], w[j] == w[j],
                                                    -w[j] if w[j] == w[j] else 0.0, j))
            kept = set(order[:keep])
            moves[i, h] = list(zip([j for j in range(keep, n) if j in kept],
                                   [j for j in range(keep) if j not in kept]))
    return moves


def within(got, want, limit, name=""):
    """Every element within its limit; the same infinities and NaN."""
    got, want, limit = (t.detach().double().cpu() for t in (got, want, limit))
    fine = want.isfinite()
    assert torch.equal(fine, got.isfinite()), f"{name}: other places are finite"
    over = ((got - want).abs() - limit)[fine]
    assert not over.numel() or over.max() <= 0, f"{name}: {over.max():.3e} over the limit"


def placed(got, want, name=""):
    """NaN in the same places, and every infinity with its sign."""
    got, want = (t.detach().double().cpu() for t in (got, want))
    assert torch.equal(got.isnan(), want.isnan()), f"{name}: NaN in other places"
    at = want.isinf() | got.isinf()
    assert torch.equal(got[at], want[at]), f"{name}: other infinities"
