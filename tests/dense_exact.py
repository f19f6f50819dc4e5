"""Dense attention from its definition in fp64 with limits for results computed from bf16
operands with fp32 sums; for biases of any size, and tight for the bias table's gradient.

Terms (u = 2^-8, half a bf16 step; first order, times 1 + 2^-6 for the rest):
  eps  relative error of P.  A score is a sum of at most 128 products accumulated in fp32, each
       addition off by at most 2^-23 of A = sum |q||k| scale, so 2^-16 A; exponential, maximum
       and logarithm less than 2^-14.  Twice: numerator and normaliser.  A bias counts into A
       relative to the row's largest one: what lies more than 64 below has no weight.
  o    P is rounded to bf16 for its product and o is rounded: (u + 2 eps) sum_j P |v| + u |o|.
  D    is summed from o and its rounding residual, which together hold 16 bits:
       e_D = sum_j (u + 2 eps) P |dP| + 2^-15 sum |dO||o|.
  dS   e = P (e_D + 2^-16 sum |dO||v|) + 2 eps |dS|; u |dS| more for its rounding, which the
       products take but the table's sums do not.
  dQ   scale sum_j (e + u |dS|) |k| + u |dQ|; dK the same over i;
  dV   (u + 2 eps) sum_i P |dO| + u |dV|.
  table  sum of e over the bucket, fp32 sums 2^-16 sum |dS|, and u |dtable|.  Of e, a row shares
       e_D and the error eps of its normaliser, the latter as a factor of its sum of dS over the
       bucket; other pairs' errors are independent of one another, but for the 2^-20 of dP's sum
       that a truncating accumulator may lose in one direction (8 additions of 2^-23).
Those hold for every element.  The roundings of different P are independent: with each uniform
within its bound, their root sum of squares is more than 1.7 standard deviations, so three times
it (5.2) is a limit for single elements too, and the whole tensor's norm stays below one times.
The table's entries get the smaller of the two limits: an entry sums over all rows, and the
first one, which adds up e_D of every row, exceeds the entry itself.
"""
import torch

U = 2.0 ** -8


def dense_exact(q, k, v, lens, scale=1.0, bias=None, starts=None, d_o=None):
    """({o, lse, dq, dk, dv, dbias}, limits of each element, limits of each norm), fp64."""
    dev, (t, hq, d), hkv = q.device, q.shape, k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    do_all = torch.zeros_like(q) if d_o is None else d_o.double()
    r = {"o": torch.zeros_like(q), "lse": q.new_full((t, hq), -torch.inf),
         "dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v)}
    if bias is not None:
        b64 = bias.double()
        r["dbias"] = torch.zeros_like(b64)
    lim = {n: torch.zeros_like(x) for n, x in r.items()}
    sq = {n: torch.zeros_like(x) for n, x in r.items()}
    end = 0
    for n in lens:
        s, end = slice(end, end + n), end + n
        dist = torch.arange(n, device=dev)
        dist = dist[:, None] - dist
        low = dist >= 0
        if bias is not None:
            at = torch.tensor(starts, device=dev)
            which = torch.bucketize(dist.clamp(min=0), at, right=True) - 1
        for h in range(hq if n else 0):
            g = h // (hq // hkv)
            qh, kg, vg, do = q[s, h], k[s, g], v[s, g], do_all[s, h]
            sc, size = scale * qh @ kg.T, scale * qh.abs() @ kg.abs().T
            if bias is not None:
                b = b64[h][which].masked_fill(~low, -torch.inf)
                gap = (b - b.amax(1, keepdim=True)).abs()
                small = torch.minimum(b.abs(), gap)
                size = size + torch.where(small <= 64, small, 0.0)  # also where it is NaN
                sc = sc + b
            sc = sc.masked_fill(~low, -torch.inf)
            p = torch.softmax(sc, 1)
            p = torch.where(torch.isneginf(sc).all(1, keepdim=True), 0.0, p)
            eps = 2 * (2.0 ** -16 * float(size[low].max()) + 2.0 ** -14)
            o, dp = p @ vg, do @ vg.T
            r["o"][s, h], r["lse"][s, h] = o, torch.logsumexp(sc, 1)
            lim["o"][s, h] = (U + eps) * (p @ vg.abs())
            sq["o"][s, h] = U * U * (p * p @ vg ** 2) + (eps * (p @ vg.abs())) ** 2
            lim["lse"][s, h] = eps + 2.0 ** -22 * r["lse"][s, h].abs()
            pd = p * dp
            small = eps * pd.abs().sum(1, True) + 2.0 ** -15 * (do * o).abs().sum(1, True)
            e_d = U * pd.abs().sum(1, True) + small
            r_d = U * U * (pd ** 2).sum(1, True) + small ** 2
            ds = p * (dp - (do * o).sum(1, True))
            f = 2.0 ** -16 * p * (do.abs() @ vg.abs().T) + eps * ds.abs()
            e = p * e_d + f
            r["dq"][s, h] = scale * ds @ kg
            lim["dq"][s, h] = scale * (e + U * ds.abs()) @ kg.abs()
            sq["dq"][s, h] = scale ** 2 * (U * U * (ds ** 2 @ kg ** 2) + r_d * (p @ kg) ** 2
                                           + (f @ kg.abs()) ** 2)
            r["dk"][s, g] += scale * ds.T @ qh
            lim["dk"][s, g] += scale * (e + U * ds.abs()).T @ qh.abs()
            sq["dk"][s, g] += scale ** 2 * (U * U * (ds.T ** 2 @ qh ** 2)
                                            + p.T ** 2 @ (r_d * qh ** 2) + (f.T @ qh.abs()) ** 2)
            r["dv"][s, g] += p.T @ do
            lim["dv"][s, g] += (U + eps) * (p.T @ do.abs())
            sq["dv"][s, g] += U * U * (p.T ** 2 @ do ** 2) + (eps * (p.T @ do.abs())) ** 2
            if bias is not None:
                nb = b64.shape[1]
                rows = q.new_zeros(n, nb).scatter_add_(1, which, p.masked_fill(~low, 0))
                sums = q.new_zeros(n, nb).scatter_add_(1, which, ds.masked_fill(~low, 0))
                r["dbias"][h] += sums.sum(0)
                f = f + 2.0 ** -16 * ds.abs()
                lim["dbias"][h].index_add_(0, which[low], (e + f)[low])
                one_way = 2.0 ** -20 * p * (do.abs() @ vg.abs().T)
                once = (eps * sums.abs()).sum(0).index_add_(0, which[low], one_way[low])
                alone = q.new_zeros(nb).index_add_(0, which[low], (f ** 2)[low])
                sq["dbias"][h] += (r_d * rows ** 2).sum(0) + alone + once ** 2
    norm = {}
    for n, x in r.items():
        if n != "lse":
            if n == "dbias":
                lim[n] = torch.minimum(lim[n], 3 * sq[n].sqrt())
            lim[n] += U * x.abs()
            sq[n] += (U * x) ** 2
            norm[n] = float(sq[n].sum().sqrt())
        lim[n] *= 1 + 2.0 ** -6
    return r, lim, norm


def compare(got, want):
    """Every output in `got` against dense_exact's result."""
    r, lim, norm = want
    for n, x in got.items():
        gap = torch.where(x.double() == r[n], 0.0, (x.double() - r[n]).abs())  # equal infinities
        assert torch.isfinite(gap).all(), f"{n}: not finite"
        over = (gap - lim[n]).flatten()
        at = int(over.argmax())
        assert float(over[at]) <= 1e-30, (
            f"{n}[{at}]: {float(x.flatten()[at]):.6g}, definition {float(r[n].flatten()[at]):.6g}, "
            f"limit {float(lim[n].flatten()[at]):.3g}")
        if x.numel() >= 64 and n in norm:
            assert float(gap.norm()) <= norm[n], f"{n}: norm {float(gap.norm())}, {norm[n]}"
