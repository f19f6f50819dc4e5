"""Dense attention from its definition in fp64, document by document and head by head,
with error bounds for results computed from bf16 operands with fp32 sums.

Bounds (u = 2^-8, half a bf16 step; first-order terms, times 1 + 2^-6 for the rest):
  P    relative eps: a score is a sum of at most 128 products accumulated in fp32, each
       addition off by at most 2^-23 of A = sum |q||k| scale, so 2^-16 A; the exponential,
       the maximum and the logarithm add less than 2^-14 for the magnitudes used here.
       Twice: numerator and normaliser.
  o    P enters the product rounded to bf16: (u + 2 eps) sum_j P |v|, and o is rounded: u |o|.
  dV   likewise (u + 2 eps) sum_i P |dO| + u |dV|.
  D    rowsum(dO o O) of the rounded o: sum |dO| e_o, plus fp32 sums 2^-16 sum |dO||o|.
  dS   (u + 2 eps) |dS| + P (e_D + 2^-16 sum |dO||v|), u being its rounding to bf16.
  dQ   scale sum_j e_dS |k| + u |dQ|; dK the same over i.
  table  its sums take dS before that rounding; u |dtable| for its own.
Those hold for every element.  Roundings of different values are independent, so the whole
tensor is held to the root of the sum of squares too (`rms`: the same terms squared, but the
fp32 terms and the error of D, which every product of a row shares, summed before squaring).
With each rounding uniform in its bound the expected square is a third of that, so a tensor of
64 or more values does not reach it.
"""
import torch

U = 2.0 ** -8


def dense_reference(q, k, v, lens, scale=1.0, bias=None, starts=None, d_o=None):
    """fp64 results {o, lse, dq, dk, dv, dbias} and their bounds {...} (CPU or GPU)."""
    dev = q.device
    T, hq, d = q.shape
    hkv = k.shape[1]
    q64, k64, v64 = q.double(), k.double(), v.double()
    z = torch.zeros
    r = {"o": z(T, hq, d, dtype=torch.float64, device=dev),
         "lse": torch.full((T, hq), -torch.inf, dtype=torch.float64, device=dev)}
    e = {"o": torch.zeros_like(r["o"]), "lse": torch.zeros_like(r["lse"])}
    if d_o is not None:
        for n, t in (("dq", q64), ("dk", k64), ("dv", v64)):
            r[n], e[n] = torch.zeros_like(t), torch.zeros_like(t)
        if bias is not None:
            r["dbias"] = torch.zeros(bias.shape, dtype=torch.float64, device=dev)
            e["dbias"] = torch.zeros_like(r["dbias"])
    w = {n: torch.zeros_like(t) for n, t in r.items()}  # squares of the rms bounds
    first = 0
    for n in lens:
        s = slice(first, first + n)
        first += n
        if n == 0:
            continue
        i = torch.arange(n, device=dev)
        dist = i[:, None] - i[None, :]
        for h in range(hq):
            g = h // (hq // hkv)
            qh, kg, vg = q64[s, h], k64[s, g], v64[s, g]
            sc = scale * (qh @ kg.T)
            a = scale * (qh.abs() @ kg.abs().T)
            if bias is not None:
                which = torch.bucketize(dist.clamp(min=0),
                                        torch.tensor(starts, device=dev), right=True) - 1
                sc = sc + bias[h].double()[which]
                b = bias[h].double().abs()
                a = a + torch.where(b > 1e3, 0.0, b)[which]  # a masking value carries no weight
            sc = sc.masked_fill(dist < 0, -torch.inf)
            lse = torch.logsumexp(sc, 1)
            p = torch.where(torch.isneginf(lse)[:, None], 0.0, (sc - lse[:, None]).exp())
            o = p @ vg
            eps = 2.0 ** -16 * float(a.max()) + 2.0 ** -14
            e_o = (U + 2 * eps) * (p @ vg.abs()) + U * o.abs()
            r["o"][s, h], r["lse"][s, h] = o, lse
            e["o"][s, h], e["lse"][s, h] = e_o, 2 * eps + 2.0 ** -22 * lse.abs()
            r_o = U * U * (p * p @ vg ** 2) + (2 * eps * (p @ vg.abs())) ** 2
            w["o"][s, h], w["lse"][s, h] = r_o, e["lse"][s, h] ** 2
            r_o = r_o + (U * o) ** 2
            if d_o is None:
                continue
            do = d_o[s, h].double()
            dp = do @ vg.T
            ds = p * (dp - (do * o).sum(1, keepdim=True))
            e_d = (do.abs() * e_o).sum(1, keepdim=True) + 2.0 ** -16 * (do * o).abs().sum(1, True)
            e_p = p * (e_d + 2.0 ** -16 * (do.abs() @ vg.abs().T)) + 2 * eps * ds.abs()
            e_ds = e_p + U * ds.abs()
            r["dq"][s, h] = scale * (ds @ kg)
            e["dq"][s, h] = scale * (e_ds @ kg.abs())
            r["dk"][s, g] += scale * (ds.T @ qh)
            e["dk"][s, g] += scale * (e_ds.T @ qh.abs())
            r["dv"][s, g] += p.T @ do
            e["dv"][s, g] += (U + 2 * eps) * (p.T @ do.abs())
            r_d = (do ** 2 * r_o).sum(1, keepdim=True)
            f = 2 * eps * ds.abs() + 2.0 ** -16 * p * (do.abs() @ vg.abs().T)  # fp32 terms
            w["dq"][s, h] = scale ** 2 * (U * U * (ds ** 2 @ kg ** 2) + r_d * (p @ kg) ** 2
                                          + (f @ kg.abs()) ** 2)
            w["dk"][s, g] += scale ** 2 * (U * U * (ds.T ** 2 @ qh ** 2)
                                           + p.T ** 2 @ (r_d * qh ** 2) + (f.T @ qh.abs()) ** 2)
            w["dv"][s, g] += U * U * (p.T ** 2 @ do ** 2) + (2 * eps * (p.T @ do.abs())) ** 2
            if bias is not None:
                low = dist >= 0
                rows = torch.zeros(n, len(starts), dtype=torch.float64, device=dev)
                rows.scatter_add_(1, which, p.masked_fill(~low, 0))
                w["dbias"][h] += (r_d * rows ** 2).sum(0)
                fsum = torch.zeros(len(starts), dtype=torch.float64, device=dev)
                w["dbias"][h] += fsum.index_add_(0, which[low], f[low]) ** 2
                r["dbias"][h].index_add_(0, which[low], ds[low])
                e["dbias"][h].index_add_(0, which[low], e_p[low])
    for n in r:
        if n not in ("o", "lse"):
            e[n] += U * r[n].abs()
        e[n] *= 1 + 2.0 ** -6
        w[n] += (U * r[n]) ** 2 if n != "lse" else 0
    e["rms"] = {n: float(t[torch.isfinite(t)].sum().sqrt()) for n, t in w.items()}
    return r, e


def check(got, ref, err, names):
    for n in names:
        x, y, b = got[n].double(), ref[n], err[n]
        assert x.shape == y.shape, n
        gap = torch.where(x == y, 0.0, (x - y).abs())  # equal infinities
        assert torch.isfinite(gap).all(), f"{n}: not finite"
        over = gap - b
        assert float(over.max()) <= 1e-30, (
            f"{n}: off by {float(gap.flatten()[over.argmax()]):.3e}, "
            f"bound {float(b.flatten()[over.argmax()]):.3e}")
        if y.numel() >= 64:
            norm = float(gap.norm())
            assert norm <= err["rms"][n], f"{n}: norm {norm:.3e}, bound {err['rms'][n]:.3e}"
