"""The definition and limits that GPU results are compared with: against independent forms, and
with planted mistakes in the bias table's gradient."""
import pytest
import torch

from dense_exact import compare, dense_exact


def _inputs(lens, hq, hkv, d, nb, seed):
    g = torch.Generator().manual_seed(seed)
    t = sum(lens)
    q, k, v, do = (torch.randn(t, h, d, generator=g) for h in (hq, hkv, hkv, hq))
    return ((q * d ** -0.5).bfloat16(), k.bfloat16(), v.bfloat16(), do.bfloat16(),
            torch.randn(hq, nb, generator=g).bfloat16())


def test_against_automatic_differentiation():
    lens, starts = [1, 30, 17], (0, 2, 9)
    q, k, v, do, bias = _inputs(lens, 4, 2, 8, 3, 1)
    bias[1] = -1e9
    bias[2, 0] = torch.finfo(torch.bfloat16).min
    bias[3, 2] = float("-inf")
    leaves = [x.double().requires_grad_(True) for x in (q, k, v, bias)]
    outs, first = [], 0
    for n in lens:
        s = slice(first, first + n)
        first += n
        i = torch.arange(n)
        dist = i[:, None] - i
        b = leaves[3][:, (dist[..., None] >= torch.tensor(starts)).sum(-1).clamp(min=1) - 1]
        sc = torch.einsum("qhd,khd->hqk", leaves[0][s], leaves[1][s].repeat_interleave(2, 1)) + b
        p = torch.softmax(sc.masked_fill(dist < 0, -torch.inf), -1)
        outs.append(torch.einsum("hqk,khd->qhd", p, leaves[2][s].repeat_interleave(2, 1)))
    o = torch.cat(outs)
    grads = torch.autograd.grad(o, leaves, do.double())
    r, _, _ = dense_exact(q, k, v, lens, 1.0, bias, starts, do)
    for x, n in zip((o, *grads), ("o", "dq", "dk", "dv", "dbias")):
        assert torch.allclose(r[n], x, rtol=1e-9, atol=1e-9), n


LAYOUTS = {
    "one": (0,), "unit": tuple(range(12)), "tile": (0, 63, 64, 65, 127, 128, 129),
    "far": (0, 1, 2, 4, 9, 40, 200, 100000), "sparse": (0, 300), "full": tuple(range(0, 640, 10)),
}


def finds_mistakes(want):
    right = want[0]["dbias"]
    compare({"dbias": right.bfloat16()}, want)
    if right.shape[1] > 1:
        for x in (0 * right, -right, right / 2, right.roll(1, 1), right.roll(1, 0)):
            with pytest.raises(AssertionError):
                compare({"dbias": x.bfloat16()}, want)


@pytest.mark.parametrize("starts", LAYOUTS.values(), ids=LAYOUTS.keys())
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (3, 3, 128), (6, 2, 128)])
def test_mistakes_in_the_table_gradient_are_found(starts, hq, hkv, d):
    """Zeros, the wrong sign, half of it, neighbouring buckets or heads exchanged.  (One bucket
    over all distances has the gradient zero, as dS of a row adds up to nothing.)"""
    lens, nb = [1, 200, 65, 513], len(starts)
    q, k, v, do, bias = _inputs(lens, hq, hkv, d, nb, 2)
    want = dense_exact(q, k, v, lens, 1.0, bias, starts, do)
    finds_mistakes(want)
    if nb == 1:
        with pytest.raises(AssertionError):
            compare({"dbias": (want[0]["dbias"] + 1.0).bfloat16()}, want)
