"""The gradient of the bias table over many items."""
import pytest
import torch

from dense_exact import compare, dense_exact
from test_dense_exact_cpu import LAYOUTS, finds_mistakes
from test_gpu_dense import _call, _inputs, _status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_sums_over_many_items(d):
    """8192 documents of 8 tokens under 64 heads of one KV head, two tokens to a tile: documents
    A, then B, then A and B with the opposite gradient.  Items of a pair have exactly opposite
    sums, so the table's gradient is zero but for the addition of some 32768 items.  n terms
    of a CTA, about 220 items of which half build up, are off by n^2 2^-48 of n/2 terms: 2^-33 of
    all CTAs' terms together.  Sums rounded to fp32 after each item are off by some 2^-22."""
    n, doc, hq, starts = 2048, 8, 64, (0, 1, 3, 5)
    x = _inputs([doc, doc], hq, 1, d, 80, nb=4)
    one = []
    for i in (0, 1):  # one document alone
        y = {m: t[i * doc:(i + 1) * doc] for m, t in x.items() if m not in ("cu", "bias")}
        y.update(bias=x["bias"], cu=torch.tensor([0, doc], dtype=torch.int32, device="cuda"))
        one.append(_call(y, starts)["dbias"].double())
    y = {m: torch.cat([x[m][:doc].repeat(n, 1, 1), x[m][doc:].repeat(n, 1, 1)] * 2)
         for m in ("q", "k", "v", "do")}
    y["do"][2 * n * doc:] *= -1
    y.update(bias=x["bias"],
             cu=torch.arange(4 * n + 1, dtype=torch.int32, device="cuda") * doc)
    got = _call(y, starts)["dbias"].double()
    assert _status() == 0
    terms = 2 * n * float(one[0].abs().max() + one[1].abs().max())
    assert float(got.abs().max()) <= 2.0 ** -32 * terms, (float(got.abs().max()), terms)
    # and the sum itself: A and B only
    y = {m: (t if m == "bias" else t[:2 * n * doc + (m == "cu") * (2 * n + 1 - 2 * n * doc)])
         for m, t in y.items()}
    got = _call(y, starts)["dbias"].double()
    want = n * (one[0] + one[1])
    # the single documents' gradients are rounded to bf16, and so is the sum
    limit = 2.0 ** -8 * (n * (one[0].abs() + one[1].abs()) + want.abs()) + 2.0 ** -20 * terms
    assert ((got - want).abs() <= limit).all()


def _against_definition(lens, hq, hkv, d, starts, seed):
    """Within limits so tight that planted mistakes in the table's gradient are found."""
    x = _inputs(lens, hq, hkv, d, seed, nb=len(starts))
    got = _call(x, starts)
    assert _status() == 0
    want = dense_exact(x["q"], x["k"], x["v"], lens, 1.0, x["bias"], starts, x["do"])
    compare(got, want)
    finds_mistakes([{n: t.cpu() for n, t in y.items()} if i < 2 else y
                    for i, y in enumerate(want)])


@pytest.mark.parametrize("starts", LAYOUTS.values(), ids=LAYOUTS.keys())
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (3, 3, 128), (6, 2, 128)])
def test_bucket_layouts(starts, hq, hkv, d):
    _against_definition([1, 200, 65, 513], hq, hkv, d, starts, 81)


@pytest.mark.parametrize("d", [64, 128])
def test_buckets_far_away(d):
    """Past the distances whose starts are kept as bits."""
    _against_definition([9300], 2, 1, d,
                        (0, 10, 4000, 4001, 4040, 8190, 8192, 8200, 8201, 8215, 9000, 9001), 82)


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (8, 1, 128), (12, 4, 64)])
def test_more_than_64_documents(hq, hkv, d):
    lens = [300, 0, 17] + [(13 * i) % 71 for i in range(70)]
    _against_definition(lens, hq, hkv, d, (0, 1, 2, 4, 8, 30, 100, 250), 83)


def test_sums_beyond_the_largest_number():
    """A gradient that overflows is infinite with its sign, as a plain sum is: 400 documents of
    two tokens, each of whose second rows adds some 6e36 to bucket 0 and takes it from bucket 1."""
    lens = [2] * 400
    x = _inputs(lens, 4, 4, 64, 84, nb=2)
    x["do"] = x["v"] * 1e36
    got = _call(x, (0, 1))["dbias"]
    want = dense_exact(x["q"], x["k"], x["v"], lens, 1.0, x["bias"], (0, 1), x["do"])[0]["dbias"]
    assert float(want[:, 0].min()) > 3.5e38 and float(want[:, 1].max()) < -3.5e38
    assert torch.equal(got.double(), want.sign() * float("inf"))
    assert _status() == 0
