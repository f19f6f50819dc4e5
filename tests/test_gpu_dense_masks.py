"""Dense attention with large finite biases: masks by a large negative value, by a type's
lowest one, and tables whose entries are far from zero."""
import pytest
import torch

from dense_exact import compare, dense_exact
from test_gpu_dense import _call, _inputs, _status

pytestmark = pytest.mark.gpu

LOWEST, HIGHEST = torch.finfo(torch.bfloat16).min, torch.finfo(torch.bfloat16).max
LENS = [1, 2, 40, 300, 130]
STARTS = (0, 3, 40, 150)


def _tables(value):
    """Where a head's large entries are; every head but the first gets them."""
    def fill(bias, columns, values):
        for c, x in zip(columns, values):
            bias[1:, c] = x
        return bias

    return {
        # a document's first tokens have no other key
        "first": lambda b: fill(b, [0], [value]),
        "last": lambda b: fill(b, [3], [value]),
        "all": lambda b: fill(b, range(4), [value] * 4),
        # a row's largest entry changes along the document
        "falling": lambda b: fill(b, range(4), [value, value / 2, value / 4, 0.5]),
        "apart": lambda b: fill(b, range(4), [value, -value, value, float("-inf")]),
    }


@pytest.mark.parametrize("where", ["first", "last", "all", "falling", "apart"])
@pytest.mark.parametrize("value", [LOWEST, -1e9, -1e5, -100.0, 1e5, HIGHEST])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (3, 3, 128), (33, 1, 128)])
def test_large_finite_biases(hq, hkv, d, value, where):
    """Every output against the definition, and the public log-sum-exp."""
    from block_sparse_attention_proxy_gb300 import make_dense_params, msa_dense_fwd

    x = _inputs(LENS, hq, hkv, d, 50, nb=4)
    x["bias"] = _tables(value)[where](x["bias"])
    got = _call(x, STARTS)
    t = sum(LENS)
    o, got["lse"] = torch.empty_like(x["q"]), torch.empty(t, hq, device="cuda")
    msa_dense_fwd(make_dense_params(t, len(LENS), hq, hkv, d, 1.0, STARTS), x["cu"], x["q"],
                  x["k"], x["v"], x["bias"], o, None, got["lse"])
    assert _status() == 0
    assert torch.equal(o, got["o"])
    compare(got, dense_exact(x["q"], x["k"], x["v"], LENS, 1.0, x["bias"], STARTS, x["do"]))


@pytest.mark.parametrize("d", [64, 128])
def test_table_far_from_zero(d):
    """A constant added to a whole table changes nothing but the log-sum-exp: a long document
    whose buckets begin inside tiles near and far, with 512 added, where bf16 still tells
    the entries apart."""
    starts = (0, 1, 2, 5, 70, 200, 201, 640, 900)
    x = _inputs([1100, 77], 4, 2, d, 51, nb=9)
    x["bias"] = x["bias"].float().mul(4).round().mul(4).bfloat16()  # multiples of 4
    want = _call(x, starts)
    x["bias"] = (x["bias"].float() + 512).bfloat16()
    got = _call(x, starts)
    exact = dense_exact(x["q"], x["k"], x["v"], [1100, 77], 1.0, x["bias"], starts, x["do"])
    compare(got, exact)
    compare(want, exact)
    assert _status() == 0


@pytest.mark.parametrize("value", [float("inf"), float("nan"), HIGHEST])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (3, 3, 128), (33, 1, 64)])
def test_buckets_that_no_pair_reaches(hq, hkv, d, value):
    """Whatever they hold, they change nothing: buckets behind the longest document, which the
    idle rows and columns of its last tile would reach."""
    lens, starts = [70, 130, 3], (0, 5, 130, 131, 200)
    x = _inputs(lens, hq, hkv, d, 52, nb=5)
    x["bias"][:, 2:] = 0
    want = _call(x, starts)
    x["bias"][:, 2:] = value
    got = _call(x, starts)
    for n in want:
        assert torch.equal(got[n], want[n]), n
    assert _status() == 0


@pytest.mark.parametrize("value", [LOWEST, -1e9, 1e5])
@pytest.mark.parametrize("hq,hkv,d", [(64, 1, 64), (40, 2, 128), (8, 2, 64)])
def test_large_tables_and_many_documents(hq, hkv, d, value):
    """Tables that do not fit beside the tiles, in batches that go document by document."""
    lens, starts = [150, 0, 3] + [(11 * i) % 23 for i in range(66)], tuple(range(0, 128, 2))
    x = _inputs(lens, hq, hkv, d, 53, nb=64)
    x["bias"][1::3, :20] = value
    x["bias"][2::3, 5:] = value
    got = _call(x, starts)
    assert _status() == 0
    compare(got, dense_exact(x["q"], x["k"], x["v"], lens, 1.0, x["bias"], starts, x["do"]))
