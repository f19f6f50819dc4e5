"""Calls of the dense attention at the edge of what it takes."""
import pytest
import torch

from dense_exact import compare, dense_exact
from test_gpu_dense import _call, _inputs, _status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu", [[0, 2 ** 32 + 60, 2 ** 32 + 128], [2 ** 32, 60, 128],
                                [0, 60 - 2 ** 32, 128]])
def test_64_bit_documents_out_of_range_are_flagged(cu):
    """In 32 bits these would be the well-formed [0, 60, 128]."""
    x = _inputs([60, 68], 4, 2, 64, 90)
    want = _call(x)
    y = dict(x, cu=x["cu"].long())
    for n, t in _call(y).items():
        assert torch.equal(t, want[n]), n
    assert _status() == 0
    y["cu"] = torch.tensor(cu, device="cuda")
    _call(y)
    assert _status() == 6
    assert _status() == 0


@pytest.mark.parametrize("last", [2 ** 31 - 1, 2 ** 31 - 200, 2 ** 25])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (33, 1, 64), (2, 2, 128)])
def test_a_last_bucket_that_no_distance_reaches(hq, hkv, d, last):
    lens, starts = [1, 400, 130], (0, 1, 90, last)
    x = _inputs(lens, hq, hkv, d, 91, nb=4)
    got = _call(x, starts)
    compare(got, dense_exact(x["q"], x["k"], x["v"], lens, 1.0, x["bias"], starts, x["do"]))
    assert not got["dbias"][:, 3].any()
    assert _status() == 0
