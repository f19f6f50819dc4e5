"""Calls of the dense attention at the edge of what it takes."""
import pytest
import torch

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
