"""Dense attention: what is not a number shows in every result that depends on it."""
import pytest
import torch

from test_gpu_dense import _call, _inputs, _status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("where", ["k", "q", "bias"])
def test_rows_that_are_not_a_number(where, d):
    """NaN in a key, a query or a bucket: lse and o of the rows that see it, and dV of every key
    that such a row sees; -inf would say that those rows have no key."""
    from block_sparse_attention_proxy_gb300 import make_dense_params, msa_dense_fwd

    lens, starts, at = [300, 140], (0, 4, 90), 133
    x = _inputs(lens, 4, 2, d, 60, nb=3)
    t = sum(lens)
    clean = _call(x, starts)
    row = torch.arange(t, device="cuda")
    if where == "k":  # KV head 0 (query heads 0, 1), first document
        x["k"][at, 0] = float("nan")
        spoilt = ((row >= at) & (row < 300))[:, None].expand(t, 2)
    elif where == "q":
        x["q"][at, :2] = float("nan")
        spoilt = (row == at)[:, None].expand(t, 2)
    else:  # distances of 90 and more
        x["bias"][:2, 2] = float("nan")
        spoilt = torch.where(row < 300, row, row - 300)[:, None].expand(t, 2) >= 90
    got = _call(x, starts)
    o, lse = torch.empty_like(x["q"]), torch.empty(t, 4, device="cuda")
    msa_dense_fwd(make_dense_params(t, 2, 4, 2, d, 1.0, starts), x["cu"], x["q"], x["k"], x["v"],
                  x["bias"], o, None, lse)
    assert _status() == 0
    assert torch.equal(torch.isnan(lse[:, :2]), spoilt)
    assert torch.isfinite(lse[:, 2:]).all()
    assert torch.equal(torch.isnan(got["o"][:, :2]).all(-1), spoilt)
    assert torch.equal(got["o"][:, :2][~spoilt], clean["o"][:, :2][~spoilt])
    for i, n in ((0, 300), (300, 140)):  # keys up to a document's last spoilt row
        last = spoilt[i:i + n, 0].nonzero().max() + 1 if spoilt[i:i + n].any() else 0
        assert torch.isnan(got["dv"][i:i + last, 0]).all()
        assert torch.equal(got["dv"][i + last:i + n], clean["dv"][i + last:i + n])
    for n in ("o", "dq", "dk", "dv"):  # the other KV head
        h = slice(2, 4) if n in ("o", "dq") else slice(1, 2)
        assert torch.equal(got[n][:, h], clean[n][:, h]), n
