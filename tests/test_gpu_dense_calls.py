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


@pytest.mark.parametrize("starts", [None, (0, 2, 70)])
def test_c_entry_points_give_the_function_s_results(starts):
    """msa_dense_fwd and msa_dense_bwd on slices of one buffer, with a workspace of the size that
    is asked for, full of NaN: the gradients of dense_attention, bit for bit; one byte less
    is refused."""
    import block_sparse_attention_proxy_gb300 as m

    lens, hq, hkv, d, nb = [190, 0, 77], 6, 2, 64, len(starts or ())
    x = _inputs(lens, hq, hkv, d, 92, nb=nb, tail=9)
    want = _call(x, starts, scale=0.5)
    t, heads = x["q"].shape[0], hq + 2 * hkv
    fused = torch.cat([x["q"], x["k"], x["v"]], 1).contiguous()
    q, k, v = fused.split([hq, hkv, hkv], 1)
    do = torch.zeros(t, 2 * hq, d, dtype=torch.bfloat16, device="cuda")[:, :hq].copy_(x["do"])
    prm = m.make_dense_params(t, len(lens), hq, hkv, d, 0.5, starts or (), heads * d, heads * d,
                              heads * d, 2 * hq * d)
    o, o_res, lse = torch.empty_like(x["q"]), torch.empty_like(x["q"]), torch.empty(
        t, hq, device="cuda")
    m.msa_dense_fwd(prm, x["cu"], q, k, v, x["bias"], o, o_res, lse)
    size = m.msa_dense_bwd_workspace_size(prm)
    ws = torch.full((size // 4,), float("nan"), device="cuda").view(torch.uint8)
    assert ws.numel() == size
    got = {"o": o, **{"d" + n: torch.full_like(x[n], float("nan")) for n in "qkv"}}
    got["dbias"] = torch.full_like(x["bias"], float("nan")) if nb else None

    def backward(ws):
        m.msa_dense_bwd(prm, x["cu"], q, k, v, x["bias"], o, o_res, lse, do, got["dq"],
                        got["dk"], got["dv"], got["dbias"], ws)

    with pytest.raises(m.MsaError) as error:
        backward(ws[:-1])
    assert error.value.status == 3
    backward(ws)
    assert _status() == 0
    for n in want:
        assert torch.equal(got[n], want[n]), n
