"""The Python calls of the dense attention's C entry points: what they refuse on the host."""
import pytest
import torch


@pytest.mark.parametrize("which", ["q", "k", "v", "dO"])
@pytest.mark.parametrize("wrong", ["slice", "stride in params", "tokens", "heads", "head dim"])
def test_tensors_that_differ_from_the_params_are_refused(which, wrong):
    """A slice whose token stride the params do not carry would be read in other rows, a
    stride that the tensor does not have behind its end."""
    import block_sparse_attention_proxy_gb300 as m

    T, hq, hkv, d = 10, 4, 2, 64
    x = {n: torch.zeros(T, h, d, dtype=torch.bfloat16)
         for n, h in (("q", hq), ("k", hkv), ("v", hkv), ("dO", hq))}
    h = x[which].shape[1]
    stride = {}
    if wrong == "slice":
        x[which] = torch.zeros(T, h + 2, d, dtype=torch.bfloat16)[:, :h]
    elif wrong == "stride in params":
        stride["do_stride" if which == "dO" else which + "_stride"] = (h + 2) * d
    else:
        at = ["tokens", "heads", "head dim"].index(wrong)
        shape = list(x[which].shape)
        shape[at] += 1
        x[which] = torch.zeros(shape, dtype=torch.bfloat16)
    prm = m.make_dense_params(T, 1, hq, hkv, d, **stride)
    cu = torch.tensor([0, T], dtype=torch.int32)
    o, o_res = torch.zeros(T, hq, d, dtype=torch.bfloat16), torch.zeros(T, hq, d).bfloat16()
    lse, kv, ws = torch.zeros(T, hq), torch.zeros(T, hkv, d).bfloat16(), torch.zeros(1 << 16)
    if which != "dO":
        with pytest.raises(ValueError):
            m.msa_dense_fwd(prm, cu, x["q"], x["k"], x["v"], None, o, o_res, lse, stream=_Null())
    with pytest.raises(ValueError):
        m.msa_dense_bwd(prm, cu, x["q"], x["k"], x["v"], None, o, o_res, lse, x["dO"], o, kv, kv,
                        None, ws, stream=_Null())


class _Null:
    cuda_stream = 0


@pytest.mark.parametrize("which", ["q", "k", "v", "bias"])
def test_forward_mode_is_refused(which):
    """It would give a product of zero: there is no forward-mode derivative."""
    import block_sparse_attention_proxy_gb300 as m

    x = {n: torch.zeros(5, 2, 64, dtype=torch.bfloat16) for n in "qkv"}
    x["bias"] = torch.zeros(2, 3, dtype=torch.bfloat16)
    cu = torch.tensor([0, 5], dtype=torch.int32)
    with torch.autograd.forward_ad.dual_level():
        x[which] = torch.autograd.forward_ad.make_dual(x[which], torch.ones_like(x[which]))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            m.dense_attention(x["q"], x["k"], x["v"], cu, bias=x["bias"], bucket_starts=(0, 1, 2))


@pytest.mark.parametrize("hq,hkv", [(64, 1), (16, 16), (1024, 16)])
def test_workspace_of_the_table_gradient(hq, hkv):
    """The sums for 64 buckets take some MB beside the rows' statistics (12 bytes each), however
    many tokens there are."""
    import block_sparse_attention_proxy_gb300 as m

    for tokens in (1000, 1 << 20):
        size = m.msa_dense_bwd_workspace_size(m.make_dense_params(
            tokens, 5, hq, hkv, 64, bucket_starts=tuple(range(64))))
        assert 0 < size - 12 * tokens * hq < (12 << 20) + 160 * hq * 64 * 8
