"""Dense attention's autograd node: what it refuses."""
import pytest
import torch

from test_gpu_dense import _inputs, _status

pytestmark = pytest.mark.gpu


def test_forward_mode_is_refused():
    """In the inputs and in the gradient that the backward gets."""
    import torch.autograd.forward_ad as fw
    from block_sparse_attention_proxy_gb300 import dense_attention

    x = _inputs([70, 5], 4, 2, 64, 70)
    q = x["q"].requires_grad_(True)
    with fw.dual_level():
        with pytest.raises(NotImplementedError, match="forward-mode"):
            dense_attention(q, fw.make_dual(x["k"], x["v"]), x["v"], x["cu"])
        o = dense_attention(q, x["k"], x["v"], x["cu"])
        with pytest.raises(NotImplementedError, match="forward-mode"):
            torch.autograd.grad(o, q, fw.make_dual(x["do"], x["do"]))
    assert _status() == 0


def test_errors_of_the_backward_are_the_package_s_own():
    """A status of the library keeps its class and number on the way through the engine."""
    from block_sparse_attention_proxy_gb300 import MsaError, dense_attention

    x = _inputs([70, 5], 4, 2, 64, 71)
    q = x["q"].requires_grad_(True)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: t[:-1]):
        o = dense_attention(q, x["k"], x["v"], x["cu"])
    for _ in range(2):
        with pytest.raises(MsaError) as error:
            torch.autograd.grad(o, q, x["do"], retain_graph=True)
        assert error.value.status == 1
    with pytest.raises(MsaError):
        o.backward(x["do"])
    assert _status() == 0
