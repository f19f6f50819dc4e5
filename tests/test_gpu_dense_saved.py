"""Dense attention whose saved tensors come back in another layout: saved-tensor hooks."""
import pytest
import torch

from test_gpu_dense import _inputs, _status

pytestmark = pytest.mark.gpu

LENS, HQ, HKV, D, STARTS = [90, 170, 1], 4, 2, 64, (0, 3, 40)


def _layer(hooks=None):
    """Gradients of a fused projection whose slices are q, k and v, and of the table."""
    from block_sparse_attention_proxy_gb300 import dense_attention

    x = _inputs(LENS, HQ, HKV, D, 40, nb=3)
    fused = torch.cat([x["q"], x["k"], x["v"]], 1).contiguous().requires_grad_(True)
    bias = x["bias"].requires_grad_(True)

    def forward():
        q, k, v = fused.split([HQ, HKV, HKV], 1)
        return dense_attention(q, k, v, x["cu"], bias=bias, bucket_starts=STARTS)

    if hooks is None:
        o = forward()
    else:
        with hooks:
            o = forward()
    return torch.autograd.grad(o, (fused, bias), x["do"])


def _off_by(t, n):
    """The same values, n elements behind an aligned address."""
    y = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)[n:].view(t.shape)
    return y.copy_(t)


HOOKS = {
    "contiguous": (lambda t: t.clone(memory_format=torch.contiguous_format), lambda t: t),
    "one buffer": (lambda t: _off_by(t, 1), lambda t: t),
    "transposed": (lambda t: t.transpose(0, -1).contiguous(), lambda t: t.transpose(0, -1)),
}


@pytest.mark.parametrize("pack,unpack", HOOKS.values(), ids=HOOKS.keys())
def test_saved_tensors_in_another_layout(pack, unpack):
    """Packed slices of a fused projection, packed off 16 bytes, packed transposed: the
    gradients are those of the call without hooks, bit for bit."""
    want = _layer()
    got = _layer(torch.autograd.graph.saved_tensors_hooks(pack, unpack))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert _status() == 0


@pytest.mark.parametrize("pinned", [False, True])
def test_activation_offload(pinned):
    want = _layer()
    for a, b in zip(_layer(torch.autograd.graph.save_on_cpu(pin_memory=pinned)), want):
        assert torch.equal(a, b)
    assert _status() == 0


@pytest.mark.parametrize("unpack", [lambda t: t.cpu(), lambda t: t[:-1], lambda t: t.double()],
                         ids=["device", "size", "type"])
def test_other_saved_tensors_are_refused(unpack):
    """On the host, before any launch."""
    from block_sparse_attention_proxy_gb300 import msa_launch_count

    launches = []

    def count(t):
        launches.append(msa_launch_count())
        return unpack(t)

    with pytest.raises(RuntimeError, match="a saved tensor"):
        _layer(torch.autograd.graph.saved_tensors_hooks(lambda t: t, count))
    assert msa_launch_count() == launches[0]
    assert _status() == 0
