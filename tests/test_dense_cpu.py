"""Dense attention without a GPU: host refusals, bucket tables, and the fp64 definition that
the GPU tests compare with, against an independent form and against differences."""
import ctypes
import os

import pytest
import torch

from dense_reference import dense_reference


@pytest.fixture(scope="module")
def m():
    import block_sparse_attention_proxy_gb300 as m

    if not os.path.exists(m.LIB_PATH):
        from block_sparse_attention_proxy_gb300 import build

        build.build()
    m.load()
    return m


def _lens_inputs(lens, hq, hkv, d, seed, nb=0):
    g = torch.Generator().manual_seed(seed)
    t = sum(lens)
    x = [torch.randn(t, h, d, generator=g, dtype=torch.float64) for h in (hq, hkv, hkv, hq)]
    return (*x, torch.randn(hq, nb, generator=g, dtype=torch.float64) if nb else None)


def test_reference_equals_sdpa():
    lens = [5, 0, 17]
    q, k, v, _, _ = _lens_inputs(lens, 4, 2, 8, 1)
    r, _ = dense_reference(q, k, v, lens, 0.3)
    first = 0
    for n in lens:
        s = slice(first, first + n)
        first += n
        o = torch.nn.functional.scaled_dot_product_attention(
            *(t[s].transpose(0, 1)[None] for t in (q, k, v)), is_causal=True, scale=0.3,
            enable_gqa=True)[0].transpose(0, 1)
        assert torch.allclose(r["o"][s], o, rtol=1e-12, atol=1e-12)


def test_reference_gradients_against_differences():
    lens, starts = [3, 9], (0, 1, 2, 6)
    q, k, v, do, bias = _lens_inputs(lens, 4, 2, 4, 2, nb=4)
    r, _ = dense_reference(q, k, v, lens, 0.7, bias, starts, do)

    def loss():
        return (dense_reference(q, k, v, lens, 0.7, bias, starts)[0]["o"] * do).sum()

    step = 1e-5
    for t, name in ((q, "dq"), (k, "dk"), (v, "dv"), (bias, "dbias")):
        flat, grad = t.view(-1), r[name].reshape(-1)
        for i in range(0, flat.numel(), 7):
            x = float(flat[i])
            flat[i] = x + step
            up = loss()
            flat[i] = x - step
            down = loss()
            flat[i] = x
            # second differences of order 1 times step^2, rounding 1e-14 / step
            assert abs(float((up - down) / (2 * step) - grad[i])) < 1e-7, (name, i)


def test_bounds_hold_a_planted_mistake():
    """The bounds reject an output with one key's weight off by a few percent."""
    from dense_reference import check

    lens = [40]
    q, k, v, do, _ = _lens_inputs(lens, 2, 1, 64, 3)
    q = q / 8
    ref, err = dense_reference(q, k, v, lens, 1.0, None, None, do)
    check(ref, ref, err, list(ref))
    wrong, _ = dense_reference(q, k * (1 + 0.1 * (torch.arange(40) == 0)[:, None, None]), v, lens,
                               1.0, None, None, do)
    for n in ("o", "dq", "dk", "dv"):
        with pytest.raises(AssertionError):
            check(wrong, ref, err, [n])


def test_log_buckets(m):
    assert m.log_buckets(8, 128) == (0, 1, 2, 3, 4, 13, 40, 128)
    for n, far in ((4, 4), (5, 9), (32, 128), (33, 33), (64, 100000)):
        s = m.log_buckets(n, far)
        assert len(s) == n and s[0] == 0 and all(a < b for a, b in zip(s, s[1:]))
        assert s[-1] >= far
    for n, far in ((3, 10), (8, 7), (0, 0)):
        with pytest.raises(ValueError):
            m.log_buckets(n, far)


def test_params_layout(m):
    assert ctypes.sizeof(m.MsaDenseParams) == 6 * 4 + 8 + 4 * 8 + 8
    assert m.MsaDenseParams.bucket_starts.offset == 24
    assert m.MsaDenseParams.softmax_scale.offset == 64


OK = dict(total_tokens=1000, num_docs=3, hq=8, hkv=2, d=64)


@pytest.mark.parametrize("change", [
    dict(num_docs=0), dict(total_tokens=-1), dict(hq=7), dict(hkv=0), dict(hq=0), dict(d=96),
    dict(hq=130, hkv=2), dict(total_tokens=1 << 25), dict(num_docs=1 << 25), dict(softmax_scale=0.0),
    dict(softmax_scale=-1.0), dict(softmax_scale=float("nan")), dict(softmax_scale=float("inf")),
    dict(softmax_scale=3e38),
    dict(bucket_starts=(1, 2)), dict(bucket_starts=(0, 2, 2)), dict(bucket_starts=(0, 5, 4)),
    dict(bucket_starts=tuple(range(65))), dict(flags=1), dict(q_stride=8 * 64 - 8),
    dict(k_stride=2 * 64 + 4), dict(v_stride=-128), dict(do_stride=1 << 38)], ids=str)
def test_parameters_refused_on_the_host(m, change):
    good, bad = m.make_dense_params(**OK), m.make_dense_params(**{**OK, **change})
    assert m.msa_dense_bwd_workspace_size(good) > 0
    assert m.msa_dense_bwd_workspace_size(bad) == 0
    p = [ctypes.c_void_p(0x1000)] * 8
    assert m.load().msa_dense_fwd(ctypes.byref(bad), *p, None) in (1, 2)


def test_pointers_and_workspace_refused_on_the_host(m):
    lib, at = m.load(), ctypes.c_void_p
    good = m.make_dense_params(**OK)
    table = m.make_dense_params(**OK, bucket_starts=(0, 4))
    need = m.msa_dense_bwd_workspace_size(good)

    def fwd(prm, i=None, to=0):
        p = [0x1000] * 8
        if i is not None:
            p[i] = to
        return lib.msa_dense_fwd(ctypes.byref(prm), *map(at, p), None)

    def bwd(prm, i=None, to=0, size=need):
        p = [0x1000] * 14
        if i is not None:
            p[i] = to
        return lib.msa_dense_bwd(ctypes.byref(prm), *map(at, p), size, None)

    for i in (0, 1, 2, 3, 5):  # cu, q, k, v, o
        assert fwd(good, i) == 1
    for i in (1, 2, 3, 5, 6, 7):  # o_res and lse too: misaligned
        assert fwd(good, i, 0x1008) == 1
    assert fwd(table, 4) == 1 and fwd(table, 4, 0x1001) == 1
    for i in (0, 1, 2, 3, 5, 6, 7, 8, 9, 10, 11, 13):
        assert bwd(good, i) == 1
    assert bwd(table, 4) == 1 and bwd(table, 12) == 1
    assert bwd(good, 13, 0x1010) == 1
    for i in (5, 6):  # o, o_res: 32 bytes
        assert fwd(good, i, 0x1010) == 1
    for i in (9, 10, 11):  # dq, dk, dv
        assert bwd(good, i, 0x1010) == 1
    assert bwd(good, size=need - 1) == 3
    empty = m.make_dense_params(**{**OK, "total_tokens": 0})
    assert fwd(empty) == 0 and bwd(empty) == 0


def test_front_end_refusals(m):
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(TypeError):  # not on a GPU
        m.dense_attention(q, q, q, cu)
    with pytest.raises(TypeError):
        m.dense_attention(q.float(), q, q, cu)
    with pytest.raises(TypeError):
        m.dense_attention(q, q, None, cu)
