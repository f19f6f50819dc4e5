"""Dense attention (dense_attention, msa_dense_fwd / msa_dense_bwd) against its fp64 definition."""
import pytest
import torch

from dense_reference import check, dense_reference

pytestmark = pytest.mark.gpu


def _inputs(lens, hq, hkv, d, seed, nb=0, tail=0, qs=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = sum(lens) + tail
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = {"q": (rnd(t, hq, d) * (qs * d ** -0.5)).bfloat16(), "k": rnd(t, hkv, d).bfloat16(),
         "v": rnd(t, hkv, d).bfloat16(), "do": rnd(t, hq, d).bfloat16(),
         "bias": rnd(hq, nb).bfloat16() if nb else None}
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    x["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    return x


def _call(x, starts=None, scale=1.0):
    """o and the gradients through autograd."""
    from block_sparse_attention_proxy_gb300 import dense_attention

    names = ["q", "k", "v"] + (["bias"] if x["bias"] is not None else [])
    leaf = {n: x[n].detach().requires_grad_(True) for n in names}
    o = dense_attention(leaf["q"], leaf["k"], leaf["v"], x["cu"], softmax_scale=scale,
                        bias=leaf.get("bias"), bucket_starts=starts)
    grads = torch.autograd.grad(o, [leaf[n] for n in names], x["do"])
    return {"o": o.detach(), **{"d" + n: g for n, g in zip(names, grads)}}


def _status():
    from block_sparse_attention_proxy_gb300 import msa_get_device_status

    return msa_get_device_status()


def _compare(x, lens, starts=None, scale=1.0):
    got = _call(x, starts, scale)
    assert _status() == 0
    ref, err = dense_reference(x["q"], x["k"], x["v"], lens, scale, x["bias"], starts, x["do"])
    check(got, ref, err, [n for n in got])
    return got


LENS = {
    "64 documents": [5 * i % 131 for i in range(64)],
    "65 documents": [129] + [7 * i % 97 for i in range(64)],
    "one": [1], "two": [2], "tile": [128], "tile+1": [129], "long": [777],
    "ragged": [1, 3, 127, 128, 129, 255, 257, 64], "empty": [0, 5, 0, 300, 0, 0, 1, 0],
    "many": [7] * 70,
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", LENS.values(), ids=LENS.keys())
def test_lengths(lens, d):
    _compare(_inputs(lens, 4, 1, d, 1), lens)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2), (6, 2), (8, 1), (10, 2), (14, 2), (16, 1),
                                    (33, 1), (64, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_head_layouts(hq, hkv, d):
    _compare(_inputs([150, 31, 260], hq, hkv, d, 2), [150, 31, 260])


STARTS = {
    "one": (0,), "unit": tuple(range(12)), "tile": (0, 63, 64, 65, 127, 128, 129),
    "far": (0, 1, 2, 4, 9, 40, 200, 100000), "sparse": (0, 300), "full": tuple(range(0, 640, 10)),
}


@pytest.mark.parametrize("starts", STARTS.values(), ids=STARTS.keys())
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (3, 3, 128), (6, 2, 128)])
def test_bias(starts, hq, hkv, d):
    lens = [1, 200, 65, 513]
    _compare(_inputs(lens, hq, hkv, d, 3, nb=len(starts)), lens, starts)


@pytest.mark.parametrize("hq,hkv", [(64, 1), (33, 1), (40, 2), (48, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_bias_of_many_heads(hq, hkv, d):
    """Groups whose table does not fit beside the tiles, up to 64 heads on one KV head."""
    lens, starts = [260, 1, 97], tuple(range(0, 256, 4))
    _compare(_inputs(lens, hq, hkv, d, 22, nb=64), lens, starts)


@pytest.mark.parametrize("d", [64, 128])
def test_bias_buckets_far_away(d):
    """Buckets that begin within one tile thousands of tokens back, past the distances whose
    starts are kept as bits."""
    lens, starts = [9300], (0, 10, 4000, 4001, 4040, 8190, 8192, 8200, 8201, 8215, 9000, 9001)
    _compare(_inputs(lens, 2, 1, d, 23, nb=len(starts)), lens, starts)


def test_softmax_scale():
    lens = [190, 77]
    x = _inputs(lens, 4, 2, 64, 4, nb=4, qs=2.0)
    _compare(x, lens, (0, 2, 8, 90), scale=0.37)


def test_peaked_scores():
    """Scores of tens: the running maximum moves in many tiles."""
    lens = [700, 300]
    x = _inputs(lens, 4, 1, 128, 5, qs=6.0)
    x["k"] *= torch.linspace(0.1, 3, sum(lens), device="cuda").bfloat16()[:, None, None]
    _compare(x, lens)


@pytest.mark.parametrize("masked", [float("-inf"), torch.finfo(torch.bfloat16).min])
def test_masking_bias(masked):
    """Distances whose bias is -inf (or the lowest value) carry no weight; a row whose only
    key is masked by -inf gives zeros and no gradient."""
    from block_sparse_attention_proxy_gb300 import (make_dense_params, msa_dense_fwd)

    lens, starts = [1, 40, 400], (0, 1, 5, 100, 200)
    x = _inputs(lens, 4, 2, 64, 6, nb=5)
    x["bias"][:, 3] = masked
    x["bias"][:2, 0] = float("-inf")  # heads 0, 1: a document's first token has no key left
    got = _compare(x, lens, starts)
    heads = torch.tensor([0, 1], device="cuda")
    firsts = x["cu"][:-1].long()
    for n in ("o", "dq"):
        assert not got[n][firsts][:, heads].any()
    t = sum(lens)
    o, lse = torch.empty_like(x["q"]), torch.empty(t, 4, device="cuda")
    msa_dense_fwd(make_dense_params(t, 3, 4, 2, 64, 1.0, starts), x["cu"], x["q"], x["k"], x["v"],
                  x["bias"], o, None, lse)
    assert torch.isneginf(lse[firsts][:, heads]).all()
    ref, err = dense_reference(x["q"], x["k"], x["v"], lens, 1.0, x["bias"], starts)
    check({"lse": lse}, ref, err, ["lse"])


@pytest.mark.parametrize("nb", [0, 3])
@pytest.mark.parametrize("lens", [[130, 60], [3] * 90], ids=["two", "many"])
def test_rows_behind_the_last_document(lens, nb):
    starts = (0, 4, 50) if nb else None
    x = _inputs(lens, 4, 2, 64, 7, nb=nb, tail=201)
    n = sum(lens)
    for name in ("q", "k", "v", "do"):
        x[name][n:] = float("nan")
    got = _call(x, starts)
    assert _status() == 0
    for name in ("o", "dq", "dk", "dv"):
        assert not got[name][n:].any(), name
    y = {k: (t if k in ("cu", "bias") else t[:n].contiguous()) for k, t in x.items()}
    alone = _call(y, starts)
    for name in alone:
        assert torch.equal(got[name][:n] if name != "dbias" else got[name], alone[name]), name


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_documents_do_not_affect_one_another(bad):
    lens = [70, 100, 200, 129]
    x = _inputs(lens, 6, 2, 128, 8)
    clean = _call(x)
    for i in (0, 2):  # spoilt documents
        s = slice(int(x["cu"][i]), int(x["cu"][i + 1]))
        for n in ("q", "k", "v", "do"):
            x[n][s] = bad
    got = _call(x)
    for i in (1, 3):
        s = slice(int(x["cu"][i]), int(x["cu"][i + 1]))
        for n in got:
            assert torch.equal(got[n][s], clean[n][s]), (n, i)


def test_strided_and_misaligned_inputs():
    """Slices of a fused projection, a broadcast gradient, a tensor off 16 bytes."""
    from block_sparse_attention_proxy_gb300 import dense_attention

    lens, hq, hkv, d = [90, 170], 4, 2, 64
    x = _inputs(lens, hq, hkv, d, 9)
    t = sum(lens)
    want = _call(x)
    fused = torch.cat([x["q"], x["k"], x["v"]], 1).contiguous().requires_grad_(True)
    q, k, v = fused.split([hq, hkv, hkv], 1)
    o = dense_attention(q, k, v, x["cu"])
    assert torch.equal(o, want["o"])
    (g,) = torch.autograd.grad(o, fused, x["do"])
    assert torch.equal(g, torch.cat([want["dq"], want["dk"], want["dv"]], 1))
    # heads before tokens, and an odd storage offset
    y = dict(x, q=x["q"].transpose(0, 1).contiguous().transpose(0, 1),
             k=torch.empty(x["k"].numel() + 1, dtype=torch.bfloat16, device="cuda")[1:]
             .view(x["k"].shape).copy_(x["k"]))
    got = _call(y)
    for n in want:
        assert torch.equal(got[n], want[n]), n
    # the gradient of a sum: every entry the same element
    one = torch.ones((), dtype=torch.bfloat16, device="cuda").expand(t, hq, d)
    got, ref = _call(dict(x, do=one)), _call(dict(x, do=one.contiguous()))
    for n in want:
        assert torch.equal(got[n], ref[n]), n


def test_no_gradient_of_some_inputs():
    from block_sparse_attention_proxy_gb300 import dense_attention

    x = _inputs([100], 4, 4, 64, 10)
    want = _call(x)
    k = x["k"].detach().requires_grad_(True)
    o = dense_attention(x["q"], k, x["v"], x["cu"])
    assert torch.equal(torch.autograd.grad(o, k, x["do"])[0], want["dk"])
    with torch.no_grad():
        assert torch.equal(dense_attention(x["q"], k, x["v"], x["cu"].long()), want["o"])


def test_repeats_bit_for_bit():
    lens = [500, 20, 900]
    starts = (0, 1, 2, 8, 30, 400)
    x = _inputs(lens, 12, 4, 64, 11, nb=6)
    a, b = _call(x, starts), _call(x, starts)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_calls_on_two_streams():
    x, y = _inputs([600, 333], 8, 2, 64, 12, nb=3), _inputs([901], 8, 2, 64, 13, nb=3)
    starts = (0, 7, 200)
    want = _call(x, starts), _call(y, starts)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a = _call(x, starts)
        with torch.cuda.stream(s2):
            b = _call(y, starts)
        torch.cuda.synchronize()
        for got, ref in zip((a, b), want):
            for n in ref:
                assert torch.equal(got[n], ref[n]), n


def test_two_captured_graphs_replay_on_new_inputs():
    """Forward and backward captured twice and replayed with new values and new document
    boundaries."""
    starts = (0, 3, 17, 300)
    shapes = [([300, 212], [500, 12]), ([77, 435], [0, 512])]
    xs = [_inputs(a, 4, 2, 64, 20 + i, nb=4) for i, (a, _) in enumerate(shapes)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for x in xs:
            _call(x, starts)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = _call(x, starts)
            graphs.append((g, out))
    torch.cuda.current_stream().wait_stream(side)
    for (x, (_, lens), i) in zip(xs, shapes, range(2)):
        new = _inputs(lens, 4, 2, 64, 30 + i, nb=4)
        for n in x:
            x[n].copy_(new[n])
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for x, (_, out) in zip(xs, graphs):
        want = _call(x, starts)
        for n in want:
            assert torch.equal(out[n], want[n]), n
    assert _status() == 0


def test_captured_backward_beside_an_eager_graph():
    """A leaf that a graph made on the default stream still holds: an error, and the capture
    ends; with that graph gone the same capture works."""
    from block_sparse_attention_proxy_gb300 import dense_attention

    x = _inputs([70], 4, 2, 64, 24)
    want = _call(x)["dq"]
    q = x["q"].detach().requires_grad_(True)
    eager = dense_attention(q, x["k"], x["v"], x["cu"])
    torch.cuda.synchronize()

    def capture():
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = dense_attention(q, x["k"], x["v"], x["cu"])
            return g, torch.autograd.grad(o, q, x["do"])[0]

    with pytest.raises(RuntimeError, match="outside the capture"):
        capture()
    assert torch.equal(torch.autograd.grad(eager, q, x["do"])[0], want)
    del eager
    g, dq = capture()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(dq, want)
    assert _status() == 0


def test_offsets_beyond_32_bits():
    """More than 2^31 elements of q: the last documents equal the same documents alone."""
    n, doc, hq, hkv, d = 280000, 70, 64, 8, 128
    lens = [doc] * (n // doc)
    x = _inputs(lens, hq, hkv, d, 14)
    assert x["q"].numel() > 2 ** 31
    got = _call(x)
    t0 = n - 3 * doc
    y = {k: t[t0:].contiguous() for k, t in x.items() if k not in ("cu", "bias")}
    y["cu"] = torch.arange(4, dtype=torch.int32, device="cuda") * doc
    y["bias"] = None
    want = _call(y)
    for name in want:
        assert torch.equal(got[name][t0:], want[name]), name
    assert _status() == 0


def test_more_items_than_the_gpu_holds():
    """Persistent CTAs go through several items of different lengths and KV heads, with
    partly filled rounds; ragged documents, 7 KV heads (no divisor of the SM count)."""
    lens = [1900, 3, 640, 1281, 129, 2000, 77]
    x = _inputs(lens, 21, 7, 64, 18, nb=9)
    _compare(x, lens, (0, 1, 3, 9, 27, 81, 243, 729, 1500))


@pytest.mark.parametrize("hq,hkv,nb", [(12, 12, 0), (10, 5, 0), (32, 16, 0), (24, 24, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_kv_heads_that_do_not_divide_the_grid(hq, hkv, nb, d):
    """More items than CTAs, rounds that end inside a slot's heads: every head of every token
    is written (the memory that the outputs get is full of NaN)."""
    lens = [1700, 5, 900, 1111]
    x = _inputs(lens, hq, hkv, d, 21, nb=nb)
    torch.cuda.synchronize()
    spoilt = [torch.full_like(x[n], float("nan")) for n in ("q", "q", "k", "k", "v")]
    spoilt.append(torch.full((64 << 20,), float("nan"), device="cuda"))
    del spoilt
    _compare(x, lens, (0, 2, 30, 400)[:nb] or None)


def test_front_end_refusals():
    from block_sparse_attention_proxy_gb300 import MsaError, dense_attention

    x = _inputs([64], 4, 2, 64, 19, nb=3)
    call = lambda **c: dense_attention(**{  # noqa: E731
        **dict(q=x["q"], k=x["k"], v=x["v"], cu_seqlens=x["cu"]), **c})
    for wrong, error in [
            (dict(q=x["q"].float()), TypeError), (dict(cu_seqlens=x["cu"].float()), TypeError),
            (dict(cu_seqlens=x["cu"].cpu()), ValueError), (dict(k=x["k"][:32]), ValueError),
            (dict(v=x["v"][:, :1]), ValueError), (dict(q=x["q"][:, :, 0]), ValueError),
            (dict(bias=x["bias"]), ValueError), (dict(bucket_starts=(0, 1, 2)), ValueError),
            (dict(bias=x["bias"], bucket_starts=(0, 1)), ValueError),
            (dict(bias=x["bias"].float(), bucket_starts=(0, 1, 2)), TypeError),
            (dict(bias=x["bias"], bucket_starts=(0, 2, 1)), MsaError),
            (dict(q=x["q"][:, :3]), MsaError), (dict(softmax_scale=0.0), MsaError),
            (dict(softmax_scale=float("nan")), MsaError),
            (dict(q=x["q"][..., :32], k=x["k"][..., :32], v=x["v"][..., :32]), MsaError)]:
        with pytest.raises(error):
            call(**wrong)
    try:
        call(softmax_scale=-1.0)
    except MsaError as e:
        assert e.status == 1
    assert _status() == 0


def test_graph_is_kept_and_differentiable_once():
    from block_sparse_attention_proxy_gb300 import dense_attention

    x = _inputs([150], 4, 2, 64, 20)
    q = x["q"].detach().requires_grad_(True)
    o = dense_attention(q, x["k"], x["v"], x["cu"])
    a = torch.autograd.grad(o, q, x["do"], retain_graph=True)[0]
    b = torch.autograd.grad(o, q, x["do"], create_graph=True)[0]
    assert torch.equal(a, b)
    with pytest.raises(RuntimeError):
        b.float().sum().backward()
    o = dense_attention(q, x["k"], x["v"], x["cu"])
    x["k"].add_(1)  # changed in place before the backward
    with pytest.raises(RuntimeError):
        torch.autograd.grad(o, q, x["do"])


def test_empty_batch():
    from block_sparse_attention_proxy_gb300 import dense_attention

    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    q, k = (torch.empty(0, h, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
            for h in (4, 2))
    bias = torch.randn(4, 2, device="cuda").bfloat16().requires_grad_(True)
    o = dense_attention(q, k, k, cu, bias=bias, bucket_starts=(0, 5))
    assert o.shape == (0, 4, 64)
    assert not torch.autograd.grad(o, bias, torch.empty_like(o))[0].any()


@pytest.mark.parametrize("cu", [[0, 90, 60, 128], [0, 64, 200], [5, 64, 128], [0, -1, 128]])
def test_malformed_documents_are_flagged(cu):
    """Found on the device: every index is checked there before it is used."""
    x = _inputs([128], 4, 2, 64, 15, nb=2)
    x["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    _call(x, (0, 9))
    assert _status() == 6
    assert _status() == 0


def test_dense_and_sparse_layers_together():
    """A dense layer feeding a sparse one, as they would be interleaved: where the sparse
    layer keeps every block, it equals the dense one, and gradients flow through both."""
    from block_sparse_attention_proxy_gb300 import dense_attention, msa_attention

    lens, hq, hkv, d = [500, 260], 4, 1, 64
    x = _inputs(lens, hq, hkv, d, 16, nb=3)
    g = torch.Generator(device="cuda").manual_seed(17)
    qp, kp = (torch.randn(sum(lens), hkv, 32, generator=g, device="cuda").bfloat16()
              for _ in range(2))
    # 4 blocks at most: top_k = 4 keeps them all
    sparse = msa_attention(x["q"], x["k"], x["v"], qp, kp, x["cu"], 4, kl_weight=0.0)
    dense = dense_attention(x["q"], x["k"], x["v"], x["cu"])
    ref, err = dense_reference(x["q"], x["k"], x["v"], lens)
    check({"o": dense}, ref, err, ["o"])
    check({"o": sparse}, ref, err, ["o"])
    leaves = [x[n].detach().requires_grad_(True) for n in ("q", "k", "v", "bias")]
    h = dense_attention(leaves[0], leaves[1], leaves[2], x["cu"], bias=leaves[3],
                        bucket_starts=(0, 4, 90))
    o = msa_attention(h, leaves[1], leaves[2], qp, kp, x["cu"], 4, kl_weight=0.0)
    grads = torch.autograd.grad(o, leaves, x["do"])
    for t, gr in zip(leaves, grads):
        assert gr.shape == t.shape and torch.isfinite(gr).all() and gr.any()
