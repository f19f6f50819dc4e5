"""Rotary positions against their definition in fp64."""
import math
import random

import pytest
import torch

from cache_reference import placed, positions_of, rotary_exact, within

pytestmark = pytest.mark.gpu

LENS = [1, 0, 5, 130, 64, 0, 33]


def _m():
    import block_sparse_attention_proxy_gb300 as m

    return m


def _rows(t, heads, d, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(t, heads, d, generator=g, device="cuda").to(dtype)


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _freq(dims, base=10000.0):
    return [base ** (-2 * i / dims) for i in range(dims // 2)]


def _check(got, x, positions, freq, **kw):
    want, limit = rotary_exact(x, positions, freq, **kw)
    within(got, want, limit)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,dims", [(64, 64), (64, 32), (128, 128), (128, 16), (80, 48), (256, 256),
                                    (16, 16), (96, 0)])
def test_layouts(dtype, interleaved, d, dims):
    m = _m()
    q, k = _rows(sum(LENS), 6, d, 1, dtype), _rows(sum(LENS), 2, d, 2, dtype)
    plan = m.rotary_plan(dims, interleaved=interleaved)
    assert plan.dims == dims
    pos = positions_of(LENS).tolist()
    for got, x in zip(m.rotary(q, k, plan, cu_seqlens=_cu(LENS)), (q, k)):
        assert got.dtype == dtype and got.is_contiguous()
        _check(got, x, pos, _freq(dims) if dims else [], interleaved=interleaved)
    assert m.msa_get_device_status() == 0


@pytest.mark.parametrize("hq,hkv", [(1, 1), (33, 1), (8, 8), (64, 8), (7, 0), (129, 3)])
@pytest.mark.parametrize("t", [1, 3, 700])
def test_heads_and_tokens(hq, hkv, t):
    m = _m()
    q, k = _rows(t, hq, 64, 3), _rows(t, hkv, 64, 4) if hkv else None
    got = m.rotary(q, k, m.rotary_plan(64), cu_seqlens=_cu([t]))
    assert hkv or got[1] is None
    for y, x in zip(got, (q, k)):
        if x is not None:
            _check(y, x, list(range(t)), _freq(64))


@pytest.mark.parametrize("positions,dtype", [
    ([0, 1, 2 ** 24 + 1, 2 ** 31 - 1, -1, -12345, -2 ** 31], torch.int32),
    ([2 ** 24 + 1, 2 ** 31, 2 ** 40 + 7, -2 ** 40, 2 ** 53 + 1, -1, 0], torch.int64)])
def test_far_positions(positions, dtype):
    """Exact turns wherever a position lies; fp32, so that a wrong turn shows."""
    m = _m()
    q = _rows(len(positions), 4, 128, 5, torch.float32)
    # frequencies rounded to 2^-64 of a turn: off by 2^-11 radians at 2^53
    got = m.rotary(q, None, m.rotary_plan(128), positions=torch.tensor(
        positions, dtype=dtype, device="cuda"))[0]
    want, limit = rotary_exact(q, positions, _freq(128))
    off = torch.tensor([abs(p) * 2.0 ** -65 * 6.2832 for p in positions], dtype=torch.float64)
    pair = (q[..., :64].abs() + q[..., 64:].abs()).double().cpu().repeat(1, 1, 2)
    within(got, want, limit + off[:, None, None] * pair)


def test_given_frequencies_amplitude_and_stretch():
    m = _m()
    r = random.Random(1)
    freq = [r.uniform(-4, 4) for _ in range(16)]
    q, at = _rows(40, 3, 64, 6, torch.float32), [r.randrange(100000) for _ in range(40)]
    plan = m.rotary_plan(32, frequencies=freq, amplitude=1.25)
    got = m.rotary(q, None, plan, positions=torch.tensor(at, device="cuda"))[0]
    _check(got, q, at, freq, amplitude=1.25)
    assert torch.equal(got[..., 32:], q[..., 32:])
    plan = m.rotary_plan(64, base=500.0, stretch=4.0)
    got = m.rotary(q, None, plan, positions=torch.tensor(at, device="cuda"))[0]
    _check(got, q, at, [f / 4 for f in _freq(64, 500.0)])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_behind_the_last_document(dtype):
    m = _m()
    q, k = _rows(50, 4, 64, 7, dtype), _rows(50, 2, 64, 8, dtype)
    q[37:] = float("nan")
    k[37:] = float("inf")
    plan = m.rotary_plan(32)
    got = m.rotary(q.requires_grad_(), k, plan, cu_seqlens=_cu([30, 7]))
    for y, x in zip(got, (q, k)):
        assert not y[37:].any()
        _check(y[:37], x[:37], positions_of([30, 7]).tolist(), _freq(32))
    g = torch.full_like(q, float("nan"))
    g[:37] = 1
    dq, = torch.autograd.grad(got[0], q, g)
    assert not dq[37:].any() and dq[:37].isfinite().all()


def test_strides():
    """Slices of a fused projection as they are; other layouts are copied."""
    m = _m()
    lens, plan = [60, 9], m.rotary_plan(128)
    fused = _rows(69, 4 + 2 + 2, 128, 9)
    q, k, v = fused.split([4, 2, 2], 1)
    want = m.rotary(q.contiguous(), k.contiguous(), plan, cu_seqlens=_cu(lens))
    odd = torch.empty(69 * 4 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(69, 4, 128)
    odd.copy_(q)
    turned = q.transpose(1, 2).contiguous().transpose(1, 2)
    for x in (q, odd, turned):
        got = m.rotary(x, k, plan, cu_seqlens=_cu(lens).long())
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    wide = _rows(1, 4, 128, 10).expand(69, 4, 128)  # every token the same row
    got = m.rotary(wide, None, plan, cu_seqlens=_cu(lens))[0]
    assert torch.equal(got, m.rotary(wide.contiguous(), None, plan, cu_seqlens=_cu(lens))[0])


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients(interleaved):
    """Against the formula, and against differences in fp32: the map is linear, so a difference of
    any size gives it, off by the roundings of two results."""
    m = _m()
    q, k = (_rows(sum(LENS), h, 64, s, torch.float32).requires_grad_() for h, s in ((4, 11), (2, 12)))
    plan, cu, pos = m.rotary_plan(48, interleaved=interleaved, amplitude=0.75), _cu(LENS), positions_of(LENS).tolist()
    y = m.rotary(q, k, plan, cu_seqlens=cu)
    up = [_rows(*x.shape, s, torch.float32) for x, s in zip(y, (13, 14))]
    grads = torch.autograd.grad(y, (q, k), up, retain_graph=True)
    for g, u in zip(grads, up):
        _check(g, u, pos, _freq(48), interleaved=interleaved, amplitude=0.75, inverse=True)
    step = _rows(*q.shape, 15, torch.float32)
    with torch.no_grad():
        far = m.rotary(q + step, None, plan, cu_seqlens=cu)[0]
    change = ((far - y[0]).double() * up[0].double()).sum()
    slope = (grads[0].double() * step.double()).sum()
    # each of the 2 results is off by 2^-21 of |a| + |b| at most
    size = (2.0 ** -20 * 4 * (q.abs() + step.abs()).double() * up[0].abs().double()).sum()
    assert abs(change - slope) <= size
    # one of the two, a broadcast gradient, another type of gradient
    one, = torch.autograd.grad(y[1], k, up[1], retain_graph=True)
    assert torch.equal(one, grads[1])
    one, = torch.autograd.grad(y[0].sum(), q, retain_graph=True)
    _check(one, torch.ones_like(q), pos, _freq(48), interleaved=interleaved, amplitude=0.75, inverse=True)
    row = _rows(1, 4, 64, 16, torch.float32).requires_grad_()  # a broadcast input
    g, = torch.autograd.grad(m.rotary(row.expand_as(q), None, plan, cu_seqlens=cu)[0], row, up[0])
    exact = grads[0].double()
    within(g[0], exact.sum(0), 2.0 ** -24 * len(pos) * exact.abs().sum(0))  # fp32 sums
    # the gradient's gradient is the rotation itself
    g, = torch.autograd.grad(y[0], q, up[0].requires_grad_(), create_graph=True)
    assert torch.equal(g, grads[0])
    back, = torch.autograd.grad(g, up[0], step)
    assert torch.equal(back, m.rotary(step, None, plan, cu_seqlens=cu)[0])
    assert m.msa_get_device_status() == 0


def test_saved_tensors_and_tangents():
    import torch.autograd.forward_ad as fw

    m = _m()
    q, plan, cu = _rows(20, 2, 64, 17).requires_grad_(), m.rotary_plan(64), _cu([20])
    g = _rows(20, 2, 64, 18)
    want, = torch.autograd.grad(m.rotary(q, None, plan, cu_seqlens=cu)[0], q, g)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.cpu(), lambda t: t.cuda()):
        y = m.rotary(q, None, plan, cu_seqlens=cu)[0]
    assert torch.equal(torch.autograd.grad(y, q, g)[0], want)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: t[:-1]):
        y = m.rotary(q, None, plan, cu_seqlens=cu)[0]
    with pytest.raises(m.MsaError):
        torch.autograd.grad(y, q, g)
    with fw.dual_level(), pytest.raises(NotImplementedError, match="forward-mode"):
        m.rotary(fw.make_dual(q, g), None, plan, cu_seqlens=cu)


def test_captured_with_its_backward():
    m = _m()
    q, k, plan, cu = _rows(90, 4, 128, 19), _rows(90, 2, 128, 20), m.rotary_plan(128), _cu([80, 10])
    up = [_rows(90, h, 128, 21) for h in (4, 2)]

    def step(x):
        y = m.rotary(*x, plan, cu_seqlens=cu)
        return [*y, *torch.autograd.grad(y, x, up)]

    want = step([q.clone().requires_grad_(), k.clone().requires_grad_()])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        x = [q.clone().requires_grad_(), k.clone().requires_grad_()]
        step(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = step(x)
        with torch.no_grad():
            for y in x:
                y.neg_()
        graph.replay()
    stream.synchronize()
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a, -b)
    for a, b in zip(got[2:], want[2:]):
        assert torch.equal(a, b)


def test_a_captured_backward_beside_a_live_graph_is_refused():
    m = _m()
    q, plan, cu = _rows(30, 2, 64, 22).requires_grad_(), m.rotary_plan(64), _cu([30])
    g = _rows(30, 2, 64, 23)
    live = m.rotary(q, None, plan, cu_seqlens=cu)[0]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with pytest.raises(RuntimeError, match="captured while"):
            with torch.cuda.graph(graph, stream=stream):
                torch.autograd.grad(m.rotary(q, None, plan, cu_seqlens=cu)[0], q, g)
    torch.cuda.synchronize()
    assert torch.autograd.grad(live, q, g)[0].isfinite().all()


def test_malformed_documents_are_flagged():
    m = _m()
    q, plan = _rows(30, 2, 64, 24), m.rotary_plan(64)
    for cu in ([1, 30], [0, 20, 10, 30], [0, 31], [0, 2 ** 32 + 30]):
        m.rotary(q, None, plan, cu_seqlens=torch.tensor(cu, device="cuda"))
        assert m.msa_get_device_status() == 6
    assert m.msa_get_device_status() == 0


def test_refusals():
    m = _m()
    q, k, plan, cu = _rows(10, 2, 64, 25), _rows(10, 1, 64, 26), m.rotary_plan(64), _cu([10])
    at = torch.arange(10, device="cuda")
    for error, call in (
            (TypeError, lambda: m.rotary(q.double(), None, plan, cu_seqlens=cu)),
            (TypeError, lambda: m.rotary(q.float(), k, plan, cu_seqlens=cu)),
            (TypeError, lambda: m.rotary(q.cpu(), None, plan, cu_seqlens=cu)),
            (TypeError, lambda: m.rotary(q, k, plan, positions=at.float())),
            (ValueError, lambda: m.rotary(q, k, plan)),
            (ValueError, lambda: m.rotary(q, k, plan, cu_seqlens=cu, positions=at)),
            (ValueError, lambda: m.rotary(q, k, plan, positions=at[:9])),
            (ValueError, lambda: m.rotary(q, k, plan, positions=at.cpu())),
            (ValueError, lambda: m.rotary(q, k[:9], plan, cu_seqlens=cu)),
            (ValueError, lambda: m.rotary(q[..., :48], None, plan, cu_seqlens=cu)),
            (ValueError, lambda: m.rotary(q[0], None, plan, cu_seqlens=cu)),
            (m.MsaError, lambda: m.rotary(_rows(4, 1, 272, 27), None, plan, positions=at[:4])),
            (m.MsaError, lambda: m.rotary(_rows(4, 1, 72, 27), None, plan, positions=at[:4]))):
        with pytest.raises(error):
            call()
    empty = m.rotary(q[:0], k[:0], plan, cu_seqlens=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert empty[0].shape == (0, 2, 64) and empty[1].shape == (0, 1, 64)
    empty = m.rotary(q[:0].requires_grad_(), k[:0], plan, positions=at[:0])
    assert empty[0].shape == (0, 2, 64)
    empty[0].sum().backward()
    assert m.msa_get_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_infinite_and_nan_elements(dtype, interleaved):
    """Each reaches its pair, with the sign that the angle gives it, and no other."""
    m = _m()
    q, r = _rows(60, 3, 64, 40, dtype), random.Random(41)
    for _ in range(200):
        value = r.choice([float("inf"), float("-inf"), float("nan")])
        q[r.randrange(60), r.randrange(3), r.randrange(64)] = value
    at = [r.randrange(0, 5000) for _ in range(60)]
    got = m.rotary(q, None, m.rotary_plan(48, interleaved=interleaved),
                   positions=torch.tensor(at, device="cuda"))[0]
    want, limit = rotary_exact(q, at, _freq(48), interleaved)
    assert want.isinf().any() and want.isnan().any()
    placed(got, want)
    within(got, want, limit)


@pytest.mark.parametrize("interleaved", [False, True])
def test_fp32_sines_keep_the_turn(interleaved):
    """Unit vectors come out as the cosine and the sine of the plan's turns.  sincospif is off by one step
    at most (2^-24 below 1) and the correction for what a float drops of the turn rounds once (2^-25);
    the turn itself is cut at 2^-32 (2^-29 radians), the second term of the angle sum is below 2^-47."""
    m = _m()
    g = torch.Generator().manual_seed(50)
    at = torch.cat([torch.arange(64), torch.randint(-2 ** 40, 2 ** 40, (8000,), generator=g)])
    x = torch.zeros(len(at), 2, 64, device="cuda")
    pair = slice(0, 64, 2) if interleaved else slice(0, 32)
    other = slice(1, 64, 2) if interleaved else slice(32, 64)
    x[:, 0, pair] = 1
    x[:, 1, other] = 1
    plan = m.rotary_plan(64, interleaved=interleaved)
    y = m.rotary(x, None, plan, positions=at.cuda())[0].double().cpu()
    turn = torch.tensor([[(f * p) % 2 ** 64 / 2 ** 64 for f in plan.frequencies] for p in at.tolist()],
                        dtype=torch.float64) * (2 * math.pi)
    limit = torch.full_like(turn, 2.0 ** -24 + 2.0 ** -25 + 2.0 ** -28)
    within(y[:, 0, pair], turn.cos(), limit)
    within(y[:, 0, other], turn.sin(), limit)
    within(y[:, 1, pair], -turn.sin(), limit)
    within(y[:, 1, other], turn.cos(), limit)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_sines_of_16_bit_results(dtype):
    """Elements that nearly cancel too.  sincospif is off by 2^-24 at most, the float that holds the turn
    by 2^-25 of half a turn, the turn itself by 2^-29 radians; the result is rounded once."""
    m = _m()
    g = torch.Generator().manual_seed(51)
    at = torch.randint(-2 ** 40, 2 ** 40, (8000,), generator=g)
    x = torch.zeros(len(at), 2, 64, device="cuda", dtype=dtype)
    x[:, 0, :32] = x[:, 1, 32:] = 1
    plan = m.rotary_plan(64)
    y = m.rotary(x, None, plan, positions=at.cuda())[0].double().cpu()
    turn = torch.tensor([[(f * p) % 2 ** 64 / 2 ** 64 for f in plan.frequencies] for p in at.tolist()],
                        dtype=torch.float64) * (2 * math.pi)
    c, s, fi = turn.cos(), turn.sin(), torch.finfo(dtype)
    assert (c.abs() < 2.0 ** -12).sum() > 10 and (s.abs() < 2.0 ** -12).sum() > 10
    off = 2.0 ** -24 + math.pi * 2.0 ** -25 + 2.0 ** -28
    for got, want in ((y[:, 0, :32], c), (y[:, 0, 32:], s), (y[:, 1, :32], -s), (y[:, 1, 32:], c)):
        within(got, want, off + fi.eps / 2 * (want.abs() + off + fi.tiny))
