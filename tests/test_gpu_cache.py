"""The paged cache (append, attention of one new token, eviction) against its definitions in fp64."""
import pytest
import torch

from cache_reference import attend_exact, evict_exact, gather, placed, rotary_exact, within

pytestmark = pytest.mark.gpu


def _m():
    import block_sparse_attention_proxy_gb300 as m

    return m


def _status():
    return _m().msa_get_device_status()


def _normal(*shape, seed, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _filled(lens, page, hkv, d, seed, spare=1, scores=True, layout="slots"):
    """A cache whose pages belong to the sequences in random order, `spare` pages of the table
    behind each sequence's last one name no page of the cache; (cache, table, lens)."""
    m = _m()
    width = max(1, max(-(-n // page) for n in lens)) + spare
    pages = sum(-(-n // page) for n in lens) + 3
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            table[b, i] = order.pop()
    shape = (pages, page, hkv, d) if layout == "slots" else (pages, hkv, page, d)
    k, v = (_normal(*shape, seed=seed + i) for i in (1, 2))
    if layout == "heads":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    weight = position = None
    if scores:
        weight = torch.rand(pages, hkv, page, device="cuda",
                            generator=torch.Generator(device="cuda").manual_seed(seed + 3))
        position = torch.zeros(pages, hkv, page, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):
            for i in range(-(-n // page)):
                position[table[b, i]] = torch.arange(i * page, (i + 1) * page, device="cuda")
    return (m.PagedCache(k, v, weight, position), table.cuda(),
            torch.tensor(lens, dtype=torch.int32, device="cuda"))


# ------------------------------ attention ---------------------------------------


def _attend(lens, hq, hkv, d, page, seed=1, scale=None, accumulate=False, layout="slots", q=None,
            spoil=True):
    m = _m()
    cache, table, n = _filled(lens, page, hkv, d, seed, layout=layout)
    if q is None:
        q = _normal(len(lens), hq, d, seed=seed + 9)
    scale = d ** -0.5 if scale is None else scale
    host = table.cpu()
    if spoil:  # what lies behind a sequence's end, on its last page and on free ones
        used = torch.zeros(cache.k.shape[:2], dtype=torch.bool)
        for b, length in enumerate(lens):
            for i in range(-(-length // page)):
                used[host[b, i], :length - i * page] = True
        for x in (cache.k, cache.v):
            x[~used.cuda()] = float("nan")
    before = cache.weight.clone()
    o = m.paged_attention(q, cache, table, n, softmax_scale=scale, accumulate=accumulate)
    assert _status() == 0
    want, limit, weights = attend_exact(q, cache.k, cache.v, table, lens, scale)
    within(o, want, limit, "o")
    if accumulate:
        exact, bound = before.double().cpu(), torch.zeros(before.shape).double()
        flat = lambda x: x.transpose(1, 2)  # noqa: E731  [pages, page, Hkv]
        for b, length in enumerate(lens):
            gain, lim = weights[b]
            at = torch.arange(length)
            at = (host[b, at // page].long(), at % page)
            flat(exact)[at] += gain.T
            flat(bound)[at] += lim.T
        within(cache.weight, exact, bound + 2.0 ** -22 * exact, "weight")
    else:
        assert torch.equal(before, cache.weight)
    return o


LENS = {
    "one entry": [1], "two": [2, 1], "tile": [128, 127, 129], "none": [0, 0],
    "ragged": [0, 1, 15, 16, 17, 255, 256, 257, 0, 1000, 0],
    "long": [5003], "many": [3 * i % 71 for i in range(700)],
    "long and short": [4001, 3, 2, 900, 1],
}


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", LENS.values(), ids=LENS.keys())
def test_lengths(lens, d, accumulate):
    _attend(lens, 4, 2, d, 16, accumulate=accumulate)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (6, 2), (5, 1), (8, 1), (9, 1), (16, 1), (24, 2),
                                    (32, 1), (33, 1), (64, 1), (40, 8)])
def test_head_layouts(hq, hkv, d, accumulate):
    _attend([300, 0, 131, 1], hq, hkv, d, 32, seed=2, accumulate=accumulate)


@pytest.mark.parametrize("layout", ["slots", "heads"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_pages(page, d, layout):
    _attend([700, 257, 40, 0, 128], 8, 2, d, page, seed=3, layout=layout, accumulate=True)


def test_peaked_scores():
    """Scores of tens that rise along the entries: the reference moves in many tiles."""
    m = _m()
    cache, table, n = _filled([3000, 700], 64, 2, 128, 4)
    rise = torch.linspace(0.1, 3, 3000, device="cuda").bfloat16()
    for b, length in enumerate([3000, 700]):
        for i in range(-(-length // 64)):
            cache.k[table[b, i]] *= rise[i * 64]
    q = _normal(2, 8, 128, seed=5, scale=0.6)
    o = m.paged_attention(q, cache, table, n)
    want, limit, _ = attend_exact(q, cache.k, cache.v, table, [3000, 700])
    within(o, want, limit)


@pytest.mark.parametrize("accumulate", [False, True])
def test_infinite_and_nan_scores(accumulate):
    """-inf takes no weight, a sequence of nothing else gives zeros; +inf and NaN give NaN, in the
    heads and sequences that they reach."""
    m = _m()
    lens = [400, 300, 200, 200, 150]
    cache, table, n = _filled(lens, 16, 2, 64, 6)
    q = _normal(5, 4, 64, seed=7)
    q[:, :, 0] = 1
    cache.k[..., 0] = 0
    page = lambda b, i: (int(table[b, i // 16]), i % 16)  # noqa: E731
    for i in list(range(128)) + [200]:
        cache.k[page(0, i)][0, 0] = float("-inf")  # a whole tile, KV head 0
    for i in range(300):
        cache.k[page(1, i)][1, 0] = float("-inf")  # every entry, KV head 1
    cache.k[page(2, 150)][0, 0] = float("inf")
    cache.k[page(3, 20)][1, 0] = float("nan")
    before = cache.weight.clone()
    o = m.paged_attention(q, cache, table, n, softmax_scale=0.125, accumulate=accumulate)
    assert _status() == 0
    want, limit, weights = attend_exact(q, cache.k, cache.v, table, lens, 0.125)
    assert not o[1, 2:].any()
    assert o[2, :2].isnan().all() and o[3, 2:].isnan().all()
    want[2, :2] = want[3, 2:] = float("nan")
    within(o, want, limit)
    if accumulate:
        for i in (5, 127, 200):
            at = page(0, i)
            assert cache.weight[at[0], 0, at[1]] == before[at[0], 0, at[1]]
        gain = (gather(cache.weight.transpose(1, 2), table[1], 300)
                - gather(before.transpose(1, 2), table[1], 300))
        assert not gain[:, 1].any()


@pytest.mark.parametrize("lens", [[300, 200, 90], [3000, 200, 1111]])
def test_weights_of_infinite_and_nan_scores(lens):
    """NaN in every entry that a head with such a score has weighed, zero gain where all scores are
    -inf: whole rows and rows that CTAs share."""
    m = _m()
    cache, table, n = _filled(lens, 32, 2, 64, 74)
    q = _normal(3, 8, 64, seed=75)
    q[:, :, 0] = 1
    cache.k[..., 0] = 0
    for b, i, h, value in ((0, 150, 0, float("inf")), (1, 20, 1, float("nan")), (2, 89, 1, float("-inf"))):
        cache.k[int(table[b, i // 32]), i % 32, h, 0] = value
    for i in range(lens[2]):
        cache.k[int(table[2, i // 32]), i % 32, 0, 0] = float("-inf")
    cache.weight.zero_()
    o = m.paged_attention(q, cache, table, n, softmax_scale=0.125, accumulate=True)
    want, _, weights = attend_exact(q, cache.k, cache.v, table, lens, 0.125)
    placed(o, want, "o")
    for b, length in enumerate(lens):
        gain = gather(cache.weight.transpose(1, 2), table[b], length).T
        placed(gain, weights[b][0], "weight")
    assert not gain[0].any() and gain[1].sum() > 3.9 and _status() == 0


def test_infinite_values():
    """An infinite element of v makes its column of o infinite, whatever its weight's roundings."""
    m = _m()
    lens = [300, 2000, 40]
    for d, hq in ((64, 4), (128, 16)):
        cache, table, n = _filled(lens, 64, 2, d, 65)
        for b, i, h, x, value in ((0, 7, 0, 3, float("inf")), (0, 299, 1, 0, float("-inf")),
                                  (1, 1500, 0, 63, float("inf")), (1, 3, 0, 63, float("inf")),
                                  (1, 9, 1, 5, float("inf")), (1, 1999, 1, 5, float("-inf"))):
            cache.v[int(table[b, i // 64]), i % 64, h, x] = value
        cache.k[int(table[0, 0]), 7, 0] = 0
        q = _normal(3, hq, d, seed=66, scale=0.1)
        q[0, 0] = 0  # all weights equal: their lower parts may be zero
        o = m.paged_attention(q, cache, table, n)
        want, limit, _ = attend_exact(q, cache.k, cache.v, table, lens)
        assert want.isinf().any() and want.isnan().any()
        assert torch.equal(o.isinf().cpu(), want.isinf()) and torch.equal(o.isnan().cpu(), want.isnan())
        assert torch.equal(o.double().cpu()[want.isinf()], want[want.isinf()])
        within(o, want, limit)


def test_scores_at_the_lowest_values():
    """Finite scores of -1e30 and below keep their weights."""
    m = _m()
    cache, table, n = _filled([300], 64, 1, 64, 8)
    cache.k.zero_()
    q = torch.zeros(1, 2, 64, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = -1e15
    cache.k[..., 0] = 1e16  # -1e31
    o = m.paged_attention(q, cache, table, n)
    v = gather(cache.v, table[0], 300).double().mean(0)
    within(o[0], v.expand(2, 64), v.abs() * 2.0 ** -8 + 2.0 ** -12)


def test_shared_pages():
    """Sequences with a common beginning read the same pages."""
    m = _m()
    cache, table, n = _filled([700, 640, 650], 64, 2, 128, 9)
    table[1, :8] = table[0, :8]
    table[2, :10] = table[0, :10]
    q = _normal(3, 8, 128, seed=10, scale=0.1)
    o = m.paged_attention(q, cache, table, n)
    want, limit, _ = attend_exact(q, cache.k, cache.v, table, [700, 640, 650])
    within(o, want, limit)


def test_strides_and_integer_types():
    m = _m()
    lens = [333, 70, 128]
    cache, table, n = _filled(lens, 32, 2, 64, 11)
    q = _normal(3, 8, 64, seed=12)
    want = m.paged_attention(q, cache, table, n)
    wide = torch.full((3, table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + table.shape[1]] = table
    fused = torch.cat([_normal(3, 2, 64, seed=13), q, q], 1)
    for qq, tt, nn in ((fused[:, 2:10], wide[:, 2:2 + table.shape[1]], n),
                       (q.transpose(1, 2).contiguous().transpose(1, 2), table.long(), n.long()),
                       (q, table.t().contiguous().t(), torch.stack([n, n], 1)[:, 0])):
        assert torch.equal(m.paged_attention(qq, cache, tt, nn), want)
    both = torch.empty(cache.k.shape[0], 32, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    both[:, :, 0], both[:, :, 1] = cache.k, cache.v  # k and v in one buffer
    one = m.PagedCache(both[:, :, 0], both[:, :, 1])
    assert torch.equal(m.paged_attention(q, one, table, n), want)


def test_repeats_bit_for_bit():
    m = _m()
    lens = [2000, 10, 5000, 0, 129]
    runs = []
    for _ in range(3):
        cache, table, n = _filled(lens, 64, 4, 128, 14)
        q = _normal(5, 16, 128, seed=15)
        runs.append((m.paged_attention(q, cache, table, n, accumulate=True), cache.weight))
    for o, w in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(w, runs[0][1])


def test_a_sequence_does_not_affect_another():
    m = _m()
    lens = [300, 4000, 17]
    cache, table, n = _filled(lens, 64, 2, 128, 16)
    q = _normal(3, 8, 128, seed=17)
    clean = m.paged_attention(q, cache, table, n)
    for i in range(-(-4000 // 64)):
        cache.k[table[1, i]] = float("nan")
        cache.v[table[1, i]] = float("inf")
    got = m.paged_attention(q, cache, table, n)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2]) and got[1].isnan().all()


def test_offsets_past_32_bits():
    """Pages beyond 2^31 elements (and bytes) of a large cache."""
    m = _m()
    pages, page, hkv, d = 70000, 256, 2, 64  # 2.3e9 elements
    k = torch.zeros(pages, page, hkv, d, dtype=torch.bfloat16, device="cuda")
    weight = torch.zeros(pages, hkv, page, device="cuda")
    position = torch.zeros(pages, hkv, page, dtype=torch.int32, device="cuda")
    cache = m.PagedCache(k, torch.zeros_like(k), weight, position)
    table = torch.tensor([[pages - 1, 3, pages - 7], [5, pages - 9, pages - 2]], dtype=torch.int32,
                         device="cuda")
    new = [600, 520]
    cu = torch.tensor([0, 600, 1120], dtype=torch.int32, device="cuda")
    x = [_normal(1120, hkv, d, seed=s) for s in (18, 19)]
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    m.cache_append(cache, *x, table, none, cu_seqlens=cu)
    n = none + torch.tensor(new, device="cuda", dtype=torch.int32)
    q = _normal(2, 6, d, seed=20, scale=0.1)
    o = m.paged_attention(q, cache, table, n, accumulate=True)
    small = m.PagedCache(*(t[table.flatten().long()].contiguous() for t in cache[:2]))
    ids = torch.arange(6, device="cuda", dtype=torch.int32).view(2, 3)
    want, limit, _ = attend_exact(q, small.k, small.v, ids, new)
    within(o, want, limit)
    for b, c in enumerate(cu[:-1].tolist()):
        assert torch.equal(gather(small.k, ids[b], new[b]), x[0][c:c + new[b]])
    total = gather(cache.weight.transpose(1, 2), table[0], 600).double().sum(0)
    assert (total - 3).abs().max() < 1e-3  # three heads to a KV head
    left = m.cache_evict(cache, table, n, 400, 30)
    assert left.tolist() == [400, 400]
    assert gather(cache.position.transpose(1, 2), table[0], 400)[:, 0].sort()[0][-30:].tolist() == \
        list(range(570, 600))
    assert _status() == 0


# ------------------------------ append ------------------------------------------


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,dims", [(64, 64), (128, 48), (128, 128), (64, 0)])
@pytest.mark.parametrize("page", [16, 128])
def test_append(page, d, dims, interleaved):
    """Ragged new tokens behind ragged lengths: rows, positions and weights of exactly those
    entries, everything else left as it was; the queries' padding zero."""
    m = _m()
    before, new = [0, 100, 15, 16, 0, 300], [40, 1, 2, 0, 0, 131]
    lens = [a + b for a, b in zip(before, new)]
    cache, table, _ = _filled(lens, page, 2, d, 21)
    t, tail, hq = sum(new), 5, 6
    q, k, v = (_normal(t + tail, h, d, seed=22 + i) for i, h in enumerate((hq, 2, 2)))
    k[t:] = float("nan")
    cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    old = [x.clone() for x in cache]
    n = torch.tensor(before, dtype=torch.int32, device="cuda")
    plan = m.rotary_plan(dims, interleaved=interleaved)
    freq = [10000.0 ** (-2 * i / dims) for i in range(dims // 2)]
    got = m.cache_append(cache, k, v, table, n, cu_seqlens=cu, plan=plan, q=q)
    assert _status() == 0 and n.tolist() == before
    at = [a + i for a, b in zip(before, new) for i in range(b)]
    within(got[:t], *rotary_exact(q[:t], at, freq, interleaved=interleaved))
    assert not got[t:].any()
    turned, limit = rotary_exact(k[:t], at, freq, interleaved=interleaved)
    expect = [x.clone() for x in old]
    row = 0
    for b, (a, more) in enumerate(zip(before, new)):
        for i in range(a, a + more):
            p, s = int(table[b, i // page]), i % page
            within(cache.k[p, s], turned[row], limit[row])
            expect[0][p, s] = cache.k[p, s]
            expect[1][p, s] = v[row]
            expect[2][p, :, s], expect[3][p, :, s] = 0, i
            row += 1
    for x, y in zip(cache, expect):
        assert torch.equal(x, y)


def test_append_one_token_each():
    """Without cu_seqlens; given positions of either type; without rotation; no weights kept."""
    m = _m()
    lens = [5, 0, 128, 63]
    cache, table, n = _filled([x + 1 for x in lens], 64, 1, 64, 25)
    n = n - 1
    k, v = _normal(4, 1, 64, seed=26), _normal(4, 1, 64, seed=27)
    at = torch.tensor([7, 100000, 2 ** 31 - 1, -3], device="cuda")
    assert m.cache_append(cache, k, v, table, n, positions=at) is None
    for b, i in enumerate(lens):
        p, s = int(table[b, i // 64]), i % 64
        assert torch.equal(cache.k[p, s], k[b]) and torch.equal(cache.v[p, s], v[b])
        assert cache.position[p, 0, s] == at[b] and cache.weight[p, 0, s] == 0
    plan = m.rotary_plan(64)
    bare = m.PagedCache(cache.k, cache.v)
    for positions in (at, at.int()):
        m.cache_append(bare, k, v, table, n, positions=positions, plan=plan)
        want, limit = rotary_exact(k, at.tolist(), [10000.0 ** (-i / 32) for i in range(32)])
        for b, i in enumerate(lens):
            within(cache.k[int(table[b, i // 64]), i % 64], want[b], limit[b])
    assert _status() == 0


def test_append_equals_rotary():
    """The same rows as rotary's, bit for bit."""
    m = _m()
    cache, table, n = _filled([200], 16, 2, 128, 28)
    q, k, v = (_normal(200, h, 128, seed=29 + h) for h in (8, 2, 3))
    v = v[:, :2]
    plan = m.rotary_plan(128, stretch=4.0, trained_length=100, amplitude=1.1)
    cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    got = m.cache_append(cache, k, v, table, n * 0, cu_seqlens=cu, plan=plan, q=q)
    want = m.rotary(q, k, plan, cu_seqlens=cu)
    assert torch.equal(got, want[0])
    assert torch.equal(gather(cache.k, table[0], 200), want[1])
    assert torch.equal(gather(cache.v, table[0], 200), v)


# ------------------------------ eviction ----------------------------------------


def _evict(lens, keep, recent, page, hkv, d, seed=40, change=None, spare=1):
    m = _m()
    cache, table, n = _filled(lens, page, hkv, d, seed, spare=spare)
    if change:
        change(cache, table)
    moves = evict_exact(cache.weight, cache.position, table.cpu(), lens, keep, recent)
    expect = [x.clone() for x in cache]
    host = table.cpu()
    for (b, h), pairs in moves.items():
        if not pairs:
            continue
        f, t = (torch.tensor(x, device="cuda") for x in zip(*pairs))
        row = host[b].cuda().long()
        of, to = (row[f // page], f % page), (row[t // page], t % page)
        for i in (0, 1):
            expect[i][to[0], to[1], h] = cache[i][of[0], of[1], h]
        for i in (2, 3):
            expect[i][to[0], h, to[1]] = cache[i][of[0], h, of[1]]
    left = m.cache_evict(cache, table, n, keep, recent)
    assert _status() == 0
    assert left.dtype == torch.int32 and left.tolist() == [min(x, keep) for x in lens]
    assert n.tolist() == lens
    for x, y, name in zip(cache, expect, cache._fields):
        assert torch.equal(x.isnan(), y.isnan()) and torch.equal(x.nan_to_num(), y.nan_to_num()), name


@pytest.mark.parametrize("lens,keep,recent", [
    ([1], 1, 0), ([2], 1, 1), ([5, 4, 3, 0], 4, 2), ([129, 128, 127, 300], 128, 16),
    ([129] * 9, 128, 128), ([1000, 999, 64, 3], 64, 0), ([1000, 700, 640], 600, 599),
    ([5000, 100, 4001], 400, 33), ([9001], 9000, 100), ([20003, 600], 1500, 7),
    ([70, 67, 65, 64, 72, 73, 74], 65, 3), ([8, 7, 2, 1], 1, 1), ([4100, 4097], 4096, 4096),
    ([30005, 30008, 30009], 30001, 0)])
@pytest.mark.parametrize("page,d", [(16, 64), (64, 128)])
def test_evict(lens, keep, recent, page, d):
    _evict(lens, keep, recent, page, 3, d)


@pytest.mark.parametrize("lens,keep,recent,spare", [
    ([60000, 49153], 2000, 100, 1), ([200001], 3001, 50, 1), ([200100], 200001, 50, 1),
    ([26000, 30000] + [50] * 160, 500, 20, 1), ([1000, 7, 903], 900, 20, 50),
    ([904, 900, 901], 900, 20, 50), ([9010, 9003], 9002, 0, 300)])
def test_evict_long_rows_and_wide_tables(lens, keep, recent, spare):
    """Ranks that fit no block, rows of several blocks, tables much wider than the lengths."""
    _evict(lens, keep, recent, 256, 1, 64, spare=spare)


@pytest.mark.parametrize("seqs", [1, 4, 8, 9])
@pytest.mark.parametrize("more", [0, 1, 5000])
@pytest.mark.parametrize("pages", [64, 300])
def test_budgets_that_no_row_can_exceed(pages, more, seqs):
    """Long tables whose every entry fits the budget, through the Python and the C call."""
    m = _m()
    cache = m.paged_cache(pages + 1, 64, 8, 64, scores=True)
    table = torch.arange(pages, device="cuda", dtype=torch.int32).repeat(seqs, 1)
    n = torch.tensor([pages * 64 - 700 * i for i in range(seqs)], device="cuda").clamp(min=0).int()
    before = [x.clone() for x in cache]
    assert torch.equal(m.cache_evict(cache, table, n, pages * 64 + more, 128), n)
    left = torch.empty_like(n)
    c, t = m.make_cache(cache), m.make_table(table, n)
    size = m.msa_cache_evict_workspace_size(c, t, pages * 64 + more)
    assert size == 256
    m.msa_cache_evict(c, t, pages * 64 + more, 128, left, n.new_empty(0))
    assert torch.equal(left, n) and _status() == 0
    for x, y in zip(cache, before):
        assert torch.equal(x, y)


def test_evict_ties_and_unusual_weights():
    """Equal weights, zeros of both signs, infinities, NaN and negative numbers."""
    def change(cache, table):
        w = cache.weight
        w.copy_((w * 4).round() / 4 - 0.25)
        w[w == 0] = torch.where(torch.rand_like(w[w == 0]) < 0.5, -0.0, 0.0)
        w[torch.rand_like(w) < 0.01] = float("inf")
        w[torch.rand_like(w) < 0.01] = float("-inf")
        w[torch.rand_like(w) < 0.01] = float("nan")
        w[torch.rand_like(w) < 0.01] = -float("nan")

    for keep in (3, 100, 500, 790):
        torch.manual_seed(keep)
        _evict([800, 640, 900], keep, min(keep, 20), 32, 2, 64, change=change)


def test_evict_positions_in_any_order():
    """After earlier evictions the newest entries lie anywhere; far positions; all equal."""
    def shuffled(cache, table):
        cache.position.copy_(torch.randperm(cache.position.numel(), device="cuda").view_as(cache.position)
                             + (2 ** 31 - 1 - cache.position.numel()))

    def equal(cache, table):
        cache.position.fill_(-2 ** 31)

    torch.manual_seed(1)
    for change in (shuffled, equal):
        _evict([500, 300], 128, 60, 32, 2, 64, change=change)


def test_many_rows():
    _evict([i % 90 for i in range(300)], 40, 10, 16, 8, 64)


# ------------------------------ together ----------------------------------------


def test_answering_under_a_budget():
    """Prompts prefilled by dense_attention and appended, then steps of append, attention with
    weights, eviction: o of every step against the definition over the entries that are left."""
    m = _m()
    hq, hkv, d, page, keep, recent = 8, 2, 64, 16, 96, 24
    new = [90, 33, 150]
    t, plan = sum(new), m.rotary_plan(64)
    cu = torch.tensor([0, 90, 123, 273], dtype=torch.int32, device="cuda")
    q, k, v = (_normal(t, h, d, seed=60 + i) for i, h in enumerate((hq, hkv, hkv)))
    cache = m.paged_cache(64, page, hkv, d, scores=True)
    table = torch.randperm(64, generator=torch.Generator().manual_seed(1))[:36].view(3, 12).int().cuda()
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    rq, rk = m.rotary(q, k, plan, cu_seqlens=cu)
    first = m.dense_attention(rq, rk, v, cu, softmax_scale=d ** -0.5)
    assert torch.equal(m.cache_append(cache, k, v, table, lens, cu_seqlens=cu, plan=plan, q=q), rq)
    lens = lens + torch.tensor(new, device="cuda", dtype=torch.int32)
    ends = (cu[1:] - 1).long()
    o = m.paged_attention(rq[ends], cache, table, lens, softmax_scale=d ** -0.5, accumulate=True)
    # both compute the last token's row: each within half a step and its weights' roundings
    within(o, first[ends], 2.0 ** -6 * first[ends].abs() + 2.0 ** -7)
    text = lens.clone()
    for step in range(40):
        q, k, v = (_normal(3, h, d, seed=100 + 3 * step + i) for i, h in enumerate((hq, hkv, hkv)))
        rq = m.cache_append(cache, k, v, table, lens, positions=text, plan=plan, q=q)
        lens += 1
        text += 1
        o = m.paged_attention(rq, cache, table, lens, softmax_scale=d ** -0.5, accumulate=True)
        want, limit, _ = attend_exact(rq, cache.k, cache.v, table, lens.tolist(), d ** -0.5)
        within(o, want, limit, f"step {step}")
        moves = evict_exact(cache.weight, cache.position, table.cpu(), lens.tolist(), keep, recent)
        lens = m.cache_evict(cache, table, lens, keep, recent)
        assert lens.max() <= keep and (step or moves)
    for b in range(3):
        at = gather(cache.position.transpose(1, 2), table[b], int(lens[b]))
        for h in range(hkv):
            seen = at[:, h].sort()[0]
            assert (seen.diff() > 0).all()  # each token once, the newest ones all there
            assert seen[-recent:].tolist() == list(range(int(text[b]) - recent, int(text[b])))
    assert _status() == 0


def test_documented_steps_under_a_budget():
    """The module's own loop, run as it stands there with a smaller budget: each entry that is left has
    the position of its token, its key turned by that, and the newest ones are among them."""
    import re

    m = _m()
    lines = [x.strip() for x in m.cache.__doc__.splitlines() if x.startswith("    ")]
    step = [x for x in lines if re.match(r"q = cache_append|lens, at|o = paged|lens = cache_evict", x)]
    assert len(step) == 4
    step = "\n".join(step).replace("keep=4096", "keep=20").replace("recent=128", "recent=3")
    plan, hq, hkv, d, steps = m.rotary_plan(64), 4, 2, 64, 50
    table = torch.arange(8, device="cuda", dtype=torch.int32).view(2, 4)
    space = dict(cache_append=m.cache_append, paged_attention=m.paged_attention, plan=plan,
                 cache_evict=m.cache_evict, cache=m.paged_cache(8, 16, hkv, d, scores=True), table=table,
                 lens=torch.zeros(2, dtype=torch.int32, device="cuda"),
                 at=torch.zeros(2, dtype=torch.int64, device="cuda"))
    keys, values = [], []
    for i in range(steps):
        space |= dict(q=_normal(2, hq, d, seed=500 + i, scale=0.2), k=_normal(2, hkv, d, seed=600 + i),
                      v=_normal(2, hkv, d, seed=700 + i))
        keys.append(m.rotary(space["k"], None, plan, positions=torch.tensor([i, i], device="cuda"))[0])
        values.append(space["v"])
        exec(step, space)
        n = min(i + 1, 20)
        assert space["lens"].tolist() == [n, n] and space["at"].tolist() == [i + 1, i + 1]
        for b in range(2):
            at = gather(space["cache"].position.transpose(1, 2), table[b], n).tolist()
            for h in range(hkv):
                own = [x[h] for x in at]
                assert len(set(own)) == n and set(range(max(0, i - 2), i + 1)) <= set(own) and max(own) == i
    for b in range(2):
        k, v, at = (gather(x, table[b], 20) for x in (space["cache"].k, space["cache"].v,
                                                     space["cache"].position.transpose(1, 2)))
        for h in range(hkv):
            for e in range(20):
                t = int(at[e, h])
                assert torch.equal(k[e, h], keys[t][b, h]) and torch.equal(v[e, h], values[t][b, h])
    assert _status() == 0


def test_captured_steps():
    """A step captured once and replayed, two graphs with workspaces of their own side by side."""
    m = _m()
    hq, hkv, d, page, keep = 8, 2, 128, 64, 250

    class Run:
        def __init__(self, seed):
            width = -(-(keep + 1) // page)
            self.table = torch.arange(4 * width, device="cuda", dtype=torch.int32).view(4, width)
            self.lens = torch.full((4,), keep, device="cuda", dtype=torch.int32)
            self.cache = m.paged_cache(4 * width, page, hkv, d, scores=True)
            self.cache.k.copy_(_normal(*self.cache.k.shape, seed=seed))
            self.cache.v.copy_(_normal(*self.cache.v.shape, seed=seed + 1))
            self.cache.position.copy_(torch.arange(page, device="cuda").expand_as(self.cache.position))
            self.text = self.lens.clone()
            self.plan = m.rotary_plan(d)
            self.q, self.k, self.v = (_normal(4, h, d, seed=seed + 2 + i)
                                      for i, h in enumerate((hq, hkv, hkv)))
            self.o = torch.zeros_like(self.q)

        def step(self):
            q = m.cache_append(self.cache, self.k, self.v, self.table, self.lens,
                               positions=self.text, plan=self.plan, q=self.q)
            self.text.add_(1)
            self.o.copy_(m.paged_attention(q, self.cache, self.table, self.lens + 1,
                                           accumulate=True))
            m.cache_evict(self.cache, self.table, self.lens + 1, keep, 50)

        def state(self):
            return [self.o.clone(), *(x.clone() for x in self.cache)]

    want = []
    for seed in (70, 80):
        run = Run(seed)
        for _ in range(6):
            run.step()
        want.append(run.state())
    runs, graphs, streams = [Run(70), Run(80)], [], []
    for run in runs:
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            run.step()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                run.step()
        graphs.append(graph)
        streams.append(stream)
    for _ in range(5):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for run, w in zip(runs, want):
        for a, b in zip(run.state(), w):
            assert torch.equal(a, b)
    assert _status() == 0


@pytest.mark.parametrize("start,hq,hkv,d,page", [
    ([5, 100, 77], 8, 2, 128, 64),             # rows of one tile: no join
    ([700, 20, 3001, 129], 8, 8, 64, 16),      # shared rows
    ([300, 2000], 64, 1, 128, 128),
])
def test_each_call_uses_all_that_the_last_one_wrote(start, hq, hkv, d, page):
    """Calls whose every input comes from the call before: in a row and captured as with the device
    idle before each."""
    m = _m()
    keep, layers, plan = max(start) - 3, 4, m.rotary_plan(d)
    q0, k0, v0 = (_normal(len(start), h, d, seed=300 + i) for i, h in enumerate((hq, hkv, hkv)))
    scale = d ** -0.5

    def build():
        out = []
        for i in range(layers):
            cache, table, n = _filled([x + 2 for x in start], page, hkv, d, 310 + 5 * i, spare=0)
            out.append((cache, table, n - 2))
        return out

    def run(state, idle):
        def done(x):
            if idle:
                torch.cuda.synchronize()
            return x
        q = q0
        for cache, table, lens in state:
            k, v = q[:, :hkv] + k0, q[:, -hkv:] + v0
            q = done(m.cache_append(cache, done(k), done(v), table, lens, plan=plan, q=q))
            o = done(m.paged_attention(q, cache, table, done(lens + 1), scale, accumulate=True))
            kept = done(m.cache_evict(cache, table, lens + 1, keep, 4))
            o2 = done(m.paged_attention(o, cache, table, kept, scale))
            q, _ = m.rotary(o2, o[:, :hkv], plan, positions=kept)
            done(q)
            q = done(m.paged_attention(q, cache, table, kept, scale)) + q
        return q

    state = build()
    want = run(state, True)
    wanted = [x.clone() for c, _, _ in state for x in c]
    for captured in (False, True):
        for _ in range(3):
            state = build()
            torch.cuda.synchronize()
            if captured:
                stream = torch.cuda.Stream()
                with torch.cuda.stream(stream):
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph, stream=stream):
                        got = run(state, False)
                    graph.replay()
                torch.cuda.synchronize()
            else:
                got = run(state, False)
            assert torch.equal(got, want)
            for a, b in zip([x for c, _, _ in state for x in c], wanted):
                assert torch.equal(a, b)
    assert _status() == 0


@pytest.mark.parametrize("captured", [False, True])
def test_streams_that_part_and_meet(captured):
    """One cache filled, read on two streams at once, copied, and evicted from where they meet."""
    m = _m()
    lens, hq, hkv, d, page = [300, 77, 1500], 8, 2, 128, 64
    plan, q0 = m.rotary_plan(d), _normal(3, hq, d, seed=400)
    k0, v0 = (_normal(3, hkv, d, seed=401 + i) for i in range(2))

    def run(cache, table, n, main, side):
        q = m.cache_append(cache, k0, v0, table, n, plan=plan, q=q0)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            a = m.paged_attention(q, cache, table, n + 1)
            a = m.rotary(a, None, plan, positions=n)[0]
        b = m.rotary(q, None, plan, positions=n)[0]
        b = m.paged_attention(b, cache, table, n + 1)
        main.wait_stream(side)
        c = m.paged_attention(a, cache, table, n + 1, accumulate=True)
        out = torch.empty_like(c)
        out.copy_(c)
        out = m.rotary(out, None, plan, positions=n)[0]
        kept = m.cache_evict(cache, table, n + 1, 64, 8)
        return a, b, c, out, kept

    def fresh():
        cache, table, n = _filled([x + 1 for x in lens], page, hkv, d, 403, spare=0)
        torch.cuda.synchronize()
        return cache, table, n - 1

    now = torch.cuda.current_stream()
    state = fresh()
    want = [*run(*state, now, now), *state[0]]
    for _ in range(3):
        main, side, state = torch.cuda.Stream(), torch.cuda.Stream(), fresh()
        torch.cuda.synchronize()
        with torch.cuda.stream(main):
            if captured:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=main):
                    got = run(*state, main, side)
                graph.replay()
            else:
                got = run(*state, main, side)
        torch.cuda.synchronize()
        for x, y in zip([*got, *state[0]], want):
            assert torch.equal(x, y)
    assert _status() == 0


@pytest.mark.parametrize("writer", ["cumsum", "cumsum of 64 bits", "eviction"])
def test_documents_that_the_last_call_wrote(writer):
    """cu_seqlens overwritten in place, by the call just before, for every rotation, its backward and
    every append: in a row and captured as with the device idle before each.  An eviction
    of rows within their budget writes their lengths, and lets the next kernel start early."""
    m = _m()
    wide = writer == "cumsum of 64 bits"
    T, seqs, layers, hq, hkv, d, page = 6000, 40, 5, 4, 2, 64, 16
    plan, g = m.rotary_plan(d), torch.Generator().manual_seed(450)
    cuts = [torch.cat([torch.tensor([0]), torch.randint(0, T + 1, (seqs - 1,), generator=g).sort()[0],
                       torch.tensor([T - 7 * i])]).clamp(max=T - 7 * i) for i in range(layers)]
    cuts = [c.to("cuda", torch.int64 if wide else torch.int32) for c in cuts]
    counts = [c.diff() for c in cuts]
    pages = -(-T // page)
    table = torch.arange(pages * seqs, device="cuda", dtype=torch.int32).view(seqs, pages)
    lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    q0, k0 = (_normal(T, h, d, seed=451 + i) for i, h in enumerate((hq, hkv)))
    # the cache whose evictions write documents: a row for each of their ends
    small = m.paged_cache(1, 256, 1, 64, scores=True)
    budget = torch.zeros(seqs + 1, T // 256 + 1, dtype=torch.int32, device="cuda")

    def run(cache, idle):
        def done(x):
            if idle:
                torch.cuda.synchronize()
            return x
        cu = torch.zeros(seqs + 1, dtype=cuts[0].dtype, device="cuda")
        out, q, k = [], q0, k0
        for i in range(layers):
            def documents():
                if writer == "eviction":
                    return done(m.cache_evict(small, budget, cuts[i], T, 0))
                done(torch.cumsum(counts[i], 0, dtype=cu.dtype, out=cu[1:]))
                return cu
            x, y = q.detach().requires_grad_(), k.detach().requires_grad_()
            fresh = documents()
            a, b = m.rotary(x, y, plan, cu_seqlens=fresh)
            done(a)
            back = torch.autograd.grad((a, b), (x, y), (q0, k0))
            done(back[0])
            fresh = documents()
            r = done(m.cache_append(cache, k, b.detach(), table, lens, cu_seqlens=fresh, plan=plan, q=q))
            out += [a.detach(), b.detach(), *back, r]
            done(cu.zero_())
            q, k = a.detach() + r, b.detach() + back[1]
        return out

    def empty():
        c = m.paged_cache(pages * seqs, page, hkv, d, scores=True)
        torch.cuda.synchronize()
        return c

    cache = empty()
    want = [*run(cache, True), *cache]
    for captured in (False, True):
        for _ in range(2):
            cache = empty()
            if captured:
                stream = torch.cuda.Stream()
                with torch.cuda.stream(stream):
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph, stream=stream):
                        got = run(cache, False)
                    graph.replay()
                torch.cuda.synchronize()
            else:
                got = run(cache, False)
            for a, b in zip([*got, *cache], want):
                assert torch.equal(a, b)
    assert _status() == 0


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("lens,hq,hkv,d,page", [([3000, 200, 0, 1020], 8, 2, 128, 64),
                                                ([9000], 16, 16, 64, 16), ([100, 900], 64, 1, 64, 256)])
def test_lengths_and_pages_changed_in_place(lens, hq, hkv, d, page, captured):
    """One table and one tensor of lengths, rewritten before each of many attentions over rows that
    CTAs share: as with the device idle before each."""
    m = _m()
    steps = 12
    cache, table0, top = _filled(lens, page, hkv, d, 460, spare=0)
    q = _normal(len(lens), hq, d, seed=470)
    weight0 = cache.weight.clone()
    at = [(top - 83 * i * i).clamp(min=0) for i in range(steps)]
    order = [torch.cat([torch.roll(r[r >= 0], i), r[r < 0]]) for i in range(steps) for r in table0]
    order = torch.stack(order).view(steps, *table0.shape).int()

    def run(idle):
        table, n, out = torch.empty_like(table0), torch.empty_like(top), []
        for i in range(steps):
            n.copy_(at[i])
            table.copy_(order[i])
            if idle:
                torch.cuda.synchronize()
            out.append(m.paged_attention(q, cache, table, n, 0.1, accumulate=i % 2 == 0))
            if idle:
                torch.cuda.synchronize()
        return out

    want, weights = run(True), cache.weight.clone()
    for _ in range(3):
        cache.weight.copy_(weight0)
        torch.cuda.synchronize()
        if captured:
            stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            with torch.cuda.stream(stream):
                with torch.cuda.graph(graph, stream=stream):
                    got = run(False)
                graph.replay()
        else:
            got = run(False)
        torch.cuda.synchronize()
        for x, y in zip([*got, cache.weight], [*want, weights]):
            assert torch.equal(x, y)
    assert _status() == 0


# ------------------------------ what is refused or flagged -----------------------


def test_bad_pages_and_lengths_are_flagged():
    """Found on the device; nothing outside the cache is touched, and the next call is sound."""
    m = _m()
    lens = [200, 90]
    for bad in ("page", "negative page", "length", "negative length"):
        cache, table, n = _filled(lens, 64, 2, 64, 50)
        q, kv = _normal(2, 4, 64, seed=51), _normal(2, 2, 64, seed=52)
        want = m.paged_attention(q, cache, table, n)
        old = [x.clone() for x in cache]
        tt, nn = table.clone(), n.clone()
        if "page" in bad:
            tt[0, 1] = cache.k.shape[0] if bad == "page" else -1
        else:
            nn[0] = table.shape[1] * 64 + 1 if bad == "length" else -1
            tt[0] = table[0, 0]  # what a length cut down to the table's reach would read
        m.paged_attention(q, cache, tt, nn, accumulate=True)
        assert _status() == 6
        m.cache_evict(cache, tt, nn, 30, 5)
        assert _status() == 6
        cache, table, n = _filled(lens, 64, 2, 64, 50)
        at = torch.full_like(n, 64) if "page" in bad else nn
        m.cache_append(cache, kv, kv, tt, at)
        assert _status() == 6
        if "page" in bad:  # sequence 0's token went nowhere
            for x, y in zip(cache, old):
                x[table[1].clamp(min=0).long()], y[table[1].clamp(min=0).long()] = 0, 0
                assert torch.equal(x, y)
        cache, table, n = _filled(lens, 64, 2, 64, 50)
        assert torch.equal(m.paged_attention(q, cache, table, n), want)
        assert _status() == 0


def test_refusals():
    m = _m()
    cache, table, n = _filled([100, 20], 64, 2, 64, 53)
    q, kv = _normal(2, 4, 64, seed=54), _normal(2, 2, 64, seed=55)
    plan, bare = m.rotary_plan(64), m.PagedCache(cache.k, cache.v)
    swap = lambda **kw: cache._replace(**kw)  # noqa: E731
    attend = lambda q=q, c=cache, t=table, n=n, **kw: m.paged_attention(q, c, t, n, **kw)  # noqa: E731
    append = lambda k=kv, v=kv, c=cache, t=table, n=n, **kw: m.cache_append(c, k, v, t, n, **kw)  # noqa: E731
    evict = lambda c=cache, keep=10, recent=2: m.cache_evict(c, table, n, keep, recent)  # noqa: E731
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    odd = torch.zeros(cache.k.numel() + 4, dtype=torch.bfloat16, device="cuda")[4:].view_as(cache.k)
    for error, call in (
            (TypeError, lambda: attend(q.float())), (TypeError, lambda: attend(c=swap(k=cache.k.half()))),
            (TypeError, lambda: attend(c=swap(k=cache.k.cpu()))), (ValueError, lambda: attend(q.cpu())),
            (ValueError, lambda: attend(q[:1])), (ValueError, lambda: attend(q[0])),
            (ValueError, lambda: attend(_normal(2, 4, 128, seed=1))),
            (ValueError, lambda: attend(c=swap(v=cache.v[:1]))),
            (ValueError, lambda: attend(c=swap(weight=cache.weight.transpose(1, 2)))),
            (TypeError, lambda: attend(c=swap(weight=cache.weight.double()))),
            (TypeError, lambda: attend(c=swap(position=cache.position.long()))),
            (TypeError, lambda: attend(t=table.float())), (ValueError, lambda: attend(t=table[0])),
            (ValueError, lambda: attend(n=n[:1])), (ValueError, lambda: attend(n=n.cpu())),
            (ValueError, lambda: attend(c=bare, accumulate=True)),
            (m.MsaError, lambda: attend(_normal(2, 3, 64, seed=1))),
            (m.MsaError, lambda: attend(_normal(2, 130, 64, seed=1))),
            (m.MsaError, lambda: attend(softmax_scale=0.0)),
            (m.MsaError, lambda: attend(softmax_scale=float("nan"))),
            (m.MsaError, lambda: attend(c=m.PagedCache(odd, cache.v))),
            (m.MsaError, lambda: attend(c=m.PagedCache(cache.k[:, :48], cache.v[:, :48]))),
            (NotImplementedError, lambda: attend(q.clone().requires_grad_())),
            (ValueError, lambda: append(k=kv[:1])), (TypeError, lambda: append(v=kv.float())),
            (ValueError, lambda: append(q=q)), (ValueError, lambda: append(q=q[:1], plan=plan)),
            (ValueError, lambda: append(cu_seqlens=cu[:2])), (TypeError, lambda: append(cu_seqlens=cu.float())),
            (ValueError, lambda: append(positions=n[:1])), (TypeError, lambda: append(positions=n.float())),
            (ValueError, lambda: append(plan=m.rotary_plan(128))),
            (NotImplementedError, lambda: append(k=kv.clone().requires_grad_())),
            (ValueError, lambda: evict(c=bare)), (ValueError, lambda: evict(c=swap(position=None))),
            (ValueError, lambda: evict(keep=0)), (ValueError, lambda: evict(recent=11)),
            (ValueError, lambda: evict(recent=-1))):
        with pytest.raises(error):
            call()
    assert _status() == 0
    none = table[:0]
    assert m.paged_attention(q[:0], cache, none, n[:0]).shape == (0, 4, 64)
    assert m.cache_evict(cache, none, n[:0], 5, 0).shape == (0,)
    assert m.cache_append(cache, kv[:0], kv[:0], none, n[:0]) is None
    with torch.no_grad():
        attend(q.clone().requires_grad_())
    version = cache.k._version
    append()
    assert cache.k._version > version
    assert _status() == 0


def test_weights_that_require_a_gradient_are_refused():
    """They are written in place; so is a tangent, which would stay as it was."""
    import torch.autograd.forward_ad as fw

    m = _m()
    cache, table, n = _filled([100, 20], 64, 2, 64, 53)
    q, kv = _normal(2, 4, 64, seed=54), _normal(2, 2, 64, seed=55)
    before = [x.clone() for x in cache]

    def calls(c):
        return (lambda: m.paged_attention(q, c, table, n, accumulate=True),
                lambda: m.cache_append(c, kv, kv, table, n), lambda: m.cache_evict(c, table, n, 10, 2))

    learned = cache._replace(weight=cache.weight.clone().requires_grad_())
    for call in calls(learned):
        with pytest.raises(NotImplementedError, match="requires a gradient"):
            call()
    with fw.dual_level():
        dual = cache._replace(weight=fw.make_dual(cache.weight, torch.ones_like(cache.weight)))
        for call in calls(dual):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
    for x, y in zip(cache, before):
        assert torch.equal(x, y)
    assert not m.paged_attention(q, learned, table, n).requires_grad  # does not write them
    with torch.no_grad():
        for call in calls(learned):
            call()
    assert _status() == 0


def test_c_entry_points_give_the_functions_results():
    """With workspaces of the size that is asked for, full of NaN; one byte less is refused."""
    m = _m()
    lens, hq = [1900, 770, 0], 6
    cache, table, n = _filled([x + 1 for x in lens], 32, 2, 64, 58)
    n = n - 1
    q, k, v = (_normal(3, h, 64, seed=59 + h) for h in (hq, 2, 3))
    v = v[:, :2]
    plan, other = m.rotary_plan(32), m.PagedCache(*(x.clone() for x in cache))
    rq = m.cache_append(cache, k, v, table, n, plan=plan, q=q)
    o = m.paged_attention(rq, cache, table, n + 1, 0.3, accumulate=True)
    left = m.cache_evict(cache, table, n + 1, 600, 9)

    c, t = m.make_cache(other), m.make_table(table, n)
    rp = m.make_rotary_params(3, hq, 2, 64, plan.frequencies)
    got = torch.empty_like(q)
    m.msa_cache_append(c, t, rp, None, None, q, k, v, got)
    assert torch.equal(got, rq)
    m.msa_rotary(m.make_rotary_params(3, hq, 0, 64, plan.frequencies), None, n, q, None, got, None)
    assert torch.equal(got, rq)
    more = n + 1
    t = m.make_table(table, more)
    prm = m.make_paged_params(hq, 0.3, accumulate=True)
    nan = lambda size: torch.full((-(-size // 4),), float("nan"), device="cuda").view(torch.uint8)[:size]  # noqa: E731
    for call, size in ((lambda ws: m.msa_paged_attention(c, t, prm, rq, got, ws),
                        m.msa_paged_attention_workspace_size(c, t, prm)),
                       (lambda ws: m.msa_cache_evict(c, t, 600, 9, n, ws),
                        m.msa_cache_evict_workspace_size(c, t, 600))):
        with pytest.raises(m.MsaError) as error:
            call(nan(size)[:-1])
        assert error.value.status == 3
        call(nan(size))
    assert _status() == 0
    assert torch.equal(got, o) and torch.equal(n, left)
    for x, y in zip(cache, other):
        assert torch.equal(x, y)


@pytest.mark.parametrize("lens,hq,hkv", [([4000, 0, 300, 129], 8, 2), ([5, 100, 0, 77], 20, 4),
                                         ([9000], 64, 1)])
def test_attention_over_its_queries(lens, hq, hkv):
    """Rows that CTAs share, rows of one CTA, and none: o may be q."""
    m = _m()
    cache, table, n = _filled(lens, 32, hkv, 64, 72, spare=0)
    q, other = _normal(len(lens), hq, 64, seed=73), m.PagedCache(*(x.clone() for x in cache))
    want = m.paged_attention(q, cache, table, n, 0.2, accumulate=True)
    c, t, p = m.make_cache(other), m.make_table(table, n), m.make_paged_params(hq, 0.2, accumulate=True)
    ws = torch.empty(m.msa_paged_attention_workspace_size(c, t, p), dtype=torch.uint8, device="cuda")
    m.msa_paged_attention(c, t, p, q, q, ws)
    assert torch.equal(q, want) and torch.equal(other.weight, cache.weight) and _status() == 0


def test_inference_mode():
    m = _m()
    with torch.inference_mode():
        cache = m.paged_cache(8, 16, 2, 64, scores=True)
        table = torch.arange(8, device="cuda", dtype=torch.int32).view(2, 4)
        lens = torch.tensor([0, 0], device="cuda", dtype=torch.int32)
        q, kv = _normal(2, 4, 64, seed=62), _normal(2, 2, 64, seed=63)
        plan = m.rotary_plan(64)
        for step in range(3):
            r = m.cache_append(cache, kv, kv, table, lens, plan=plan, q=q)
            lens = lens + 1
            o = m.paged_attention(r, cache, table, lens, accumulate=True)
        assert m.cache_evict(cache, table, lens, 2, 1).tolist() == [2, 2]
        assert (o.view(2, 2, 2, 64) == kv[:, :, None]).all()  # all values are the same
        assert m.rotary(q, None, plan, positions=lens)[0].shape == q.shape
    before = cache.k.clone()
    with torch.no_grad(), pytest.raises(RuntimeError, match="[Ii]nference"):
        m.cache_append(cache, kv, kv, table, lens)
    assert torch.equal(cache.k, before) and _status() == 0


def test_two_streams():
    """Calls that share nothing but the library, at once."""
    m = _m()
    cache, table, n = _filled([4000, 100, 2500], 64, 4, 128, 56)
    q = [_normal(3, 16, 128, seed=57 + i) for i in range(2)]
    want = [m.paged_attention(x, cache, table, n) for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(m.paged_attention(q[i], cache, table, n))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)
