"""Rotary positions and the paged cache without a GPU: plans, and what the C entry points refuse
before any CUDA call."""
import ctypes
import math
import os
import re
from fractions import Fraction

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import block_sparse_attention_proxy_gb300 as m

    if not os.path.exists(m.LIB_PATH):
        from block_sparse_attention_proxy_gb300 import build

        build.build()
    m.load()
    return m


@pytest.fixture(autouse=True)
def _without_a_gpu():
    """Some calls below pass every check on the host, with pointers of nothing: only where there is no
    GPU are they refused all the same."""
    if torch.cuda.is_available():
        pytest.skip("for machines without a GPU")


# ------------------------------ plans -------------------------------------------


@pytest.mark.parametrize("dims,kw", [(64, {}), (128, dict(base=1e6)), (32, dict(stretch=4.0)),
                                     (128, dict(stretch=8.0, trained_length=4096)),
                                     (16, dict(frequencies=[0.0, -1.0, 1e-9, 7.5, 6.25, 1, 2, 3]))])
def test_plan_frequencies(m, dims, kw):
    """Whole numbers within half of 2^-64 of a turn of the frequency, and the rule behind it."""
    plan = m.rotary_plan(dims, **kw)
    assert plan.dims == dims and len(plan.frequencies) == dims // 2
    two_pi = Fraction(int("6283185307179586476925286766559005768394338798750"), 10 ** 48)
    for i, word in enumerate(plan.frequencies):
        if "frequencies" in kw:
            f = kw["frequencies"][i]
        else:
            f = kw.get("base", 10000.0) ** (-2 * i / dims)
            s, part = kw.get("stretch", 1.0), 0.0
            if "trained_length" in kw:
                part = min(1.0, max(0.0, (4096 * f / (2 * math.pi) - 1) / 31))
            f *= part + (1 - part) / s
        off = Fraction(word, 2 ** 64) - Fraction(f) / two_pi
        off -= round(off)
        assert abs(off) <= Fraction(1, 2 ** 60) * 2 + abs(Fraction(f)) * Fraction(1, 2 ** 50)


def test_plan_stretch_leaves_fast_pairs(m):
    plain, far = m.rotary_plan(128), m.rotary_plan(128, stretch=16.0, trained_length=2048)
    assert far.frequencies[0] == plain.frequencies[0]
    assert abs(far.frequencies[-1] * 16 - plain.frequencies[-1]) <= 16
    ratio = [a / b for a, b in zip(plain.frequencies, far.frequencies)]
    assert all(1 - 1e-9 <= x <= 16 + 1e-9 for x in ratio)
    assert all(a <= b + 1e-9 for a, b in zip(ratio, ratio[1:]))


def test_plan_refusals(m):
    for kw in (dict(dims=8), dict(dims=24), dict(dims=-16), dict(dims=272), dict(dims=16, base=0),
               dict(dims=16, stretch=0), dict(dims=16, stretch=float("inf")),
               dict(dims=16, amplitude=float("nan")), dict(dims=16, trained_length=0),
               dict(dims=16, trained_length=10, low=3, high=3), dict(dims=16, frequencies=[1.0] * 7),
               dict(dims=16, frequencies=[float("nan")] * 8),
               dict(dims=16, frequencies=[1.0] * 8, stretch=2.0)):
        with pytest.raises(ValueError):
            m.rotary_plan(**kw)


def test_cpu_tensors_are_refused(m):
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        m.rotary(q, None, m.rotary_plan(64), positions=torch.arange(4))
    cache = m.paged_cache(2, 16, 2, 64, scores=True, device="cpu")
    table, lens = torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    for call in (lambda: m.paged_attention(q, cache, table, lens),
                 lambda: m.cache_append(cache, q, q, table, lens),
                 lambda: m.cache_evict(cache, table, lens, 1, 0)):
        with pytest.raises(TypeError):
            call()


# ------------------------------ C entry points ----------------------------------

P = 0x10000  # never read: every call below is refused first


def _cache(m, **kw):
    given = dict(k=P, v=P, weight=P, position=P, num_pages=9, page_size=64, hkv=2, d=64,
                 k_page_stride=8192, k_slot_stride=128, k_head_stride=64, v_page_stride=8192,
                 v_slot_stride=128, v_head_stride=64)
    return m._abi.MsaCache(**{**given, **kw})


def _table(m, **kw):
    return m._abi.MsaTable(**{**dict(pages=P, lens=P, num_seqs=3, max_pages=16, stride=16), **kw})


BAD_CACHES = [(1, dict(num_pages=0)), (1, dict(hkv=0)), (2, dict(d=96)), (2, dict(d=256)),
              (2, dict(page_size=8)), (2, dict(page_size=48)), (2, dict(page_size=512)),
              (2, dict(page_size=0)), (2, dict(hkv=1025)), (1, dict(k_page_stride=0)),
              (1, dict(k_slot_stride=-128)), (1, dict(v_head_stride=60)),
              (1, dict(v_page_stride=1 << 38))]
BAD_TABLES = [(1, dict(num_seqs=-1)), (1, dict(max_pages=0)), (1, dict(stride=15)),
              (2, dict(num_seqs=1 << 20)), (2, dict(max_pages=1 << 24, stride=1 << 24))]


def _calls(m, cache, table, hq=4, keep=500, recent=2, ws=1 << 30, **ptr):
    """Status of attention and eviction with everything else in order."""
    lib, by = m.load(), ctypes.byref
    p = m.make_paged_params(hq)
    at = {**dict(q=P, o=P, room=P, new=2 * P), **ptr}
    return (lib.msa_paged_attention(by(cache), by(table), by(p), at["q"], at["o"], at["room"], ws, None),
            lib.msa_cache_evict(by(cache), by(table), keep, recent, at["new"], at["room"], ws, None))


@pytest.mark.parametrize("status,kw", BAD_CACHES)
def test_bad_caches(m, status, kw):
    assert _calls(m, _cache(m, **kw), _table(m)) == (status, status)
    rp = m.make_rotary_params(3, 4, kw.get("hkv", 2), kw.get("d", 64), [1] * 8)
    assert m.load().msa_cache_append(ctypes.byref(_cache(m, **kw)), ctypes.byref(_table(m)),
                                     ctypes.byref(rp), 0, None, None, P, P, P, P, None) == status
    assert m.msa_paged_attention_workspace_size(_cache(m, **kw), _table(m), m.make_paged_params(4)) == 0
    assert m.msa_cache_evict_workspace_size(_cache(m, **kw), _table(m), 10) == 0


@pytest.mark.parametrize("status,kw", BAD_TABLES)
def test_bad_tables(m, status, kw):
    assert _calls(m, _cache(m), _table(m, **kw)) == (status, status)


def test_strides_of_single_rows_do_not_matter(m):
    """Of a dimension of size 1; the calls get as far as their workspace."""
    cache = _cache(m, num_pages=1, hkv=1, k_page_stride=1, v_head_stride=-3)
    assert _calls(m, cache, _table(m, num_seqs=1, stride=0), ws=0) == (3, 3)


def test_bad_pointers_and_workspaces(m):
    ok = _cache(m), _table(m)
    for kw in (dict(k=0), dict(v=P + 8), dict(weight=P + 2)):
        assert _calls(m, _cache(m, **kw), ok[1]) == (1, 1)
    for kw in (dict(pages=0), dict(lens=0), dict(lens=P + 1)):
        assert _calls(m, ok[0], _table(m, **kw)) == (1, 1)
    for kw in (dict(q=0), dict(q=P + 8), dict(o=0), dict(room=0), dict(room=P + 16)):
        assert _calls(m, *ok, **kw)[0] == 1
    for kw in (dict(new=0), dict(new=P), dict(new=P + 8), dict(room=0)):  # new lengths over the old
        assert _calls(m, *ok, **kw)[1] == 1
    prm = m.make_paged_params(4)
    assert _calls(m, *ok, ws=m.msa_paged_attention_workspace_size(*ok, prm) - 1)[0] == 3
    assert _calls(m, *ok, ws=m.msa_cache_evict_workspace_size(*ok, 500) - 1)[1] == 3


def test_bad_numbers(m):
    ok = _cache(m), _table(m)
    for hq, status in ((0, 1), (3, 1), (-2, 1), (130, 2), (2048, 2)):
        assert _calls(m, *ok, hq=hq)[0] == status
    for keep, recent in ((0, 0), (-1, 0), (5, 6), (5, -1)):
        assert _calls(m, *ok, keep=keep, recent=recent)[1] == 1
    assert _calls(m, _cache(m, weight=0), ok[1])[1] == 1
    assert _calls(m, _cache(m, position=0), ok[1])[1] == 1
    lib, by = m.load(), ctypes.byref
    for kw, status in ((dict(softmax_scale=0.0), 1), (dict(softmax_scale=float("inf")), 1),
                       (dict(softmax_scale=3e38), 1), (dict(flags=1), 1), (dict(q_stride=252), 1),
                       (dict(q_stride=64), 1)):
        p = m.make_paged_params(4, **kw)
        assert lib.msa_paged_attention(by(ok[0]), by(ok[1]), by(p), P, P, P, 1 << 30, None) == status
    p = m.make_paged_params(4, accumulate=True)
    assert m.msa_paged_attention_workspace_size(_cache(m, weight=0), ok[1], p) == 0
    many = _cache(m, hkv=1024, page_size=256), _table(m, max_pages=(1 << 22) - 1, stride=1 << 22)
    assert m.msa_paged_attention_workspace_size(*many, m.make_paged_params(1024)) == 0
    huge = _table(m, num_seqs=(1 << 20) - 1, max_pages=1 << 20, stride=1 << 20)
    assert m.msa_paged_attention_workspace_size(_cache(m), huge, p) == 0
    empty = _table(m, num_seqs=0)
    assert _calls(m, ok[0], empty, ws=0) == (0, 0)


def test_workspace_of_the_weights(m):
    """4 bytes a query head for every entry that the table names (a row's rounded up to 128), beside
    the shared rows' parts."""
    plain = m.msa_paged_attention_workspace_size(_cache(m), _table(m), m.make_paged_params(4))
    prm = m.make_paged_params(4, accumulate=True)
    for pages in (16, 17, 64):
        more = m.msa_paged_attention_workspace_size(_cache(m), _table(m, max_pages=pages, stride=pages),
                                                    prm) - plain
        assert 0 <= more - 3 * 4 * -(-pages * 64 // 128) * 128 * 4 <= 512
    assert 256 < plain < 4 << 20
    short = _table(m, max_pages=8, stride=8)  # rows that one CTA takes whole need none
    assert m.msa_paged_attention_workspace_size(_cache(m), short, m.make_paged_params(4)) == 256
    assert m.msa_cache_evict_workspace_size(_cache(m), short, 256) == 256  # few moves
    assert m.msa_cache_evict_workspace_size(_cache(m), _table(m), 257) > 6 * 2 * 257 * 8


def test_bad_rotations(m):
    lib, by = m.load(), ctypes.byref
    base = dict(total_tokens=10, hq=2, hkv=1, d=64, frequencies=[1] * 16)

    def call(cu=None, pos=P, q=P, k=8 * P, qo=32 * P, ko=64 * P, **kw):
        p = m.make_rotary_params(**{**base, **kw})
        return lib.msa_rotary(by(p), cu, pos, q, k, qo, ko, None)

    for kw in (dict(pos=None), dict(cu=P, num_docs=1), dict(num_docs=1), dict(cu=P, pos=None),
               dict(total_tokens=-1), dict(hq=-1), dict(hq=0, hkv=0), dict(interleaved=2),
               dict(inverse=2), dict(dtype=3), dict(position_bytes=2), dict(flags=1),
               dict(amplitude=float("inf")), dict(frequencies=[1] * 40), dict(q_stride=100),
               dict(q_stride=64), dict(k_stride=60), dict(q=0), dict(k=0), dict(qo=0), dict(ko=0),
               dict(q=P + 8), dict(ko=64 * P + 2), dict(pos=P + 1),
               dict(pos=P + 4, position_bytes=8), dict(qo=P), dict(ko=P + 32), dict(qo=8 * P),
               dict(cu=P + 2, pos=None, num_docs=1)):
        assert call(**kw) == 1, kw
    for kw in (dict(d=72, frequencies=[1] * 16), dict(d=272), dict(frequencies=[1] * 4),
               dict(hq=2048), dict(hq=3000), dict(total_tokens=1 << 25), dict(d=0, frequencies=[])):
        assert call(**kw) == 2, kw
    assert call(total_tokens=0, q=0, k=0) == 0
    assert call(total_tokens=0, q=0, k=0, pos=None) == 0  # of an empty tensor
    assert call(total_tokens=0, pos=None, num_docs=3, cu=P) == 0
    assert call(total_tokens=0, pos=None, dtype=3) == 1


def test_bad_appends(m):
    lib, by = m.load(), ctypes.byref

    def call(cu=None, pos=None, q=P, k=8 * P, v=9 * P, qo=32 * P, v_stride=0, **kw):
        p = m.make_rotary_params(**{**dict(total_tokens=3, hq=4, hkv=2, d=64, frequencies=[1] * 16),
                                    **kw})
        return lib.msa_cache_append(by(_cache(m)), by(_table(m)), by(p), v_stride, cu, pos, q, k, v,
                                    qo, None)

    for kw in (dict(hkv=1), dict(d=128), dict(dtype=1), dict(inverse=True), dict(total_tokens=4),
               dict(cu=P, num_docs=2), dict(cu=P), dict(num_docs=3), dict(v_stride=100),
               dict(v_stride=64), dict(k=0), dict(v=0), dict(v=9 * P + 8), dict(q=0), dict(qo=0),
               dict(qo=8 * P), dict(qo=9 * P), dict(pos=P + 2)):
        assert call(**kw) == 1, kw
    assert call(cu=P, num_docs=3, total_tokens=0, q=0, k=0, v=0) == 0


CUTS = r"""
#include <cstdio>
#include "cache_common.cuh"
using namespace msa;
// Every tile belongs to one team, every team with tiles has per or per + 1 of them in a row.
int main() {
  uint64_t r = 1;
  for (int k = 0; k < 4000; ++k) {
    r = r * 6364136223846793005ull + 1442695040888963407ull;
    const int teams = 1 + (int)((r >> 33) % 320);
    const long long total = k < 1000 ? k : (long long)((r >> 20) % (k % 2 ? 100000 : 1ll << 40));
    const PagedCuts c(total, teams);
    if (c.n != (total < teams ? total : teams) || c.cut(0) != 0 || c.cut(c.n) != total ||
        c.cut(c.n + 5) != total)
      return std::printf("%lld tiles, %d teams: ends\n", total, teams), 1;
    for (int i = 0; i < c.n; ++i) {
      const long long a = c.cut(i), b = c.cut(i + 1), n = b - a;
      if (n < 1 || n < c.per || n > c.per + 1 || c.team_of(a) != i || c.team_of(b - 1) != i ||
          c.team_of(a + n / 2) != i)
        return std::printf("%lld tiles, %d teams: team %d\n", total, teams, i), 1;
    }
  }
  for (long long a : {0ll, 7ll, 1ll << 31, (1ll << 32) - 1, 1ll << 32, 1ll << 52})
    for (long long b : {1ll, 3ll, (1ll << 32) - 1, 1ll << 32, 1ll << 33})
      if (quotient(a, b) != a / b) return std::printf("%lld / %lld\n", a, b), 1;
  return 0;
}
"""


def test_tiles_are_shared_out_without_gaps(tmp_path):
    from test_dense_host_cpu import run

    run(tmp_path, CUTS)


def test_struct_layouts(m):
    """As in the header on both machines: 10 + 1 (padding none) words, pointers and strides of 8 bytes."""
    a = m._abi
    assert ctypes.sizeof(a.MsaRotaryParams) == 10 * 4 + 8 + 2 * 8 + 2 * 4
    assert ctypes.sizeof(a.MsaCache) == 4 * 8 + 4 * 4 + 6 * 8
    assert ctypes.sizeof(a.MsaTable) == 2 * 8 + 2 * 4 + 8
    assert ctypes.sizeof(a.MsaPagedParams) == 2 * 4 + 8 + 2 * 4


def test_kernels_that_start_early_read_by_plain_loads():
    """They may be on the GPU before their inputs are written: read-only loads, which may move ahead of
    the wait for those, are not for them."""
    import block_sparse_attention_proxy_gb300 as package

    csrc = os.path.join(os.path.dirname(package.__file__), "csrc")
    early = []
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as f:
            code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
        if name != "cache_common.cuh" and "launch_early(" not in code:
            continue
        early.append(name)
        for word in ("__ldg", "ld.global.nc", "__restrict__", "doc_of_token(", "doc_of_block("):
            assert word not in code, f"{name}: {word}"
    assert early == ["cache_common.cuh", "k_evict.cu", "k_paged.cu", "k_rotary.cu"]


def _evict(m, cache, table, keep, room, ws):
    return m.load().msa_cache_evict(ctypes.byref(cache), ctypes.byref(table), keep, 0, 64 * P, room, ws,
                                    None)


@pytest.mark.parametrize("seqs,hkv", [(1, 1), (4, 8), (8, 8), (100, 8)])
@pytest.mark.parametrize("pages,keep", [(64, 4096), (64, 5000), (512, 32768), (4096, 1 << 30),
                                        (16, 1024)])
def test_budgets_that_no_row_can_exceed(m, seqs, hkv, pages, keep):
    """Nothing can move: no workspace is asked for, and none is missed."""
    cache, table = _cache(m, hkv=hkv), _table(m, num_seqs=seqs, max_pages=pages, stride=pages)
    assert m.msa_cache_evict_workspace_size(cache, table, keep) == 256
    assert _evict(m, cache, table, keep, None, 0) == 4  # there is no device


def test_sizes_of_256_say_that_nothing_is_used(m):
    """Every eviction that uses its workspace asks for more."""
    cache = _cache(m)
    for seqs in (1, 30, 32):
        for pages in (3, 17, 64, 700):
            table = _table(m, num_seqs=seqs, max_pages=pages, stride=pages)
            for keep in {1, 64, pages * 64 - 1, pages * 64, pages * 64 + 1, pages * 32}:
                size = m.msa_cache_evict_workspace_size(cache, table, keep)
                if size == 256:
                    assert _evict(m, cache, table, keep, None, 0) == 4
                else:
                    assert size > 256 and _evict(m, cache, table, keep, None, 0) == 1
                    assert _evict(m, cache, table, keep, P, size - 1) == 3


def test_rotated_rows_over_each_other_are_refused(m):
    """q_out [10, 2, 64] and k_out [10, 1, 64] of bf16: 2560 and 1280 bytes."""
    p = m.make_rotary_params(10, 2, 1, 64, [1] * 16)
    alone = {hq: m.make_rotary_params(10, hq, 2 - hq, 64, [1] * 16) for hq in (0, 2)}

    def call(qo, ko, p=p):
        return m.load().msa_rotary(ctypes.byref(p), None, P, P, 8 * P, qo, ko, None)

    far = 64 * P
    for ko in (far, far + 2544, far - 1264):
        assert call(far, ko) == 1
    for ko in (far + 2560, far - 1280):
        assert call(far, ko) == 4  # there is no device
    assert call(far, None, alone[2]) == 4 and call(None, far, alone[0]) == 4


def test_attention_over_its_queries(m):
    """o over q [3, 4, 64] itself is taken as far as its workspace; over a part of it, or over rows of
    another stride, it is refused."""
    cache, table = _cache(m), _table(m)

    def call(q, o, stride=0):
        p = m.make_paged_params(4, q_stride=stride)
        return m.load().msa_paged_attention(ctypes.byref(cache), ctypes.byref(table), ctypes.byref(p), q,
                                            o, P, 0, None)

    size = 3 * 4 * 64 * 2
    for o in (0, size, -size):
        assert call(64 * P, 64 * P + o) == 3
        assert call(64 * P, 64 * P + o, 256) == 3
    for o in (16, 512, size - 16, 16 - size):
        assert call(64 * P, 64 * P + o) == 1
    assert call(64 * P, 64 * P, 512) == 1 and call(64 * P, 64 * P + 2 * 512 * 2 + 496, 512) == 1
    assert call(64 * P, 64 * P + 2 * 512 * 2 + 512, 512) == 3
    table = _table(m, num_seqs=1)  # of one row any stride
    assert call(64 * P, 64 * P, 512) == 3 and call(64 * P, 64 * P + 16, 512) == 1


def test_the_join_reads_past_l1_before_its_wait():
    """What it works out ahead of its wait rests on lengths and pages that it has not waited for."""
    import block_sparse_attention_proxy_gb300 as package

    with open(os.path.join(os.path.dirname(package.__file__), "csrc", "k_paged.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    join = code[code.index("k_paged_join(const"):]
    ahead = join[:join.index("wait_for_previous()")]
    assert "paged_span<true>(" in ahead and "PagedWalk<true> w" in ahead
    for word in ("fetch(", "<false>", "cache_len(", "cache_page(", "tiles_of(", "PagedWalk w"):
        assert word not in ahead, word


def test_placed_finds_planted_mistakes():
    from cache_reference import placed

    inf, nan = float("inf"), float("nan")
    want = torch.tensor([1.0, inf, -inf, nan])
    placed(want + torch.tensor([0.5, 0, 0, 0]), want)
    for wrong in ([1.0, -inf, -inf, nan], [1.0, nan, -inf, nan], [1.0, inf, -inf, inf],
                  [1.0, inf, -inf, 0.0], [inf, inf, -inf, nan], [1.0, 3e38, -inf, nan]):
        with pytest.raises(AssertionError):
            placed(torch.tensor(wrong), want)


def _half_a_unit(words, doubles):
    """Whether every whole number lies within half of 2^-64 of a turn of its frequency (and 2^-150
    for the literal of 2 pi, right to 2^-157 of itself)."""
    two_pi = Fraction(int("6283185307179586476925286766559005768394338798750"), 10 ** 48)
    for word, f in zip(words, doubles, strict=True):
        off = Fraction(word, 2 ** 64) - Fraction(f) / two_pi
        if abs(off - round(off)) > Fraction(1, 2 ** 65) + Fraction(1, 2 ** 150):
            return False
    return True


@pytest.mark.parametrize("dims,kw", [(64, {}), (128, {}), (256, dict(base=1e6)), (16, dict(base=0.5)),
                                     (32, dict(stretch=4.0)),
                                     (128, dict(stretch=8.0, trained_length=4096)),
                                     (16, dict(frequencies=[0.0, -1.0, 1e-9, 7.5, 6.25, 1, 2, 3])),
                                     (16, dict(frequencies=[5e-324, -1e-20, 1e15, -3.7e9, 0.1, 2.0 ** -60,
                                                            6.283185307179586, -6.283185307179587]))])
def test_plan_frequencies_to_half_a_unit(m, dims, kw):
    """Of the doubles that the documented rule gives, in its order of operations."""
    if "frequencies" in kw:
        doubles = [float(f) for f in kw["frequencies"]]
    else:
        doubles, s = [], kw.get("stretch", 1.0)
        for i in range(dims // 2):
            f = kw.get("base", 10000.0) ** (-2 * i / dims)
            part = 0.0
            if "trained_length" in kw:
                turns = kw["trained_length"] * f / (2 * math.pi)
                part = min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
            doubles.append(f * (part + (1 - part) / s))
    assert _half_a_unit(m.rotary_plan(dims, **kw).frequencies, doubles)


@pytest.mark.parametrize("dims", [64, 128])
def test_half_a_unit_finds_plans_of_64_bit_floats(m, dims):
    doubles = [10000.0 ** (-2 * i / dims) for i in range(dims // 2)]
    rounded = [int(f / (2 * math.pi) % 1 * 2.0 ** 64) for f in doubles]
    assert not _half_a_unit(rounded, doubles)
    words = list(m.rotary_plan(dims).frequencies)
    for i in (0, dims // 4, dims // 2 - 1):
        for by in (-1, 1):
            assert not _half_a_unit(words[:i] + [words[i] + by] + words[i + 1:], doubles)
