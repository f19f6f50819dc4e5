"""Measured cases of the operators around a paged key-value cache: rotary positions (for
training and for the cache), appending to the cache, attention of one new token over it, and
eviction from it by accumulated attention weight.

A case names its operator ("op"), its sizes and its variant. The cache's tensors, one page table
row and one length a sequence:
  k, v      [pages, page, Hkv, d]  bf16, entry i of a sequence in page table[b, i // page]
  weight    [pages, Hkv, page]     fp32, attention weight that the entry has received so far
  position  [pages, Hkv, page]     int32, the entry's position in its text

`run` computes either the framework's operators (`own`) or their plain form: elementary
torch operations in fp32 (angles in fp64), rounded once.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decoding step of 64 conversations, far into their texts
        _rotary("rotary_step", "forward", 64, 64, 0.0, 32, 8, 128, 128),
        # the packed batch of the varlen workload, training
        _rotary("rotary_train_varlen", "train", 8, 32768, 0.45, 16, 4, 128, 128),
        # many short documents, half of each head rotated in neighbouring pairs, odd lengths,
        # frequencies stretched for longer texts than the model was trained on
        _rotary("rotary_train_part", "train", 61, 24001, 0.6, 8, 1, 64, 32, interleaved=True,
                stretch=8.0, trained=4096),
        # the long workload's tokens at fp32
        _rotary("rotary_long_fp32", "forward", 1, 131072, 0.0, 8, 2, 128, 128, dtype="fp32",
                stretch=4.0),
        # one decoding step of 64 conversations: new keys rotated and stored, queries rotated
        _append("append_step", 64, 1, 4000, 32, 8, 128, 64),
        # eight ragged prompts enter the cache
        _append("append_prompts", 8, 4096, 0, 16, 4, 128, 64),
        # a handful of short conversations: latency counts
        _attend("attend_short", 4, 103, 0.9, 32, 8, 128, 64),
        # a full batch of ragged conversations
        _attend("attend_batch", 64, 4096, 0.8, 32, 8, 128, 64),
        # one long text
        _attend("attend_long", 1, 131072, 0.0, 32, 8, 128, 128),
        # heads that share no keys, small pages, weights accumulated for eviction
        _attend("attend_mha_weights", 23, 2047, 0.7, 12, 12, 64, 16, weights=True),
        # a decoding step under a budget: one entry in, the least attended one out
        _evict("evict_step", 48, 4097, 0.0, 4096, 128, 8, 128, 64, step=True),
        # prompts cut down to a budget
        _evict("evict_prompts", 4, 32768, 0.3, 4096, 512, 8, 128, 64),
    ]


def _rotary(name, direction, docs, tokens, ragged, hq, hkv, d, dims, interleaved=False,
            stretch=1.0, trained=0, dtype="bf16"):
    return dict(name=name, op="rotary", direction=direction, docs=docs, tokens=tokens,
                ragged=ragged, hq=hq, hkv=hkv, d=d, dims=dims, interleaved=interleaved,
                stretch=stretch, trained=trained, dtype=dtype)


def _append(name, seqs, new, before, hq, hkv, d, page):
    """`new` tokens a sequence (ragged if more than one) behind about `before` entries."""
    return dict(name=name, op="append", seqs=seqs, new=new, before=before, hq=hq, hkv=hkv, d=d,
                page=page)


def _attend(name, seqs, length, ragged, hq, hkv, d, page, weights=False):
    """`length`: mean of the sequences' lengths."""
    return dict(name=name, op="attend", seqs=seqs, length=length, ragged=ragged, hq=hq, hkv=hkv,
                d=d, page=page, weights=weights)


def _evict(name, seqs, length, ragged, keep, recent, hkv, d, page, step=False):
    return dict(name=name, op="evict", seqs=seqs, length=length, ragged=ragged, keep=keep,
                recent=recent, hkv=hkv, d=d, page=page, step=step)


HEADS = ((4, 1), (4, 4), (6, 2), (8, 1), (8, 8), (10, 2), (12, 4), (16, 1), (16, 2), (16, 4),
         (24, 2), (32, 1), (32, 8), (64, 1))


def draw(rng):
    while True:
        op = rng.choice(("rotary", "append", "attend", "attend", "evict"))
        hq, hkv = rng.choice(HEADS)
        d, page = rng.choice((64, 128)), rng.choice((16, 32, 64, 128, 256))
        ragged = round(rng.uniform(0, 0.9), 2)
        if op == "rotary":
            tokens = int(2 ** rng.uniform(0, 17))
            d = rng.choice((32, 64, 80, 96, 128, 256))
            case = _rotary("", rng.choice(("forward", "train")), min(tokens, int(2 ** rng.uniform(0, 6))),
                           tokens, ragged, hq, hkv, d, 16 * rng.randint(1, d // 16),
                           rng.random() < 0.5, round(rng.uniform(1, 16), 1),
                           rng.choice((0, 1000, 8192)), rng.choice(("bf16", "bf16", "fp16", "fp32")))
        elif op == "append":
            case = _append("", int(2 ** rng.uniform(0, 8)), rng.choice((1, int(2 ** rng.uniform(0, 13)))),
                           rng.choice((0, int(2 ** rng.uniform(0, 12)))), hq, hkv, d, page)
        elif op == "attend":
            case = _attend("", int(2 ** rng.uniform(0, 7)), int(2 ** rng.uniform(0, 17)), ragged,
                           hq, hkv, d, page, rng.random() < 0.4)
        else:
            step = rng.random() < 0.5
            keep = int(2 ** rng.uniform(3, 13))
            length = keep + 1 if step else int(keep * 2 ** rng.uniform(0.1, 4))
            case = _evict("", int(2 ** rng.uniform(0, 6)), length, 0.0 if step else ragged, keep,
                          rng.randint(0, keep // 2), hkv, d, page, step)
        del case["name"]
        most = {"rotary": 4e8, "append": 2e8, "attend": 1e9, "evict": 3e8}
        if work(case)["bytes"] > most[op]:
            continue
        if op == "attend" and max(lengths(case)) * case["seqs"] * hkv * d > 6e8:
            continue
        if op == "append" and case["seqs"] * (case["new"] + case["before"]) * hkv * d > 6e8:
            continue
        if op == "evict" and sum(lengths(case)) * hkv * d > 3e8:
            continue
        return case


def _spread(n, total, ragged, least):
    """n lengths that add up to `total`, the same for every seed of the inputs."""
    r = random.Random("%d %d %.3f" % (n, total, ragged))
    share = [1 + ragged * r.uniform(-1, 1) for _ in range(n)]
    lens = [max(least, int(total * s / sum(share))) for s in share]
    lens[-1] = max(least, lens[-1] + total - sum(lens))
    return lens


def lengths(case):
    """Rotary: the documents'. Others: entries of each sequence before the call (append), or
    that the call sees."""
    if case["op"] == "rotary":
        n, total = case["docs"], case["tokens"]
        lens = _spread(n, total, case["ragged"], 1)
        while sum(lens) > total:
            lens[lens.index(max(lens))] -= 1
        return lens
    if case["op"] == "append":
        return _spread(case["seqs"], case["seqs"] * case["before"], 0.9, 0)
    return _spread(case["seqs"], case["seqs"] * case["length"], case["ragged"], 1)


def new_lengths(case):
    """Append: tokens that come in for each sequence."""
    if case["new"] == 1:
        return [1] * case["seqs"]
    return _spread(case["seqs"], case["seqs"] * case["new"], 0.6, 1)


def moved(case):
    """Evict: rows that a random choice of entries moves, on average, over all sequences and heads."""
    rows = 0.0
    for n in lengths(case):
        if n > case["keep"]:
            left = (case["keep"] - case["recent"]) / (n - case["recent"])  # chance to stay
            rows += min(case["recent"], n - case["keep"])  # recent ones behind the budget
            rows += max(0, n - case["recent"] - case["keep"]) * left
    return rows * case["hkv"]


def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "rotary":
        size = case["tokens"] * (case["hq"] + hkv) * d
        passes = 2 if case["direction"] == "train" else 1
        per = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": passes * 2 * size * per,
                "flops": passes * 3 * size * case["dims"] / d}
    if case["op"] == "append":  # q in and out, k and v in and out, weight and position out
        t = sum(new_lengths(case))
        return {"bytes": t * (4 * case["hq"] * d + 8 * hkv * d + 8 * hkv),
                "flops": t * 3 * (case["hq"] + hkv) * d}
    n = sum(lengths(case))
    if case["op"] == "attend":  # k and v in, q in, o out, the weights updated
        size = n * hkv * (4 * d + (8 if case["weights"] else 0)) + 4 * case["seqs"] * case["hq"] * d
        return {"bytes": size, "flops": 4 * n * case["hq"] * d}
    # weights and positions in; the moved rows of k, v, weight and position in and out
    size = n * hkv * 8 + moved(case) * 2 * (4 * d + 8)
    if case["step"]:  # the new entry in and out
        size += case["seqs"] * hkv * (8 * d + 8)
    return {"bytes": size, "flops": n * hkv}


def frequencies(case):
    """Radians a position of each rotated pair: powers of the base; divided by `stretch`, or, for a
    model trained on `trained` positions, only as far as a pair turns less than 32 times
    over those, fully where it turns less than once."""
    freq = []
    for i in range(case["dims"] // 2):
        f = 10000.0 ** (-2 * i / case["dims"])
        part = 0.0
        if case["trained"]:
            part = min(1.0, max(0.0, (case["trained"] * f / (2 * math.pi) - 1) / (32 - 1)))
        freq.append(f * (part + (1 - part) / case["stretch"]))
    return freq


CACHE = {"dims": 0, "stretch": 1.0, "trained": 0, "interleaved": False}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def ends(lens):
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        return ints(cu)

    hkv, d = case["hkv"], case["d"]
    state = {"case": dict(case), "op": case["op"]}
    if case["op"] == "rotary":
        dtype, t, hq = DTYPES[case["dtype"]], case["tokens"], case["hq"]
        state.update(train=case["direction"] == "train", dims=case["dims"],
                     interleaved=case["interleaved"])
        state["freq"] = torch.tensor(frequencies(case), dtype=torch.float64, device="cuda")
        state["q"], state["k"] = (normal(t, h, d, dtype=dtype) for h in (hq, hkv))
        if t == case["docs"]:  # one token each: positions far into the texts
            state["positions"] = torch.randint(0, 1 << 20, (t,), generator=g, device="cuda",
                                               dtype=torch.int32)
            state["cu"] = None
        else:
            state["positions"], state["cu"] = None, ends(lengths(case))
        if state["train"]:
            state["dq"], state["dk"] = (normal(t, h, d, dtype=dtype) for h in (hq, hkv))
            state["leaves"] = [state[n].requires_grad_(True) for n in ("q", "k")]
        return state

    # the cache: pages of the sequences in random order
    page, lens = case["page"], lengths(case)
    seen = [n + m for n, m in zip(lens, new_lengths(case))] if case["op"] == "append" else lens
    width = -(-max(seen) // page)
    pages = case["seqs"] * width
    state["table"] = torch.randperm(pages, generator=g, device="cuda").int().view(-1, width)
    state["lens"] = ints(lens)
    state["longest"] = max(seen)
    state["k"], state["v"] = (normal(pages, page, hkv, d) for _ in range(2))
    state["weight"] = state["position"] = None
    if case["op"] == "append":
        state["weight"] = torch.zeros(pages, hkv, page, device="cuda")
        state["position"] = torch.zeros(pages, hkv, page, dtype=torch.int32, device="cuda")
        t = sum(new_lengths(case))
        state["q"] = normal(t, case["hq"], d, scale=d ** -0.5)
        state["new_k"], state["new_v"] = (normal(t, hkv, d) for _ in range(2))
        state["cu"] = None if case["new"] == 1 else ends(new_lengths(case))
        state["freq"] = torch.tensor(frequencies(dict(CACHE, dims=d)), dtype=torch.float64,
                                     device="cuda")
    if case["op"] == "attend":
        state["q"] = normal(case["seqs"], case["hq"], d, scale=d ** -0.5)
        if case["weights"]:
            state["weight"] = torch.rand(pages, hkv, page, generator=g, device="cuda")
    if case["op"] == "evict":
        # accumulated weights: mostly small, a few entries hold most
        state["scores"] = torch.rand(pages, hkv, page, generator=g, device="cuda") ** 8
        at = torch.arange(width * page, device="cuda", dtype=torch.int32).view(width, 1, page)
        state["positions"] = torch.empty(pages, hkv, page, dtype=torch.int32, device="cuda")
        state["positions"][state["table"].long()] = at.expand(-1, hkv, -1)
        state["weight"], state["position"] = state["scores"].clone(), state["positions"].clone()
        if case["step"]:
            state["before"] = state["lens"] - 1
            state["next"] = state["before"].clone()
            state["new_k"], state["new_v"] = (normal(case["seqs"], hkv, d) for _ in range(2))
    return state


def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return _plain(state)


def _own(state):
    import block_sparse_attention_proxy_gb300 as m

    s, case = state, state["case"]
    if s["op"] in ("rotary", "append") and "plan" not in s:  # a program makes it once
        c = case if s["op"] == "rotary" else dict(CACHE, dims=case["d"])
        s["plan"] = m.rotary_plan(c["dims"], interleaved=c["interleaved"], stretch=c["stretch"],
                                  trained_length=c["trained"] or None)
    if s["op"] == "rotary":
        if not s["train"]:
            with torch.no_grad():
                return list(m.rotary(s["q"], s["k"], s["plan"], cu_seqlens=s["cu"],
                                     positions=s["positions"]))
        y = m.rotary(s["q"], s["k"], s["plan"], cu_seqlens=s["cu"], positions=s["positions"])
        return [*y, *torch.autograd.grad(y, s["leaves"], (s["dq"], s["dk"]))]
    cache = m.PagedCache(s["k"], s["v"], s["weight"], s["position"])
    if s["op"] == "append":
        q = m.cache_append(cache, s["new_k"], s["new_v"], s["table"], s["lens"],
                           cu_seqlens=s["cu"], plan=s["plan"], q=s["q"])
        return [q, *cache]
    if s["op"] == "attend":
        o = m.paged_attention(s["q"], cache, s["table"], s["lens"], accumulate=case["weights"])
        return [o, s["weight"]] if case["weights"] else [o]
    if case["step"]:
        s["next"].add_(1)
        m.cache_append(cache, s["new_k"], s["new_v"], s["table"], s["before"],
                       positions=s["next"])
    else:  # a prompt's scores come from its prefill
        s["weight"].copy_(s["scores"])
        s["position"].copy_(s["positions"])
    kept = m.cache_evict(cache, s["table"], s["lens"], case["keep"], case["recent"])
    return [*cache, kept]


def _turn(x, angle, dims, interleaved, back=False):
    """Rotates the first `dims` elements of x's rows by the angles [rows, dims / 2], in fp32."""
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if back:
        sin = -sin
    y = x.float()
    out = y.clone()
    a, b = ((slice(0, dims, 2), slice(1, dims, 2)) if interleaved else
            (slice(0, dims // 2), slice(dims // 2, dims)))
    out[..., a] = y[..., a] * cos - y[..., b] * sin
    out[..., b] = y[..., b] * cos + y[..., a] * sin
    return out.to(x.dtype)


def _text_positions(cu, t):
    token = torch.arange(t, device=cu.device)
    doc = torch.searchsorted(cu[1:].long(), token, right=True)
    return doc, token - cu.long()[doc]


def _plain(state):
    s = state
    if s["op"] == "rotary":
        at = s["positions"] if s["cu"] is None else _text_positions(s["cu"], s["q"].shape[0])[1]
        angle = at.double()[:, None] * s["freq"]
        out = [_turn(s[n], angle, s["dims"], s["interleaved"]) for n in ("q", "k")]
        if s["train"]:
            out += [_turn(s[n], angle, s["dims"], s["interleaved"], True) for n in ("dq", "dk")]
        return out
    if s["op"] == "append":
        return _plain_append(s, s["new_k"], s["new_v"], s["lens"], None, s["q"])
    if s["op"] == "attend":
        return _plain_attend(s)
    if s["case"]["step"]:
        s["next"].add_(1)
        _plain_append(s, s["new_k"], s["new_v"], s["before"], s["next"], None)
    else:
        s["weight"].copy_(s["scores"])
        s["position"].copy_(s["positions"])
    return _plain_evict(s)


def _plain_append(s, k, v, lens, positions, q):
    t, page = k.shape[0], s["k"].shape[1]
    if s.get("cu") is None:
        seq, slot = torch.arange(t, device=k.device), lens.long()
    else:
        seq, slot = _text_positions(s["cu"], t)
        slot = slot + lens.long()[seq]
    if positions is None:
        positions = slot
        angle = positions.double()[:, None] * s["freq"]
        q, k = (_turn(x, angle, k.shape[2], False) for x in (q, k))
    where = s["table"].long()[seq, slot // page]
    s["k"][where, slot % page] = k
    s["v"][where, slot % page] = v
    s["weight"][where, :, slot % page] = 0.0
    s["position"][where, :, slot % page] = positions.int()[:, None]
    return [q, s["k"], s["v"], s["weight"], s["position"]]


def _plain_attend(s):
    q, n = s["q"], s["longest"]
    (b, hq, d), (_, page, hkv, _) = q.shape, s["k"].shape
    table = s["table"].long()
    at = torch.arange(n, device=q.device)
    there = at < s["lens"][:, None]
    k, v = (s[x][table].view(b, -1, hkv, d)[:, :n].permute(0, 2, 1, 3).float() for x in ("k", "v"))
    p = q.view(b, hkv, -1, d).float() @ k.transpose(-1, -2)
    p.masked_fill_(~there[:, None, None], float("-inf"))
    p -= p.amax(-1, keepdim=True)
    p = p.exp_()
    p /= p.sum(-1, keepdim=True)
    o = (p @ v).view(b, hq, d).to(q.dtype)
    if s["weight"] is None:
        return [o]
    index = (table[:, at // page][:, None], torch.arange(hkv, device=q.device)[None, :, None],
             (at % page)[None, None])
    s["weight"].index_put_(index, p.sum(2), accumulate=True)
    return [o, s["weight"]]


def _plain_evict(s):
    case, table, lens = s["case"], s["table"].long(), s["lens"]
    keep, recent = case["keep"], case["recent"]
    (b, width), (_, hkv, page) = table.shape, s["weight"].shape
    n = width * page
    at = torch.arange(n, device=lens.device)
    there = (at < lens[:, None])[:, None]
    w, pos = (s[x][table].transpose(1, 2).reshape(b, hkv, n) for x in ("weight", "position"))
    newest = torch.where(there, pos, -1).amax(-1, keepdim=True)
    w = torch.where(there, torch.where(pos > newest - recent, float("inf"), w), float("-inf"))
    order = torch.argsort(w, dim=-1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(-1, order, at.expand(b, hkv, n))
    kept = (rank < keep) & there
    into = (at < keep) & ~kept & there  # evicted entries below the budget take ...
    out = (at >= keep) & kept           # ... the kept ones from behind it, in order
    src, dst = out.nonzero(), into.nonzero()
    for name, axis in (("k", 1), ("v", 1), ("weight", 2), ("position", 2)):
        x = s[name] if axis == 2 else s[name].transpose(1, 2)
        x[table[dst[:, 0], dst[:, 2] // page], dst[:, 1], dst[:, 2] % page] = \
            x[table[src[:, 0], src[:, 2] // page], src[:, 1], src[:, 2] % page]
    return [s["k"], s["v"], s["weight"], s["position"], lens.clamp(max=keep)]


def exact(case, seed):
    """The outputs from the definitions, sequence by sequence, in fp64 on whole numbers' indexes."""
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, s)
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    return _exact_evict(case, s)


def _complex_turn(x, positions, freq, interleaved):
    """Each pair as one complex number, times exp(i position frequency)."""
    y = x.detach().double()
    half = len(freq)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       torch.outer(positions.double(), torch.tensor(freq, dtype=torch.float64,
                                                                    device=x.device)))
    if interleaved:
        z = torch.complex(y[..., 0:2 * half:2], y[..., 1:2 * half:2]) * turn[:, None]
        first = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :half], y[..., half:2 * half]) * turn[:, None]
        first = torch.cat((z.real, z.imag), -1)
    return torch.cat((first, y[..., 2 * half:]), -1)


def _exact_rotary(case, s):
    if s["cu"] is None:
        at = s["positions"]
    else:
        at = torch.cat([torch.arange(n, device="cuda") for n in lengths(case)])
    freq = frequencies(case)
    out = [_complex_turn(s[n], at, freq, case["interleaved"]) for n in ("q", "k")]
    if s["train"]:
        out += [_complex_turn(s[n], -at, freq, case["interleaved"]) for n in ("dq", "dk")]
    return out


def _exact_append(case, s):
    before, new, page = lengths(case), new_lengths(case), case["page"]
    at = torch.cat([torch.arange(a, a + n, device="cuda") for a, n in zip(before, new)])
    freq = frequencies(dict(CACHE, dims=case["d"]))
    q, k = (_complex_turn(s[n], at, freq, False) for n in ("q", "new_k"))
    # every entry's row in the flattened pages
    row = torch.cat([s["table"][i].long()[torch.arange(a, a + n, device="cuda") // page]
                     for i, (a, n) in enumerate(zip(before, new))]) * page + at % page
    k_all, v_all = s["k"].double(), s["v"].double()
    k_all.view(-1, case["hkv"], case["d"])[row] = k
    v_all.view(-1, case["hkv"], case["d"])[row] = s["new_v"].double()
    position = s["position"].clone()
    position[row // page, :, row % page] = at.int()[:, None]
    return [q, k_all, v_all, s["weight"].double(), position]


def _exact_attend(case, s):
    page, group = case["page"], case["hq"] // case["hkv"]
    o = s["q"].double()
    weight = None if s["weight"] is None else s["weight"].double()
    for b, n in enumerate(lengths(case)):
        pages = s["table"][b, :-(-n // page)].long()
        k, v = (s[x][pages].flatten(0, 1)[:n].double() for x in ("k", "v"))
        for h in range(case["hkv"]):
            heads = slice(h * group, (h + 1) * group)
            score = k[:, h] @ s["q"][b, heads].double().T
            prob = (score - torch.logsumexp(score, 0)).exp()
            o[b, heads] = prob.T @ v[:, h]
            if weight is not None:
                more = torch.zeros(pages.numel() * page, dtype=torch.float64, device="cuda")
                more[:n] = prob.sum(1)
                weight[pages, h] += more.view(-1, page)
    return [o] if weight is None else [o, weight]


def _exact_evict(case, s):
    page, keep, recent = case["page"], case["keep"], case["recent"]
    if sum(lengths(case)) * case["hkv"] > 3e6:
        return None
    if case["step"]:
        for b, n in enumerate(lengths(case)):
            p, i = int(s["table"][b, (n - 1) // page]), (n - 1) % page
            s["k"][p, i], s["v"][p, i] = s["new_k"][b], s["new_v"][b]
            s["weight"][p, :, i], s["position"][p, :, i] = 0.0, n
    left = []
    for b, n in enumerate(lengths(case)):
        left.append(min(n, keep))
        if n <= keep:
            continue
        pages = s["table"][b].long()
        for h in range(case["hkv"]):
            w = s["weight"][pages, h].flatten()[:n].tolist()
            pos = s["position"][pages, h].flatten()[:n].tolist()
            newest = max(pos)
            w = [math.inf if p > newest - recent else x for x, p in zip(w, pos)]
            kept = set(sorted(range(n), key=lambda i: (-w[i], i))[:keep])
            src = torch.tensor([i for i in range(keep, n) if i in kept], dtype=torch.long, device="cuda")
            dst = torch.tensor([i for i in range(keep) if i not in kept], dtype=torch.long, device="cuda")
            to, of = pages[dst // page], pages[src // page]
            for name in ("k", "v"):
                s[name][to, dst % page, h] = s[name][of, src % page, h].clone()
            for name in ("weight", "position"):
                s[name][to, h, dst % page] = s[name][of, h, src % page].clone()
    return [s["k"].double(), s["v"].double(), s["weight"].double(), s["position"],
            torch.tensor(left, dtype=torch.int32, device="cuda")]
