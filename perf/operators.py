"""Measured cases of the dense attention operators: packed causal attention with
grouped heads, forward and backward, without and with a learned relative
position bias by distance buckets.

A case is a packed batch of documents (lengths from `lengths(case)`), its head
layout, the head dim, the direction ("forward": no gradient is asked for;
"train": forward and the gradients of every input) and, for the bias, the
number of buckets and the distance from which the last bucket holds.

`run` computes either the framework's operator (`own`) or its plain form: the
batch padded to [documents, heads, longest, d], the whole score matrix in fp32,
softmax and products written out, each result rounded once to bf16.
"""
import bisect
import random

import torch

own = False

# fp64 work (operations) above which the exact values would take too long
_EXACT_OPS = 8e12


def listed():
    return [
        # a handful of chat-sized prompts answered at once: launch latency counts
        _case("forward_short", "forward", 8, 412, 0.9, 32, 8, 128),
        # the packed batch of the varlen workload (8 ragged documents), inference
        _case("forward_varlen", "forward", 8, 32768, 0.45, 16, 4, 128),
        # one long prompt
        _case("forward_long", "forward", 1, 32768, 0.0, 8, 2, 128),
        # heads that share no keys, d = 64, odd lengths
        _case("forward_mha_odd", "forward", 3, 10007, 0.5, 12, 12, 64),
        # the tiny training step: one document, four heads on one KV head
        _case("train_tiny", "train", 1, 1024, 0.0, 4, 1, 64),
        # many short documents, all heads on one KV head
        _case("train_documents", "train", 61, 24001, 0.6, 8, 1, 64),
        # the packed batch of the varlen workload, training
        _case("train_varlen", "train", 8, 32768, 0.45, 16, 4, 128),
        # a dense layer between sparse ones: the long workload's heads
        _case("train_long", "train", 1, 16384, 0.0, 32, 8, 128),
        # short prompts with 32 buckets that saturate at distance 128
        _case("bias_forward_short", "forward", 12, 1203, 0.8, 8, 8, 64, 32, 128),
        # a long prompt whose buckets reach far beyond one key tile
        _case("bias_forward_long", "forward", 1, 16384, 0.0, 16, 4, 128, 32, 4096),
        # training on ragged documents, three heads to a KV head
        _case("bias_train_documents", "train", 23, 16001, 0.7, 12, 4, 64, 32, 128),
        # training on one document with 64 buckets over its whole length
        _case("bias_train_long", "train", 1, 8192, 0.0, 16, 4, 128, 64, 8192),
    ]


def _case(name, direction, docs, tokens, ragged, hq, hkv, d, buckets=0, far=0):
    return dict(name=name, direction=direction, docs=docs, tokens=tokens, ragged=ragged, hq=hq,
                hkv=hkv, d=d, buckets=buckets, far=far)


def draw(rng):
    while True:
        direction = rng.choice(("forward", "train"))
        hq, hkv = rng.choice(((4, 1), (4, 4), (6, 2), (8, 1), (8, 8), (10, 2), (12, 4), (16, 2),
                              (16, 4), (32, 8)))
        tokens = int(2 ** rng.uniform(5, 15))
        docs = min(tokens, int(2 ** rng.uniform(0, 6)))
        buckets, far = 0, 0
        if rng.random() < 0.5:
            buckets = rng.choice((8, 16, 32, 48, 64))
            far = int(2 ** rng.uniform(7, 13))
        case = _case("", direction, docs, tokens, round(rng.uniform(0, 0.9), 2), hq, hkv,
                     rng.choice((64, 128)), buckets, far)
        del case["name"]
        longest = max(lengths(case))
        if (work(case)["flops"] <= 7.6e12 and docs * hq * longest * longest <= 32 * 16384 ** 2
                and longest <= (16384 if buckets or direction == "train" else 32768)):
            return case


def lengths(case):
    """Document lengths of the packed batch: the same for every seed of the inputs."""
    n, total = case["docs"], case["tokens"]
    r = random.Random("%d %d %.3f" % (n, total, case["ragged"]))
    share = [1 + case["ragged"] * r.uniform(-1, 1) for _ in range(n)]
    lens = [max(1, int(total * s / sum(share))) for s in share]
    while sum(lens) > total:
        lens[lens.index(max(lens))] -= 1
    lens[-1] += total - sum(lens)
    return lens


def bucket_starts(buckets, far):
    """First distance of each bucket: one distance per bucket up to half of them, then
    spaced evenly in the logarithm up to `far`, where the last one begins."""
    half = buckets // 2
    starts = list(range(half))
    for i in range(buckets - half):
        at = round(half * (far / half) ** (i / (buckets - half - 1)))
        starts.append(max(at, starts[-1] + 1))
    return tuple(starts)


def work(case):
    lens = lengths(case)
    t, d, hq, hkv = case["tokens"], case["d"], case["hq"], case["hkv"]
    pairs = hq * sum(n * (n + 1) // 2 for n in lens)
    rows_q, rows_kv = t * hq * d * 2, t * hkv * d * 2
    table = hq * case["buckets"] * 2
    if case["direction"] == "train":  # q, dO in and o, dq out; k, v in and dk, dv out
        return {"bytes": 4 * rows_q + 4 * rows_kv + 2 * table, "flops": 14 * d * pairs}
    return {"bytes": 2 * rows_q + 2 * rows_kv + table, "flops": 4 * d * pairs}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]

    def normal(*shape, scale=1.0):
        x = torch.randn(*shape, generator=g, device="cuda") * scale
        return x.to(torch.bfloat16)

    cu = [0]
    for n in lengths(case):
        cu.append(cu[-1] + n)
    train = case["direction"] == "train"
    state = {
        "q": normal(t, hq, d, scale=d ** -0.5), "k": normal(t, hkv, d), "v": normal(t, hkv, d),
        "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"),
        "longest": max(lengths(case)), "train": train, "bias": None, "starts": None,
        "do": normal(t, hq, d) if train else None,
    }
    if case["buckets"]:
        state["bias"] = normal(hq, case["buckets"], scale=0.5)
        state["starts"] = bucket_starts(case["buckets"], case["far"])
    if train:
        state["leaves"] = [state[n].requires_grad_(True) for n in ("q", "k", "v", "bias")
                           if state[n] is not None]
    return state


def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return _plain(state)


def _own(state):
    from block_sparse_attention_proxy_gb300 import dense_attention

    if not state["train"]:
        with torch.no_grad():
            return [dense_attention(state["q"], state["k"], state["v"], state["cu"],
                                    bias=state["bias"], bucket_starts=state["starts"])]
    o = dense_attention(state["q"], state["k"], state["v"], state["cu"], bias=state["bias"],
                        bucket_starts=state["starts"])
    return [o, *torch.autograd.grad(o, state["leaves"], state["do"])]


def _plain(state):
    q, k, v, cu, n = state["q"], state["k"], state["v"], state["cu"].long(), state["longest"]
    t, hq, d = q.shape
    hkv, docs = k.shape[1], cu.numel() - 1
    pos = torch.arange(n, device=q.device)
    at = (cu[:-1, None] + pos).clamp(max=t - 1)
    there = (pos < (cu[1:] - cu[:-1])[:, None])[:, :, None, None]
    token = torch.arange(t, device=q.device)
    doc = torch.searchsorted(cu[1:], token, right=True)
    at_doc = token - cu[doc]

    def padded(x):  # [tokens, heads, d] -> [documents, kv heads, heads of one * longest, d]
        x = torch.where(there, x.float()[at], 0.0)
        return x.transpose(1, 2).reshape(docs, hkv, -1, d)

    def packed(x):  # and back, rounded once
        return x.view(docs, -1, n, d)[doc, :, at_doc].to(torch.bfloat16)

    qp, kp, vp = padded(q), padded(k), padded(v)
    s = (qp @ kp.transpose(-1, -2)).view(docs, hq, n, n)
    dist = pos[:, None] - pos
    if state["bias"] is not None:
        starts = torch.tensor(state["starts"], device=q.device)
        bucket = torch.searchsorted(starts, pos, right=True) - 1  # of each distance
        s += state["bias"].float()[:, bucket][:, dist.clamp(min=0)]
    s.masked_fill_(dist < 0, float("-inf"))
    s -= s.amax(-1, keepdim=True)
    p = s.exp_()
    p /= p.sum(-1, keepdim=True)
    p4 = p.view(docs, hkv, -1, n)
    o = packed(p4 @ vp)
    if not state["train"]:
        return [o]
    dop = padded(state["do"])
    dv = p4.transpose(-1, -2) @ dop
    dp = (dop @ vp.transpose(-1, -2)).view(docs, hq, n, n)
    dp -= (p * dp).sum(-1, keepdim=True)
    ds = dp.mul_(p)
    ds4 = ds.view(docs, hkv, -1, n)
    out = [o, packed(ds4 @ kp), packed(ds4.transpose(-1, -2) @ qp), packed(dv)]
    if state["bias"] is not None:
        # sums over equal distances: keys reversed, each row shifted by its position
        skew = torch.cat((ds.flip(-1), torch.zeros_like(ds)), -1).view(docs, hq, -1)
        skew = skew[..., : n * (2 * n - 1)].view(docs, hq, n, 2 * n - 1)
        by_dist = skew.sum((0, 2), dtype=torch.float64)[:, n - 1:]
        table = torch.zeros(hq, len(state["starts"]), dtype=torch.float64, device=q.device)
        out.append(table.index_add_(1, bucket, by_dist).to(torch.bfloat16))
    return out


def exact(case, seed):
    """The outputs from the definition, head by head and document by document, in fp64."""
    lens = lengths(case)
    train, hq, hkv, d = case["direction"] == "train", case["hq"], case["hkv"], case["d"]
    if sum(n * n for n in lens) * hq * d * (14 if train else 4) > _EXACT_OPS:
        return None
    state = prepare(case, seed)
    q, k, v = (state[n].detach().double() for n in ("q", "k", "v"))
    o = torch.zeros_like(q)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    starts = state["starts"]
    table = dtable = None
    if starts:
        table = state["bias"].detach().double()
        dtable = torch.zeros_like(table)
    first = 0
    for n in lens:
        rows = slice(first, first + n)
        first += n
        causal = torch.ones(n, n, dtype=torch.bool, device=q.device).tril_()
        if starts:
            which = torch.tensor([bisect.bisect_right(starts, i) - 1 for i in range(n)],
                                 device=q.device)
            i = torch.arange(n, device=q.device)
            gap = (i[:, None] - i[None, :]).clamp_(min=0)
        for h in range(hq):
            g = h // (hq // hkv)
            logit = q[rows, h] @ k[rows, g].T
            if starts:
                logit += table[h, which][gap]
            logit[~causal] = -torch.inf
            prob = (logit - torch.logsumexp(logit, 1, keepdim=True)).exp_()
            del logit
            o[rows, h] = prob @ v[rows, g]
            if not train:
                continue
            do = state["do"][rows, h].double()
            dv[rows, g] += prob.T @ do
            # dS = P (dP - D), D = dO . O of the row
            dlogit = prob * (do @ v[rows, g].T - (do * o[rows, h]).sum(1, keepdim=True))
            dq[rows, h] = dlogit @ k[rows, g]
            dk[rows, g] += dlogit.T @ q[rows, h]
            if starts:
                beyond = [dlogit.tril(-s).sum() if s < n else dlogit.new_zeros(())
                          for s in (*starts, n)]
                beyond = torch.stack(beyond)
                dtable[h] += beyond[:-1] - beyond[1:]
    if not train:
        return [o]
    return [o, dq, dk, dv] + ([dtable] if starts else [])
