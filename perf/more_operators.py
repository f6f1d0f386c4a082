"""Operators for long and for drafted decoding over the paged 8-bit cache: cases, plain forms and 64-bit values.

Five operators beside those of the serving path (one fp32 scale for each block
of 16 tokens of a head, as there):

* tree    attention of a tree of drafted tokens over the cache: each new token
          sees the cached ones and those new ones whose bits it is given;
* sinks   attention with a sliding window and a few first tokens that stay
          visible;
          both also give the logarithm of each row's sum of exponentials;
* weigh   the attention weight that each cached token gets from the new queries,
          summed over them and over the query heads that share its head;
* evict   a budget of tokens for each sequence and head: the first ones, the
          last ones and the heaviest of the rest are kept and moved together
          into other pages (and read back as numbers: codes are returned as the
          values they stand for);
* adjust  logits before sampling: penalties for repeated tokens, biases and the
          bit masks of a grammar.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 16           # tokens that share a scale


def _q4():
    import quantized_weight_q4_gb300 as q4
    return q4


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one user's small draft of full precision: latency
        dict(name="tree-one", op="tree", type="f32", seqs=1, new_lo=13, new_hi=13, ctx_lo=777, ctx_hi=777, q_heads=32,
             kv_heads=32, dim=128, page=64, window=0, sinks=0),
        # a serving batch that checks drafts of different sizes at once, shared heads
        dict(name="tree-batch", op="tree", type="bf16", seqs=16, new_lo=5, new_hi=61, ctx_lo=300, ctx_hi=6001,
             q_heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0),
        # one user beyond the window: latency
        dict(name="sinks-one", op="sinks", type="f32", seqs=1, new_lo=1, new_hi=1, ctx_lo=3001, ctx_hi=3001, q_heads=16,
             kv_heads=4, dim=64, page=16, window=1000, sinks=4),
        # a serving batch of long-running sequences, one token each
        dict(name="sinks-batch", op="sinks", type="bf16", seqs=64, new_lo=1, new_hi=1, ctx_lo=900, ctx_hi=16001,
             q_heads=32, kv_heads=8, dim=128, page=64, window=4096, sinks=4),
        # a long prompt under the window
        dict(name="sinks-prompt", op="sinks", type="bf16", seqs=1, new_lo=9001, new_hi=9001, ctx_lo=0, ctx_hi=0,
             q_heads=32, kv_heads=8, dim=128, page=64, window=1024, sinks=4),
        # one token's weights over a short sequence: latency
        dict(name="weigh-one", op="weigh", type="f32", seqs=1, new_lo=1, new_hi=1, ctx_lo=389, ctx_hi=389, q_heads=32,
             kv_heads=32, dim=128, page=64, window=0, sinks=0),
        # the last tokens of a batch weigh all that its sequences hold, before some of it is dropped
        dict(name="weigh-batch", op="weigh", type="bf16", seqs=64, new_lo=1, new_hi=2, ctx_lo=50, ctx_hi=8191,
             q_heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0),
        # a whole prompt weighs itself
        dict(name="weigh-prompt", op="weigh", type="bf16", seqs=1, new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0,
             q_heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0),
        # one document cut to a third of it
        dict(name="evict-one", op="evict", seqs=1, ctx_lo=100003, ctx_hi=100003, keep=32768, kv_heads=8, dim=128,
             page=64, sinks=4, recent=1024),
        # a batch whose sequences have outgrown their budget, and some that have not
        dict(name="evict-batch", op="evict", seqs=48, ctx_lo=1500, ctx_hi=8191, keep=2048, kv_heads=8, dim=128, page=64,
             sinks=4, recent=256),
        # one user's row of logits, penalties only
        dict(name="adjust-one", op="adjust", type="f32", rows=1, vocab=32000, history=391, bias=0, grammar=False),
        # a serving batch: long histories, biases, and grammars on half of the rows
        dict(name="adjust-batch", op="adjust", type="bf16", rows=200, vocab=128007, history=8000, bias=100,
             grammar=True),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["tree", "tree", "sinks", "sinks", "weigh", "weigh", "evict", "adjust"])
    kind = rng.choice(["f32", "bf16"])
    if op == "adjust":
        return dict(op=op, type=kind, rows=_log(rng, 1, 120), vocab=_log(rng, 500, 128000),
                    history=_log(rng, 1, 8000), bias=rng.choice([0, 1, 300]), grammar=rng.random() < 0.5)
    kv_heads = rng.choice([1, 2, 4, 8])
    c = dict(op=op, kv_heads=kv_heads, dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]))
    if op == "evict":
        hi = _log(rng, 200, 8000)
        c.update(seqs=_log(rng, 1, 40), ctx_lo=_log(rng, 1, 150), ctx_hi=hi, keep=rng.randint(100, hi),
                 sinks=rng.randint(0, 20), recent=_log(rng, 1, 80))
        return c
    c.update(type=kind, q_heads=kv_heads * rng.choice([1, 3, 4, 8] if kv_heads <= 4 else [1, 4]))
    if op == "tree":
        windowed = rng.random() < 0.3
        c.update(seqs=_log(rng, 1, 16), new_lo=1, new_hi=_log(rng, 2, 64), ctx_lo=_log(rng, 1, 300),
                 ctx_hi=_log(rng, 301, 5000), window=700 if windowed else 0, sinks=3 if windowed else 0)
        return c
    form = rng.choice(["single", "few", "prompts"])
    window = rng.choice([300, 1000]) if op == "sinks" else rng.choice([0, 0, 777])
    c.update(window=window, sinks=rng.choice([1, 4, 37]) if window else 0)
    if form == "prompts":
        c.update(type="bf16", seqs=rng.randint(1, 4), new_lo=_log(rng, 2, 100), new_hi=_log(rng, 101, 2500), ctx_lo=0,
                 ctx_hi=_log(rng, 1, 4000))
    else:
        c.update(seqs=_log(rng, 1, 60), new_lo=1, new_hi=1 if form == "single" else rng.randint(2, 16),
                 ctx_lo=_log(rng, 1, 500), ctx_hi=_log(rng, 501, 8000))
    return c


# -------------------------------------------------------------------- inputs
def _lengths(case):
    """New tokens and tokens in all of each sequence: the same for every seed."""
    import random
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    new, total = [], []
    for i in range(case["seqs"]):
        n = r.randint(case["new_lo"], case["new_hi"]) if "new_lo" in case else 0
        c = r.randint(case["ctx_lo"], case["ctx_hi"])
        if i == 0:   # the extremes are always there
            n, c = case.get("new_hi", 0), case["ctx_hi"]
        new.append(n)
        total.append(n + c)
    return new, total


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _seen(case):
    """Pairs of a new and a cached token that sees it, and cached tokens that any new one sees."""
    new, total = _lengths(case)
    w, sinks = case["window"], case["sinks"]
    pairs = tokens = 0
    for n, t in zip(new, total):
        if case["op"] == "tree":          # half of the draft, on an average; its positions hardly move the window
            each = min(t - n, w + sinks) if w else t - n
            pairs += n * each + n * (n + 1) // 4
            tokens += each + n
            continue
        for p in (range(t - n, t) if n < 64 or w else ()):
            pairs += min(p + 1, w + min(sinks, max(0, p + 1 - w))) if w else p + 1
        if not (n < 64 or w):
            pairs += (t - n + 1 + t) * n // 2
        tokens += min(t, n + w - 1 + sinks) if w else t
    return pairs, tokens


def work(case):
    if case["op"] == "adjust":
        size, n = 4 if case["type"] == "f32" else 2, case["rows"] * case["vocab"]
        b = 2 * n * size + case["rows"] * (2 * case["history"] // 3 + 2 * case["bias"]) * 4
        return {"bytes": b + (n // 16 if case["grammar"] else 0), "flops": 4 * n}
    new, total = _lengths(case)
    heads, dim = case["kv_heads"], case["dim"]
    token = heads * (dim + 4 / BLOCK)     # codes and scales of a cached token's keys (or values)
    if case["op"] == "evict":
        kept = sum(min(t, case["keep"]) for t in total)
        # all weights and the kept tokens in; list, weights, codes out; and as numbers
        n = sum(total) * heads * 4 + kept * heads * 8 + 4 * kept * token + 4 * kept * heads * dim
        return {"bytes": int(n), "flops": 4 * kept * heads * dim}
    size = 4 if case["type"] == "f32" else 2
    pairs, tokens = _seen(case)
    T, q_heads = sum(new), case["q_heads"]
    if case["op"] == "weigh":
        n = T * q_heads * (dim * size + 4) + tokens * token + sum(total) * heads * 4
        return {"bytes": int(n), "flops": 2 * q_heads * dim * pairs}
    n = T * q_heads * (2 * dim * size + 4) + 2 * tokens * token
    return {"bytes": int(n), "flops": 4 * q_heads * dim * pairs}


def _draft(rng, n):
    """A tree of n drafted tokens, parents first: for each node, bits of itself and of those before it on its path."""
    bits = []
    for i in range(n):
        parent = max(-1, i - 1 - int(rng.random() ** 2 * 8))
        bits.append((bits[parent] if parent >= 0 else 0) | 1 << i)
    return bits


def _word(bits, i):
    w = bits >> (32 * i) & 0xffffffff
    return w - (1 << 32) if w >> 31 else w


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 29)
    kind = torch.float32 if case.get("type") == "f32" else torch.bfloat16

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=dev, dtype=torch.int32)

    if case["op"] == "adjust":
        rows, vocab, most = case["rows"], case["vocab"], case["history"]
        s = dict(case=case, logits=(normal(rows, vocab) * 2.5).to(kind))
        # what a text repeats: a few tokens often, many once
        s["history"] = (uniform(rows, most) ** 4 * vocab).int().clamp_(max=vocab - 1)
        at = torch.arange(rows, device=dev)
        s["history_len"] = torch.where(at == 0, most, whole(most // 3, most + 1, rows)).int()
        s["prompt_len"] = (s["history_len"] * uniform(rows)).int()
        s["repetition"] = torch.where(at % 3 == 1, 1.0, 1 + 0.3 * uniform(rows))
        s["presence"] = torch.where(at % 2 == 1, 0.0, uniform(rows))
        s["frequency"] = torch.where(at % 4 == 3, 0.0, 0.5 * uniform(rows) - 0.1)
        s["bias_index"] = s["bias"] = s["mask"] = s["mask_row"] = None
        if case["bias"]:
            # distinct tokens of a request, then padding
            first = whole(0, vocab, rows, 1)
            step = max(1, vocab // case["bias"])
            index = (first + torch.arange(case["bias"], device=dev) * step) % vocab
            index = torch.where(torch.arange(case["bias"], device=dev) * step < vocab, index, -1)
            s["bias_index"] = torch.where(uniform(rows, case["bias"]) < 0.7, index, -1).int().contiguous()
            s["bias"] = 4 * normal(rows, case["bias"])
        if case["grammar"]:
            # a state of a grammar allows some words of the vocabulary's bits whole, some in part, most not at all
            states = max(1, rows // 3)
            words = -(-vocab // 32)
            some = whole(-2 ** 31, 2 ** 31 - 1, states, words)
            pick = uniform(states, words)
            s["mask"] = torch.where(pick < 0.6, 0, torch.where(pick < 0.8, -1, some)).int().contiguous()
            s["mask_row"] = torch.where(at % 2 == 0, whole(0, states, rows), -1).int()
        s["out"] = torch.empty(rows, vocab, dtype=kind, device=dev)
        return s

    new, total = _lengths(case)
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    evict = case["op"] == "evict"
    count = [min(t, case["keep"]) for t in total] if evict else []
    used = [-(-t // page) for t in total]
    to = [-(-n // page) for n in count]              # the pages that kept tokens move to
    pages = sum(used) + sum(to) + 2
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)

    def table_of(need, skip):
        at = torch.tensor(_starts(need)[:-1])[:, None] + skip
        rank = torch.arange(max(max(need), 1))[None, :] + at
        return order[torch.minimum(rank, torch.tensor(pages - 1)).to(dev)].contiguous()

    def codes():
        x = torch.empty(pages, heads, page, dim, dtype=torch.int8, device=dev)
        flat = x.view(-1)
        for lo in range(0, flat.numel(), 1 << 27):
            part = flat[lo:lo + (1 << 27)]
            part.copy_((normal(part.numel()) * 30).round_().clamp_(-127, 127))
        return x

    s = dict(case=case, table=table_of(used, 0), k=codes(), v=codes(),
             k_scale=(0.8 + 0.4 * uniform(pages, heads, page // BLOCK)) / 30,
             v_scale=(0.8 + 0.4 * uniform(pages, heads, page // BLOCK)) / 30,
             kv_len=torch.tensor(total, dtype=torch.int32, device=dev),
             new=new, total=total, most_new=max(new), most_kv=max(total))
    if case["op"] == "weigh":
        s["weight"] = 1e-4 * uniform(pages, heads, page)           # of tokens that were there before
    if evict:
        s["weight"] = (2 * normal(pages, heads, page)).exp_()      # a few tokens get most of the weight
        s["to_table"] = table_of(to, sum(used))
        s["budget"] = torch.full((len(total),), case["keep"], dtype=torch.int32, device=dev)
        s["kept"] = torch.zeros(len(total), heads, max(count), dtype=torch.int32, device=dev)
        s["count"] = torch.empty(len(total), dtype=torch.int32, device=dev)
        s["counts"] = count
        s["zero"] = torch.zeros(len(total), dtype=torch.int32, device=dev)
        s["back"] = torch.tensor(_starts(count), dtype=torch.int32, device=dev)
        s["k_out"] = torch.empty(sum(count), heads, dim, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.empty(sum(count), heads, dim, dtype=torch.bfloat16, device=dev)
        return s
    T = sum(new)
    s["cu"] = torch.tensor(_starts(new), dtype=torch.int32, device=dev)
    s["q"] = (1.5 * normal(T, case["q_heads"], dim)).to(kind)
    s["tree"] = None
    if case["op"] == "tree":
        import random
        r = random.Random(int(seed) * 31 + 7)
        words = -(-s["most_new"] // 32)
        bits = sum((_draft(r, n) for n in new), [])
        s["tree"] = torch.tensor([[_word(x, i) for i in range(words)] for x in bits], dtype=torch.int32, device=dev)
    s["lse"] = torch.empty(T, case["q_heads"], dtype=torch.float32, device=dev)
    if case["op"] == "weigh":
        s["lse"].copy_(_plain_attention(s, values=False)[1])       # as the attention before gave it
        s["held"] = torch.zeros(len(total), dtype=torch.int32, device=dev)   # weights begin anew
    else:
        s["out"] = torch.empty(T, case["q_heads"], dim, dtype=kind, device=dev)
    return s


# --------------------------------------------------------------- plain forms
def _owner(cu, n):
    """The sequence of each of n packed tokens, and the token's place within it."""
    i = torch.arange(n, device=cu.device)
    b = torch.searchsorted(cu[1:].long(), i, right=True)
    return b, i - cu[b]


def _bits(words, n):
    """Bits of int32 words as truth values [..., n]."""
    i = torch.arange(n, device=words.device)
    return (words.long()[..., i // 32] >> (i % 32)) & 1 > 0


def _plain_scores(s):
    """Masked scores [B, heads, group, N, L] of all sequences side by side; the owners of the packed rows."""
    case = s["case"]
    dev = s["q"].device
    B, N, L, dim = len(s["new"]), s["most_new"], s["most_kv"], case["dim"]
    heads, group = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    kpos = torch.arange(L, device=dev)
    at = s["table"][:, kpos // case["page"]].long()
    slot = (kpos % case["page"])[None, :].expand(B, L)
    k = s["k"][at, :, slot].float() * s["k_scale"][at, :, slot // BLOCK][..., None]     # [B, L, heads, dim]
    b, i = _owner(s["cu"], s["q"].shape[0])
    q = torch.zeros(B, N, heads, group, dim, device=dev)
    q[b, i] = s["q"].float().unflatten(1, (heads, group))
    n = s["cu"][1:] - s["cu"][:-1]
    base = (s["kv_len"] - n)[:, None]                       # cached tokens before the new ones
    qpos = base + torch.arange(N, device=dev)
    drafted = None
    if s["tree"] is not None:
        drafted = torch.zeros(B, N, N, dtype=torch.bool, device=dev)
        drafted[b, i] = _bits(s["tree"], N)
        qpos = base + drafted.sum(-1) - 1                   # as many tokens as its path has
    seen = kpos <= qpos[..., None]
    if case["window"]:
        seen &= (kpos > qpos[..., None] - case["window"]) | (kpos < case["sinks"])
    if drafted is not None:
        j = kpos - base                                     # place among the new tokens
        new = torch.take_along_dim(drafted, j.clamp(0, N - 1)[:, None, :], 2)
        seen = torch.where((j >= 0)[:, None, :], new & (j < n[:, None])[:, None, :], seen)
    q = q.permute(0, 2, 3, 1, 4).reshape(B, heads, group * N, dim)
    p = (q @ k.permute(0, 2, 3, 1)).mul_(dim ** -0.5).view(B, heads, group, N, L)
    return p.masked_fill_(~seen[:, None, None], -math.inf), at, slot, b, i


def _plain_attention(s, values=True):
    case = s["case"]
    p, at, slot, b, i = _plain_scores(s)
    B, heads, group, N, L = p.shape
    top = p.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top)[..., 0].permute(0, 3, 1, 2)[b, i].flatten(1)
    if not values:
        return None, lse
    p = p.div_(torch.where(total > 0, total, 1.0)).view(B, heads, group * N, L)
    v = s["v"][at, :, slot].float() * s["v_scale"][at, :, slot // BLOCK][..., None]
    o = (p @ v.permute(0, 2, 1, 3)).view(B, heads, group, N, case["dim"]).permute(0, 3, 1, 2, 4)
    return o[b, i].reshape(s["q"].shape).to(s["q"].dtype), lse


def _plain_weigh(s):
    p, at, slot, b, i = _plain_scores(s)
    B, heads, group, N, L = p.shape
    lse = torch.full((B, N, heads, group), math.inf, device=p.device)
    lse[b, i] = s["lse"].unflatten(1, (heads, group))
    got = p.sub_(lse.permute(0, 2, 3, 1)[..., None]).exp_().sum((2, 3))              # [B, heads, L]
    kpos = torch.arange(L, device=p.device)
    had = s["weight"][at, :, slot].transpose(1, 2)
    got += torch.where((kpos < s["held"][:, None])[:, None], had, 0.0)
    own_token = kpos < s["kv_len"][:, None]
    at, slot = at[own_token], slot[own_token]
    s["weight"][at, :, slot] = got.transpose(1, 2)[own_token]
    return s["weight"]


def _plain_evict(s):
    case = s["case"]
    dev = s["k"].device
    B, L, page, heads = len(s["total"]), s["most_kv"], case["page"], case["kv_heads"]
    count = torch.minimum(s["kv_len"], s["budget"])
    kpos = torch.arange(L, device=dev)
    at, slot = s["table"][:, kpos // page].long(), (kpos % page)[None, :].expand(B, L)
    w = s["weight"][at, :, slot].transpose(1, 2)                                     # [B, heads, L]
    first = torch.minimum(count, torch.tensor(case["sinks"], device=dev))
    last = torch.minimum(count - first, torch.tensor(case["recent"], device=dev))
    must = (kpos < first[:, None]) | (kpos >= (s["kv_len"] - last)[:, None])
    w = torch.where(must[:, None], math.inf, w)
    w = torch.where((kpos < s["kv_len"][:, None])[:, None], w, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True)[1]
    n = s["kept"].shape[-1]
    i = torch.arange(n, device=dev)
    kept = torch.where(i < count[:, None, None], order[..., :n], L).sort(-1)[0]      # [B, heads, n]
    exists = i < count[:, None]
    kept = torch.where(exists[:, None], kept, 0)
    s["kept"].copy_(kept)
    s["count"].copy_(count)
    # sources and places of all kept tokens
    b = torch.arange(B, device=dev)[:, None, None]
    h = torch.arange(heads, device=dev)[None, :, None]
    src, src_slot = s["table"].long()[b, kept // page], kept % page
    to = s["to_table"].long()[b, (i // page)[None, None].expand(B, heads, n)]
    to_slot = (i % page)[None, None].expand(B, heads, n)
    exists = exists[:, None].expand(B, heads, n)
    h = h.expand(B, heads, n)
    s["weight"][to[exists], h[exists], to_slot[exists]] = s["weight"][src, h, src_slot][exists]
    out = []
    back_b, back_i = _owner(s["back"], s["k_out"].shape[0])
    for x in ("k", "v"):
        codes, scale = s[x], s[x + "_scale"]
        was = torch.where(exists, scale[src, h, src_slot // BLOCK], 0.0)
        pad = -n % BLOCK
        now = torch.nn.functional.pad(was, (0, pad)).unflatten(-1, (-1, BLOCK)).amax(-1)   # a block's largest scale
        now = now.repeat_interleave(BLOCK, -1)[..., :n]
        ratio = torch.where(now > 0, was / now, 0.0)
        rows = (codes[src, h, src_slot].float() * ratio[..., None]).round()
        codes[to[exists], h[exists], to_slot[exists]] = rows[exists].to(torch.int8)
        scale[to[exists], h[exists], (to_slot // BLOCK)[exists]] = now[exists]
        out.append((rows * now[..., None])[back_b, :, back_i].to(torch.bfloat16))
    return {"kept": s["kept"], "count": s["count"], "weight": s["weight"], "k": out[0], "v": out[1]}


def _plain_adjust(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    i = torch.arange(s["history"].shape[1], device=x.device)
    known = (i < s["history_len"][:, None]).float()
    said = known * (i >= s["prompt_len"][:, None])
    seen = torch.zeros_like(x).scatter_add_(1, s["history"].long(), known) > 0
    times = torch.zeros_like(x).scatter_add_(1, s["history"].long(), said)
    again = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / again, x * again), x)
    x = x - s["frequency"][:, None] * times
    x = torch.where(times > 0, x - s["presence"][:, None], x)
    if s["bias"] is not None:
        at = s["bias_index"].long()
        x = x + torch.zeros_like(x).scatter_add_(1, at.clamp(min=0), torch.where(at >= 0, s["bias"], 0.0))
    if s["mask"] is not None:
        row = s["mask_row"].long()
        allowed = _bits(s["mask"], vocab)[row.clamp(min=0)] | (row < 0)[:, None]
        x = torch.where(allowed, x, -math.inf)
    return x.to(s["logits"].dtype)


def run(state):
    s, case = state, state["case"]
    if case["op"] == "adjust":
        if own:
            _q4().q4_adjust_logits(s["out"], s["logits"], history=s["history"], history_len=s["history_len"],
                                   prompt_len=s["prompt_len"], repetition=s["repetition"], presence=s["presence"],
                                   frequency=s["frequency"], bias_index=s["bias_index"], bias=s["bias"],
                                   mask=s["mask"], mask_row=s["mask_row"])
            return {"logits": s["out"]}
        return {"logits": _plain_adjust(s)}
    if own:
        q4 = _q4()
        cache = q4.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if case["op"] == "evict":
        if own:
            q4.q4_kv_select(s["kept"], s["count"], s["weight"], cache, s["table"], s["kv_len"], s["budget"],
                            max_kv=s["most_kv"], sinks=case["sinks"], recent=case["recent"])
            q4.q4_kv_compact(cache, s["table"], s["kv_len"], s["kept"], s["count"], weight=s["weight"],
                             to_table=s["to_table"])
            q4.q4_kv_gather(s["k_out"], s["v_out"], cache, s["to_table"], s["zero"], s["back"])
            return {"kept": s["kept"], "count": s["count"], "weight": s["weight"], "k": s["k_out"], "v": s["v_out"]}
        return _plain_evict(s)
    if case["op"] == "weigh":
        if own:
            q4.q4_kv_weigh(s["weight"], s["q"], s["lse"], cache, s["table"], s["kv_len"], s["cu"], max_q=s["most_new"],
                           max_kv=s["most_kv"], held=s["held"], window=case["window"], sinks=case["sinks"])
            return {"weight": s["weight"]}
        return {"weight": _plain_weigh(s)}
    if own:
        q4.q4_kv_attention(s["out"], s["q"], cache, s["table"], s["kv_len"], s["cu"], max_q=s["most_new"],
                           max_kv=s["most_kv"], window=case["window"], sinks=case["sinks"], tree=s["tree"],
                           lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    out, lse = _plain_attention(s)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------ 64-bit values
def _held(s, x, b, pos, h):
    """Cached keys or values (x) of head h at positions pos of sequence b."""
    page = s["case"]["page"]
    p, t = s["table"][b].long()[pos // page], pos % page
    return s[x][p, h, t].double() * s[x + "_scale"][p, h, t // BLOCK].double()[..., None]


def _exact_rows(s):
    """For each sequence, query head and run of rows: their place, scores in 64 bits and who sees what."""
    case = s["case"]
    group, w = case["q_heads"] // case["kv_heads"], case["window"]
    at = 0
    for b, (n, t) in enumerate(zip(s["new"], s["total"])):
        pos = torch.arange(t, device=s["q"].device)
        for lo in range(0, n, 2048):
            hi = min(n, lo + 2048)
            place = torch.arange(t - n + lo, t - n + hi, device=pos.device)
            if s["tree"] is not None:
                words = s["tree"][at + lo:at + hi].long() & 0xffffffff
                path = torch.stack([(words[:, j // 32] >> (j % 32)) % 2 for j in range(n)], 1) == 1
                place = t - n - 1 + path.sum(1)
            see = pos[None, :] <= place[:, None]
            if w:
                see = see & ((place[:, None] - pos[None, :] < w) | (pos < case["sinks"])[None, :])
            if s["tree"] is not None:
                see[:, t - n:] = path
            for h in range(case["q_heads"]):
                k = _held(s, "k", b, pos, h // group)
                score = s["q"][at + lo:at + hi, h].double() @ k.T / math.sqrt(case["dim"])
                yield b, h, slice(at + lo, at + hi), pos, torch.where(see, score, -math.inf)
        at += n


def _exact_attention(s):
    case = s["case"]
    group = case["q_heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=s["q"].device)
    for b, h, rows, pos, score in _exact_rows(s):
        lse[rows, h] = torch.logsumexp(score, -1)
        p = torch.softmax(score, -1).nan_to_num(0.0)       # a row that sees nothing
        out[rows, h] = p @ _held(s, "v", b, pos, h // group)
    return {"out": out, "lse": lse}


def _exact_weigh(s):
    case = s["case"]
    page, group = case["page"], case["q_heads"] // case["kv_heads"]
    weight = s["weight"].double()
    for b, t in enumerate(s["total"]):
        pos = torch.arange(t, device=weight.device)
        fresh = pos >= s["held"][b]
        p, slot = s["table"][b].long()[pos // page], pos % page
        weight[p, :, slot] = torch.where(fresh[:, None], 0.0, weight[p, :, slot])
    for b, h, rows, pos, score in _exact_rows(s):
        p, slot = s["table"][b].long()[pos // page], pos % page
        weight[p, h // group, slot] += torch.exp(score - s["lse"][rows, h].double()[:, None]).sum(0)
    return {"weight": weight}


def _exact_evict(s):
    case = s["case"]
    page, heads = case["page"], case["kv_heads"]
    weight, kept = s["weight"].double(), torch.zeros_like(s["kept"])
    ks, vs = [], []
    for b, (t, n) in enumerate(zip(s["total"], s["counts"])):
        first = min(case["sinks"], n)
        last = min(case["recent"], n - first)
        pos = torch.arange(t, device=weight.device)
        w = s["weight"][s["table"][b].long()[pos // page], :, pos % page].double().T        # [heads, t]
        middle = torch.sort(-w[:, first:t - last], dim=-1, stable=True)[1][:, :n - first - last] + first
        ends = torch.cat([pos[:first], pos[t - last:]])
        keep = torch.cat([middle, ends.expand(heads, -1)], 1).sort(-1)[0]
        kept[b, :, :n] = keep
        i = torch.arange(n, device=weight.device)
        to = s["to_table"][b].long()[i // page]
        both = {"k": [], "v": []}
        for h in range(heads):
            weight[to, h, i % page] = w[h, keep[h]]
            for x in both:
                p, slot = s["table"][b].long()[keep[h] // page], keep[h] % page
                scale = s[x + "_scale"][p, h, slot // BLOCK].double()
                step = torch.stack([part.max() for part in scale.split(BLOCK)]).repeat_interleave(BLOCK)[:n]
                code = (s[x][p, h, slot].double() * (scale / step)[:, None]).round()
                both[x].append(code * step[:, None])
        ks.append(torch.stack(both["k"], 1))
        vs.append(torch.stack(both["v"], 1))
    count = torch.tensor(s["counts"], dtype=torch.int32)
    return {"kept": kept, "count": count, "weight": weight, "k": torch.cat(ks), "v": torch.cat(vs)}


def _exact_adjust(s):
    out = s["logits"].double()
    vocab = out.shape[1]
    for r in range(out.shape[0]):
        n, prompt = int(s["history_len"][r]), int(s["prompt_len"][r])
        text = s["history"][r, :n].long()
        row = out[r]
        ids = torch.unique(text)
        again, x = float(s["repetition"][r]), row[ids]
        row[ids] = torch.where(x > 0, x / again, x * again)
        times = torch.bincount(text[prompt:], minlength=vocab)
        row -= times * float(s["frequency"][r]) + (times > 0) * float(s["presence"][r])
        if s["bias"] is not None:
            used = s["bias_index"][r] >= 0
            row[s["bias_index"][r][used].long()] += s["bias"][r][used].double()
        if s["mask"] is not None and int(s["mask_row"][r]) >= 0:
            words = s["mask"][int(s["mask_row"][r])].cpu().numpy().view("uint8")
            allowed = torch.from_numpy(np.unpackbits(words, bitorder="little")[:vocab]).to(out.device)
            row[allowed == 0] = -math.inf
    return {"logits": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_attention, "sinks": _exact_attention, "weigh": _exact_weigh, "evict": _exact_evict,
            "adjust": _exact_adjust}[case["op"]](s)
