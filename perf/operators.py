"""Serving operators around the quantised matmuls: cases, plain forms and 64-bit values.

Four operators that a decode step needs between its Q4_0 projections and its
next token, over a paged key/value cache held in 8 bits (one fp32 scale for
each block of 16 tokens of a head):

* append     new tokens' queries, keys and values: optional RMS norm of each
             head's queries and keys, position rotation, the rotated queries
             out, keys and values quantised into the cache's pages;
* gather     cached keys and values back as numbers (copying a sequence out,
             looking at what a cache holds);
* attention  the new tokens' queries over the cached tokens;
* sample     one token a row from its logits: temperature, top-k, top-p, min-p,
             from a given uniform number.

A cache's codes are returned as the values they stand for: an append case
appends and then gathers the blocks that it wrote.
"""

import math

import torch

own = False

BLOCK = 16           # tokens that share a scale
TINY = 2.0 ** -110   # scales below this are stored as zero
WEIGHT_BITS = 40     # sampling weights: exp(z - max) in units of 2^-40


def _q4():
    import quantized_weight_q4_gb300 as q4
    return q4


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one user, one token, full-precision activations, 32 heads of 128 without sharing
        # (hidden size 4096): the smallest call of a decode loop
        dict(name="append-one", op="append", type="f32", seqs=1, new_lo=1, new_hi=1, ctx_lo=613, ctx_hi=613,
             q_heads=32, kv_heads=32, dim=128, page=64, rope=128, style="pairs", norm=False),
        # prompts of several users in one batch, ragged, some continuing a partly filled block;
        # shared heads, norms of queries and keys
        dict(name="append-prompts", op="append", type="bf16", seqs=7, new_lo=211, new_hi=4001, ctx_lo=0, ctx_hi=1500,
             q_heads=32, kv_heads=8, dim=128, page=64, rope=128, style="halves", norm=True),
        # looking at one short sequence
        dict(name="gather-one", op="gather", type="f32", seqs=1, ctx_lo=333, ctx_hi=333, kv_heads=8, dim=128, page=16),
        # moving a batch of sequences out of the cache
        dict(name="gather-batch", op="gather", type="bf16", seqs=24, ctx_lo=100, ctx_hi=6001, kv_heads=8, dim=128,
             page=64),
        # one user early in an answer: latency
        dict(name="attend-one-short", op="attention", type="f32", seqs=1, new_lo=1, new_hi=1, ctx_lo=389, ctx_hi=389,
             q_heads=32, kv_heads=32, dim=128, page=64, window=0),
        # one user deep in a long document: the long axis has to be split
        dict(name="attend-one-long", op="attention", type="bf16", seqs=1, new_lo=1, new_hi=1, ctx_lo=131070,
             ctx_hi=131070, q_heads=32, kv_heads=8, dim=128, page=64, window=0),
        # a serving batch, one token each, ragged contexts
        dict(name="attend-batch", op="attention", type="bf16", seqs=64, new_lo=1, new_hi=1, ctx_lo=50, ctx_hi=8191,
             q_heads=32, kv_heads=8, dim=128, page=64, window=0),
        # checking several drafted tokens a sequence at once, small heads, small pages, a sliding window
        dict(name="attend-drafts", op="attention", type="f32", seqs=12, new_lo=2, new_hi=5, ctx_lo=700, ctx_hi=5000,
             q_heads=16, kv_heads=4, dim=64, page=16, window=2048),
        # pieces of prompts on top of contexts of several lengths, in one batch with single tokens
        dict(name="attend-chunks", op="attention", type="bf16", seqs=6, new_lo=1, new_hi=1537, ctx_lo=0, ctx_hi=9000,
             q_heads=32, kv_heads=8, dim=128, page=64, window=0),
        # one long prompt from nothing
        dict(name="attend-prompt", op="attention", type="bf16", seqs=1, new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0,
             q_heads=32, kv_heads=8, dim=128, page=64, window=0),
        # the end of one user's decode step
        dict(name="sample-one", op="sample", type="f32", rows=1, vocab=32000, greedy=False),
        # a serving batch, every row with settings of its own, some greedy, an odd vocabulary
        dict(name="sample-batch", op="sample", type="bf16", rows=200, vocab=128007, greedy=True),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["append", "append", "gather", "attention", "attention", "attention", "sample"])
    kind = rng.choice(["f32", "bf16"])
    if op == "sample":
        return dict(op=op, type=kind, rows=_log(rng, 1, 96), vocab=_log(rng, 500, 128000), greedy=rng.random() < 0.5)
    kv_heads = rng.choice([1, 2, 4, 8])
    c = dict(op=op, type=kind, kv_heads=kv_heads, dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]))
    if op == "gather":
        c.update(seqs=_log(rng, 1, 24), ctx_lo=_log(rng, 1, 400), ctx_hi=_log(rng, 401, 6000))
        return c
    c.update(q_heads=kv_heads * rng.choice([1, 3, 4, 8] if kv_heads <= 4 else [1, 4]))
    if op == "append":
        long = rng.random() < 0.5
        c.update(seqs=_log(rng, 1, 7 if long else 64), new_lo=1, new_hi=_log(rng, 2, 2000) if long else 1,
                 ctx_lo=0, ctx_hi=_log(rng, 1, 1500), rope=c["dim"] // rng.choice([1, 1, 2]),
                 style=rng.choice(["halves", "pairs"]), norm=rng.random() < 0.5)
        return c
    form = rng.choice(["single", "single", "drafts", "prompts"])
    if form == "prompts":
        c.update(type="bf16", seqs=rng.randint(1, 4), new_lo=_log(rng, 2, 100), new_hi=_log(rng, 101, 2500),
                 ctx_lo=0, ctx_hi=_log(rng, 1, 4000), window=rng.choice([0, 0, 1000]))
    else:
        top = 1 if form == "single" else rng.randint(2, 8)
        c.update(seqs=_log(rng, 1, 60), new_lo=1, new_hi=top, ctx_lo=_log(rng, 1, 500), ctx_hi=_log(rng, 501, 8000),
                 window=rng.choice([0, 0, 777]))
    return c


# -------------------------------------------------------------------- inputs
def _lengths(case):
    """New tokens and cached tokens (after the append) of each sequence: the same for every seed."""
    import random
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    new, total = [], []
    for i in range(case["seqs"]):
        n = r.randint(case["new_lo"], case["new_hi"]) if "new_lo" in case else 0
        c = r.randint(case["ctx_lo"], case["ctx_hi"])
        if i == 0:   # the extremes are always there
            n, c = case.get("new_hi", 0), case["ctx_hi"]
        new.append(n)
        total.append(n + c + (n + c == 3 * 1024))
    return new, total


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _visible(new, total, window):
    """Keys seen by all new queries together (causal, at most `window` of them each)."""
    seen = 0
    for n, t in zip(new, total):
        first, last = t - n + 1, t
        if window and last > window:
            short = max(0, window - first + 1)   # queries that see fewer than `window` keys
            seen += sum(range(first, first + short)) + (n - short) * window
        else:
            seen += (first + last) * n // 2
    return seen


def _read_keys(new, total, window):
    """Cached tokens that at least one new query sees."""
    return sum(min(t, n + window - 1) if window else t for n, t in zip(new, total))


def work(case):
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * size + case["rows"] * 28, "flops": 4 * n}
    new, total = _lengths(case)
    heads, dim = case["kv_heads"], case["dim"]
    token = 2 * heads * (dim + 4 / BLOCK)    # codes and scales of one cached token
    if case["op"] == "gather":
        return {"bytes": int(sum(total) * (token + 2 * heads * dim * size)), "flops": 2 * sum(total) * heads * dim}
    T, q_heads = sum(new), case["q_heads"]
    if case["op"] == "append":
        first = [(t - n) // BLOCK * BLOCK for n, t in zip(new, total)]
        back = sum(t - f for t, f in zip(total, first))       # tokens of the blocks written
        n = T * (2 * q_heads + 2 * heads) * dim * size        # queries in and out, keys and values in
        n += back * (token + 2 * heads * dim * size) + T * case["rope"] * 4
        return {"bytes": int(n), "flops": T * (q_heads + heads) * dim * 6}
    n = 2 * T * q_heads * dim * size + _read_keys(new, total, case["window"]) * token
    return {"bytes": int(n), "flops": 4 * q_heads * dim * _visible(new, total, case["window"])}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    kind = torch.float32 if case["type"] == "f32" else torch.bfloat16

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    if case["op"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        logits = normal(rows, vocab) * 2.5
        top = torch.randint(0, vocab, (rows, 40), generator=g, device=dev)
        logits.scatter_add_(1, top, 6 + 3 * normal(rows, 40))       # some likely tokens, as a trained model gives
        s = dict(case=case, logits=logits.to(kind), u=uniform(rows))
        s["temperature"] = 0.5 + uniform(rows)
        s["top_k"] = torch.randint(1, 200, (rows,), generator=g, device=dev, dtype=torch.int32)
        s["top_p"] = 0.6 + 0.39 * uniform(rows)
        s["min_p"] = 0.05 * uniform(rows)
        at = torch.arange(rows, device=dev)
        s["top_k"] = torch.where(at % 3 == 1, 0, s["top_k"])         # off on some rows, as requests differ
        s["top_p"] = torch.where(at % 4 == 2, 1.0, s["top_p"])
        s["min_p"] = torch.where(at % 2 == 1, 0.0, s["min_p"])
        if case["greedy"]:
            s["temperature"] = torch.where(at % 5 == 3, 0.0, s["temperature"])
        s["tokens"] = torch.empty(rows, dtype=torch.int32, device=dev)
        s["probs"] = torch.empty(rows, dtype=torch.float32, device=dev)
        return s

    new, total = _lengths(case)
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    used = [-(-t // page) for t in total]
    pages, most = sum(used) + 2, max(max(used), 1)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(len(total), most, dtype=torch.int32)
    at = _starts(used)
    rank = torch.arange(most)[None, :] + torch.tensor(at[:-1])[:, None]
    table = order[torch.minimum(rank, torch.tensor(pages - 1)).to(dev)].contiguous()

    def codes():
        x = torch.empty(pages, heads, page, dim, dtype=torch.int8, device=dev)
        flat = x.view(-1)
        for lo in range(0, flat.numel(), 1 << 27):
            part = flat[lo:lo + (1 << 27)]
            part.copy_((normal(part.numel()) * 30).round_().clamp_(-127, 127))
        return x

    s = dict(case=case, table=table, k=codes(), v=codes(),
             k_scale=(0.8 + 0.4 * uniform(pages, heads, page // BLOCK)) / 30,
             v_scale=(0.8 + 0.4 * uniform(pages, heads, page // BLOCK)) / 30,
             kv_len=torch.tensor(total, dtype=torch.int32, device=dev),
             new=new, total=total, most_new=max(new), most_kv=max(total))
    T = sum(new)
    s["cu"] = torch.tensor(_starts(new), dtype=torch.int32, device=dev)
    if case["op"] == "gather":
        first, count = [0] * len(total), total
    elif case["op"] == "append":
        first = [(t - n) // BLOCK * BLOCK for n, t in zip(new, total)]
        count = [t - f for t, f in zip(total, first)]
        q_heads = case["q_heads"]
        # queries, keys and values as one projection gives them: three slices of each row, and some columns that
        # belong to something else
        rows = normal(T, (q_heads + 2 * heads) * dim + 32).to(kind)
        s["q"] = rows[:, :q_heads * dim].unflatten(1, (q_heads, dim))
        s["knew"] = rows[:, q_heads * dim:(q_heads + heads) * dim].unflatten(1, (heads, dim))
        s["vnew"] = rows[:, (q_heads + heads) * dim:-32].unflatten(1, (heads, dim))
        half = case["rope"] // 2
        turn = torch.arange(max(total), dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half) / half)
        s["cos"], s["sin"] = turn.cos().float().to(dev), turn.sin().float().to(dev)
        s["q_norm"] = 1 + 0.1 * normal(dim) if case["norm"] else None
        s["k_norm"] = 1 + 0.1 * normal(dim) if case["norm"] else None
        s["q_out"] = torch.empty(T, q_heads, dim, dtype=kind, device=dev)
    else:
        s["q"] = (1.5 * normal(T, case["q_heads"], dim)).to(kind)
        s["out"] = torch.empty(T, case["q_heads"], dim, dtype=kind, device=dev)
        return s
    s["first"] = torch.tensor(first, dtype=torch.int32, device=dev)
    s["back"] = torch.tensor(_starts(count), dtype=torch.int32, device=dev)
    s["k_out"] = torch.empty(sum(count), heads, dim, dtype=kind, device=dev)
    s["v_out"] = torch.empty(sum(count), heads, dim, dtype=kind, device=dev)
    return s


# --------------------------------------------------------------- plain forms
def _owner(cu, n):
    """The sequence of each of n packed tokens, and the token's place within it."""
    i = torch.arange(n, device=cu.device)
    b = torch.searchsorted(cu[1:].long(), i, right=True)
    return b, i - cu[b]


def _plain_gather(s):
    case = s["case"]
    b, i = _owner(s["back"], s["k_out"].shape[0])
    pos = s["first"][b] + i
    at, slot = s["table"][b, pos // case["page"]].long(), pos % case["page"]
    kind = s["k_out"].dtype
    k = s["k"][at, :, slot].float() * s["k_scale"][at, :, slot // BLOCK][..., None]
    v = s["v"][at, :, slot].float() * s["v_scale"][at, :, slot // BLOCK][..., None]
    return k.to(kind), v.to(kind)


def _sum_pairs(x):
    """Sum over the last axis (a power of two), neighbours first: the order is part of the definition."""
    while x.shape[-1] > 1:
        x = x[..., 0::2] + x[..., 1::2]
    return x


def _norm(x, weight):
    mean = _sum_pairs(x * x) / x.shape[-1]
    return x * (1.0 / torch.sqrt(mean + 1e-6)) * weight


def _rotate(x, cos, sin, style):
    """The first 2 * cos.shape[-1] elements of each head, turned in pairs; the others stay."""
    n = 2 * cos.shape[-1]
    c, s = cos[:, None, :], sin[:, None, :]
    part, rest = x[..., :n], x[..., n:]
    if style == "halves":
        a, b = part[..., :n // 2], part[..., n // 2:]
        return torch.cat([a * c - b * s, b * c + a * s, rest], -1)
    a, b = part[..., 0::2], part[..., 1::2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), rest], -1)


def _plain_store(codes, scale, x, at, slot, lead, fresh, page):
    """Quantise x [T, heads, dim] into the cache. lead: the first new token of each block."""
    heads, dim = x.shape[1], x.shape[2]
    blocks = page // BLOCK
    key = (at[:, None] * heads + torch.arange(heads, device=x.device)) * blocks + (slot // BLOCK)[:, None]
    most = torch.zeros(scale.numel(), device=x.device).scatter_reduce(0, key.flatten(), x.abs().amax(-1).flatten(),
                                                                      "amax")
    touched = key[lead].flatten()                       # each block once
    was = torch.where(fresh[lead].repeat_interleave(heads), 0.0, scale.view(-1)[touched])
    now = torch.maximum(was, most[touched] / 127.0)
    now = torch.where(now < TINY, 0.0, now)
    ratio = torch.where(now > 0, was / now, 0.0)
    rows = codes.view(-1, BLOCK, dim)
    rows[touched] = (rows[touched].float() * ratio[:, None, None]).round().to(torch.int8)
    scale.view(-1)[touched] = now
    inverse = torch.where(now > 0, 1.0 / now, 0.0)
    each = torch.zeros_like(most)
    each[touched] = inverse
    rows[key, (slot % BLOCK)[:, None]] = (x * each[key][..., None]).round().clamp(-127, 127).to(torch.int8)


def _plain_append(s):
    case = s["case"]
    T = s["q"].shape[0]
    b, i = _owner(s["cu"], T)
    n = (s["cu"][1:] - s["cu"][:-1])[b]
    start = s["kv_len"][b] - n
    pos = start + i
    q, k, v = s["q"].float(), s["knew"].float(), s["vnew"].float()
    if case["norm"]:
        q, k = _norm(q, s["q_norm"]), _norm(k, s["k_norm"])
    cos, sin = s["cos"][pos], s["sin"][pos]
    q, k = _rotate(q, cos, sin, case["style"]), _rotate(k, cos, sin, case["style"])
    at, slot = s["table"][b, pos // case["page"]].long(), (pos % case["page"]).long()
    lead = (i == 0) | (pos % BLOCK == 0)
    fresh = pos // BLOCK * BLOCK >= start              # no earlier token in the block
    _plain_store(s["k"], s["k_scale"], k, at, slot, lead, fresh, case["page"])
    _plain_store(s["v"], s["v_scale"], v, at, slot, lead, fresh, case["page"])
    return q.to(s["q_out"].dtype)


def _plain_attention(s):
    case = s["case"]
    dev, kind = s["q"].device, s["q"].dtype
    B, N, L, dim = len(s["new"]), s["most_new"], s["most_kv"], case["dim"]
    heads, group = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    kpos = torch.arange(L, device=dev)
    at = s["table"][:, kpos // case["page"]].long()
    slot = (kpos % case["page"])[None, :].expand(B, L)
    k = s["k"][at, :, slot].float() * s["k_scale"][at, :, slot // BLOCK][..., None]     # [B, L, heads, dim]
    v = s["v"][at, :, slot].float() * s["v_scale"][at, :, slot // BLOCK][..., None]
    b, i = _owner(s["cu"], s["q"].shape[0])
    q = torch.zeros(B, N, heads, group, dim, device=dev)
    q[b, i] = s["q"].float().unflatten(1, (heads, group))
    n = s["cu"][1:] - s["cu"][:-1]
    qpos = (s["kv_len"] - n)[:, None] + torch.arange(N, device=dev)
    seen = kpos <= qpos[..., None]
    if case["window"]:
        seen &= kpos > qpos[..., None] - case["window"]
    q = q.permute(0, 2, 3, 1, 4).reshape(B, heads, group * N, dim)
    p = (q @ k.permute(0, 2, 3, 1)).mul_(dim ** -0.5).view(B, heads, group, N, L)
    p.masked_fill_(~seen[:, None, None], -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True)).view(B, heads, group * N, L)
    o = (p @ v.permute(0, 2, 1, 3)).view(B, heads, group, N, dim).permute(0, 3, 1, 2, 4)
    return o[b, i].reshape(s["q"].shape).to(kind)


def _plain_sample(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    greedy = s["temperature"] < 1e-5
    z = x * torch.where(greedy, 1.0, 1.0 / s["temperature"])[:, None]
    e = (z - z.amax(-1, keepdim=True)).exp()
    w = (e * 2.0 ** WEIGHT_BITS).long()                    # whole numbers: sums do not depend on their order
    order = torch.sort(z, dim=-1, descending=True, stable=True)[1]
    most = torch.where(greedy, 1, torch.where(s["top_k"] > 0, s["top_k"], vocab))
    ranked = torch.where(torch.arange(vocab, device=x.device) < most[:, None], w.gather(1, order), 0)
    before = ranked.cumsum(-1) - ranked
    whole = ranked.sum(-1)
    part = (s["top_p"].double() * whole.double()).ceil().long()
    part = torch.where(s["top_p"] < 1, part, whole).clamp(min=1)
    keep = (before < part[:, None]) & (e.gather(1, order) >= s["min_p"][:, None])
    kept = torch.zeros_like(w).scatter(1, order, torch.where(keep, ranked, 0))
    upto = kept.cumsum(-1)
    whole = upto[:, -1]
    r = torch.minimum((s["u"].double() * whole.double()).long(), whole - 1)
    token = (upto <= r[:, None]).sum(-1)
    prob = kept.gather(1, token[:, None])[:, 0].float() / whole.float()
    return token.to(torch.int32), prob


def run(state):
    s, case = state, state["case"]
    if case["op"] == "sample":
        if own:
            _q4().q4_sample(s["tokens"], s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                            top_p=s["top_p"], min_p=s["min_p"], probs=s["probs"])
            return {"tokens": s["tokens"], "probs": s["probs"]}
        token, prob = _plain_sample(s)
        return {"tokens": token, "probs": prob}
    if own:
        q4 = _q4()
        cache = q4.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if case["op"] == "attention":
        if own:
            q4.q4_kv_attention(s["out"], s["q"], cache, s["table"], s["kv_len"], s["cu"], max_q=s["most_new"],
                               max_kv=s["most_kv"], window=case["window"])
            return {"out": s["out"]}
        return {"out": _plain_attention(s)}
    found = {}
    if case["op"] == "append":
        if own:
            q4.q4_kv_append(cache, s["q_out"], s["q"], s["knew"], s["vnew"], s["table"], s["kv_len"], s["cu"],
                            cos=s["cos"], sin=s["sin"],
                            rope_style=q4.Q4_ROPE_HALVES if case["style"] == "halves" else q4.Q4_ROPE_PAIRS,
                            q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6)
            found["q"] = s["q_out"]
        else:
            found["q"] = _plain_append(s)
    if own:
        q4.q4_kv_gather(s["k_out"], s["v_out"], cache, s["table"], s["first"], s["back"])
        return {**found, "k": s["k_out"], "v": s["v_out"]}
    k, v = _plain_gather(s)
    return {**found, "k": k, "v": v}


# ------------------------------------------------------------ 64-bit values
def _tokens(s, b, lo, hi):
    """Cache row, slot and block of tokens lo..hi-1 of sequence b."""
    page = s["case"]["page"]
    pos = torch.arange(lo, hi, device=s["table"].device)
    return s["table"][b].long()[pos // page], pos % page, (pos % page) // BLOCK


def _held(s, b, lo, hi):
    p, t, j = _tokens(s, b, lo, hi)
    return [s[x][p, :, t].double() * s[x + "_scale"][p, :, j].double()[..., None] for x in ("k", "v")]


def _exact_gather(s):
    ks, vs = [], []
    for b in range(len(s["total"])):
        k, v = _held(s, b, int(s["first"][b]), s["total"][b])
        ks.append(k)
        vs.append(v)
    return torch.cat(ks), torch.cat(vs)


def _exact_turn(x, pos, case, weight):
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
    half = case["rope"] // 2
    ang = pos.double()[:, None] * 10000.0 ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    turn = torch.polar(torch.ones_like(ang), ang)[:, None, :]
    part = x[..., :2 * half]
    if case["style"] == "halves":
        z = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * turn
        done = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(part.unflatten(-1, (half, 2)).contiguous()) * turn
        done = torch.view_as_real(z).flatten(-2)
    return torch.cat([done, x[..., 2 * half:]], -1)


def _exact_append(s):
    case = s["case"]
    qs, at = [], 0
    out = {"k": [], "v": []}
    for b, (n, t) in enumerate(zip(s["new"], s["total"])):
        rows = slice(at, at + n)
        at += n
        pos = torch.arange(t - n, t, device=s["q"].device)
        qs.append(_exact_turn(s["q"][rows].double(), pos, case, s["q_norm"]))
        lo = (t - n) // BLOCK * BLOCK
        had = t - n - lo                                    # earlier tokens of the first block
        p, slot, j = _tokens(s, b, lo, t)
        for x, fresh in (("k", _exact_turn(s["knew"][rows].double(), pos, case, s["k_norm"])),
                         ("v", s["vnew"][rows].double())):
            pad = -(t - lo) % BLOCK
            shape = (had, *fresh.shape[1:])
            rowsx = torch.cat([torch.zeros(shape, device=fresh.device, dtype=torch.float64), fresh,
                               torch.zeros(pad, *fresh.shape[1:], device=fresh.device, dtype=torch.float64)])
            blocks = rowsx.unflatten(0, (-1, BLOCK))        # [blocks, 16, heads, dim]
            step = blocks.abs().amax((1, 3)) / 127
            old = s[x + "_scale"][p[0], :, j[0]].double()
            if had:
                step[0] = torch.maximum(step[0], old)
            code = (blocks / step[:, None, :, None].clamp(min=1e-300)).round().clamp(-127, 127)
            if had:
                kept = s[x][p[:had], :, slot[:had]].double()
                code[0, :had] = (kept * (old / step[0])[None, :, None]).round()
            out[x].append((code * step[:, None, :, None]).flatten(0, 1)[:t - lo])
    return {"q": torch.cat(qs), "k": torch.cat(out["k"]), "v": torch.cat(out["v"])}


def _exact_attention(s):
    case = s["case"]
    group, dim = case["q_heads"] // case["kv_heads"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    at = 0
    for b, (n, t) in enumerate(zip(s["new"], s["total"])):
        q = s["q"][at:at + n].double()
        k, v = _held(s, b, 0, t)
        for lo in range(0, n, 2048):
            hi = min(n, lo + 2048)
            qpos = torch.arange(t - n + lo, t - n + hi, device=q.device)[:, None]
            kpos = torch.arange(t, device=q.device)[None, :]
            seen = kpos <= qpos
            if case["window"]:
                seen &= kpos > qpos - case["window"]
            for h in range(case["q_heads"]):
                score = q[lo:hi, h] @ k[:, h // group].T / math.sqrt(dim)
                p = torch.softmax(torch.where(seen, score, -math.inf), -1)
                out[at + lo:at + hi, h] = p @ v[:, h // group]
        at += n
    return out


def _exact_sample(s):
    tokens, probs = [], []
    for r in range(s["logits"].shape[0]):
        t = float(s["temperature"][r])
        z = s["logits"][r].double()
        k = int(s["top_k"][r]) or z.numel()
        if t < 1e-5:
            t, k = 1.0, 1
        p = torch.softmax(z / t, -1)
        p, order = torch.sort(p, descending=True, stable=True)
        p, order = p[:k] / p[:k].sum(), order[:k]
        keep = (p.cumsum(-1) - p < float(s["top_p"][r])) & (p / p[0] >= float(s["min_p"][r]))
        p = torch.zeros_like(z).scatter(0, order, torch.where(keep, p, 0.0))
        p = p / p.sum()
        token = int((p.cumsum(-1) <= float(s["u"][r])).sum().clamp(max=z.numel() - 1))
        tokens.append(token)
        probs.append(p[token])
    return {"tokens": torch.tensor(tokens, dtype=torch.int32), "probs": torch.stack(probs)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    if case["op"] == "attention":
        return {"out": _exact_attention(s)}
    if case["op"] == "append":
        return _exact_append(s)
    k, v = _exact_gather(s)
    return {"k": k, "v": v}
