"""The operators for long and drafted decoding as a decode loop runs them: drafts checked
and their accepted path kept, a cache held to a budget step by step (eagerly and from a
captured graph), logits adjusted before sampling."""

import os

import numpy as np
import pytest

from gpu_util import device, torch
from long_util import attend, draft, select, slots, visible, words_of
from serve_util import dev, f32, i32, rng, starts
from test_gpu_kv_attention import bound

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


class Held:
    """A cache's values as the reference wants them: read back from the device."""

    def __init__(self, cache, table, heads):
        self.cache, self.table, self.heads = cache, table, heads

    def values(self, b, n):
        k, v = (torch.empty(max(n, 1), self.heads, self.cache.dim, device=device()) for _ in range(2))
        if n:
            q4.q4_kv_gather(k, v, self.cache, self.table[b:b + 1], i32([0]), i32([0, n]))
        torch.cuda.synchronize()
        return k[:n].double().cpu().numpy(), v[:n].double().cpu().numpy()


def tables(n, half):
    ang = torch.arange(n)[:, None] * 10000.0 ** (-torch.arange(half) / half)
    return ang.cos().float().to(device()), ang.sin().float().to(device())


def turned(x, pos, half):
    """Keys at their positions in 64 bits (pairs half of a head apart)."""
    ang = pos[:, None] * 10000.0 ** (-np.arange(half) / half)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = x[..., :half], x[..., half:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_drafts_and_their_accepted_paths(kind):
    """Three sequences, two rounds of drafts and a single token after them.  Before: each draft's rows against 64-bit
    attention over what the cache holds.  After: the cache holds the accepted tokens at consecutive places, turned by
    their positions."""
    B, Hq, heads, D, page = 3, 8, 2, 64, 16
    g = rng(91, 1)
    cache = q4.KVCache.empty(B * 12, heads, D, page)
    table = i32(g.permutation(B * 12).reshape(B, 12))
    cos, sin = tables(400, D // 2)
    lens = [0] * B
    truth = [[np.zeros((0, heads, D)), np.zeros((0, heads, D))] for _ in range(B)]     # accepted keys (turned), values
    most = [0.0, 0.0]                 # largest key and value that a block may have had
    held = Held(cache, table, heads)
    name = "f32" if kind is torch.float32 else "bf16"

    def rows(n):
        x = [torch.from_numpy((g.standard_normal((n, h, D))).astype(f32)).to(device()).to(kind) for h in (Hq, heads, heads)]
        return x, [t.double().cpu().numpy() for t in x]

    def step(new, trees, kept):
        T = sum(new)
        (q, k, v), (_, k64, v64) = rows(T)
        depth = [t.sum(1) - 1 for t in trees]
        places = np.concatenate([lens[b] + depth[b] for b in range(B)])
        for b in range(B):
            lens[b] += new[b]
        kv_len, cu = i32(lens), i32(starts(new))
        turned_q, out = torch.empty_like(q), torch.empty_like(q)
        q4.q4_kv_append(cache, turned_q, q, k, v, table, kv_len, cu, cos=cos, sin=sin, positions=i32(places))
        words = max(1, -(-max(new) // 32))
        lse = torch.empty(T, Hq, device=device())
        q4.q4_kv_attention(out, turned_q, cache, table, kv_len, cu, max(new), 192,
                           tree=dev(np.concatenate([words_of(t, words) for t in trees if len(t)])), lse=lse)
        sees = [visible(n, t, tree=trees[b]) for b, (n, t) in enumerate(zip(new, lens))]
        ref, ref_lse, mag, big = attend(held, turned_q.double().cpu().numpy(), new, lens, D ** -0.5, sees)
        assert np.all(np.abs(out.double().cpu().numpy() - ref) <= bound(ref, mag, big, D, max(lens), name))
        # scores of up to 100 in 64 bits against fp32 arithmetic: see the bounds of the sums' own tests
        assert np.all(np.abs(lse.double().cpu().numpy() - ref_lse) <= 2.0 ** -13)
        # the accepted paths: a list for all heads alike
        first = [t - n for n, t in zip(new, lens)]
        lists = np.zeros((B, 1, max(max(len(p) for p in kept), 1)), np.int32)
        for b in range(B):
            lists[b, 0, :len(kept[b])] = first[b] + np.asarray(kept[b], np.int64)
            lo = sum(new[:b])
            take = lo + np.asarray(kept[b], np.int64)
            both = turned(k64[lo:lo + new[b]], places[lo:lo + new[b]], D // 2), v64[lo:lo + new[b]]
            most[:] = [max(m, np.abs(x).max()) if new[b] else m for m, x in zip(most, both)]
            truth[b][0] = np.concatenate([truth[b][0], turned(k64[take], places[take], D // 2)])
            truth[b][1] = np.concatenate([truth[b][1], v64[take]])
        q4.q4_kv_compact(cache, table, kv_len, dev(lists), i32([len(p) for p in kept]), first=i32(first))
        for b in range(B):
            lens[b] = first[b] + len(kept[b])

    chain = lambda n: np.tril(np.ones((n, n), bool))
    step([20, 37, 5], [chain(20), chain(37), chain(5)], [range(20), range(37), range(5)])      # prompts: all is kept
    for seed in (1, 2):
        trees = [draft(n, seed + n) for n in (9, 17, 4)]
        paths = [np.flatnonzero(t[-1 - seed]) for t in trees]
        step([9, 17, 4], trees, paths)
    step([1, 0, 1], [chain(1), chain(0), chain(1)], [[0], [], [0]])
    assert q4.q4_get_device_status() == q4.Q4_OK
    for b in range(B):
        assert lens[b] == len(truth[b][0])
        k, v = held.values(b, lens[b])
        for got, want, top in ((k, truth[b][0], most[0]), (v, truth[b][1], most[1])):
            # a code is off by half a step when it is made, and by half of the new one whenever its block's scale grows:
            # by an append to its block, or by tokens that a compaction moves beside it.  A token here meets the append
            # that makes it, the compaction that moves it, and up to one of each of the next round in its block
            assert np.all(np.abs(got - want) <= 4 * 0.5 * top / 127 + 1e-5)


def test_a_cache_held_to_a_budget():
    """A prompt weighs itself and is cut to the budget; then each step appends a token at its own position, attends, adds
    its weights and leaves one token out: eagerly, and the same steps from one captured graph, bit for bit."""
    B, Hq, heads, D, page, budget, steps = 2, 4, 2, 64, 16, 40, 6
    g = rng(92, 1)
    lens = [90, 61]
    cos, sin = tables(400, D // 2)
    T = sum(lens)
    data = [(g.standard_normal((T + steps * B, h, D))).astype(f32) for h in (Hq, heads, heads)]
    runs = []
    for graphed in (False, True):
        cache = q4.KVCache.empty(B * 8, heads, D, page)
        for x in (cache.k, cache.v, cache.k_scale, cache.v_scale):
            x.zero_()
        table = i32(rng(92, 2).permutation(B * 8).reshape(B, 8))
        weight = torch.zeros(B * 8, heads, page, device=device())
        held = Held(cache, table, heads)
        q, k, v = (dev(x[:T]) for x in data)
        kv_len, cu = i32(lens), i32(starts(lens))
        turned_q, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(T, Hq, device=device())
        q4.q4_kv_append(cache, turned_q, q, k, v, table, kv_len, cu, cos=cos, sin=sin)
        q4.q4_kv_attention(out, turned_q, cache, table, kv_len, cu, max(lens), max(lens), lse=lse)
        q4.q4_kv_weigh(weight, turned_q, lse, cache, table, kv_len, cu, max(lens), max(lens))
        kept = torch.zeros(B, heads, budget, dtype=torch.int32, device=device())
        count, room = torch.empty(B, dtype=torch.int32, device=device()), i32([budget] * B)
        q4.q4_kv_select(kept, count, weight, cache, table, kv_len, room, max(lens), sinks=2, recent=8)
        w = weight.cpu().numpy()
        before = [held.values(b, lens[b]) for b in range(B)]
        q4.q4_kv_compact(cache, table, kv_len, kept, count, weight=weight)
        kv_len.copy_(count)
        torch.cuda.synchronize()
        for b in range(B):
            at, slot = table.cpu().numpy()[b, np.arange(lens[b]) // page], np.arange(lens[b]) % page
            after = held.values(b, budget)
            for h in range(heads):
                want = select(w[at, h, slot], budget, 2, 8)
                assert np.array_equal(kept[b, h].cpu().numpy(), want)
                for x in (0, 1):   # the moved tokens' codes are rounded once more, to a step that some block had
                    step = np.abs(before[b][x][:, h]).max() / 127
                    assert np.all(np.abs(after[x][:, h] - before[b][x][want, h]) <= 0.5 * step * 1.0001)
        # steps
        one = i32(range(B + 1))
        q1, k1, v1 = (torch.empty(B, h, D, device=device()) for h in (Hq, heads, heads))
        place = i32([n - 1 for n in lens])
        t1, o1, l1 = torch.empty_like(q1), torch.empty_like(q1), torch.empty(B, Hq, device=device())
        ws = torch.zeros(q4.q4_kv_attention_workspace_size(cache, Hq, B, B, 1, budget + 1), dtype=torch.uint8, device=device())

        def step():
            kv_len.add_(1)
            place.add_(1)
            q4.q4_kv_append(cache, t1, q1, k1, v1, table, kv_len, one, cos=cos, sin=sin, positions=place)
            q4.q4_kv_attention(o1, t1, cache, table, kv_len, one, 1, budget + 1, lse=l1, workspace=ws)
            q4.q4_kv_weigh(weight, t1, l1, cache, table, kv_len, one, 1, budget + 1)
            q4.q4_kv_select(kept, count, weight, cache, table, kv_len, room, budget + 1, sinks=2, recent=8)
            q4.q4_kv_compact(cache, table, kv_len, kept, count, weight=weight)
            kv_len.copy_(count)

        if graphed:
            stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                step()
        seen = []
        for i in range(steps):
            for x, to in zip(data, (q1, k1, v1)):
                to.copy_(dev(x[T + i * B:T + (i + 1) * B]))
            torch.cuda.synchronize()
            past = [held.values(b, budget) for b in range(B)]
            graph.replay() if graphed else step()
            torch.cuda.synchronize()
            seen.append([x.clone() for x in (o1, l1, kept, weight, cache.k, cache.v_scale)])
            if graphed:
                continue
            for b in range(B):    # attention over what was there and the new token, at its own position
                new_k = turned(data[1][T + i * B + b][None].astype(np.float64), np.array([lens[b] + i]), D // 2)
                kk = np.concatenate([past[b][0], new_k])
                vv = np.concatenate([past[b][1], data[2][T + i * B + b][None].astype(np.float64)])
                for h in range(Hq):
                    s = kk[:, h // 2] @ t1[b, h].double().cpu().numpy() * D ** -0.5
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    want = p @ vv[:, h // 2]
                    # half a step of 1/127 for the new token, as much for those whose block's scale it raised: of keys
                    # times |q|_1 in the score, of values in the sum
                    slack = np.abs(t1[b, h].double().cpu().numpy()).sum() * D ** -0.5 * np.abs(kk).max() / 127 * 0.5
                    far = 2 * np.expm1(slack) * (p @ np.abs(vv[:, h // 2])) + 0.5 * np.abs(vv).max() / 127 + 1e-5
                    assert np.all(np.abs(o1[b, h].double().cpu().numpy() - want) <= far)
        assert kv_len.tolist() == [budget] * B and place.tolist() == [n - 1 + steps for n in lens]
        assert q4.q4_get_device_status() == q4.Q4_OK
        runs.append(seen)
    for a, b in zip(*runs):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_graphs_share_one_workspace():
    """Captured apart, replayed one after another on one stream: drafts in one, single tokens in the other."""
    Hq, heads, D, page, n = 8, 1, 128, 64, 30
    g = rng(93, 1)
    cache = q4.KVCache(dev(g.integers(-127, 128, (20, heads, page, D)).astype(np.int8)),
                       dev(g.integers(-127, 128, (20, heads, page, D)).astype(np.int8)),
                       torch.full((20, heads, page // 16), 0.03, device=device()), torch.full((20, heads, page // 16), 0.03, device=device()))
    table = i32(g.permutation(20)[None])
    qs = [dev(g.standard_normal((m, Hq, D)).astype(f32)).to(torch.bfloat16) for m in (n, 1)]
    tree = dev(words_of(draft(n, 3), 1))
    kv_len = i32([1000])
    cus = [i32([0, n]), i32([0, 1])]
    ws = torch.zeros(q4.q4_kv_attention_workspace_size(cache, Hq, 1, n, n, 1280), dtype=torch.uint8, device=device())
    outs = [torch.empty_like(q) for q in qs]
    calls = [lambda: q4.q4_kv_attention(outs[0], qs[0], cache, table, kv_len, cus[0], n, 1280, tree=tree, workspace=ws),
             lambda: q4.q4_kv_attention(outs[1], qs[1], cache, table, kv_len, cus[1], 1, 1280, window=300, sinks=4, workspace=ws)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = []
    for call in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            call()
    for length in (1000, 40, 1279, 700):
        kv_len.fill_(length)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for i in (0, 1, 1, 0):
                graphs[i].replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for i, call in enumerate(calls):
            call()
            torch.cuda.synchronize()
            assert torch.equal(outs[i], got[i])
    assert q4.q4_get_device_status() == q4.Q4_OK


def test_logits_of_a_decode_loop():
    """Penalties over a history that grows on the device, in place, then sampling: captured, against plain steps."""
    T, V, most = 3, 1000, 64
    g = rng(94, 1)
    base = dev(g.standard_normal((T, V)).astype(f32) * 2)
    logits, tokens, u = torch.empty_like(base), torch.empty(T, dtype=torch.int32, device=device()), torch.full((T,), 0.4, device=device())
    history = torch.full((T, most), -1, dtype=torch.int32, device=device())
    length = torch.zeros(T, dtype=torch.int32, device=device())
    twice, once = torch.full((T,), 1.5, device=device()), torch.full((T,), 0.5, device=device())
    zero = torch.zeros(T, device=device())

    def step():
        logits.copy_(base)
        q4.q4_adjust_logits(logits, logits, history=history, history_len=length, repetition=twice, presence=once, frequency=once)
        q4.q4_sample(tokens, logits, u, temperature=zero)
        history.scatter_(1, length.long()[:, None], tokens[:, None])
        length.add_(1)

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step()
    said = [[] for _ in range(T)]
    host = base.cpu().numpy()
    for _ in range(20):
        graph.replay()
        torch.cuda.synchronize()
        for t in range(T):
            x = host[t].copy()
            for v in set(said[t]):
                y = x[v] / f32(1.5) if x[v] > 0 else x[v] * f32(1.5)
                x[v] = y - f32(0.5) * f32(said[t].count(v)) - f32(0.5)
            said[t].append(int(x.argmax()))
            assert int(tokens[t]) == said[t][-1]
    assert all(len(set(s)) > 3 for s in said)


def test_the_example_with_penalties(monkeypatch):
    """With an infinite penalty no later token of a greedy sequence is one that the sequence has."""
    monkeypatch.syspath_prepend(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decode
    gen = torch.Generator("cuda").manual_seed(3)
    m = decode.Decoder(layers=1, hidden=256, heads=2, kv_heads=1, dim=64, inner=512, vocab=512, seqs=2, max_tokens=128,
                       page_tokens=16, seed=4)
    prompts = [torch.randint(0, m.vocab, (n,), generator=gen, device=device(), dtype=torch.int32) for n in (5, 30)]
    settings = dict(temperature=torch.zeros(2, device=device()))
    u = torch.zeros(2, device=device())
    tokens, _ = m.prompts(prompts, u, settings)
    history = torch.full((2, 128), -1, dtype=torch.int32, device=device())
    for row, p in zip(history, prompts):
        row[:p.numel()] = p
    length = i32([5, 30])
    history.scatter_(1, length.long()[:, None], tokens[:, None])
    length += 1
    penalties = dict(history=history, history_len=length, presence=torch.full((2,), float("inf"), device=device()))
    graph, _ = m.capture_step(tokens, u, settings, penalties)
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert length.tolist() == [26, 51]
    for row, n in zip(history.tolist(), (5, 30)):
        assert len(set(row[n + 1:n + 21])) == 20 and not set(row[n + 1:n + 21]) & set(row[:n + 1])
    assert q4.q4_get_device_status() == q4.Q4_OK
