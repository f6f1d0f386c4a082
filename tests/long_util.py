"""64-bit references of the operators for long and drafted decoding (numpy)."""

import numpy as np

from serve_util import BLOCK, f32, rng


def draft(n, seed):
    """A random tree of n drafted tokens, parents first: bool [n, n], whom each one sees (its path, itself included)."""
    g = rng(seed, 77)
    see = np.zeros((n, n), bool)
    for i in range(n):
        parent = int(g.integers(-1, i)) if i else -1
        if parent >= 0:
            see[i] = see[parent]
        see[i, i] = True
    return see


def words_of(see, words):
    """int32 words of bool rows; columns past the words are lost."""
    n, m = see.shape
    bits = np.zeros((n, words * 32), bool)
    bits[:, :min(m, words * 32)] = see[:, :words * 32]
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32).reshape(n, words)


def visible(n, length, causal=True, window=0, sinks=0, tree=None):
    """bool [n, length]: what each of the n new tokens of a sequence of `length` sees."""
    length = max(length, 0)
    base = length - n
    j = np.arange(length)
    see = np.zeros((n, length), bool)
    for i in range(n):
        place = base + i if tree is None else base - 1 + int(tree[i].sum())
        if not causal:
            see[i] = True
            continue
        row = j <= place
        if window:
            row &= (j > place - window) | (j < sinks)
        if tree is not None:
            for k in range(max(base, 0), length):
                row[k] = tree[i, k - base]
        see[i] = row
    return see


def attend(cache, q, new, lens, scale, sees):
    """64-bit attention under given visibility: out, lse, and what the bounds need: sum p|v|, largest |scale| sum|q k|."""
    T, Hq, D = q.shape
    group = Hq // cache.heads
    out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    big, lse = np.zeros((T, Hq, 1)), np.full((T, Hq), -np.inf)
    t = 0
    for b, (n, length) in enumerate(zip(new, lens)):
        k, v = cache.values(b, max(length, 0))
        for h in range(Hq):
            x = q[t:t + n, h].astype(np.float64)
            s = x @ k[:, h // group].T * scale
            a = np.abs(x) @ np.abs(k[:, h // group]).T * abs(scale)
            for i in range(n):
                see = np.flatnonzero(sees[b][i])
                if len(see):
                    top = s[i, see].max()
                    e = np.exp(s[i, see] - top)
                    lse[t + i, h] = top + np.log(e.sum())
                    p = e / e.sum()
                    out[t + i, h] = p @ v[see, h // group]
                    mag[t + i, h] = p @ np.abs(v[see, h // group])
                    big[t + i, h] = a[i, see].max()
        t += n
    return out, lse, mag, big


def weigh(cache, q, lse, new, lens, scale, sees):
    """Weights that tokens get, [heads, length] for each sequence, and the bound of their error.  A score is off by
    at most (D + 8) 2^-23 big, the exponent's multiplication and addition by 2^-23 of score and lse each, the
    exponential by 2^-22; m terms are added in fp32."""
    T, Hq, D = q.shape
    group = Hq // cache.heads
    sums, bounds = [], []
    t = 0
    for b, (n, length) in enumerate(zip(new, lens)):
        k, _ = cache.values(b, max(length, 0))
        w, e = np.zeros((cache.heads, max(length, 0))), np.zeros((cache.heads, max(length, 0)))
        for i in range(n):
            for h in range(Hq):
                if not np.isfinite(lse[t + i, h]):
                    continue
                x = q[t + i, h].astype(np.float64)
                s, a = k[:, h // group] @ x * scale, np.abs(k[:, h // group]) @ np.abs(x) * abs(scale)
                p = np.where(sees[b][i], np.exp(np.where(sees[b][i], s - lse[t + i, h], -np.inf)), 0.0)
                w[h // group] += p
                e[h // group] += p * ((D + 8) * 2.0 ** -23 * a + 2.0 ** -22 * (a + abs(lse[t + i, h]) + 2))
        t += n
        sums.append(w)
        bounds.append(e + (n * group + 8) * 2.0 ** -23 * w + 1e-30)
    return sums, bounds


def slots(cache, b, n):
    """Pages and slots of the first n tokens of sequence b."""
    i = np.arange(n)
    return cache.table[b, i // cache.page], i % cache.page


def select(weights, budget, sinks, recent):
    """Positions kept of one head, ascending."""
    n = len(weights)
    count = max(0, min(n, budget))
    head = min(count, sinks)
    tail = min(count - head, recent)
    w = np.where(np.isnan(weights), -np.inf, weights.astype(np.float64)) + 0.0
    low = np.isnan(weights)                       # below -inf
    rest = sorted(range(head, n - tail), key=lambda i: (low[i], -w[i], i))[:count - head - tail]
    return np.array(sorted([*range(head), *rest, *range(n - tail, n)]), np.int64)


def move(codes, scales, table, to_table, page, first, kept, heads):
    """Codes and scales (copies) of one sequence after a compaction: kept [heads][count] positions."""
    codes, scales = codes.copy(), scales.copy()
    old, olds = codes.copy(), scales.copy()
    count = len(kept[0])
    for h in range(heads):
        at = first // BLOCK * BLOCK
        while at < first + count:
            places = range(at, min(at + BLOCK, first + count))
            p = to_table[at // page]
            was = []
            for x in places:
                if x < first:
                    was.append((old[p, h, x % page], olds[p, h, (x % page) // BLOCK]))
                else:
                    y = kept[h][x - first]
                    s = table[y // page]
                    was.append((old[s, h, y % page], olds[s, h, (y % page) // BLOCK]))
            now = max(f32(s) for _, s in was)
            for x, (c, s) in zip(places, was):
                ratio = f32(s) / f32(now) if now > 0 else f32(0)
                codes[p, h, x % page] = np.rint(c.astype(f32) * ratio).astype(np.int8)
            scales[p, h, (at % page) // BLOCK] = now
            at += BLOCK
    return codes, scales


def adjust(logits, history=None, n=None, prompt=0, r=1.0, f=0.0, p=0.0, bias=(), mask=None):
    """One row in fp32, one operation a step.  bias: (token, value) pairs; mask: bool [V] or None."""
    x = logits.astype(f32).copy()
    V = len(x)
    if history is not None:
        known = history[:n]
        inside = (known >= 0) & (known < V)
        seen = np.zeros(V, bool)
        seen[known[inside]] = True
        said = np.bincount(known[prompt:][inside[prompt:]], minlength=V).astype(f32)
        with np.errstate(all="ignore"):
            y = np.where(x > 0, x / f32(r), x * f32(r))
            x = np.where(seen, y, x)
            x = np.where(said > 0, x - f32(f) * said - f32(p), x)
    last = {}
    for t, v in bias:
        if 0 <= t < V:
            last[t] = f32(v)
    for t, v in last.items():
        x[t] = x[t] + v
    if mask is not None:
        x = np.where(mask, x, f32(-np.inf))
    return x.astype(f32)
