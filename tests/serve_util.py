"""Inputs and 64-bit references of the serving operators' tests (numpy)."""

import numpy as np

from gpu_util import device, torch

import quantized_weight_q4_gb300 as q4

BLOCK = 16
f32 = np.float32


def rng(*seed):
    return np.random.Generator(np.random.PCG64(list(seed)))


def bf16(x):
    """fp32 values rounded to bf16 (as fp32)."""
    return torch.from_numpy(np.ascontiguousarray(x, f32)).to(torch.bfloat16).float().numpy()


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).to(device())
    return t if dtype is None else t.to(dtype)


def i32(x):
    return dev(np.asarray(x, np.int32))


class Cache:
    """A cache of random codes for sequences of the given lengths, on the host and the device.
    extra: pages that no sequence uses.  NaN scales mark blocks that hold no token."""

    def __init__(self, lens, heads, dim, page, seed, extra=3, spread=1.0):
        g = rng(seed, 1)
        used = [-(-max(n, 0) // page) for n in lens]
        self.pages = sum(used) + extra
        order = g.permutation(self.pages)
        self.table = np.full((len(lens), max(max(used), 1) + 1), -7, np.int32)
        at = 0
        self.k = np.clip(np.rint(g.standard_normal((self.pages, heads, page, dim)) * 30), -127, 127).astype(np.int8)
        self.v = np.clip(np.rint(g.standard_normal((self.pages, heads, page, dim)) * 30), -127, 127).astype(np.int8)
        shape = (self.pages, heads, page // BLOCK)
        self.ks = np.full(shape, np.nan, f32)
        self.vs = np.full(shape, np.nan, f32)
        for b, n in enumerate(lens):
            for i in range(used[b]):
                p = order[at]
                at += 1
                self.table[b, i] = p
                blocks = min(page // BLOCK, -(-(n - i * page) // BLOCK))
                for s in (self.ks, self.vs):
                    s[p, :, :blocks] = (0.02 + 0.03 * g.random((heads, blocks))) * spread ** g.uniform(-1, 1, (heads, blocks))
        self.lens, self.heads, self.dim, self.page = list(lens), heads, dim, page

    def to_device(self):
        c = q4.KVCache(dev(self.k), dev(self.v), dev(self.ks), dev(self.vs))
        return c, dev(self.table)

    def values(self, b, n):
        """Keys and values of the first n tokens of sequence b, [n, heads, dim] in 64 bits."""
        out = []
        for codes, scale in ((self.k, self.ks), (self.v, self.vs)):
            x = np.zeros((n, self.heads, self.dim))
            for t in range(n):
                p, s = self.table[b, t // self.page], t % self.page
                x[t] = codes[p, :, s].astype(np.float64) * scale[p, :, s // BLOCK].astype(np.float64)[:, None]
            out.append(x)
        return out


def starts(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def attention(cache, q, new, lens, scale, causal=True, window=0):
    """64-bit attention, with what its error bound needs: (out, sum p|v|, largest |scale| * sum|q k|),
    each [T, Hq, dim] or [T, Hq, 1]."""
    T, Hq, D = q.shape
    group = Hq // cache.heads
    out, mag, big = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq, 1))
    t = 0
    for b, (n, length) in enumerate(zip(new, lens)):
        k, v = cache.values(b, max(length, 0))
        for j in range(n):
            pos = length - n + j
            see = np.arange(max(length, 0))
            if causal:
                see = see[see <= pos]
                if window:
                    see = see[see > pos - window]
            if len(see):
                kk, vv = k[see], v[see]
                for h in range(Hq):
                    x = q[t, h].astype(np.float64)
                    s = kk[:, h // group] @ x * scale
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    out[t, h] = p @ vv[:, h // group]
                    mag[t, h] = p @ np.abs(vv[:, h // group])
                    big[t, h] = abs(scale) * (np.abs(kk[:, h // group]) @ np.abs(x)).max()
            t += 1
    return out, mag, big
