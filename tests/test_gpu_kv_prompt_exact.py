"""Prompt attention over the paged 8-bit cache: the products of the codes are
exact, and blocks that a query does not see take no part in its accuracy.

Bound on the relative error (norms over all outputs; a single row gets four times as much): the
weights are fp16 (2^-11 each), the result is bf16 (2^-8 at most for an element,
evenly spread: 2^-8 / sqrt(3)), scores and sums are fp32 (below 2^-12 here:
scores of up to 100 with 2^-22 each step of 16 elements)."""

import numpy as np
import pytest

from gpu_util import device, torch
from serve_util import Cache, bf16, dev, f32, i32, rng, starts

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu

REL = 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -11 + 2.0 ** -12


def run(c, q, new, lens, window=0, causal=True):
    cache, table = c.to_device()
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=device())
    q4.q4_kv_attention(out, dev(q, torch.bfloat16), cache, table, i32(lens), i32(starts(new)), max(new), max(lens),
                       window=window, causal=causal)
    assert q4.q4_get_device_status() == q4.Q4_OK
    return out.float().cpu().numpy().astype(np.float64)


def reference(c, q, new, lens, window=0, causal=True):
    T, Hq, D = q.shape
    out, at = np.zeros((T, Hq, D)), 0
    for b, (n, t) in enumerate(zip(new, lens)):
        k, v = c.values(b, t)
        pos, see = np.arange(t - n, t)[:, None], np.arange(t)[None, :]
        ok = see <= pos if causal else np.ones((n, t), bool)
        if window:
            ok = ok & (see > pos - window)
        for h in range(Hq):
            g = h // (Hq // c.heads)
            s = np.where(ok, q[at:at + n, h].astype(np.float64) @ k[:, g].T * D ** -0.5, -np.inf)
            p = np.exp(s - np.maximum(s.max(1, keepdims=True), -1e300))
            out[at:at + n, h] = p @ v[:, g] / np.maximum(p.sum(1, keepdims=True), 1e-300)
        at += n
    return out


def rows_off(got, want):
    """Relative error of each row [token, head]."""
    return np.linalg.norm(got - want, axis=-1) / np.maximum(np.linalg.norm(want, axis=-1), 1e-300)


@pytest.mark.parametrize("D", [64, 128])
def test_a_channel_that_stands_out(D):
    """Keys with one channel near 100 (as a bias leaves them) and a query element of 8 on it: a key's rounding to
    11 bits would move scores by up to 0.02 and the outputs by about a percent."""
    g = rng(D, 71)
    n, t = 300, 900
    c = Cache([t], 4, D, 64, 72)
    keys = g.standard_normal((t, 4, D))
    keys[..., 7] = 100 + g.standard_normal((t, 4))
    for i in range(0, t, 16):
        p, s = c.table[0, i // 64], i % 64
        blk = keys[i:i + 16]
        step = np.abs(blk).max((0, 2)) / 127
        c.ks[p, :, s // 16] = step
        codes = np.rint(blk / step[None, :, None]).astype(np.int8)
        c.k[p, :, s:s + len(blk)] = codes.transpose(1, 0, 2)
    q = g.standard_normal((n, 16, D)).astype(f32)
    q[..., 7] = 8
    q = bf16(q)
    got, want = run(c, q, [n], [t]), reference(c, q, [n], [t])
    assert np.linalg.norm(got - want) <= REL * np.linalg.norm(want), np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("big", [2.0 ** 12, 2.0 ** 40])
@pytest.mark.parametrize("at", [0, 260, 280])
def test_large_scales_that_no_query_sees(at, big):
    """A block whose scales are far above the others', before every query's window: it costs no accuracy."""
    n, t, window, D = 300, 700, 100, 64     # the first query, at 400, sees 301 ..
    c = Cache([t], 1, D, 16, 73)
    q = bf16((1.5 * rng(74).standard_normal((n, 16, D))).astype(f32))
    p, s = c.table[0, at // 16], at % 16 // 16
    c.ks[p, :, s] *= big
    c.vs[p, :, s] *= big
    got, want = run(c, q, [n], [t], window), reference(c, q, [n], [t], window)
    assert np.all(rows_off(got, want) <= 4 * REL)
    assert np.linalg.norm(got - want) <= REL * np.linalg.norm(want)


def test_large_scales_that_some_queries_see():
    """Causal: queries before a block of large values keep their accuracy, those after it see it."""
    n = t = 400
    D = 128
    c = Cache([t], 1, D, 64, 75)
    for p, s in ((c.table[0, 3], 1),):       # tokens 208 .. 223
        c.vs[p, :, s] *= 2.0 ** 30
    q = bf16((1.5 * rng(76).standard_normal((n, 8, D))).astype(f32))
    got, want = run(c, q, [n], [t]), reference(c, q, [n], [t])
    assert np.all(rows_off(got, want) <= 4 * REL)
    for lo, hi in ((0, 208), (208, 400)):
        assert np.linalg.norm((got - want)[lo:hi]) <= REL * np.linalg.norm(want[lo:hi])


def test_blocks_of_zeros():
    """Scales of 0 (all values of a block are zero, and in one case all keys): their weights count."""
    n, t, D = 280, 530, 64
    c = Cache([t], 2, D, 64, 77)
    for i in (0, 5, 11, 12, 13, 14, 15, 16, 17, 18, 19, 30):      # 12 .. 19 with 11: whole tiles of 128 tokens
        p, s = c.table[0, i * 16 // 64], i * 16 % 64 // 16
        c.vs[p, :, s] = 0
        if i == 5:
            c.ks[p, :, s] = 0
    q = bf16((1.5 * rng(78).standard_normal((n, 16, D))).astype(f32))
    got, want = run(c, q, [n], [t]), reference(c, q, [n], [t])
    assert np.all(rows_off(got, want) <= 4 * REL)
    c.vs[...] = np.where(np.isnan(c.vs), c.vs, 0)
    assert np.all(run(c, q, [n], [t]) == 0)


def test_four_query_heads_a_kv_head():
    """Pieces of a few hundred tokens on a context, four query heads a kv head, in one batch with a single token."""
    new, ctx = [420, 1, 300], [1500, 900, 37]
    lens = [a + b for a, b in zip(new, ctx)]
    c = Cache(lens, 2, 128, 64, 79, spread=3.0)
    q = bf16((1.5 * rng(80).standard_normal((sum(new), 8, 128))).astype(f32))
    got, want = run(c, q, new, lens), reference(c, q, new, lens)
    assert np.all(rows_off(got, want) <= 4 * REL)
    assert np.linalg.norm(got - want) <= REL * np.linalg.norm(want)
