"""The paged 8-bit cache: appending (norm, rotation, quantisation) and reading
back, against a step-by-step fp32 host model of the definition (bit for bit)
and against 64-bit values."""

import numpy as np
import pytest

from gpu_util import device, torch
from serve_util import BLOCK, bf16, dev, f32, i32, rng, starts

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


def norm(x, w, eps):
    s = x * x
    while s.shape[-1] > 1:
        s = s[..., 0::2] + s[..., 1::2]
    r = f32(1) / np.sqrt(s / f32(x.shape[-1]) + f32(eps))
    return x * r * w


def rotate(x, c, s, pairs):
    n = 2 * c.shape[-1]
    y = x.copy()
    c, s = c[:, None, :], s[:, None, :]
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if pairs else (x[..., :n // 2], x[..., n // 2:n])
    ya, yb = a * c - b * s, b * c + a * s
    if pairs:
        y[..., 0:n:2], y[..., 1:n:2] = ya, yb
    else:
        y[..., :n // 2], y[..., n // 2:n] = ya, yb
    return y


class HostCache:
    """The definition, one block at a time, in fp32 numpy."""

    def __init__(self, pages, heads, dim, page, seed):
        g = rng(seed, 2)
        self.k = g.integers(-127, 128, (pages, heads, page, dim)).astype(np.int8)
        self.v = g.integers(-127, 128, (pages, heads, page, dim)).astype(np.int8)
        self.ks = (g.random((pages, heads, page // BLOCK)) * 0.02).astype(f32)
        self.vs = (g.random((pages, heads, page // BLOCK)) * 0.02).astype(f32)
        self.page = page

    def to_device(self):
        return q4.KVCache(dev(self.k), dev(self.v), dev(self.ks), dev(self.vs))

    def append(self, table, x, start, what):
        """x: [n, heads, dim] fp32, at positions start .. of the sequence with this table row."""
        codes, scales = (self.k, self.ks) if what == "k" else (self.v, self.vs)
        n = len(x)
        for blk in range(start // BLOCK, (start + n - 1) // BLOCK + 1):
            lo, hi = max(start, blk * BLOCK), min(start + n, (blk + 1) * BLOCK)
            pg, off = table[blk * BLOCK // self.page], blk * BLOCK % self.page
            for h in range(x.shape[1]):
                rows = x[lo - start:hi - start, h]
                m = np.abs(rows).max()
                s0 = scales[pg, h, off // BLOCK] if lo > blk * BLOCK else f32(0)
                s = max(s0, f32(m * (f32(1) / f32(127))))
                if s < f32(2.0 ** -110):
                    s = f32(0)
                ratio = f32(s0 / s) if s > 0 else f32(0)
                inv = f32(f32(1) / s) if s > 0 else f32(0)
                old = codes[pg, h, off:off + lo - blk * BLOCK].astype(f32)
                codes[pg, h, off:off + lo - blk * BLOCK] = np.rint(old * ratio).astype(np.int8)
                codes[pg, h, off + lo - blk * BLOCK:off + hi - blk * BLOCK] = np.clip(np.rint(rows * inv), -127, 127).astype(np.int8)
                scales[pg, h, off // BLOCK] = s


def tables(n, rows, seed=0):
    ang = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(n // 2) / (n // 2))
    return np.cos(ang).astype(f32), np.sin(ang).astype(f32)


CASES = [
    # new tokens, earlier tokens, Hq, heads, dim, page, rotated, pairs, norms, type
    ([1], [0], 1, 1, 64, 16, 64, False, False, "f32"),
    ([1], [15], 4, 2, 128, 16, 128, True, False, "f32"),
    ([1, 1, 1, 1], [16, 31, 0, 7], 8, 2, 128, 64, 128, False, True, "bf16"),
    ([17, 1, 33, 2], [5, 0, 31, 14], 6, 2, 64, 32, 32, True, True, "bf16"),
    ([0, 40, 0, 3], [9, 0, 0, 45], 3, 3, 128, 128, 64, False, True, "f32"),
    ([130], [3], 5, 1, 64, 256, 8, True, False, "f32"),
    ([16, 64, 15], [0, 16, 1], 32, 8, 128, 64, 128, False, True, "bf16"),
    ([2] * 70, list(range(70)), 2, 1, 64, 16, 0, False, False, "bf16"),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_append_and_gather_bit_exact(case):
    new, ctx, Hq, heads, D, page, R, pairs, norms, kind = CASES[case]
    g = rng(case, 3)
    lens = [a + b for a, b in zip(new, ctx)]
    used = [-(-n // page) for n in lens]
    host = HostCache(sum(used) + 2, heads, D, page, case)
    order = g.permutation(sum(used) + 2)
    table = np.zeros((len(new), max(used)), np.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    cache = host.to_device()
    T, cu = sum(new), starts(new)
    gap = 8
    wide = g.standard_normal((T, (Hq + 2 * heads) * D + gap)).astype(f32)
    wide[:, :: 7] *= 9
    td = torch.float32 if kind == "f32" else torch.bfloat16
    if kind == "bf16":
        wide = bf16(wide)
    rows = dev(wide, td)
    q = rows[:, :Hq * D].unflatten(1, (Hq, D))
    k = rows[:, Hq * D:(Hq + heads) * D].unflatten(1, (heads, D))
    v = rows[:, (Hq + heads) * D:(Hq + 2 * heads) * D].unflatten(1, (heads, D))
    qn = (1 + 0.2 * g.standard_normal(D)).astype(f32) if norms else None
    kn = (1 + 0.2 * g.standard_normal(D)).astype(f32) if norms else None
    cos, sin = tables(R, max(lens)) if R else (None, None)
    out = torch.full((T, Hq, D), float("nan"), dtype=td, device=device())
    q4.q4_kv_append(cache, out, q, k, v, dev(table), i32(lens), i32(cu),
                    cos=None if cos is None else dev(cos), sin=None if sin is None else dev(sin),
                    rope_style=q4.Q4_ROPE_PAIRS if pairs else q4.Q4_ROPE_HALVES,
                    q_norm=None if qn is None else dev(qn), k_norm=None if kn is None else dev(kn), eps=1e-5)
    torch.cuda.synchronize()
    assert q4.q4_get_device_status() == q4.Q4_OK

    hq = wide[:, :Hq * D].reshape(T, Hq, D)
    hk = wide[:, Hq * D:(Hq + heads) * D].reshape(T, heads, D)
    hv = wide[:, (Hq + heads) * D:(Hq + 2 * heads) * D].reshape(T, heads, D)
    pos = np.concatenate([np.arange(c, c + n) for n, c in zip(new, ctx)]).astype(int)
    if norms:
        hq, hk = norm(hq, qn, 1e-5), norm(hk, kn, 1e-5)
    if R:
        hq, hk = rotate(hq, cos[pos], sin[pos], pairs), rotate(hk, cos[pos], sin[pos], pairs)
    for b, (n, c) in enumerate(zip(new, ctx)):
        if n:
            host.append(table[b], hk[cu[b]:cu[b + 1]], c, "k")
            host.append(table[b], hv[cu[b]:cu[b + 1]], c, "v")
    want = hq if kind == "f32" else bf16(hq)
    assert np.array_equal(out.float().cpu().numpy(), want)
    # the whole cache, untouched blocks too
    for got, ref in ((cache.k, host.k), (cache.v, host.v), (cache.k_scale, host.ks), (cache.v_scale, host.vs)):
        assert np.array_equal(got.cpu().numpy(), ref)

    # reading back, from an odd token on, into rows that no sequence owns as well
    first = [min(3, n) for n in lens]
    count = [n - f for n, f in zip(lens, first)]
    cu2 = starts(count)
    for td2 in (torch.float32, torch.bfloat16):
        ko, vo = (torch.full((int(cu2[-1]) + 2, heads, D), float("nan"), dtype=td2, device=device()) for _ in range(2))
        q4.q4_kv_gather(ko, vo, cache, dev(table), i32(first), i32(cu2))
        for got, codes, scales in ((ko, host.k, host.ks), (vo, host.v, host.vs)):
            ref = np.zeros((int(cu2[-1]) + 2, heads, D), f32)
            for b in range(len(new)):
                for i in range(count[b]):
                    t = first[b] + i
                    p = table[b, t // page]
                    ref[cu2[b] + i] = codes[p, :, t % page].astype(f32) * scales[p, :, t % page // BLOCK, None]
            assert np.array_equal(got.float().cpu().numpy(), ref if td2 == torch.float32 else bf16(ref))
    assert q4.q4_get_device_status() == q4.Q4_OK


def test_token_by_token_stays_within_the_steps():
    """Tokens appended one call at a time: a value is at most half a step off when it is stored and
    half a step more each time its block's scale grows (at most 15 times)."""
    g = rng(77)
    D, n = 64, 40
    cache = q4.KVCache.empty(3, 1, D, 16, device=device())
    table = i32([[2, 0, 1]])
    x = (g.standard_normal((n, 1, D)) * np.exp(g.standard_normal((n, 1, 1)))).astype(f32)
    for t in range(n):
        row = dev(x[t:t + 1])
        q4.q4_kv_append(cache, None, None, row, row, table, i32([t + 1]), i32([0, 1]))
    ko, vo = (torch.empty((n, 1, D), device=device()) for _ in range(2))
    q4.q4_kv_gather(ko, vo, cache, table, i32([0]), i32([0, n]))
    ko, vo = ko.cpu().numpy(), vo.cpu().numpy()
    assert np.array_equal(ko, vo)
    for blk in range(0, n, BLOCK):
        rows = x[blk:blk + BLOCK, 0]
        peak = np.maximum.accumulate(np.abs(rows).max(1))
        grew = np.array([(np.diff(peak[t:]) > 0).sum() for t in range(len(rows))])
        step = peak[-1] / 127
        err = np.abs(ko[blk:blk + BLOCK, 0] - rows).max(1)
        assert np.all(err <= step * 0.5001 * (1 + grew)), (blk, err / step, grew)
        assert np.all(np.abs(ko[blk:blk + BLOCK]).max() <= peak[-1] * (1 + 1e-6))


def test_zero_tiny_and_odd_values():
    D = 64
    cache = q4.KVCache.empty(1, 2, D, 16, device=device())
    x = np.zeros((3, 2, D), f32)
    x[1, 1] = 1e-36                       # below 127 * 2^-110
    one = dev(x)
    q4.q4_kv_append(cache, None, None, one, one, i32([[0]]), i32([3]), i32([0, 3]))
    assert q4.q4_get_device_status() == q4.Q4_OK
    assert np.all(cache.k_scale.cpu().numpy() == 0) and np.all(cache.k.cpu().numpy()[:, :, :3] == 0)
    x[:] = rng(5).standard_normal(x.shape)
    x[0, 0, 3], x[2, 0, 9], x[1, 1, 0] = np.nan, np.inf, -np.inf
    bad, good = dev(x), dev(np.ones_like(x))
    q4.q4_kv_append(cache, None, None, bad, good, i32([[0]]), i32([3]), i32([0, 3]))
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE
    assert q4.q4_last_device_flags() == q4.Q4_DEVERR_VALUE
    k = cache.k.cpu().numpy()[0, :, :3]
    assert k[0, 0, 3] == 0 and k[0, 2, 9] == 127 and k[1, 1, 0] == -127
    assert np.all(np.isfinite(cache.k_scale.cpu().numpy()))
    assert np.all(cache.v.cpu().numpy()[0, :, :3] == 127)
    assert q4.q4_get_device_status() == q4.Q4_OK


def test_bad_pages_and_positions_are_skipped():
    D = 64
    cache = q4.KVCache.empty(2, 1, D, 16, device=device())
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t.zero_()
    x = dev(np.ones((6, 1, D), f32))
    out = torch.full((6, 1, D), float("nan"), device=device())
    cos, sin = tables(D, 20)
    # sequence 0: page out of range; 1: fine; 2: one token beyond the rotation table; 3: table too short
    q4.q4_kv_append(cache, out, x, x, x, i32([[2], [1], [0], [0]]), i32([1, 3, 21, 17]), i32([0, 1, 4, 5, 6]),
                    cos=dev(cos), sin=dev(sin))
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
    codes = cache.v.cpu().numpy()
    assert np.all(codes[0] == 0) and np.all(codes[1, 0, :3] == 127) and np.all(codes[1, 0, 3:] == 0)
    o = out.cpu().numpy()
    assert np.all(o[4] == 0) and np.all(o[1] == 1) and np.isfinite(o).all()
    # more new tokens than the sequence holds: those before position 0 have no place
    q4.q4_kv_append(cache, out, x, x, x, i32([[0]]), i32([2]), i32([0, 6]))
    assert q4.q4_get_device_status() == q4.Q4_OK
    assert np.all(cache.v.cpu().numpy()[0, 0, :2] == 127) and np.all(cache.v.cpu().numpy()[0, 0, 2:] == 0)
    assert np.all(out.cpu().numpy()[:4] == 0) and np.all(out.cpu().numpy()[4:] == 1)


def test_cache_beyond_32_bit_offsets():
    """Pages whose codes lie past 2^32 bytes."""
    D, heads, page = 128, 8, 256
    pages = (1 << 32) // (heads * page * D) + 3
    cache = q4.KVCache.empty(pages, heads, D, page, device=device())
    x = rng(9).standard_normal((20, heads, D)).astype(f32)
    k = dev(x)
    table = i32([[pages - 1]])
    q4.q4_kv_append(cache, None, None, k, k, table, i32([20]), i32([0, 20]))
    ko, vo = (torch.empty((20, heads, D), device=device()) for _ in range(2))
    q4.q4_kv_gather(ko, vo, cache, table, i32([0]), i32([0, 20]))
    step = np.concatenate([np.abs(x[:16]).max((0, 2), keepdims=True).repeat(16, 0),
                           np.abs(x[16:]).max((0, 2), keepdims=True).repeat(4, 0)]) / 127
    assert np.all(np.abs(ko.cpu().numpy() - x) <= 0.5001 * step)
    assert torch.equal(ko, vo)
    q = torch.zeros((1, heads, D), device=device())
    out = torch.empty_like(q)
    q4.q4_kv_attention(out, q, cache, table, i32([20]), i32([0, 1]), 1, 20)
    assert np.allclose(out.cpu().numpy()[0], vo.cpu().numpy().mean(0), atol=1e-5)
    assert q4.q4_get_device_status() == q4.Q4_OK


def test_runs_in_a_graph_and_on_another_stream():
    D = 64
    cache = q4.KVCache.empty(2, 2, D, 16, device=device())
    x = dev(rng(3).standard_normal((2, 2, D)).astype(f32))
    table, lens, cu = i32([[0], [1]]), i32([1, 1]), i32([0, 1, 2])
    ko, vo = (torch.empty((4, 2, D), device=device()) for _ in range(2))
    first, cu2 = i32([0, 0]), i32([0, 2, 4])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        q4.q4_kv_append(cache, None, None, x, x, table, lens, cu)
        q4.q4_kv_gather(ko, vo, cache, table, first, cu2)
    for step in (1, 2):
        lens.fill_(step)
        g.replay()
    torch.cuda.synchronize()
    a = ko.cpu().numpy().reshape(2, 2, 2, D)
    assert np.array_equal(a[:, 0], a[:, 1]) and np.isfinite(a).all() and np.abs(a).max() > 0.5
    assert q4.q4_get_device_status() == q4.Q4_OK


@pytest.mark.parametrize("D", [64, 128])
def test_norm_weights_off_16_bytes_give_the_same(D):
    """Norm weights are aligned to a float: the same bits wherever they start."""
    g = rng(D, 8)
    T, Hq, heads = 37, 5, 2
    host = HostCache(2, heads, D, 64, 8)
    x = dev(g.standard_normal((T, Hq + 2 * heads, D)).astype(f32), torch.float32)
    w = dev((1 + g.standard_normal(2 * D + 3)).astype(f32), torch.float32)
    table, n, cu = i32([[1]]), i32([T]), i32([0, T])
    got = []
    for off in (0, 1, 2, 3):
        w_here = torch.empty(2 * D + off, dtype=torch.float32, device=device())[off:]
        w_here.copy_(w[:2 * D])
        cache = host.to_device()
        out = torch.empty((T, Hq, D), dtype=torch.float32, device=device())
        q4.q4_kv_append(cache, out, x[:, :Hq], x[:, Hq:Hq + heads], x[:, Hq + heads:], table, n, cu,
                        q_norm=w_here[:D], k_norm=w_here[D:])
        torch.cuda.synchronize()
        got.append((out, cache.k[1], cache.k_scale[1], cache.v[1]))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
    assert q4.q4_get_device_status() == q4.Q4_OK
