"""Choosing and moving cached tokens, bit for bit against plain numpy."""

import numpy as np
import pytest

from gpu_util import device, torch
from long_util import move, select, slots
from serve_util import BLOCK, Cache, dev, f32, i32, rng

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


def weights(c, seed, ties=False):
    g = rng(seed, 9)
    w = np.exp(2 * g.standard_normal((c.pages, c.heads, c.page))).astype(f32)
    return np.round(w * 2) if ties else w


def run_select(c, w, budget, sinks, recent, width=None, max_kv=None, table=None, lens=None):
    cache, tab = c.to_device()
    lens = c.lens if lens is None else lens
    B = len(lens)
    width = width or max(max(budget), max(lens), 1)
    kept = torch.full((B, c.heads, width), -9, dtype=torch.int32, device=device())
    count = torch.full((B,), -9, dtype=torch.int32, device=device())
    q4.q4_kv_select(kept, count, dev(w.astype(f32)), cache, tab if table is None else dev(table), i32(lens), i32(budget),
                    max_kv or max(max(lens), 1), sinks=sinks, recent=recent)
    torch.cuda.synchronize()
    return kept.cpu().numpy(), count.cpu().numpy()


def check_select(c, w, budget, sinks, recent, width=None, max_kv=None):
    kept, count = run_select(c, w, budget, sinks, recent, width, max_kv)
    assert q4.q4_get_device_status() == q4.Q4_OK
    for b, n in enumerate(c.lens):
        p, s = slots(c, b, max(n, 0))
        for h in range(c.heads):
            want = select(w[p, h, s], min(budget[b], width or budget[b]), sinks, recent)
            assert count[b] == len(want)
            assert np.array_equal(kept[b, h, :len(want)], want), (b, h)
            assert np.all(kept[b, h, len(want):] == -9)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 511, 512, 513, 1025, 3001, 9000])
def test_select_lengths(n):
    c = Cache([n], 2, 64, 64, n)
    w = weights(c, n)
    for budget in {1, n // 2, n - 1, n, n + 5}:
        check_select(c, w, [budget], 0, 0)
        check_select(c, w, [budget], 3, 10)


@pytest.mark.parametrize("page", [16, 128, 256])
@pytest.mark.parametrize("heads", [1, 3, 8])
def test_select_batches(heads, page):
    c = Cache([700, 0, 5, 1300, 64, 2000], heads, 64, page, heads)
    check_select(c, weights(c, heads), [100, 7, 5, 1299, 0, 600], 4, 50)
    check_select(c, weights(c, heads, ties=True), [300, 0, 2, 1000, 63, 600], 2, 8)


@pytest.mark.parametrize("seqs,heads,n", [(1, 1, 9003), (2, 2, 2049), (3, 8, 5001), (10, 8, 2500), (5, 32, 8190), (1, 2, 16385)])
def test_select_launch_shapes(seqs, heads, n):
    """One CTA a (sequence, head), clusters with an SM for each CTA, and clusters that share SMs."""
    c = Cache([n - 37 * b for b in range(seqs)], heads, 64, 64, seqs + heads)
    check_select(c, weights(c, seqs), [n // 3 + b for b in range(seqs)], 5, 17)
    check_select(c, weights(c, n, ties=True), [n // 7] * seqs, 1, 130)


@pytest.mark.parametrize("many", [1.0, 0.5])
def test_select_mostly_equal_weights(many):
    """Many tokens at the cut, in every CTA of a cluster: the first of them stay."""
    c = Cache([7003, 6000], 4, 64, 64, 5)
    w = np.where(rng(17, 4).random((c.pages, c.heads, c.page)) < many, f32(0.25), weights(c, 3))
    check_select(c, w, [3001, 4500], 3, 9)


@pytest.mark.parametrize("sinks,recent", [(0, 0), (10, 0), (0, 10), (10, 20), (30, 30), (100, 5), (5, 100), (1000, 1000)])
def test_select_first_and_last(sinks, recent):
    """Also where the budget is less than both together."""
    c = Cache([90, 40], 2, 64, 16, sinks)
    check_select(c, weights(c, recent), [25, 25], sinks, recent)


@pytest.mark.parametrize("n", [100, 3000, 20000])
def test_select_equal_weights(n):
    """All equal; two values; zeros of both signs."""
    c = Cache([n], 1, 64, 64, n)
    for w in (np.zeros((c.pages, 1, 64)), np.full((c.pages, 1, 64), 0.1), rng(n, 3).integers(0, 2, (c.pages, 1, 64)),
              np.where(rng(n, 4).random((c.pages, 1, 64)) < 0.5, 0.0, -0.0)):
        check_select(c, w.astype(f32), [n // 3], 1, 7)


def test_select_any_number():
    """Negative, infinite, tiny and missing numbers, in the order of numbers; neighbours in the last bit."""
    c = Cache([800], 2, 64, 32, 5)
    g = rng(5, 5)
    w = g.standard_normal((c.pages, 2, 32)).astype(f32)
    w.flat[g.integers(0, w.size, 300)] = g.choice(np.array([np.inf, -np.inf, np.nan, 1e-45, -1e-45, 3e38], f32), 300)
    for budget in (1, 30, 400, 700, 790):
        check_select(c, w, [budget], 0, 0)
    w = (np.full(w.shape, 0x3f800000, np.int32) + g.integers(0, 7, w.shape).astype(np.int32)).view(f32)
    check_select(c, w, [350], 0, 3)


def test_select_narrow_lists_and_wrong_bounds():
    """A list narrower than the budget; a bound on the lengths far too large, and one too small."""
    c = Cache([900, 300], 2, 64, 64, 6)
    w = weights(c, 6)
    check_select(c, w, [500, 500], 4, 9, width=77)
    check_select(c, w, [500, 100], 4, 9, max_kv=1 << 20)
    check_select(c, w, [500, 100], 4, 9, max_kv=10)


def test_select_a_long_sequence():
    """More tokens than the shared memory of a cluster, in one sequence."""
    n = 400_000
    c = Cache.__new__(Cache)
    c.lens, c.heads, c.dim, c.page, c.pages = [n], 1, 64, 256, -(-n // 256)
    c.table = rng(1, 1).permutation(c.pages).astype(np.int32)[None]
    c.k = c.v = np.zeros((c.pages, 1, 256, 64), np.int8)
    c.ks = c.vs = np.zeros((c.pages, 1, 16), f32)
    check_select(c, weights(c, 8, ties=True), [150_001], 4, 1000)


def test_select_pages_outside_the_cache():
    c = Cache([200], 2, 64, 16, 7)
    w = weights(c, 7)
    table = c.table.copy()
    table[0, 4] = -1
    kept, count = run_select(c, w, [60], 2, 3, table=table)
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
    p, s = slots(c, 0, 200)
    for h in range(2):
        v = w[p, h, s].copy()
        v[64:80] = np.nan
        assert np.array_equal(kept[0, h, :60], select(v, 60, 2, 3))


def test_lengths_past_the_table():
    """Work goes by what the table has, whatever the lengths say."""
    c = Cache([64], 2, 64, 16, 15)
    w = weights(c, 15)
    table = c.table[:, :4].copy()
    kept, count = run_select(c, w, [1 << 30], 0, 3, table=table, lens=[2 ** 31 - 1], width=70, max_kv=64)
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
    assert count.tolist() == [64] and np.array_equal(kept[0, :, :64], np.tile(np.arange(64), (2, 1)))
    cache, _ = c.to_device()
    q, lse = torch.zeros(40, 8, 64, dtype=torch.bfloat16, device=device()), torch.zeros(40, 8, device=device())
    tree = torch.zeros(40, 2, dtype=torch.int32, device=device())
    out = torch.empty_like(q)
    for n in (1, 40):
        q4.q4_kv_attention(out[:n], q[:n], cache, dev(table), i32([2 ** 31 - 1]), i32([0, n]), n, 64, tree=tree[:n].contiguous(),
                           lse=lse[:n]) if n > 2 else None
        weight = torch.ones(c.pages, 2, 16, device=device())
        q4.q4_kv_weigh(weight, q[:n], torch.zeros_like(lse[:n]), cache, dev(table), i32([2 ** 31 - 1]), i32([0, n]), n, 64)
        torch.cuda.synchronize()
        assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
        got = weight.cpu().numpy()[c.table[0, :4]]
        assert np.all(got == 1 + 4 * n)          # all queries see all that is there, four heads of them: exp(0) each


# ------------------------------------------------------------------ moving
def check_move(c, kept, first, seed, to=False, head_lists=True, ragged=0):
    """kept[b][h]: positions.  All of the cache is compared: what is not to change, too."""
    B, heads = len(c.lens), c.heads
    count = [len(k[0]) for k in kept]
    width = max(max(count), 1) + ragged
    w = weights(c, seed)
    lists = np.full((B, heads if head_lists else 1, width), -5, np.int32)
    for b in range(B):
        for h in range(lists.shape[1]):
            lists[b, h, :count[b]] = kept[b][h]
    to_table = None
    codes = [c.k, c.v]
    scales = [np.where(np.isnan(c.ks), 0, c.ks), np.where(np.isnan(c.vs), 0, c.vs)]
    if to:
        need = [-(-(f + n) // c.page) for f, n in zip(first, count)]
        extra = sum(need)
        g = rng(seed, 31)
        codes = [np.concatenate([x, g.integers(-127, 128, (extra, *x.shape[1:])).astype(np.int8)]) for x in codes]
        scales = [np.concatenate([x, (0.01 + 0.05 * g.random((extra, *x.shape[1:]))).astype(f32)]) for x in scales]
        w = np.concatenate([w, np.full((extra, *w.shape[1:]), -1, f32)])
        to_table = np.full((B, max(max(need), 1)), -3, np.int32)
        at = c.pages
        for b in range(B):
            to_table[b, :need[b]] = range(at, at + need[b])
            at += need[b]
    cache = q4.KVCache(dev(codes[0]), dev(codes[1]), dev(scales[0].astype(f32)), dev(scales[1].astype(f32)))
    wd = dev(w)
    q4.q4_kv_compact(cache, dev(c.table), i32(c.lens), dev(lists), i32(count), weight=wd,
                     first=None if not any(first) else i32(first), to_table=None if to_table is None else dev(to_table))
    torch.cuda.synchronize()
    assert q4.q4_get_device_status() == q4.Q4_OK
    want_w = w.copy()
    for x, (cs, ss) in enumerate(zip(codes, scales)):
        cs, ss = cs.copy(), ss.astype(f32)
        for b in range(B):
            target = c.table[b] if to_table is None else to_table[b]
            cs, ss = move(cs, ss, c.table[b], target, c.page, first[b], kept[b] if head_lists else [kept[b][0]] * heads, heads)
            if x == 0:
                old = want_w.copy()
                for h in range(heads):
                    src = np.asarray(kept[b][h if head_lists else 0], np.int64)
                    dst = first[b] + np.arange(len(src))
                    want_w[target[dst // c.page], h, dst % c.page] = old[c.table[b][src // c.page], h, src % c.page]
        got, got_s = (cache.k, cache.k_scale) if x == 0 else (cache.v, cache.v_scale)
        assert np.array_equal(got_s.cpu().numpy(), ss)
        assert np.array_equal(got.cpu().numpy(), cs)
    assert np.array_equal(wd.cpu().numpy(), want_w)


def random_kept(c, first, count, seed, same=False):
    g = rng(seed, 12)
    out = []
    for b, n in enumerate(c.lens):
        one = lambda: np.sort(g.choice(np.arange(first[b], n), min(count[b], max(n - first[b], 0)), replace=False))
        out.append([one()] * c.heads if same else [one() for _ in range(c.heads)])
    return out


@pytest.mark.parametrize("to", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,count", [(1, 1), (2, 1), (16, 16), (17, 3), (40, 39), (129, 100), (300, 128), (700, 129), (900, 600)])
def test_move(n, count, D, to):
    c = Cache([n], 2, D, 32 if n % 2 else 64, n, spread=8.0)
    check_move(c, random_kept(c, [0], [count], n), [0], n, to=to, ragged=n % 3)


@pytest.mark.parametrize("to", [False, True])
@pytest.mark.parametrize("page", [16, 256])
def test_move_batches(page, to):
    lens = [500, 0, 33, 1, 800, 260]
    c = Cache(lens, 3, 64, page, page, spread=8.0)
    count = [100, 0, 33, 1, 777, 0]
    check_move(c, random_kept(c, [0] * 6, count, page), [0] * 6, page, to=to)


@pytest.mark.parametrize("first", [1, 5, 15, 16, 17, 100])
def test_move_the_accepted_path_of_a_draft(first):
    """All heads alike, behind tokens that stay, which share a block with the first of them."""
    lens = [first + 40, first + 7, first]
    c = Cache(lens, 2, 128, 64, first, spread=8.0)
    check_move(c, random_kept(c, [first] * 3, [6, 7, 0], first, same=True), [first] * 3, first, head_lists=False)
    # into another page, where the block has earlier tokens of its own
    check_move(c, random_kept(c, [first] * 3, [30, 1, 0], first, same=True), [first] * 3, first, to=True, head_lists=False)


def test_move_nothing_changes():
    """A list that keeps all: codes, scales and weights stay."""
    c = Cache([300], 2, 64, 64, 9)
    check_move(c, [[np.arange(300)] * 2], [0], 9)
    check_move(c, [[np.arange(290)] * 2], [0], 9)
    # an untouched beginning
    check_move(c, [[np.r_[0:200, 210:300]] * 2], [0], 9)


@pytest.mark.parametrize("to", [False, True])
def test_move_rounds_products_first(to):
    """Millions of codes: some products lie so near a half that rounding them to fp32 first, or not, decides the code."""
    n = 30_000
    c = Cache.__new__(Cache)
    g = rng(17, 1)
    c.lens, c.heads, c.dim, c.page, c.pages = [n], 1, 128, 256, -(-n // 256)
    c.table = g.permutation(c.pages).astype(np.int32)[None]
    c.k, c.v = (g.integers(-127, 128, (c.pages, 1, 256, 128)).astype(np.int8) for _ in range(2))
    c.ks, c.vs = ((0.02 + 0.03 * g.random((c.pages, 1, 16))).astype(f32) for _ in range(2))
    check_move(c, random_kept(c, [0], [20_000], 17), [0], 17, to=to)


def test_move_zero_scales():
    c = Cache([200], 2, 64, 64, 10)
    c.ks[c.table[0, 0]] = 0
    c.ks[c.table[0, 2], 0, 1] = 0
    check_move(c, random_kept(c, [0], [150], 10), [0], 10)
    c.ks[:] = 0
    check_move(c, random_kept(c, [0], [150], 10), [0], 10, to=True)


def test_move_bad_entries():
    """Entries out of bounds and pages outside the cache become zeros; the others move."""
    c = Cache([100], 2, 64, 16, 11)
    kept = np.array([[[0, 3, 50, 120, 99]]], np.int32)      # 120 is past the end
    cache, table = c.to_device()
    q4.q4_kv_compact(cache, table, i32([100]), dev(kept), i32([5]))
    torch.cuda.synchronize()
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
    got = cache.k.cpu().numpy()[c.table[0, 0]]
    assert np.all(got[:, 3] == 0) and np.array_equal(got[:, 5:], c.k[c.table[0, 0]][:, 5:])
    for to_first in (0, 2):                                 # entry below its place
        cache, table = c.to_device()
        q4.q4_kv_compact(cache, table, i32([100]), dev(np.array([[[1, 3]]], np.int32)), i32([2]), first=i32([to_first]))
        torch.cuda.synchronize()
        assert (q4.q4_get_device_status() == q4.Q4_OK) == (to_first == 0)
    cache, table = c.to_device()
    t = c.table.copy()
    t[0, 2] = -1
    q4.q4_kv_compact(cache, dev(t), i32([100]), dev(np.array([[[1, 33, 60]]], np.int32)), i32([3]))
    torch.cuda.synchronize()
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE
    got = cache.v.cpu().numpy()[c.table[0, 0]]
    assert np.all(got[:, 1] == 0)
    cache, table = c.to_device()
    q4.q4_kv_compact(cache, table, i32([100]), dev(np.array([[[1, 33, 60]]], np.int32)), i32([3]), to_table=i32([[-1]]))
    torch.cuda.synchronize()
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE
    assert np.array_equal(cache.k.cpu().numpy(), c.k)


# ------------------------------------------------------- positions of their own
@pytest.mark.parametrize("style", [q4.Q4_ROPE_HALVES, q4.Q4_ROPE_PAIRS])
@pytest.mark.parametrize("rope", [64, 32])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_append_at_positions(kind, rope, style):
    """Positions equal to the slots give what no positions give; others give what a table in their order gives."""
    new, ctx, Hq, heads, D = [5, 1, 40], [3, 0, 30], 4, 2, 64
    lens = [a + b for a, b in zip(new, ctx)]
    c = Cache(lens, heads, D, 16, 13)
    g = rng(13, 5)
    T = sum(new)
    q, k, v = (dev(g.standard_normal((T, n, D)).astype(f32)).to(kind) for n in (Hq, heads, heads))
    ang = g.random((200, rope // 2))
    cos, sin = dev(np.cos(ang).astype(f32)), dev(np.sin(ang).astype(f32))
    norm = dev(g.random(D).astype(f32))
    place = np.concatenate([np.arange(b, b + n) for n, b in zip(new, ctx)])
    cu = i32(np.concatenate([[0], np.cumsum(new)]))

    def run(cos, sin, positions):
        cache, table = c.to_device()
        cache.k_scale.nan_to_num_(0.0)
        cache.v_scale.nan_to_num_(0.0)
        out = torch.empty_like(q)
        q4.q4_kv_append(cache, out, q, k, v, table, i32(lens), cu, cos=cos, sin=sin, rope_style=style, q_norm=norm,
                        k_norm=norm, positions=positions)
        torch.cuda.synchronize()
        assert q4.q4_get_device_status() == q4.Q4_OK
        return [out, cache.k, cache.v, cache.k_scale, cache.v_scale]

    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))
    plain = run(cos, sin, None)
    assert same(plain, run(cos, sin, i32(place)))
    # every token one place further on: the tables moved by one
    assert same(run(cos[1:].contiguous(), sin[1:].contiguous(), None), run(cos, sin, i32(place + 1)))
    far = i32(g.integers(0, 200, T))
    got = run(cos, sin, far)
    rows = far.long()
    # a table of the tokens' own rows, at their slots: one sequence at a time
    at = 0
    for b, n in enumerate(new):
        cb, sb = (torch.zeros(lens[b], rope // 2, device=device()) for _ in range(2))
        cb[ctx[b]:], sb[ctx[b]:] = cos[rows[at:at + n]], sin[rows[at:at + n]]
        cache, table = c.to_device()
        out = torch.empty_like(q[at:at + n])
        q4.q4_kv_append(cache, out, q[at:at + n], k[at:at + n], v[at:at + n], table[b:b + 1], i32(lens[b:b + 1]),
                        i32([0, n]), cos=cb, sin=sb, rope_style=style, q_norm=norm, k_norm=norm)
        torch.cuda.synchronize()
        assert torch.equal(out, got[0][at:at + n])
        for p in c.table[b, :-(-lens[b] // 16)]:
            assert torch.equal(cache.k[p], got[1][p]) and torch.equal(cache.v[p], got[2][p])
        at += n


def test_append_at_positions_outside_the_tables():
    c = Cache([20], 1, 64, 16, 14)
    g = rng(14, 5)
    q, k, v = (dev(g.standard_normal((20, 1, 64)).astype(f32)) for _ in range(3))
    cos, sin = torch.ones(9, 32, device=device()), torch.zeros(9, 32, device=device())
    for bad in (9, -1, 1 << 30):
        pos = np.zeros(20, np.int32)
        pos[7] = bad
        cache, table = c.to_device()
        out = torch.empty_like(q)
        q4.q4_kv_append(cache, out, q, k, v, table, i32([20]), i32([0, 20]), cos=cos, sin=sin, positions=i32(pos))
        torch.cuda.synchronize()
        assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
        want = q.clone()
        want[7] = 0
        assert torch.equal(out, want)
        held = cache.k.cpu().numpy()[c.table[0, 0], 0], cache.v.cpu().numpy()[c.table[0, 0], 0]
        for x, y in zip(held, (k, v)):
            assert np.all(x[7] == 0)
            y = y.cpu().numpy()[:16, 0].copy()
            y[7] = 0
            s = np.abs(y).max() * f32(1 / 127)
            assert np.array_equal(x, np.rint(y * (f32(1) / s)).astype(np.int8))
