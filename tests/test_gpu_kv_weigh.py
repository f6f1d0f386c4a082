"""Attention weights of cached tokens against 64-bit sums."""

import numpy as np
import pytest

from gpu_util import device, torch
from long_util import attend, slots, visible, weigh
from serve_util import Cache, bf16, dev, f32, i32, rng, starts

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


def check(new, ctx, Hq, heads, D, page, kind, seed, window=0, sinks=0, causal=True, scale=None, held=None, q_gain=1.5,
          spread=1.0, break_rows=(), max_q=None, pad=2):
    lens = [a + b for a, b in zip(new, ctx)]
    c = Cache(lens, heads, D, page, seed, spread=spread)
    g = rng(seed, 5)
    T = sum(new)
    q = (q_gain * g.standard_normal((T, Hq, D))).astype(f32)
    if kind == "bf16":
        q = bf16(q)
    td = {"f32": torch.float32, "bf16": torch.bfloat16}[kind]
    sc = D ** -0.5 if scale is None else scale
    sees = [visible(n, t, causal, window, sinks) for n, t in zip(new, lens)]
    lse = attend(c, q, new, lens, sc, sees)[1].astype(f32)
    sent = q.copy()
    for r, what in break_rows:           # rows that add nothing: what they hold does not matter
        lse[r] = what
        sent[r] = np.nan if np.isnan(what) else np.inf
    cache, table = c.to_device()
    before = (g.random((c.pages, heads, page)) * 3).astype(f32)
    weight = dev(before)
    wide = torch.full((T + pad, Hq * D + 16), float("nan"), dtype=td, device=device())
    wide[:T, 8:8 + Hq * D] = dev(sent.reshape(T, Hq * D), td)
    qd = wide[:, 8:8 + Hq * D].unflatten(1, (Hq, D))
    lse_d = torch.cat([dev(lse), torch.zeros(pad, Hq, device=device())])
    had = [max(0, t - n) for n, t in zip(new, lens)] if held is None else [max(0, min(h, t)) for h, t in zip(held, lens)]
    q4.q4_kv_weigh(weight, qd, lse_d, cache, table, i32(lens), i32(starts(new)), max_q or max(max(new), 1), max(max(lens), 1),
                   held=None if held is None else i32(held), scale=scale, causal=causal, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert q4.q4_get_device_status() == q4.Q4_OK
    got = weight.cpu().numpy()
    sums, bounds = weigh(c, q, lse.astype(np.float64), new, lens, sc, sees)
    untouched = np.ones(before.shape, bool)
    for b, t in enumerate(lens):
        if t <= 0:
            continue
        p, s = slots(c, b, t)
        old = np.where(np.arange(t) < had[b], before[p, :, s].T.astype(np.float64), 0.0)
        want = old + sums[b]
        tol = bounds[b] + 2.0 ** -23 * want
        err = np.abs(got[p, :, s].T - want)
        assert np.all(err <= tol), (b, float(np.max(err / tol)), np.argwhere(~(err <= tol))[:3])
        untouched[p, :, s] = False
    assert np.array_equal(got[untouched], before[untouched])
    again = dev(before)
    q4.q4_kv_weigh(again, qd, lse_d, cache, table, i32(lens), i32(starts(new)), max_q or max(max(new), 1), max(max(lens), 1),
                   held=None if held is None else i32(held), scale=scale, causal=causal, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert torch.equal(again, weight)            # the same bits each time


KINDS = ["f32", "bf16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 129, 300, 700])
def test_single_token_lengths(n, D, kind):
    check([1], [n - 1], 4, 2, D, 16 if n % 2 else 64, kind, n)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,heads", [(1, 1), (8, 8), (8, 1), (6, 2), (7, 1), (9, 1), (24, 2), (48, 2)])
def test_head_layouts(Hq, heads, kind):
    check([1, 3], [40, 133], Hq, heads, 64, 32, kind, Hq * 100 + heads)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_ragged_batch_and_pages(page, kind):
    check([1, 3, 0, 2, 5, 1, 4], [0, 100, 30, 0, 256, 513, 12], 8, 2, 128, page, kind, page)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (16, 16), (33, 5), (100, 40), (1000, 4)])
def test_windows_and_sinks(window, sinks, kind):
    check([1, 4, 20], [200, 61, 0], 4, 2, 64, 32, kind, window, window=window, sinks=sinks)
    check([1, 30], [400, 100], 4, 2, 64, 32, kind, window + 1, window=window, sinks=sinks, held=[0, 0])


@pytest.mark.parametrize("kind", KINDS)
def test_what_is_held(kind):
    """From nothing, from inside the sequence, all of it, out of its bounds; sequences without queries."""
    check([2, 0, 1, 3], [50, 77, 20, 0], 4, 2, 64, 16, kind, 3, held=[0, 40, 21, 99])
    check([2, 0, 1, 3], [50, 77, 20, 0], 4, 2, 64, 16, kind, 4, held=[51, 0, -5, 1], window=8, sinks=2)


@pytest.mark.parametrize("kind", KINDS)
def test_every_query_sees_everything(kind):
    check([3, 1, 17], [50, 0, 3], 4, 2, 64, 16, kind, 8, causal=False)
    check([7, 2], [-4, 30], 4, 2, 64, 16, kind, 9)       # fewer tokens than queries


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,ctx", [(17, 0), (33, 100), (65, 3), (130, 0), (200, 77), (300, 300)])
def test_prompts(n, ctx, kind):
    check([n], [ctx], 4, 1, 128, 64, kind, n)
    check([n, 1, 40], [ctx, 200, 0], 8, 2, 64, 32, kind, n + 1, window=90, sinks=5, held=[0, 0, 0])


@pytest.mark.parametrize("kind", KINDS)
def test_sharp_scores_and_uneven_scales(kind):
    check([1, 3], [500, 90], 4, 2, 128, 64, kind, 51, q_gain=20)
    check([1, 3], [500, 90], 4, 2, 64, 64, kind, 52, spread=100.0, q_gain=0.05)
    check([2], [90], 2, 2, 64, 64, kind, 53, scale=-0.3)
    check([200], [90], 8, 1, 128, 64, kind, 54, q_gain=10, spread=10.0)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_without_a_sum_add_nothing(kind):
    check([4, 30], [50, 20], 4, 2, 64, 16, kind, 6, break_rows=[(1, -np.inf), (3, np.nan), (10, np.inf)])
    check([150], [20], 8, 1, 128, 16, kind, 7, break_rows=[(0, -np.inf), (77, np.nan), (149, np.inf)])


@pytest.mark.parametrize("Hq,heads", [(3, 1), (14, 2), (9, 1), (16, 1), (64, 1), (5, 5), (130, 1), (300, 1)])
def test_prompts_of_any_group(Hq, heads):
    """Tiles of queries that whole tokens do not fill, and groups as large as a tile or larger."""
    check([90, 1, 70], [300, 40, 0], Hq, heads, 64, 32, "bf16", Hq)
    check([130], [7], Hq, heads, 128, 64, "bf16", Hq + 1, window=50, sinks=3, held=[0])


def test_more_prompts_than_clusters():
    """Several turns of work for each cluster, of unlike sizes, some without a query that sees the tokens."""
    new = [70 + 13 * i for i in range(24)]
    check(new, [(97 * i) % 700 for i in range(24)], 8, 4, 64, 64, "bf16", 81)
    check(new, [(97 * i) % 700 for i in range(24)], 8, 4, 64, 64, "bf16", 82, window=30, held=[(61 * i) % 900 for i in range(24)])


def test_prompts_of_other_masks_and_lengths():
    check([200], [333], 8, 2, 128, 64, "bf16", 83, causal=False)
    check([300], [-40], 8, 2, 64, 64, "bf16", 84)        # fewer tokens than queries
    check([150, 100], [1000, 600], 8, 1, 64, 16, "bf16", 85, window=40, sinks=300, held=[1100, 0])
    check([0], [300], 8, 1, 64, 16, "bf16", 86, held=[100], max_q=500, pad=200)   # no query at all
    check([1], [300], 8, 1, 64, 16, "bf16", 87, max_q=500, pad=200)
    check([2, 0, 1], [300, 50, 700], 8, 1, 64, 16, "bf16", 88, max_q=500, held=[3, 4, 5], pad=200)


def test_weights_of_a_prompt_add_up():
    """Every query row's weights add to one: with attention's own sums, all of them to T * Hq."""
    n, Hq, heads, D, page = 600, 8, 2, 128, 64
    c = Cache([n], heads, D, page, 71)
    cache, table = c.to_device()
    q = dev(rng(71, 5).standard_normal((n, Hq, D)).astype(f32)).to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(n, Hq, device=device())
    q4.q4_kv_attention(out, q, cache, table, i32([n]), i32([0, n]), n, n, lse=lse)
    weight = torch.zeros(c.pages, heads, page, device=device())
    q4.q4_kv_weigh(weight, q, lse, cache, table, i32([n]), i32([0, n]), n, n)
    torch.cuda.synchronize()
    p, s = slots(c, 0, n)
    total = weight.cpu().numpy()[p, :, s].sum(0, dtype=np.float64)
    assert np.all(np.abs(total - n * Hq / heads) <= 1e-5 * n * Hq / heads)


def test_pages_outside_the_cache():
    c = Cache([100], 2, 64, 16, 72)
    c.table[0, 3] = 1 << 20
    cache, table = c.to_device()
    weight = torch.full((c.pages, 2, 16), 5.0, device=device())
    q, lse = torch.zeros(1, 4, 64, device=device()), torch.zeros(1, 4, device=device())
    q4.q4_kv_weigh(weight, q, lse, cache, table, i32([100]), i32([0, 1]), 1, 100)
    torch.cuda.synchronize()
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
    got = weight.cpu().numpy()
    for i in range(7):
        if i == 3:
            continue
        rows = min(16, 100 - 16 * i)
        want = np.where(np.arange(rows) + 16 * i < 99, 7.0, 2.0)     # two query heads, weight 1 each
        assert np.array_equal(got[c.table[0, i], 0, :rows], want)


def test_captured_and_on_another_stream():
    n = 200
    c = Cache([n], 2, 64, 16, 73)
    cache, table = c.to_device()
    q = dev(rng(73, 5).standard_normal((1, 4, 64)).astype(f32))
    lse = torch.full((1, 4), 5.0, device=device())
    lens, cu = i32([n]), i32([0, 1])
    weight, want = torch.zeros(c.pages, 2, 16, device=device()), torch.zeros(c.pages, 2, 16, device=device())
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        q4.q4_kv_weigh(weight, q, lse, cache, table, lens, cu, 1, n)
    for length in (n, 17, 100):
        lens.fill_(length)
        graph.replay()
        q4.q4_kv_weigh(want, q, lse, cache, table, lens, cu, 1, n)
    torch.cuda.synchronize()
    assert torch.equal(weight, want) and float(weight.sum()) > 0
