"""Attention over the cache with a tree of drafted tokens, with first tokens that a
window leaves visible, and the sums of exponentials, against 64-bit attention."""

import numpy as np
import pytest

from gpu_util import device, torch
from long_util import attend, draft, visible, words_of
from serve_util import Cache, bf16, dev, f32, i32, rng, starts
from test_gpu_kv_attention import bound

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


def lse_bound(lse, big, D, n, kind):
    """A score is off by (D + 8) 2^-23 big and its scaling by 2^-22 (big + 1); n exponentials (2^-22 each) are added
    in fp32; the logarithm and the reference's addition round three times.  On the tensor cores (bf16) an
    exponent also has the logarithm of a value scale, up to 64 in size, that is taken out again: 2^-17."""
    d = (D + 8) * 2.0 ** -23 * big[..., 0] + 2.0 ** -22 * (big[..., 0] + 1)
    return d + (n + 16) * 2.0 ** -23 + 2.0 ** -20 + 3 * 2.0 ** -23 * np.abs(lse) + (2.0 ** -17 if kind == "bf16" else 0)


def floor(c, n, kind):
    """Where the heaviest tokens' values are zero, weights matter that fp16 cannot hold relative to them.  A weight is
    held as w = unit * p * scale / top, top at most twice the largest scale, and rounded by 2^-25 at most where w is
    subnormal: 2^-25 / unit * top * |code| of the result for each of n tokens, |code| <= 127.  unit is 2^7 for bf16;
    fp32's second term is rounded 2^11 times finer, at a unit of 2^9."""
    return n * (2.0 ** -32 if kind == "bf16" else 2.0 ** -45) * 2 * np.nanmax(c.vs) * 127


def check(new, ctx, Hq, heads, D, page, kind, seed, window=0, sinks=0, trees=None, words=None, causal=True, scale=None,
          q_gain=1.5, spread=1.0, max_q=None, workspace=False, hide=None, pad=2):
    lens = [a + b for a, b in zip(new, ctx)]
    c = Cache(lens, heads, D, page, seed, spread=spread)
    g = rng(seed, 5)
    T = sum(new)
    q = (q_gain * g.standard_normal((T, Hq, D))).astype(f32)
    if kind == "bf16":
        q = bf16(q)
    td = {"f32": torch.float32, "bf16": torch.bfloat16}[kind]
    sees = [visible(n, t, causal, window, sinks, None if trees is None else trees[b])
            for b, (n, t) in enumerate(zip(new, lens))]
    if hide is not None:         # pages that nobody sees have left the table
        c.table = c.table.copy()
        full = c.table.copy()
        for b, see in enumerate(sees):
            any_seen = see.any(0)
            for i in range(-(-lens[b] // page)):
                if not any_seen[i * page:(i + 1) * page].any():
                    c.table[b, i] = hide
    cache, table = c.to_device()
    if hide is not None:
        c.table = full
    qd = torch.cat([dev(q, td), torch.full((pad, Hq, D), float("nan"), dtype=td, device=device())])
    tree = None
    if trees is not None:
        words = words or max(1, -(-max(new) // 32))
        rows = [words_of(t, words) for t in trees if len(t)]
        tree = dev(np.concatenate([*rows, np.full((pad, words), -1, np.int32)]))
    out = torch.full((T + pad, Hq, D), float("nan"), dtype=td, device=device())
    lse = torch.full((T + pad, Hq), float("nan"), device=device())
    args = (max_q or max(new), max(max(lens), 1))
    ws = None
    if workspace:
        ws = torch.zeros(q4.q4_kv_attention_workspace_size(cache, Hq, len(new), T + pad, *args), dtype=torch.uint8,
                         device=device())
    for _ in range(2):
        q4.q4_kv_attention(out, qd, cache, table, i32(lens), i32(starts(new)), *args, scale=scale, causal=causal,
                           window=window, sinks=sinks, tree=tree, lse=lse, workspace=ws)
    again = torch.full_like(out, float("nan"))
    q4.q4_kv_attention(again, qd, cache, table, i32(lens), i32(starts(new)), *args, scale=scale, causal=causal,
                       window=window, sinks=sinks, tree=tree, workspace=ws)
    torch.cuda.synchronize()
    assert q4.q4_get_device_status() == q4.Q4_OK
    if tree is not None or (sinks and window):
        assert torch.equal(out, again)
    got, got_lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.all(got[T:] == 0) and np.all(got_lse[T:] == -np.inf)
    ref, ref_lse, mag, big = attend(c, q, new, lens, D ** -0.5 if scale is None else scale, sees)
    n = max(max(lens), 1)
    err, tol = np.abs(got[:T] - ref), bound(ref, mag, big, D, n, kind) + floor(c, n, kind)
    assert np.all(err <= tol), (float(np.max(err / tol)), np.argwhere(~(err <= tol))[:3])
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(got_lse[:T]), empty) and np.all(got[:T][empty] == 0)
    ref_lse, got_lse = np.where(empty, 0, ref_lse), np.where(empty, 0, got_lse[:T])
    err, tol = np.abs(got_lse - ref_lse), lse_bound(ref_lse, big, D, n, kind)
    assert np.all(err <= tol), (float(np.max(err / tol)), np.argwhere(~(err <= tol))[:3])


KINDS = ["f32", "bf16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,ctx", [(1, 0), (1, 1), (2, 14), (7, 9), (13, 100), (16, 16), (17, 0), (31, 33), (32, 1),
                                   (33, 500), (64, 63), (65, 200)])
def test_tree_sizes(n, ctx, D, kind):
    check([n], [ctx], 4, 2, D, 16 if n % 2 else 64, kind, n + ctx, trees=[draft(n, n)])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,heads", [(1, 1), (8, 1), (6, 2), (24, 2), (8, 8)])
def test_tree_batches_and_heads(Hq, heads, kind):
    new, ctx = [5, 0, 19, 1, 40, 3], [30, 12, 0, 700, 129, 256]
    check(new, ctx, Hq, heads, 64, 32, kind, Hq, trees=[draft(n, i) for i, n in enumerate(new)], workspace=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (40, 4), (100, 33), (1000, 7)])
def test_tree_under_a_window(window, sinks, kind):
    """Long and short paths, some longer than the window."""
    new, ctx = [30, 9, 2], [300, 41, 0]
    chain = np.tril(np.ones((30, 30), bool))
    check(new, ctx, 4, 2, 64, 16, kind, window, window=window, sinks=sinks, trees=[chain, draft(9, 1), draft(2, 2)])


@pytest.mark.parametrize("kind", KINDS)
def test_tree_rows_that_see_little(kind):
    """No bit at all (with and without earlier tokens), only another's bit, bits past the sequence's end, fewer
    words than tokens."""
    new, ctx = [40, 5, 3], [20, 0, 0]
    a = draft(40, 3)
    a[4] = False
    a[7] = False
    a[7, 39] = True
    b = np.zeros((5, 40), bool)
    b[1, :] = True                    # bits from 5 on belong to nobody
    b[2, 6] = True
    tree = [a, b[:, :5], np.zeros((3, 3), bool)]
    check(new, ctx, 4, 2, 64, 16, kind, 9, trees=tree, words=2)
    # one word: nodes from 32 on are seen by nobody
    short = a.copy()
    short[:, 32:] = False
    lens = [60]
    c = Cache(lens, 2, 64, 16, 11)
    cache, table = c.to_device()
    q = bf16(rng(11, 5).standard_normal((40, 4, 64)))
    out = torch.empty(40, 4, 64, dtype=torch.bfloat16, device=device())
    q4.q4_kv_attention(out, dev(q, torch.bfloat16), cache, table, i32(lens), i32([0, 40]), 40, 60,
                       tree=dev(words_of(a, 1)))
    want = torch.empty_like(out)
    q4.q4_kv_attention(want, dev(q, torch.bfloat16), cache, table, i32(lens), i32([0, 40]), 40, 60,
                       tree=dev(words_of(short, 2)))
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # bits behind a sequence's last token
    late = torch.empty_like(out[:5])
    tree = torch.full((5, 3), -1, dtype=torch.int32, device=device())
    lens = [5]
    q4.q4_kv_attention(late, dev(q[:5], torch.bfloat16), cache, table, i32(lens), i32([0, 5]), 5, 60, tree=tree)
    full = torch.empty_like(late)
    q4.q4_kv_attention(full, dev(q[:5], torch.bfloat16), cache, table, i32(lens), i32([0, 5]), 5, 60, causal=False)
    torch.cuda.synchronize()
    assert float((late.float() - full.float()).abs().max()) <= 2.0 ** -5   # two roundings to bf16 of values up to 127 * 0.05


def test_a_chain_is_the_causal_mask():
    """A draft without branches gives what causal attention gives: the same bits in fp32; bf16 calls take another
    form for drafts, and both results are within the bound of the 64-bit one, so within twice it of each other."""
    n, ctx = 50, 70
    c = Cache([n + ctx], 2, 128, 64, 5)
    cache, table = c.to_device()
    for kind in (torch.float32, torch.bfloat16):
        q = dev(rng(5, 5).standard_normal((n, 8, 128)).astype(f32)).to(kind)
        a, b = torch.empty_like(q), torch.empty_like(q)
        tree = dev(words_of(np.tril(np.ones((n, n), bool)), 2))
        q4.q4_kv_attention(a, q, cache, table, i32([n + ctx]), i32([0, n]), n, n + ctx, tree=tree)
        q4.q4_kv_attention(b, q, cache, table, i32([n + ctx]), i32([0, n]), n, n + ctx)
        torch.cuda.synchronize()
        if kind is torch.float32:
            assert torch.equal(a, b)
            continue
        ref, _, mag, big = attend(c, q.float().cpu().numpy(), [n], [n + ctx], 128 ** -0.5, [visible(n, n + ctx)])
        far = np.abs(a.double().cpu().numpy() - b.double().cpu().numpy())
        assert np.all(far <= 2 * bound(ref, mag, big, 128, n + ctx, "bf16"))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 1), (2, 16), (16, 4), (33, 17), (100, 128), (50, 300), (300, 1), (1000, 4)])
def test_sinks(window, sinks, kind):
    check([1, 4, 20, 1], [200, 61, 0, 700], 4, 2, 64, 32, kind, window, window=window, sinks=sinks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_sinks_of_single_tokens(page, kind):
    """Pages before the window have left the table, with any entry in their place."""
    for hide in (-1, 1 << 20):
        check([1] * 5, [900, 3, 130, 511, 64], 8, 2, 128, page, kind, page, window=70, sinks=5, hide=hide)


@pytest.mark.parametrize("hide", [-1, 1 << 20])
def test_sinks_of_a_prompt(hide):
    """The tensor-core form, sinks in a tile of their own, beside the window and across tiles."""
    for window, sinks, new, ctx in ((40, 4, 300, 400), (200, 130, 260, 150), (128, 128, 500, 0), (30, 1, 257, 600)):
        check([new], [ctx], 8, 1, 128, 64, "bf16", window, window=window, sinks=sinks, hide=hide)
    check([150, 1, 300], [200, 500, 0], 8, 1, 64, 16, "bf16", 3, window=100, sinks=20, hide=hide, workspace=True)


def test_large_trees_on_the_tensor_cores():
    """Trees with so many rows that they take the other form, alone and beside single tokens."""
    check([130], [300], 16, 1, 128, 64, "bf16", 1, trees=[draft(130, 1)])
    check([300], [77], 8, 1, 64, 16, "bf16", 2, trees=[draft(300, 2)], window=60, sinks=3)
    new = [100, 1, 0, 90]
    check(new, [500, 200, 3, 0], 16, 1, 128, 32, "bf16", 3, trees=[draft(n, i) for i, n in enumerate(new)],
          workspace=True)


@pytest.mark.parametrize("D", [64, 128])
def test_drafts_cut_between_ctas(D):
    """More tiles than CTAs, long and short sequences, tiles of rows that are partly empty, shares to join."""
    new, ctx = [30, 3, 70, 1, 9, 64, 5, 33], [2500, 100, 900, 4000, 0, 1300, 700, 60]
    trees = [draft(n, i) for i, n in enumerate(new)]
    check(new, ctx, 8, 2, D, 64, "bf16", 5, trees=trees, workspace=True)
    check(new, ctx, 12, 4, D, 16, "bf16", 6, trees=trees, window=500, sinks=200, hide=-1)
    check([40], [5000], 4, 1, D, 256, "bf16", 7, trees=[draft(40, 9)])
    check([1] * 20 + [17], [333 * i % 1500 for i in range(21)], 4, 1, D, 32, "bf16", 8)


def test_drafts_of_uneven_scales():
    """Blocks of very large and very small values, seen by some rows only; scores of up to hundreds."""
    for seed in range(3):
        check([37, 5], [300, 90], 8, 2, 128, 64, "bf16", 60 + seed, trees=[draft(37, seed), draft(5, seed)], spread=100.0, q_gain=0.05)
        check([37, 5], [300, 90], 8, 2, 64, 64, "bf16", 70 + seed, trees=[draft(37, seed), draft(5, seed)], q_gain=20)
        check([300], [90], 8, 2, 64, 16, "bf16", 80 + seed, window=20, sinks=3, spread=1000.0, q_gain=0.01)


@pytest.mark.parametrize("kind", KINDS)
def test_sums_alone(kind):
    """lse without any mask of these, causal or not, with scales far apart; queries that see nothing."""
    check([1, 3, 20], [500, 90, 0], 4, 2, 64, 64, kind, 52, spread=100.0, q_gain=0.05)
    check([3, 1, 17], [50, 0, 3], 4, 2, 128, 16, kind, 8, causal=False)
    check([1, 3], [500, 90], 4, 2, 128, 64, kind, 51, q_gain=20)
    check([300], [100], 8, 1, 128, 64, kind, 53)
    check([7, 2], [-4, 30], 4, 2, 64, 16, kind, 54)      # fewer tokens than queries
    check([2], [90], 2, 2, 64, 64, kind, 55, scale=-0.3)


def test_streams_graphs_and_workspaces():
    """Captured on another stream with a workspace, replayed as lengths grow, beside an eager call."""
    n, most = 6, 400
    c = Cache([most], 2, 64, 16, 21)
    cache, table = c.to_device()
    q = dev(rng(21, 5).standard_normal((n, 4, 64)).astype(f32))
    tree = draft(n, 4)
    words = dev(words_of(tree, 1))
    lens, cu = i32([100]), i32([0, n])
    ws = torch.zeros(q4.q4_kv_attention_workspace_size(cache, 4, 1, n, n, most), dtype=torch.uint8, device=device())
    out, lse = torch.empty_like(q), torch.empty(n, 4, device=device())
    stream = torch.cuda.Stream()
    call = lambda: q4.q4_kv_attention(out, q, cache, table, lens, cu, n, most, window=50, sinks=3, tree=words, lse=lse,
                                      workspace=ws)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    for length in (100, 6, 7, 399, 64):
        lens.fill_(length)
        graph.replay()
        other, other_lse = torch.empty_like(q), torch.empty_like(lse)
        q4.q4_kv_attention(other, q, cache, table, lens, cu, n, most, window=50, sinks=3, tree=words, lse=other_lse)
        torch.cuda.synchronize()
        assert torch.equal(out, other) and torch.equal(lse, other_lse)
        see = [visible(n, length, True, 50, 3, tree)]
        ref, ref_lse, mag, big = attend(c, q.cpu().numpy(), [n], [length], 64 ** -0.5, see)
        assert np.all(np.abs(out.cpu().numpy() - ref) <= bound(ref, mag, big, 64, length, "f32"))
