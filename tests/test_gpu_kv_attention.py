"""Attention over the paged 8-bit cache against 64-bit attention over the
values that the cache holds."""

import numpy as np
import pytest

from gpu_util import device, torch
from serve_util import Cache, attention, bf16, dev, f32, i32, rng, starts

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


def bound(ref, mag, big, D, n, kind):
    """Error allowed to each output.  A score is a sum of D products added in fp32 (truncating at worst),
    then scaled: off by at most d = (D + 8) 2^-23 big + 2^-22 (big + 1).  Every weight is then off by
    a factor within d, and so is their sum; n of them are added in fp32.  The half-precision terms of
    fp32 calls hold 22 bits.  bf16 calls round each weight to fp16 (2^-11), keys and values may be rounded
    to fp16 once each (scores: 2^-11 big / sqrt(D) on average over a head's elements, taken as 2^-12 big),
    and the result to bf16 (2^-9)."""
    d = (D + 8) * 2.0 ** -23 * big + 2.0 ** -22 * (big + 1)
    rel = 2 * d + (n + 16) * 2.0 ** -23 + 2.0 ** -20
    if kind == "f32":
        return rel * mag + 1e-30
    return (rel + 2.0 ** -10 + 2 * 2.0 ** -12 * big) * mag + 2.0 ** -8 * np.abs(ref) + 1e-30


def check(new, ctx, Hq, heads, D, page, kind, seed, window=0, causal=True, scale=None, q_gain=1.5, spread=1.0,
          out_kind=None, max_q=None, stream=None, workspace=False):
    lens = [a + b for a, b in zip(new, ctx)]
    c = Cache(lens, heads, D, page, seed, spread=spread)
    g = rng(seed, 5)
    T = sum(new)
    q = (q_gain * g.standard_normal((T, Hq, D))).astype(f32)
    if kind == "bf16":
        q = bf16(q)
    td = {"f32": torch.float32, "bf16": torch.bfloat16}
    cache, table = c.to_device()
    wide = torch.zeros((T, Hq * D + 16), dtype=td[kind], device=device())
    wide[:, 8:8 + Hq * D] = dev(q.reshape(T, -1), td[kind])
    qd = wide[:, 8:8 + Hq * D].unflatten(1, (Hq, D))
    out_kind = out_kind or kind
    out = torch.full((T + 2, Hq, D), float("nan"), dtype=td[out_kind], device=device())
    # two rows more than the sequences have: zeros
    qpad = torch.cat([qd, torch.full((2, Hq, D), float("nan"), dtype=td[kind], device=device())])
    sc = D ** -0.5 if scale is None else scale
    ws = None
    args = (max_q or max(new), max(max(lens), 1))
    if workspace:
        ws = torch.zeros(q4.q4_kv_attention_workspace_size(cache, Hq, len(new), T + 2, *args), dtype=torch.uint8,
                         device=device())
    lens_d, cu_d = i32(lens), i32(starts(new))
    for _ in range(2):
        q4.q4_kv_attention(out, qpad, cache, table, lens_d, cu_d, *args, scale=scale, causal=causal, window=window,
                           workspace=ws)
    q4.q4_kv_attention(out[:T], qd, cache, table, lens_d, cu_d, *args, scale=scale, causal=causal, window=window,
                       workspace=ws)
    torch.cuda.synchronize()
    assert q4.q4_get_device_status() == q4.Q4_OK
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.all(got[T:] == 0)
    ref, mag, big = attention(c, q, new, lens, sc, causal, window)
    tol = bound(ref, mag, big, D, max(max(lens), 1), "f32" if kind == out_kind == "f32" else "bf16")
    err = np.abs(got[:T] - ref)
    assert np.all(err <= tol), (float(np.max(err - tol)), np.argwhere(~(err <= tol))[:3], float(np.max(err / tol)))
    return got[:T], ref


LENGTHS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 300, 700]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n", LENGTHS)
def test_single_token_lengths(n, kind, D):
    check([1], [n - 1], 4, 2, D, 16 if n % 2 else 64, kind, n)


@pytest.mark.parametrize("Hq,heads", [(1, 1), (8, 8), (8, 1), (6, 2), (7, 1), (16, 1), (24, 2), (48, 2)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_head_layouts(Hq, heads, kind):
    check([1, 1], [40, 133], Hq, heads, 64, 32, kind, Hq * 100 + heads)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_ragged_batch_and_pages(page, kind):
    new = [1, 3, 0, 2, 5, 1, 4]
    ctx = [0, 100, 30, 0, 256, 513, 12]
    check(new, ctx, 8, 2, 128, page, kind, page)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("window", [1, 2, 16, 33, 100, 1000])
def test_windows(window, kind):
    check([1, 4, 20], [200, 61, 0], 4, 2, 64, 32, kind, window, window=window)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_every_query_sees_everything(kind):
    check([3, 1, 17], [50, 0, 3], 4, 2, 64, 16, kind, 8, causal=False)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_short_prompts(kind):
    check([37, 1, 66], [0, 0, 21], 4, 1, 128, 64, kind, 31)


def test_mixed_types():
    check([1, 2], [77, 5], 4, 2, 64, 16, "f32", 41, out_kind="bf16")
    check([1, 2], [77, 5], 4, 2, 64, 16, "bf16", 42, out_kind="f32")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_sharp_scores_and_uneven_scales(kind):
    """Scores of up to hundreds, block scales up to 1e4 apart, a negative scale."""
    check([1, 3], [500, 90], 4, 2, 128, 64, kind, 51, q_gain=20)
    check([1, 3], [500, 90], 4, 2, 64, 64, kind, 52, spread=100.0, q_gain=0.05)
    check([2], [90], 2, 2, 64, 64, kind, 53, scale=-0.3)
    check([2], [90], 2, 2, 64, 64, kind, 54, scale=0.0)


def test_queries_of_any_size():
    for gain in (1e-30, 1e-8, 1e6, 1e20):
        check([1], [40], 2, 1, 64, 16, "f32", 61, q_gain=gain, scale=0.1 / gain)


def test_long_axis_is_split_and_joined():
    got, ref = check([1, 2], [9000, 5000], 4, 1, 64, 64, "f32", 71, workspace=True)
    assert np.linalg.norm(got - ref) <= 5e-6 * np.linalg.norm(ref)


def test_nothing_to_see():
    """Empty sequences, and new tokens before position 0 (more new tokens than the sequence holds)."""
    c = Cache([0, 3, 20], 1, 64, 16, 81)
    cache, table = c.to_device()
    q = dev(rng(82).standard_normal((9, 2, 64)).astype(f32))
    out = torch.full((9, 2, 64), float("nan"), device=device())
    # sequence 0: 2 new tokens, none held; 1: 6 new tokens, 3 held; 2: one
    q4.q4_kv_attention(out, q, cache, table, i32([0, 3, 20]), i32([0, 2, 8, 9]), 6, 20)
    assert q4.q4_get_device_status() == q4.Q4_OK
    got = out.cpu().numpy()
    assert np.all(got[:5] == 0)
    ref, mag, big = attention(c, q.cpu().numpy()[5:], [0, 3, 1], [0, 3, 20], 64 ** -0.5)
    assert np.all(np.abs(got[5:] - ref) <= bound(ref, mag, big, 64, 20, "f32"))


def test_a_missing_page_is_not_seen():
    c = Cache([40], 1, 64, 16, 91)
    cache, table = c.to_device()
    q = torch.zeros((1, 1, 64), device=device())
    out = torch.empty_like(q)
    table[0, 1] = c.pages
    q4.q4_kv_attention(out, q, cache, table, i32([40]), i32([0, 1]), 1, 40)
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
    v = c.values(0, 40)[1][:, 0]
    want = np.concatenate([v[:16], v[32:]]).mean(0)
    assert np.allclose(out.cpu().numpy()[0, 0], want, atol=1e-5)


def test_a_bad_query_stays_in_its_row():
    c = Cache([40, 40], 2, 64, 16, 95)
    cache, table = c.to_device()
    x = rng(96).standard_normal((4, 4, 64)).astype(f32)
    good, bad = x.copy(), x.copy()
    bad[1, 2, 5], bad[2, 0, 0] = np.nan, np.inf
    outs = []
    for q in (good, bad):
        out = torch.empty((4, 4, 64), device=device())
        q4.q4_kv_attention(out, dev(q), cache, table, i32([40, 40]), i32([0, 2, 4]), 2, 40)
        outs.append(out.cpu().numpy())
    assert np.isnan(outs[1][1, 2]).all() and np.isnan(outs[1][2, 0]).all()
    same = np.ones((4, 4), bool)
    same[1, 2] = same[2, 0] = False
    assert np.array_equal(outs[0][same], outs[1][same])


def test_same_bits_each_time_and_in_a_graph():
    new, ctx = [1, 1, 1], [3000, 10, 777]
    lens = [a + b for a, b in zip(new, ctx)]
    c = Cache(lens, 2, 128, 64, 101)
    cache, table = c.to_device()
    q = dev(rng(102).standard_normal((3, 8, 128)).astype(f32))
    lens_d, cu_d = i32(lens), i32(starts(new))
    outs = []
    for _ in range(3):
        out = torch.empty((3, 8, 128), device=device())
        q4.q4_kv_attention(out, q, cache, table, lens_d, cu_d, 1, 4096)
        outs.append(out.cpu().numpy())
    assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])
    ws = torch.zeros(q4.q4_kv_attention_workspace_size(cache, 8, 3, 3, 1, 4096), dtype=torch.uint8, device=device())
    out = torch.empty((3, 8, 128), device=device())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        q4.q4_kv_attention(out, q, cache, table, lens_d, cu_d, 1, 4096, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), outs[0])
    # the captured call follows the lengths on the device
    lens_d.copy_(i32([50, 11, 778]))
    g.replay()
    torch.cuda.synchronize()
    ref, mag, big = attention(c, q.cpu().numpy(), new, [50, 11, 778], 128 ** -0.5)
    assert np.all(np.abs(out.cpu().numpy() - ref) <= bound(ref, mag, big, 128, 778, "f32"))


def test_two_streams_do_not_share_scratch():
    c = Cache([6000], 1, 64, 64, 111)
    cache, table = c.to_device()
    qs = [dev(rng(112, i).standard_normal((1, 4, 64)).astype(f32)) for i in range(2)]
    lens, cu = i32([6000]), i32([0, 1])
    want = []
    for q in qs:
        out = torch.empty((1, 4, 64), device=device())
        q4.q4_kv_attention(out, q, cache, table, lens, cu, 1, 6000)
        want.append(out.cpu().numpy())
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [torch.empty((1, 4, 64), device=device()) for _ in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, out, s in zip(qs, outs, streams):
            q4.q4_kv_attention(out, q, cache, table, lens, cu, 1, 6000, stream=s)
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert np.array_equal(out.cpu().numpy(), w)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind,Hq", [("f32", 4), ("bf16", 3), ("bf16", 16)])
def test_one_long_among_many_short(kind, Hq, D):
    """More sequences than SMs, and one cut into hundreds of shares."""
    ctx = [i % 40 for i in range(181)]
    ctx[77] = 100_000
    check([1] * 181, ctx, Hq, 1, D, 64, kind, 300 + D + Hq)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("Hq", [1, 3, 4, 5, 8, 9, 16])
def test_few_rows_joined_from_many_shares(Hq, kind, D):
    check([1], [30_000], Hq, 1, D, 128, kind, 400 + D + Hq)
