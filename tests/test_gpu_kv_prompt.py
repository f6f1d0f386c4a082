"""Prompt attention over the paged 8-bit cache (the tensor-core form, bf16),
alone and in batches with single tokens, against 64-bit attention.  A sequence
of more than 1024 query rows (new tokens x query heads that share a kv head)
takes that form whatever its length; most cases have one."""

import numpy as np
import pytest

from gpu_util import device, torch
from serve_util import Cache, bf16, dev, f32, i32, rng, starts

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


def reference(c, q, new, lens, scale, window, causal):
    """64-bit outputs and their error bounds.

    Keys and values are rounded to fp16 (2^-11 each), weights too (2^-11, and 2^-32 of the largest where fp16
    runs out of exponents), sums are fp32, the result is rounded to bf16 (2^-9).  A score is off by at most
    2^-11 sum|q k| scale; its D terms' roundings are independent, so by a D^-1/2 of that times a few: a quarter
    is allowed (D >= 64), for the weight and for the weights' sum."""
    T, Hq, D = q.shape
    group = Hq // c.heads
    out, tol = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    at = 0
    for b, (n, t) in enumerate(zip(new, lens)):
        k, v = c.values(b, max(t, 0))
        pos, see = np.arange(t - n, t)[:, None], np.arange(max(t, 0))[None, :]
        ok = (see <= pos) if causal else np.ones((n, max(t, 0)), bool)
        if window:
            ok &= see > pos - window
        for h in range(Hq):
            kk, vv, x = k[:, h // group], v[:, h // group], q[at:at + n, h].astype(np.float64)
            if not ok.size:
                continue
            s = np.where(ok, x @ kk.T * scale, -np.inf)
            p = np.exp(s - np.maximum(s.max(1, keepdims=True), -1e300))
            l = p.sum(1, keepdims=True)
            p = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
            o = p @ vv
            big = np.where(ok, np.abs(x) @ np.abs(kk).T * abs(scale), 0).max(1, keepdims=True)
            mag = p @ np.abs(vv)
            rel = 3 * 2.0 ** -11 + 2 * 2.0 ** -13 * big + (t + D) * 2.0 ** -23 + 2.0 ** -20
            out[at:at + n, h] = o
            tol[at:at + n, h] = rel * mag + 2.0 ** -8 * np.abs(o) + 2.0 ** -32 * (ok @ np.abs(vv)) + 1e-30
        at += n
    return out, tol


def check(new, ctx, Hq, heads, D, page, seed, window=0, causal=True, scale=None, q_gain=1.5, spread=1.0, total_kv=0,
          pad=3):
    lens = [a + b for a, b in zip(new, ctx)]
    c = Cache(lens, heads, D, page, seed, spread=spread)
    T = sum(new)
    q = bf16((q_gain * rng(seed, 5).standard_normal((T, Hq, D))).astype(f32))
    cache, table = c.to_device()
    qd = torch.full((T + pad, Hq, D), float("nan"), dtype=torch.bfloat16, device=device())
    qd[:T] = dev(q, torch.bfloat16)
    out = torch.full((T + pad, Hq, D), float("nan"), dtype=torch.bfloat16, device=device())
    sc = D ** -0.5 if scale is None else scale
    for _ in range(2):
        q4.q4_kv_attention(out, qd, cache, table, i32(lens), i32(starts(new)), max(new), max(max(lens), 1), total_kv=total_kv,
                           scale=scale, causal=causal, window=window)
    torch.cuda.synchronize()
    assert q4.q4_get_device_status() == q4.Q4_OK
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.all(got[T:] == 0)
    ref, tol = reference(c, q, new, lens, sc, window, causal)
    err = np.abs(got[:T] - ref)
    assert np.all(err <= tol), (float(np.max(err / tol)), np.argwhere(~(err <= tol))[:4], int((~(err <= tol)).sum()))
    rel = np.linalg.norm(got[:T] - ref) / np.linalg.norm(ref)
    assert rel <= 3e-3, rel       # bf16 results: 2^-9 / sqrt(3) = 1.1e-3 .. 1.7e-3 on average
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,ctx", [(65, 0), (128, 0), (129, 0), (200, 56), (100, 1000), (257, 127), (300, 84), (513, 0)])
def test_lengths(n, ctx, D):
    check([n], [ctx], 16, 1, D, 64, n + ctx)


@pytest.mark.parametrize("Hq,heads", [(1, 1), (4, 4), (8, 1), (6, 2), (7, 1), (12, 4)])
def test_head_layouts(Hq, heads):
    check([1030 * heads // Hq + 1], [33], Hq, heads, 64, 32, Hq)


def test_a_token_of_many_heads():
    """One kv head shared by more query rows than a tile holds."""
    check([3, 1], [50, 400], 400, 1, 64, 16, 9)


@pytest.mark.parametrize("page", [16, 128, 256])
def test_ragged_batch_with_single_tokens(page):
    check([1, 140, 0, 33, 1, 300, 2], [700, 0, 20, 5, 0, 129, 50], 32, 2, 128, page, page)


def test_sum_of_lengths_bounds_the_workspace():
    new, ctx = [1, 140, 90], [2000, 0, 38]
    check(new, ctx, 32, 2, 128, 64, 17, total_kv=sum(new) + sum(ctx))


@pytest.mark.parametrize("window", [1, 16, 100, 128, 300])
def test_windows(window):
    check([280, 90], [300, 0], 16, 2, 64, 64, window, window=window)


def test_every_query_sees_everything():
    check([140, 70], [50, 0], 32, 2, 64, 16, 8, causal=False)


def test_scales_and_sharpness():
    check([130], [200], 16, 2, 128, 64, 51, q_gain=4)
    check([130], [200], 16, 2, 64, 64, 52, spread=20.0)
    check([130], [60], 16, 2, 64, 64, 53, scale=-0.2)
    check([130], [60], 16, 2, 64, 64, 54, scale=0.0)


def test_growing_maxima_rescale_the_sums():
    """Scores that rise from token to token: the running maximum moves in nearly every tile."""
    D, n = 64, 700
    c = Cache([n], 1, D, 64, 61)
    cache, table = c.to_device()
    k, _ = c.values(0, n)
    q = np.zeros((200, 6, D), f32)
    # a direction along which the keys grow with their position
    c.k[...] = 0
    for t in range(n):
        c.k[c.table[0, t // 64], :, t % 64, 0] = t * 127 // n
    c.ks[...] = 0.5
    cache, table = c.to_device()
    q[..., 0] = 16.0
    out = torch.empty((200, 6, D), dtype=torch.bfloat16, device=device())
    q4.q4_kv_attention(out, dev(q, torch.bfloat16), cache, table, i32([n]), i32([0, 200]), 200, n, scale=1.0)
    ref, tol = reference(c, q, [200], [n], 1.0, 0, True)
    got = out.float().cpu().numpy()
    # scores are multiples of 8 and exact: nothing of their bound is needed
    assert np.all(np.abs(got - ref) <= 2.0 ** -7 * np.abs(ref) + 2.0 ** -9 * np.abs(c.values(0, n)[1]).max())
    assert q4.q4_get_device_status() == q4.Q4_OK


def test_nothing_to_see_and_missing_pages():
    c = Cache([0, 30, 300], 1, 64, 16, 81)
    cache, table = c.to_device()
    new = [70, 100, 120]
    q = bf16(rng(82).standard_normal((290, 16, 64)).astype(f32))
    out = torch.full((290, 16, 64), float("nan"), dtype=torch.bfloat16, device=device())
    args = (i32([0, 30, 300]), i32(starts(new)), 120, 300)
    q4.q4_kv_attention(out, dev(q, torch.bfloat16), cache, table, *args)
    assert q4.q4_get_device_status() == q4.Q4_OK
    got = out.float().cpu().numpy()
    assert np.all(got[:140] == 0)        # no tokens; and 70 new tokens before position 0
    ref, tol = reference(c, q[140:], [0, 30, 120], [0, 30, 300], 64 ** -0.5, 0, True)
    assert np.all(np.abs(got[140:] - ref) <= tol)
    # tokens 16..31 and 160..175 of the last sequence have no page: not seen
    table[2, 1], table[2, 10] = -1, c.pages + 5
    q4.q4_kv_attention(out, dev(q, torch.bfloat16), cache, table, *args)
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
    got = out.float().cpu().numpy()[170:]
    k, v = c.values(2, 300)
    seen = np.ones(300, bool)
    seen[16:32] = seen[160:176] = False
    for j in (0, 60, 119):
        for h in range(16):
            ok = seen & (np.arange(300) <= 180 + j)
            p = np.exp(k[ok, 0] @ q[170 + j, h].astype(np.float64) / 8)
            want = p @ v[ok, 0] / p.sum()
            assert np.allclose(got[j, h], want, rtol=0.02, atol=0.02)


def test_longer_sequences_than_the_call_says():
    """kv_len above max_kv: zeros and an error, nothing out of range."""
    c = Cache([300, 300], 1, 64, 16, 91)
    cache, table = c.to_device()
    q = dev(rng(92).standard_normal((200, 16, 64)).astype(f32), torch.bfloat16)
    out = torch.full((200, 16, 64), float("nan"), dtype=torch.bfloat16, device=device())
    q4.q4_kv_attention(out, q, cache, table, i32([300, 300]), i32([0, 100, 200]), 100, 120)
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
    assert np.all(out.float().cpu().numpy() == 0)


def test_a_bad_query_stays_in_its_row():
    c = Cache([150], 2, 64, 16, 95)
    cache, table = c.to_device()
    x = rng(96).standard_normal((150, 16, 64)).astype(f32)
    bad = x.copy()
    bad[50, 2, 5], bad[140, 0, 0] = np.nan, np.inf
    outs = []
    for q in (x, bad):
        out = torch.empty((150, 16, 64), dtype=torch.bfloat16, device=device())
        q4.q4_kv_attention(out, dev(q, torch.bfloat16), cache, table, i32([150]), i32([0, 150]), 150, 150)
        outs.append(out.float().cpu().numpy())
    assert np.isnan(outs[1][50, 2]).all() and np.isnan(outs[1][140, 0]).all()
    same = np.ones((150, 16), bool)
    same[50, 2] = same[140, 0] = False
    assert np.array_equal(outs[0][same], outs[1][same])


def test_in_a_graph():
    c = Cache([700, 300], 2, 128, 64, 101)
    cache, table = c.to_device()
    new = [130, 1]
    q = bf16(rng(102).standard_normal((131, 16, 128)).astype(f32))
    lens, cu = i32([700, 300]), i32(starts(new))
    qd = dev(q, torch.bfloat16)
    ws = torch.zeros(q4.q4_kv_attention_workspace_size(cache, 16, 2, 131, 130, 700), dtype=torch.uint8, device=device())
    out = torch.empty((131, 16, 128), dtype=torch.bfloat16, device=device())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        q4.q4_kv_attention(out, qd, cache, table, lens, cu, 130, 700, workspace=ws)
    for ls in ([700, 300], [131, 2], [555, 299]):
        lens.copy_(i32(ls))
        g.replay()
        torch.cuda.synchronize()
        ref, tol = reference(c, q, new, ls, 128 ** -0.5, 0, True)
        assert np.all(np.abs(out.float().cpu().numpy() - ref) <= tol)
    assert q4.q4_get_device_status() == q4.Q4_OK
