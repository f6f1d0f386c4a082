"""Appending at the end of the rotation tables: tokens inside them are stored,
keys and values, whatever their neighbours; tokens beyond them are not."""

import numpy as np
import pytest

from gpu_util import device, torch
from serve_util import dev, f32, i32, rng

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


def tables(dim, n):
    ang = np.arange(n)[:, None] * 100.0 ** (-np.arange(dim // 2) / (dim // 2))
    return dev(np.cos(ang).astype(f32)), dev(np.sin(ang).astype(f32))


def filled(pages, heads, D, page):
    """A cache with marks: codes 99 and scales 7."""
    cache = q4.KVCache.empty(pages, heads, D, page, device=device())
    cache.k.fill_(99), cache.v.fill_(99), cache.k_scale.fill_(7), cache.v_scale.fill_(7)
    return cache


@pytest.mark.parametrize("style", [q4.Q4_ROPE_HALVES, q4.Q4_ROPE_PAIRS])
@pytest.mark.parametrize("part", [1, 2])
@pytest.mark.parametrize("start,end,limit", [(0, 40, 20), (5, 29, 20), (17, 24, 20), (0, 64, 31), (3, 50, 16), (0, 20, 33)])
def test_tokens_inside_the_tables_are_stored(start, end, limit, part, style):
    D, heads, Hq = 64, 2, 2
    rot = D // part
    x = rng(start, end, limit).standard_normal((end, Hq + 2 * heads, D)).astype(f32)
    table = i32([[1, 0, 3, 2]])
    caches = []
    for top in (limit, 64):        # short tables, and tables for all
        cos, sin = tables(rot, top)
        cache = filled(4, heads, D, 16)
        at = 0
        if start:                  # earlier tokens, inside both tables
            first = dev(x[:start])
            q4.q4_kv_append(cache, None, None, first[:, Hq:Hq + heads], first[:, Hq + heads:], table, i32([start]),
                            i32([0, start]), cos=cos, sin=sin, rope_style=style)
            at = start
        # the call with all tables is given the tokens inside the short ones only
        stop = end if top == limit else min(end, limit)
        new = dev(x[at:stop])
        out = torch.full((stop - at, Hq, D), float("nan"), device=device())
        q4.q4_kv_append(cache, out, new[:, :Hq], new[:, Hq:Hq + heads], new[:, Hq + heads:], table, i32([stop]),
                        i32([0, stop - at]), cos=cos, sin=sin, rope_style=style)
        beyond = stop > top
        assert q4.q4_get_device_status() == (q4.Q4_ERR_DEVICE if beyond else q4.Q4_OK)
        if beyond:
            assert q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
        caches.append((cache, out))
    (got, q_got), (want, q_want) = caches
    inside = q_want.shape[0]
    assert torch.equal(q_got[:inside], q_want) and bool((q_got[inside:] == 0).all())
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(got, name), getattr(want, name)), name


def test_attention_over_the_tokens_inside():
    """Tokens inside the table can be attended after a call that also had some beyond it."""
    D, limit, T = 64, 20, 37
    x = rng(9).standard_normal((T, 3, D)).astype(f32)
    cache = q4.KVCache.empty(3, 1, D, 16, device=device())
    cache.k_scale.fill_(float("nan")), cache.v_scale.fill_(float("nan"))
    cos, sin = tables(D, limit)
    xd = dev(x)
    q4.q4_kv_append(cache, None, None, xd[:, 1:2], xd[:, 2:3], i32([[0, 1, 2]]), i32([T]), i32([0, T]), cos=cos, sin=sin)
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE
    out = torch.full((1, 1, D), float("nan"), device=device())
    q4.q4_kv_attention(out, xd[:1, :1], cache, i32([[0, 1, 2]]), i32([limit]), i32([0, 1]), 1, limit)
    k, v = (torch.empty((limit, 1, D), device=device()) for _ in range(2))
    q4.q4_kv_gather(k, v, cache, i32([[0, 1, 2]]), i32([0]), i32([0, limit]))
    k, v = (t[:, 0].double().cpu().numpy() for t in (k, v))
    p = np.exp(k @ x[0, 0].astype(np.float64) * D ** -0.5)
    want = p @ v / p.sum()
    # values are within half a step of a code of what was given, sums in fp32
    step = np.abs(x[:32, 2]).max() / 127
    assert np.all(np.abs(v - x[:limit, 2]) <= 0.51 * step)
    assert np.all(np.abs(out.cpu().numpy()[0, 0] - want) <= 1e-5)
    assert q4.q4_get_device_status() == q4.Q4_OK
