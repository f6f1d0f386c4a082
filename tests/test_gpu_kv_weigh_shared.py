"""Weights of sequences that share the pages of a prefix: a call of their own each, one after another, adds them up."""

import numpy as np
import pytest

from gpu_util import device, torch
from long_util import visible, weigh
from serve_util import Cache, bf16, dev, f32, i32, rng, starts

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,n", [("f32", 1), ("bf16", 1), ("bf16", 40)])
@pytest.mark.parametrize("page", [16, 64])
def test_calls_of_their_own_add_up(kind, n, page):
    td, D, Hq, prefix = torch.float32 if kind == "f32" else torch.bfloat16, 64, 8, 192
    lens = [prefix + 77, prefix + n, prefix + 130]
    c = Cache(lens, 2, D, page, n + page)
    shared = prefix // page
    c.table[1:, :shared] = c.table[0, :shared]       # one prefix, read by all
    cache, table = c.to_device()
    q = (1.5 * rng(n, page).standard_normal((3 * n, Hq, D))).astype(f32)
    q = bf16(q) if kind == "bf16" else q
    qd, new = dev(q, td), [n] * 3
    lse = torch.empty(3 * n, Hq, device=device())
    out = torch.empty_like(qd)
    q4.q4_kv_attention(out, qd, cache, table, i32(lens), i32(starts(new)), n, max(lens), lse=lse)   # reading: all at once
    sees = [visible(n, t) for t in lens]
    sums, bounds = weigh(c, q, lse.double().cpu().numpy(), new, lens, D ** -0.5, sees)
    first = None
    for turn in range(2):
        weight = torch.full((c.pages, 2, page), 7.0, device=device())
        for b, length in enumerate(lens):
            at = slice(b * n, (b + 1) * n)
            q4.q4_kv_weigh(weight, qd[at], lse[at], cache, table[b:b + 1], i32([length]), i32([0, n]), n, length,
                           held=i32([0 if b == 0 else prefix]))
        first = weight if first is None else first
        assert torch.equal(weight, first)
    assert q4.q4_get_device_status() == q4.Q4_OK
    got = first.cpu().numpy().astype(np.float64)
    for b, length in enumerate(lens):
        j = np.arange(length)
        mine = got[c.table[b, j // page], :, j % page].T
        want, tol = sums[b].copy(), bounds[b].copy()
        for x in range(3):
            if x != b:
                want[:, :prefix] += sums[x][:, :prefix]
                tol[:, :prefix] += bounds[x][:, :prefix]
        tol += 3 * 2.0 ** -23 * want         # an addition a call
        assert np.all(np.abs(mine - want) <= tol), b
