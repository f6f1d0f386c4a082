"""Attention without a causal mask where a sequence has more new queries than
cached tokens: every query sees all cached tokens, in both forms."""

import copy

import numpy as np
import pytest

from gpu_util import device, torch
from serve_util import Cache, attention, bf16, dev, f32, i32, rng, starts

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("new,lens,Hq,heads", [([7], [3], 2, 1), ([40, 1, 20], [17, 1, 0], 4, 2), ([150], [33], 16, 2),
                                               ([70, 2], [5, 40], 16, 1)])
def test_more_queries_than_tokens(new, lens, Hq, heads, kind):
    D = 64
    td = torch.float32 if kind == "f32" else torch.bfloat16
    c = Cache(lens, heads, D, 16, sum(new))
    q = bf16(rng(sum(lens), 3).standard_normal((sum(new), Hq, D)).astype(f32))
    cache, table = c.to_device()
    out = torch.full(q.shape, float("nan"), dtype=td, device=device())
    q4.q4_kv_attention(out, dev(q, td), cache, table, i32(lens), i32(starts(new)), max(new), max(lens), causal=False)
    assert q4.q4_get_device_status() == q4.Q4_OK
    # 64-bit attention takes lengths of at least the new tokens: one query at a time
    want = np.zeros(q.shape)
    mag = np.zeros(q.shape)
    at = 0
    for b, (n, t) in enumerate(zip(new, lens)):
        for j in range(n):
            if t:
                one = copy.copy(c)
                one.table = c.table[b:b + 1]
                parts = attention(one, q[at + j:at + j + 1], [1], [t], D ** -0.5, causal=False)
                want[at + j], mag[at + j] = parts[0][0], parts[1][0]
        at += n
    got = out.float().cpu().numpy()
    # fp32: as the other tests' fp32 calls; bf16: fp16 weights and a bf16 result
    tol = 2.0 ** -16 * mag + 1e-30 if kind == "f32" else 2.0 ** -10 * mag + 2.0 ** -8 * np.abs(want) + 1e-30
    assert np.all(np.abs(got - want) <= tol)
