"""The first 4 KB of an attention workspace: zero before the first call, and after every call."""

import numpy as np
import pytest

from gpu_util import device, torch
from long_util import draft, words_of
from serve_util import Cache, bf16, dev, f32, i32, rng, starts

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("new,ctx", [([1], [5000]), ([40], [5000]), ([33] * 5, [2000, 9, 700, 1500, 4]),
                                     ([1, 300, 60], [900, 10, 3000]), ([2] * 70, [50 * i + 1 for i in range(70)])])
def test_counters_return_to_zero(new, ctx, kind):
    """Long sequences are cut over many CTAs, which count in the header how many have handed in their share."""
    td = torch.float32 if kind == "f32" else torch.bfloat16
    lens, T = [a + b for a, b in zip(new, ctx)], sum(new)
    c = Cache(lens, 2, 64, 64, T)
    cache, table = c.to_device()
    q = dev(bf16(rng(T, 3).standard_normal((T, 8, 64)).astype(f32)), td)
    words = -(-max(new) // 32)
    tree = dev(np.concatenate([words_of(draft(n, n), words) for n in new]))
    size = q4.q4_kv_attention_workspace_size(cache, 8, len(new), T, max(new), max(lens))
    ws = torch.zeros(size, dtype=torch.uint8, device=device())
    lse = torch.empty(T, 8, device=device())
    firsts = []
    for turn in range(2):
        for more in ({}, {"lse": lse}, {"tree": tree}, {"window": 100, "sinks": 3}):
            out = torch.full_like(q, float("nan"))
            q4.q4_kv_attention(out, q, cache, table, i32(lens), i32(starts(new)), max(new), max(lens), workspace=ws, **more)
            assert not ws[:4096].any(), more
            firsts.append(out)
    for a, b in zip(firsts[:4], firsts[4:]):
        assert torch.equal(a, b)
    assert q4.q4_get_device_status() == q4.Q4_OK
