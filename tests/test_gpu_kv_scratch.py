"""The attention's memory: library scratch that grows, and workspace sizes."""

import numpy as np
import pytest

from gpu_util import device, torch
from serve_util import Cache, bf16, dev, f32, i32, rng, starts

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu

MB = 1 << 20


def test_growing_scratch_is_not_kept():
    """A prompt in pieces with a growing bound: one buffer of the stream, not one for every size that was asked for."""
    c = Cache([300], 8, 128, 64, 1)
    cache, table = c.to_device()
    q = dev(bf16(rng(2).standard_normal((300, 32, 128)).astype(f32)), torch.bfloat16)
    out, first = torch.empty_like(q), torch.empty_like(q)
    lens, cu = i32([300]), i32([0, 300])
    q4.q4_release_scratch()
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    bounds = [int(2000 * 1.3 ** i) for i in range(16)]      # up to 102,000 tokens
    for bound in bounds:
        q4.q4_kv_attention(out, q, cache, table, lens, cu, 300, bound)
        if bound == bounds[0]:
            first.copy_(out)
        assert torch.equal(first, out)
    torch.cuda.synchronize()
    taken = before - torch.cuda.mem_get_info()[0]
    need = q4.q4_kv_attention_workspace_size(cache, 32, 1, 300, 300, bounds[-1])
    assert need >= bounds[-1] * 8 * 128 * 4
    assert taken <= need * 1.25 + 64 * MB, (taken / MB, need / MB)
    q4.q4_release_scratch()
    assert before - torch.cuda.mem_get_info()[0] <= 64 * MB
    assert q4.q4_get_device_status() == q4.Q4_OK


def test_workspace_of_few_new_tokens_on_long_sequences():
    """Calls that take the form without copies of the cache need no room for them: 64 sequences of up to 131,072
    tokens with 5 new ones and 8 query heads a kv head."""
    cache = q4.KVCache.empty(4, 8, 128, 64, device=device())
    assert q4.q4_kv_attention_workspace_size(cache, 64, 64, 320, 5, 131072) <= 512 * MB
    # prompts have the room for all their tokens: 8 heads of 128 as fp16, keys and values
    assert q4.q4_kv_attention_workspace_size(cache, 64, 4, 4096, 1024, 65536) >= 4 * 65536 * 8 * 128 * 4


@pytest.mark.parametrize("D", [64, 128])
def test_workspace_serves_smaller_calls(D):
    """A workspace of the size for some bounds takes every call within them."""
    g = rng(D, 31)
    heads, group = 2, 8
    cache = q4.KVCache.empty(64, heads, D, 64, device=device())
    for t in (cache.k, cache.v):
        t.fill_(3)
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(0.01)
    calls = 0
    for B, max_q, max_kv in [(1, 40, 100000), (8, 12, 50000), (40, 5, 20000), (64, 9, 30000), (64, 16, 3000), (6, 200, 5000)]:
        T = B * max_q
        size = q4.q4_kv_attention_workspace_size(cache, heads * group, B, T, max_q, max_kv)
        assert size <= 3000 * MB
        ws = torch.zeros(size, dtype=torch.uint8, device=device())
        tries = [(B, max_q, max_kv), (B, max_q, 300), (B, max_q, 800), (B, max_q, 2000), (1, max_q, max_kv)]
        tries += [(int(g.integers(1, B + 1)), int(g.integers(1, max_q + 1)), int(np.exp(g.uniform(0, np.log(max_kv)))) + 1)
                  for _ in range(40)]
        for b, n, kv in tries:
            kv = min(kv, max_kv)
            q = torch.zeros((b * n, heads * group, D), dtype=torch.bfloat16, device=device())
            out = torch.full_like(q, float("nan"))
            have = min(kv, 64)
            q4.q4_kv_attention(out, q, cache, i32(np.arange(b)[:, None]), i32([have] * b), i32(starts([n] * b)), n, kv,
                               workspace=ws)
            # queries before the first token see nothing; the others an average of equal values
            want = (np.arange(n) >= n - have).astype(f32) * bf16(f32(0.03))
            got = out.float().cpu().numpy().reshape(b, n, -1)
            assert np.all(np.abs(got - want[None, :, None]) <= 2.0 ** -8 * 0.03)
            calls += 1
    assert calls == 6 * 45 and q4.q4_get_device_status() == q4.Q4_OK


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_workspace_at_any_16_bytes(kind):
    """A workspace starts at a multiple of 16 bytes, no more: the same bits wherever that is."""
    td = torch.float32 if kind == "f32" else torch.bfloat16
    new, lens = [150, 1], [400, 77]
    c = Cache(lens, 2, 128, 64, 5)
    cache, table = c.to_device()
    q = dev(bf16(rng(6).standard_normal((151, 16, 128)).astype(f32)), td)
    size = q4.q4_kv_attention_workspace_size(cache, 16, 2, 151, 150, 400)
    outs = []
    for off in (0, 16, 48, 240):
        ws = torch.zeros(size + off, dtype=torch.uint8, device=device())[off:]
        out = torch.full_like(q, float("nan"))
        for _ in range(2):
            q4.q4_kv_attention(out, q, cache, table, i32(lens), i32(starts(new)), 150, 400, workspace=ws)
        outs.append(out)
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    assert q4.q4_get_device_status() == q4.Q4_OK
