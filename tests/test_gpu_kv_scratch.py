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
