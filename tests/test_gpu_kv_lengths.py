"""Lengths on the device that are far beyond the call's bounds: an error and
zeros, nothing out of range."""

import numpy as np
import pytest

from gpu_util import device, torch
from serve_util import Cache, bf16, dev, f32, i32, rng, starts

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("lens", [[MOST], [300, MOST], [MOST, 300], [MOST] * 3 + [300], [1 << 30] * 40 + [300],
                                  [MOST - 127] * 16, [-5, MOST]])
def test_lengths_that_no_cache_has(lens):
    n, D, B = 140, 64, len(lens)
    c = Cache([300], 1, D, 16, 3)
    cache, table = c.to_device()
    q = bf16(rng(B).standard_normal((n * B, 16, D)).astype(f32))
    qd = dev(q, torch.bfloat16)
    ws = torch.zeros(q4.q4_kv_attention_workspace_size(cache, 16, B, n * B, n, 400), dtype=torch.uint8, device=device())
    out = torch.full_like(qd, float("nan"))
    q4.q4_kv_attention(out, qd, cache, table.repeat(B, 1), i32(lens), i32(starts([n] * B)), n, 400, workspace=ws)
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
    got = out.float().cpu().numpy().reshape(B, n, 16, D)
    alone = torch.full((n, 16, D), float("nan"), dtype=torch.bfloat16, device=device())
    for b, length in enumerate(lens):
        if length == 300 and max(lens[:b], default=0) < 1000:    # before the lengths that do not fit
            q4.q4_kv_attention(alone, qd[b * n:(b + 1) * n], cache, table, i32([300]), i32([0, n]), n, 400, workspace=ws)
            assert np.array_equal(got[b], alone.float().cpu().numpy())
        else:
            assert np.all(got[b] == 0)
    assert q4.q4_get_device_status() == q4.Q4_OK
