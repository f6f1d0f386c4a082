"""Sampling at an infinite temperature: every finite logit has the same weight,
and infinities (0 * inf is a NaN) have none, whatever stands beside them."""

import numpy as np
import pytest

from gpu_util import device, torch
from serve_util import bf16, dev, f32, i32, rng

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("V", [9, 500, 5003])
def test_infinite_temperature(V, kind):
    g = rng(V, 41)
    rows = 24
    x = bf16(g.standard_normal((rows, V)).astype(f32))
    for r in range(rows):
        odd = g.permutation(V)[:1 + (V - 2) * (r % 4) // 3]     # up to all but one
        x[r, odd] = g.choice([np.inf, np.inf, -np.inf, np.nan], len(odd))
    u = g.random(rows).astype(f32)
    want = []
    for r in range(rows):
        finite = np.flatnonzero(np.isfinite(x[r]))
        want.append(finite[int(np.floor(float(u[r]) * len(finite)))])
    tokens = torch.full((rows,), -5, dtype=torch.int32, device=device())
    probs = torch.zeros(rows, device=device())
    q4.q4_sample(tokens, dev(x, torch.float32 if kind == "f32" else torch.bfloat16), dev(u),
                 temperature=dev(np.full(rows, np.inf, f32)), probs=probs)
    assert np.array_equal(tokens.cpu().numpy(), want)
    n = np.isfinite(x).sum(1)
    assert np.allclose(probs.cpu().numpy(), 1 / n, rtol=1e-6)
    # with a limit: the first of the equal ones by index
    q4.q4_sample(tokens, dev(x, torch.float32 if kind == "f32" else torch.bfloat16), dev(np.full(rows, 0.999, f32)),
                 temperature=dev(np.full(rows, np.inf, f32)), top_k=i32([3] * rows))
    assert np.array_equal(tokens.cpu().numpy(), [np.flatnonzero(np.isfinite(r))[:3][-1] for r in x])
    assert q4.q4_get_device_status() == q4.Q4_OK
