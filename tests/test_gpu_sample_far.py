"""Sampling where the cut lies far below the largest logit, and rows that leave
most of a cluster's last CTA empty."""

import numpy as np
import pytest

from gpu_util import device, torch
from serve_util import bf16, dev, f32, i32, rng

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu

BELOW_ONE = np.float32(1) - np.float32(2.0 ** -24)


def sample(logits, u, kind, **settings):
    T = logits.shape[0]
    td = torch.float32 if kind == "f32" else torch.bfloat16
    tokens = torch.full((T,), -5, dtype=torch.int32, device=device())
    args = {n: dev(np.asarray(v, f32)) for n, v in settings.items()}
    q4.q4_sample(tokens, dev(logits, td), dev(np.asarray(u, f32)), **args)
    torch.cuda.synchronize()
    assert q4.q4_get_device_status() == q4.Q4_OK
    return tokens.cpu().numpy()


@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n", [4000, 30000, 100000])
def test_cut_far_below_the_largest(n, kind, shuffled):
    """One likely token and n between 14.5 and 20 nats below it, top-p alone: the cut lies among the far ones.

    The last kept token by index is taken by the largest u below 1: u * (all) is at most all - all 2^-24 + 1, and the
    token's weight is above all 2^-23.  Weights are whole numbers of 2^-40; the reference's sums may differ from the
    kernel's by n roundings of expf, within 2^-22 of the far weight, far less than the margin that is kept from
    the step's ends."""
    g = rng(n, 21)
    far = -14.5 - 5.5 * g.random(n)
    z = np.concatenate([[0.0], far]).astype(f32)
    if kind == "bf16":
        z = bf16(z)
    z[1:] = np.sort(z[1:])[::-1]
    order = np.arange(n + 1)
    if shuffled:
        order = g.permutation(n + 1)                 # where each of the ranking stands
        placed = np.empty_like(z)
        # equal logits are ranked by index
        for v in np.unique(z):
            same = np.flatnonzero(z == v)
            order[same] = np.sort(order[same])
        placed[order] = z
    else:
        placed = z
    w = np.floor(np.exp(z.astype(np.float64)) * 2.0 ** 40)
    upto, whole = np.cumsum(w), w.sum()
    light = int((w > whole * 2.0 ** -23).sum())     # those heavy enough to aim at
    ps, want = [], []
    for at in np.linspace(2, light - 2, 9).astype(int):
        # an fp32 limit inside the step of rank `at`
        for r in range(at, light):
            p = f32((upto[r] - w[r] / 2) / whole)
            target = np.ceil(float(p) * whole)
            if upto[r] - w[r] * 0.8 < target < upto[r] - w[r] * 0.2:
                kept = order[:r + 1]
                last = kept[np.argmax(kept)]
                if w[np.flatnonzero(order == last)[0]] > whole * 2.0 ** -23:
                    ps.append(p), want.append(last)
                break
    assert len(ps) >= 5
    got = sample(np.tile(placed, (len(ps), 1)), [BELOW_ONE] * len(ps), kind, top_p=ps)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("V", [4097, 4099, 8193, 16385])
def test_rows_that_leave_a_cta_nearly_empty(V, kind):
    """The last CTA of a row's cluster has an element or a few and is ready long before the others."""
    g = rng(V, 22)
    rows = 1500
    x = g.standard_normal((rows, V)).astype(f32)
    x[::2, V - 1] = 50                               # the largest in the last CTA,
    x[1::2, 3] = 50                                  # or in the first
    if kind == "bf16":
        x = bf16(x)
    want = np.where(np.arange(rows) % 2 == 0, V - 1, 3)
    for _ in range(3):
        got = sample(x, np.full(rows, 0.5), kind, temperature=np.where(np.arange(rows) % 3 == 0, 0, 1.0))
        assert np.array_equal(got, want)
