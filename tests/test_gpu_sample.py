"""Sampling against a 64-bit reference.  The reference's kept set and the tokens'
intervals are known; a uniform number is put in the middle of an interval (and
a top-p limit between two steps).  Uniform numbers are fp32, so a token less
likely than their spacing cannot be aimed at: the token has to be kept, and its
interval has to hold the fp32 number, up to the weights' own rounding."""

import numpy as np
import pytest

from gpu_util import device, torch
from serve_util import bf16, dev, f32, i32, rng

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


def kept(logits, t=1.0, k=0, p=1.0, m=0.0):
    """Ranking and kept probabilities (by index, sum 1) of one row, in 64 bits."""
    z = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    if t < 1e-5:
        t, k = 1.0, 1
    # the definition's z is one fp32 product
    z = (z.astype(f32) * f32(f32(1) / f32(t))).astype(np.float64)
    e = np.exp(z - z.max())
    e[e < 2.0 ** -40] = 0
    order = np.lexsort((np.arange(len(z)), -z))
    n = len(z) if k <= 0 else min(k, len(z))
    r = np.zeros(len(z), bool)
    r[:n] = True
    w = np.where(r, e[order], 0)
    before = np.cumsum(w) - w
    if p < 1:
        r &= before < max(p * w.sum(), 1e-300)
        r[0] = True
    r &= e[order] >= min(m, 1.0)
    out = np.zeros(len(z))
    out[order] = np.where(r, w, 0)
    return order, out / out.sum()


def sample(logits, u, kind="f32", stride=None, **settings):
    T, V = logits.shape
    td = torch.float32 if kind == "f32" else torch.bfloat16
    wide = torch.full((T, stride or V), 50.0, dtype=td, device=device())
    wide[:, :V] = dev(logits, td)
    tokens = torch.full((T,), -5, dtype=torch.int32, device=device())
    probs = torch.full((T,), float("nan"), device=device())
    args = {n: (i32(v) if n == "top_k" else dev(np.asarray(v, f32))) for n, v in settings.items()}
    q4.q4_sample(tokens, wide[:, :V], dev(np.asarray(u, f32)), probs=probs, **args)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), probs.cpu().numpy()


def middle(p, token):
    c = np.cumsum(p)
    return c[token] - p[token] / 2


def check(got, probs, us, ps):
    """Row by row: the token is kept, its interval holds u, its probability is p's.  Weights are exact
    to 2 ulp of exp and one of its argument (|z| < 100: 2^-18 at worst, 2^-22 on average); a running
    sum of probabilities is within the average."""
    for r, (token, u, p) in enumerate(zip(got, us, ps)):
        assert p[token] > 0, (r, token)
        hi = np.cumsum(p)[token]
        assert hi - p[token] - 2.0 ** -22 <= f32(u) <= hi + 2.0 ** -22, (r, token, u, hi, p[token])
        assert abs(probs[r] - p[token]) <= 2e-5 * p[token], (r, token)


def pick(g, p):
    """A kept token whose interval is wide enough to aim at, and a u inside it."""
    likely = np.flatnonzero(p > 1e-4)
    token = int(g.choice(likely))
    return token, middle(p, token)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 31, 500, 4096, 4097, 32000, 50257, 128007, 327672])
def test_temperature_alone(V, kind):
    g = rng(V, 1)
    rows = 7
    logits = (g.standard_normal((rows, V)) * 2).astype(f32)
    logits[:, g.integers(0, V, 5)] += 7
    if kind == "bf16":
        logits = bf16(logits)
    temp = g.uniform(0.5, 1.5, rows).astype(f32)
    want, us, ps = [], [], []
    for r in range(rows):
        _, p = kept(logits[r], float(temp[r]))
        token, u = pick(g, p)
        want.append(token), us.append(u), ps.append(p)
    got, probs = sample(logits, us, kind, temperature=temp)
    assert np.array_equal(got, want)
    check(got, probs, us, ps)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("V", [3, 700, 9001, 60000])
def test_limits(V, kind):
    """top-k, top-p and min-p, alone and together: a token in the middle of the kept ones, the first
    and the last of the ranking."""
    g = rng(V, 2)
    rows = 24
    logits = (g.standard_normal((rows, V)) * 2.5).astype(f32)
    if kind == "bf16":
        logits = bf16(logits)          # many equal logits: ties go by index
    temp = g.uniform(0.6, 1.4, rows).astype(f32)
    top_k = np.where(np.arange(rows) % 2 == 0, g.integers(1, min(V, 300) + 1, rows), 0)
    min_p = np.where(np.arange(rows) % 3 == 0, g.uniform(0.01, 0.3, rows), 0).astype(f32)
    top_p, want, us, ps = np.ones(rows, f32), [], [], []
    for r in range(rows):
        if r % 4 < 3 and V > 1:
            # a limit in the middle of a step of the ranking after top-k
            order, p = kept(logits[r], float(temp[r]), int(top_k[r]))
            c = np.cumsum(p[order])
            at = np.searchsorted(c, g.uniform(0.2, 0.98))
            at = min(at, int((p > 0).sum()) - 1)
            top_p[r] = c[at] - p[order][at] / 2
        order, p = kept(logits[r], float(temp[r]), int(top_k[r]), float(top_p[r]), float(min_p[r]))
        e = p / p.max()
        assert min_p[r] == 0 or np.abs(e[e > 0] - min_p[r]).min() > 1e-6
        n = int((p > 0).sum())
        token = int(order[[0, n - 1, n // 2][r % 3]])
        want.append(token), us.append(middle(p, token)), ps.append(p)
    got, probs = sample(logits, us, kind, stride=V + 3, temperature=temp, top_k=top_k, top_p=top_p, min_p=min_p)
    aimed = [p[t] > 1e-5 for p, t in zip(ps, want)]
    assert np.array_equal(got[aimed], np.array(want)[aimed])
    check(got, probs, us, ps)


def test_equal_logits():
    V = 20000
    flat = np.zeros((4, V), f32)
    got, probs = sample(flat, [0.0, 0.5, 0.99999, 0.25], top_k=[0, 0, 7, 1000], top_p=[1, 0.5, 1, 0.1])
    # exact integer arithmetic of the definition: 10000 kept, the middle of them; 7; and 101, as fp32's 0.1 is
    # above 0.1
    assert list(got) == [0, 5000, 6, 25]
    assert np.allclose(probs, [1 / V, 1 / 10000, 1 / 7, 1 / 101], rtol=1e-6)


def test_greedy_and_ties():
    g = rng(11)
    logits = g.standard_normal((5, 3001)).astype(f32)
    logits[1, 40] = logits[1, 2000] = 9
    logits[2, 0] = logits[2, 3000] = np.inf
    logits[3, 3000] = 8
    logits[4, 5] = np.nan
    got, probs = sample(logits, [0.999] * 5, temperature=[0, 1e-6, -1, 0, float("nan")])
    assert list(got) == [int(logits[0].argmax()), 40, 0, 3000, int(np.nanargmax(logits[4]))]
    assert np.all(probs == 1)


def test_masked_rows():
    g = rng(12)
    logits = g.standard_normal((6, 5000)).astype(f32)
    logits[0] = -np.inf
    logits[1] = np.nan
    logits[2], logits[2, 4321] = -np.inf, -5.0
    logits[3], logits[3, 17] = np.finfo(f32).min, 0.0
    logits[4, 100:] = -np.inf
    logits[5] = np.finfo(f32).min
    u = [0.5, 0.5, 0.7, 0.9999, 0.0, 0.5]
    for extra in ({}, {"top_p": [0.9] * 6, "top_k": [50] * 6}):
        got, probs = sample(logits, u, **extra)
        assert list(got[:4]) == [-1, -1, 4321, 17] and list(probs[:4]) == [0, 0, 1, 1]
        assert got[4] < 100 and 0 <= got[5] < 5000
    _, p = kept(logits[4])
    assert got[4] == np.flatnonzero(p)[0] or extra


def test_codes_that_share_a_fine_bin():
    """Logits that differ in their last bits only: the cut has to be found on the code itself."""
    V = 6000
    g = rng(13)
    base = np.float32(3.0).view(np.int32) if hasattr(np.float32(3.0), "view") else 0
    bits = base + g.permutation(V).astype(np.int32) % 1500
    z = bits.astype(np.int32).view(f32)
    z = np.concatenate([[np.float32(8.0)], z]).astype(f32)
    ks = [2, 3, 700, 3001, 5990]
    logits = np.tile(z, (len(ks), 1))
    want, us = [], []
    for k in ks:
        order, p = kept(z, 1.0, k)
        token = int(order[k - 1])
        want.append(token), us.append(middle(p, token))
    got, _ = sample(logits, us, top_k=ks)
    assert list(got) == want


def test_extreme_u_and_settings():
    g = rng(14)
    logits = g.standard_normal((7, 900)).astype(f32)
    u = [0.0, 1.0, np.float32(1) - np.float32(2.0 ** -24), -3.0, float("nan"), 0.5, 0.5]
    got, _ = sample(logits, u, top_p=[1, 1, 1, 1, 1, 0.0, -1.0], min_p=[0, 0, 0, 0, 0, 5.0, 0])
    assert got[0] == 0 and got[1] == 899 and got[2] == 899 and got[3] == 0 and got[4] == 0
    assert got[5] == logits[5].argmax() and got[6] == logits[6].argmax()


def test_distribution():
    """Many uniform numbers over one row: frequencies follow the kept probabilities (6 sigma)."""
    g = rng(15)
    row = (g.standard_normal(300) * 2).astype(f32)
    n = 20000
    u = (np.arange(n) + 0.5) / n
    got, _ = sample(np.tile(row, (n, 1)), u, top_k=[40] * n, temperature=[0.8] * n)
    _, p = kept(row, 0.8, 40)
    count = np.bincount(got, minlength=300)
    assert np.all(np.abs(count - n * p) <= 2)      # evenly spread u: within a step at each end
    assert q4.q4_get_device_status() == q4.Q4_OK
