"""Drafts on the tensor cores where many tiles have blocks that do not exist or whose pages are missing: which tokens a
tile has goes from the warp that looks blocks up to the warps that widen codes and those of the softmax."""

import numpy as np
import pytest

from gpu_util import device, torch
from long_util import attend, draft, visible, words_of
from serve_util import Cache, bf16, dev, f32, i32, rng, starts
from test_gpu_kv_attention import bound
from test_gpu_kv_masks import floor, lse_bound

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
def test_missing_pages_of_many_drafts(D, page):
    g = rng(D, page, 9)
    new = [int(n) for n in g.integers(5, 34, 24)]
    ctx = [int(n) for n in g.integers(1, 700, 24)]
    lens = [a + b for a, b in zip(new, ctx)]
    c = Cache(lens, 2, D, page, 21)
    q = bf16(1.5 * g.standard_normal((sum(new), 8, D)).astype(f32))
    trees = [draft(n, b) for b, n in enumerate(new)]
    sees = [visible(n, t, tree=trees[b]) for b, (n, t) in enumerate(zip(new, lens))]
    broken = c.table.copy()
    for b, t in enumerate(lens):
        for i in range(ctx[b] // page):              # of the tokens before the draft
            if g.random() < 0.3:
                broken[b, i] = (-1, c.pages)[i % 2]
                sees[b][:, i * page:(i + 1) * page] = False
    cache, _ = c.to_device()
    td, words = torch.bfloat16, max(1, -(-max(new) // 32))
    tree = dev(np.concatenate([words_of(t, words) for t in trees]))
    qd, cu, table, n_kv = dev(q, td), i32(starts(new)), dev(broken), max(lens)
    first = None
    for turn in range(60):
        out, lse = torch.full_like(qd, float("nan")), torch.full((sum(new), 8), float("nan"), device=device())
        q4.q4_kv_attention(out, qd, cache, table, i32(lens), cu, max(new), n_kv, tree=tree, lse=lse)
        if first is None:
            first = out, lse
            assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
        else:
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1]), turn
    q4.q4_get_device_status()
    ref, ref_lse, mag, big = attend(c, q, new, lens, D ** -0.5, sees)
    err, tol = np.abs(first[0].double().cpu().numpy() - ref), bound(ref, mag, big, D, n_kv, "bf16") + floor(c, n_kv, "bf16")
    assert np.all(err <= tol), float(np.max(err / tol))
    err, tol = np.abs(first[1].double().cpu().numpy() - ref_lse), lse_bound(ref_lse, big, D, n_kv, "bf16")
    assert np.all(err <= tol), float(np.max(err / tol))
