"""Lengths on the device that are past the page table: attention over the tokens that it has, in every form, and the
error recorded by that call alone."""

import numpy as np
import pytest

from gpu_util import device, torch
from serve_util import Cache, dev, f32, i32

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu

HAVE = 64            # tokens of the table
LENS = [65, 200, 1 << 30, 2 ** 31 - 17, 2 ** 31 - 1]


def sees(n, length, extra, window, sinks):
    """bool [n, HAVE]."""
    j = np.arange(HAVE)
    place = np.array([length - n - 1 if extra == "tree" else length - n + i for i in range(n)], np.int64)[:, None]
    see = j <= place
    if window:
        see &= (j > place - window) | (j < sinks)
    return see


@pytest.mark.parametrize("extra", ["none", "lse", "sinks", "tree"])
@pytest.mark.parametrize("kind,n", [("f32", 1), ("f32", 13), ("bf16", 1), ("bf16", 3), ("bf16", 40)])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_goes_by_what_the_table_has(kind, n, extra, D):
    if extra == "none" and n == 40:
        pytest.skip("the form for prompts has bounds of its own: tests/test_gpu_kv_lengths.py")
    td = torch.float32 if kind == "f32" else torch.bfloat16
    c = Cache([HAVE], 2, D, 16, 15)
    cache, _ = c.to_device()
    table = dev(np.ascontiguousarray(c.table[:, :HAVE // 16]))
    _, v = c.values(0, HAVE)
    window, sinks = (24, 4) if extra == "sinks" else (0, 0)
    q = torch.zeros(n, 8, D, dtype=td, device=device())      # equal weights for all that a row sees
    more = {}
    if extra == "tree":
        more["tree"] = torch.zeros(n, 2, dtype=torch.int32, device=device())
    if extra == "sinks":
        more.update(window=window, sinks=sinks)
    assert q4.q4_get_device_status() == q4.Q4_OK
    for length in [HAVE] + LENS:
        out = torch.full_like(q, float("nan"))
        lse = torch.full((n, 8), float("nan"), device=device())
        if extra != "none":
            more["lse"] = lse
        q4.q4_kv_attention(out, q, cache, table, i32([length]), i32([0, n]), n, HAVE, **more)
        torch.cuda.synchronize()
        status, flags = q4.q4_get_device_status(), q4.q4_last_device_flags()
        if length > HAVE:
            assert status == q4.Q4_ERR_DEVICE and flags == q4.Q4_DEVERR_INDEX, length
        else:
            assert status == q4.Q4_OK
        see = sees(n, length, extra, window, sinks)
        got, sums = out.double().cpu().numpy(), lse.cpu().numpy()
        for i in range(n):
            m = int(see[i].sum())
            for h in range(8):
                if m == 0:
                    assert np.all(got[i, h] == 0) and (extra == "none" or sums[i, h] == -np.inf), (length, i)
                    continue
                want, mag = v[see[i], h // 4].mean(0), np.abs(v[see[i], h // 4]).mean(0)
                # fp32: weights of 22 bits, 64 terms in fp32; bf16: weights rounded to fp16 (2^-11), the result to bf16 (2^-8)
                tol = 2.0 ** -18 * mag if kind == "f32" else 1.01 * (2.0 ** -11 * mag + 2.0 ** -8 * np.abs(want))
                assert np.all(np.abs(got[i, h] - want) <= tol), (length, i, h)
                if extra != "none":      # a logarithm below 8, to a few units of 2^-22
                    assert abs(sums[i, h] - np.log(f32(m))) <= 2.0 ** -20, (length, i, h)
