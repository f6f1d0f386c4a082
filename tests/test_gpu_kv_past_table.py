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


@pytest.mark.parametrize("kind,n", [("f32", 1), ("bf16", 2), ("bf16", 40)])
def test_a_table_of_two_billion_tokens(kind, n):
    """Positions next to 2^31: counted up to 2^30, the bound of every call, whatever the table has room for."""
    td, page, D = torch.float32 if kind == "f32" else torch.bfloat16, 256, 64
    c = Cache([page], 1, D, page, 16)
    cache, _ = c.to_device()
    table = torch.full((1, (1 << 31) // page), -1, dtype=torch.int32, device=device())
    table[0, 0] = int(c.table[0, 0])
    q, lse = torch.zeros(n, 4, D, dtype=td, device=device()), torch.zeros(n, 4, device=device())
    weight = torch.ones(c.pages, 1, page, device=device())
    assert q4.q4_get_device_status() == q4.Q4_OK
    for length in (1 << 30, 2 ** 31 - 200, 2 ** 31 - 1):
        args = cache, table, i32([length]), i32([0, n]), n, 1 << 30
        weight.fill_(1)
        q4.q4_kv_weigh(weight, q, torch.zeros_like(lse), *args)
        assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
        got = weight.cpu().numpy()      # all that is there gets an exp(0) of every row; other slots stay
        assert np.all(got[c.table[0, 0]] == 1 + 4 * n) and np.all(np.delete(got, c.table[0, 0], 0) == 1)
        out = torch.empty_like(q)
        q4.q4_kv_attention(out, q, *args, lse=lse)
        assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
        assert np.all(np.abs(lse.cpu().numpy() - np.log(f32(page))) <= 2.0 ** -20)
