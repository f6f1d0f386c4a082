"""Penalties, biases and masks on logits, bit for bit against plain fp32 steps."""

import numpy as np
import pytest

from gpu_util import device, torch
from long_util import adjust
from serve_util import bf16, dev, f32, i32, rng

import quantized_weight_q4_gb300 as q4

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "bf16": torch.bfloat16}


def check(T, V, kind, seed, width=0, nbias=0, masks=0, out_kind=None, requests=None, prompts=True, in_place=False, pad=0,
          odd=None, parts=("repetition", "frequency", "presence"), hot=1.0):
    g = rng(seed, 3)
    out_kind = out_kind or kind
    x = (g.standard_normal((T, V)) * 3).astype(f32)
    x.flat[g.integers(0, x.size, max(1, x.size // 50))] = 0.0
    if odd is not None:
        x.flat[g.integers(0, x.size, max(1, x.size // 20))] = g.choice(np.array(odd, f32), max(1, x.size // 20))
    if kind == "bf16":
        x = bf16(x)
    R = requests or T
    req = g.integers(-1, R, T).astype(np.int32) if requests else np.arange(T, dtype=np.int32)
    a, row = {}, [dict() for _ in range(T)]
    if width:
        history = np.minimum((g.random((R, width)) ** hot * V), V + 3).astype(np.int32)
        history[g.random((R, width)) < 0.05] = -1
        history[g.random((R, width)) < 0.02] = V
        n = g.integers(0, width + 1, T).astype(np.int32)
        n[0] = width
        a.update(history=dev(history), history_len=i32(n))
        prompt = np.zeros(T, np.int32)
        if prompts:
            prompt = (n * g.random(T)).astype(np.int32)
            prompt[T // 2] = n[T // 2]
            a["prompt_len"] = i32(prompt)
        values = dict(repetition=(0.7 + g.random(T)).astype(f32), frequency=(g.random(T) - 0.3).astype(f32),
                      presence=(g.random(T) - 0.2).astype(f32))
        a.update({k: dev(values[k]) for k in parts})
        for t in range(T):
            if req[t] >= 0:
                row[t] = dict(history=history[req[t]], n=n[t], prompt=prompt[t],
                              r=values["repetition"][t] if "repetition" in parts else 1.0,
                              f=values["frequency"][t] if "frequency" in parts else 0.0,
                              p=values["presence"][t] if "presence" in parts else 0.0)
    if nbias:
        index = g.integers(-2, V + 2, (R, nbias)).astype(np.int32)       # some twice, some outside
        if nbias > 2:
            index[:, -1] = index[:, 0]
        bias = (4 * g.standard_normal((R, nbias))).astype(f32)
        a.update(bias_index=dev(index), bias=dev(bias))
        for t in range(T):
            if req[t] >= 0:
                row[t]["bias"] = list(zip(index[req[t]], bias[req[t]]))
    if requests:
        a["request"] = i32(req)
    if masks:
        words = -(-V // 32)
        bits = g.integers(-2 ** 31, 2 ** 31, (masks, words)).astype(np.int32)
        bits[0] = 0
        which = g.integers(-1, masks, T).astype(np.int32)
        which[0] = 0
        a.update(mask=dev(bits), mask_row=i32(which))
        allowed = np.unpackbits(bits.view(np.uint8), axis=1, bitorder="little")[:, :V].astype(bool)
        for t in range(T):
            if which[t] >= 0:
                row[t]["mask"] = allowed[which[t]]
    wide = torch.zeros(T, V + pad, dtype=TD[kind], device=device())
    logits = wide[:, pad // 2:pad // 2 + V]
    logits.copy_(dev(x))
    out = logits if in_place else torch.full((T, V + pad), float("nan"), dtype=TD[out_kind], device=device())[:, pad - pad // 2:][:, :V]
    q4.q4_adjust_logits(out, logits, **a)
    torch.cuda.synchronize()
    assert q4.q4_get_device_status() == q4.Q4_OK
    want = np.stack([adjust(x[t], **row[t]) for t in range(T)])
    want = torch.from_numpy(want).to(TD[out_kind]).float().numpy()
    got = out.float().cpu().numpy()
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    assert np.all(same), (np.argwhere(~same)[:5], got[~same][:5], want[~same][:5])
    if pad and in_place:
        assert float(wide[:, :pad // 2].abs().max()) == 0 and float(wide[:, pad // 2 + V:].abs().max()) == 0


KINDS = ["f32", "bf16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 32, 33, 255, 1000, 1023, 1025, 4096, 32000, 50257, 128007])
def test_vocabularies(V, kind):
    check(3, V, kind, V, width=200, nbias=5, masks=2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 2, 37, 200])
def test_rows(T, kind):
    check(T, 5003, kind, T, width=300, nbias=20, masks=3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pad,in_place", [(1, False), (8, False), (13, False), (0, True), (8, True), (3, True)])
def test_strides_and_in_place(pad, in_place, kind):
    check(5, 1001, kind, pad, width=50, nbias=3, masks=2, pad=pad, in_place=in_place)
    check(1, 2048, kind, pad, width=50, nbias=3, masks=2, pad=pad, in_place=in_place)


def test_mixed_types():
    check(4, 3001, "bf16", 1, width=100, nbias=4, masks=2, out_kind="f32")
    check(4, 3001, "f32", 2, width=100, nbias=4, masks=2, out_kind="bf16", pad=8)


@pytest.mark.parametrize("kind", KINDS)
def test_each_alone(kind):
    check(4, 2000, kind, 1, width=500)
    check(4, 2000, kind, 2, nbias=7)
    check(4, 2000, kind, 3, masks=4)
    check(4, 2000, kind, 4)
    for part in ("repetition", "frequency", "presence"):
        check(4, 2000, kind, 5, width=500, parts=(part,))
    check(4, 2000, kind, 6, width=500, parts=())
    check(4, 2000, kind, 7, width=500, prompts=False)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_that_share_requests(kind):
    """Several rows a request (drafted tokens), each with a history of its own length; rows without a request."""
    check(30, 3000, kind, 1, width=400, nbias=9, masks=5, requests=4)
    check(30, 3000, kind, 2, nbias=9, requests=3)
    check(2, 3000, kind, 3, width=40, requests=9)


def test_long_histories_and_many_biases():
    check(60, 128007, "bf16", 4, width=2000, nbias=50, masks=20, hot=4.0)
    check(60, 128007, "f32", 5, width=2000, nbias=50, masks=20, hot=4.0, out_kind="bf16")
    check(2, 40000, "f32", 1, width=100_000, hot=3.0)
    check(1, 300, "f32", 2, width=524287, nbias=4095)
    check(2, 327672, "bf16", 3, width=3000, nbias=300, masks=1)


@pytest.mark.parametrize("kind", KINDS)
def test_numbers_that_are_none(kind):
    check(6, 3000, kind, 8, width=800, nbias=30, masks=2, odd=[np.inf, -np.inf, np.nan, -0.0, 3e38, -3e38, 1e-40])


def test_rows_that_are_not_there():
    x = torch.randn(3, 100, device=device())
    out = torch.empty_like(x)
    hist = i32([[1, 2, 3]])
    q4.q4_adjust_logits(out, x, history=hist, history_len=i32([3, 3, 3]), request=i32([0, 1, -1]),
                        presence=torch.ones(3, device=device()))
    torch.cuda.synchronize()
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE and q4.q4_last_device_flags() == q4.Q4_DEVERR_INDEX
    assert torch.equal(out[1:], x[1:]) and not torch.equal(out[0], x[0])
    mask = torch.zeros(2, 4, dtype=torch.int32, device=device())
    q4.q4_adjust_logits(out, x, mask=mask, mask_row=i32([1, 2, -7]))
    torch.cuda.synchronize()
    assert q4.q4_get_device_status() == q4.Q4_ERR_DEVICE
    assert torch.equal(out[1:], x[1:]) and bool(torch.isneginf(out[0]).all())


def test_then_sampled():
    """A row whose mask leaves one token gives that token."""
    g = rng(9, 9)
    T, V = 20, 5000
    x = dev(g.standard_normal((T, V)).astype(f32))
    pick = g.integers(0, V, T)
    bits = np.zeros((T, -(-V // 32) * 32), bool)
    bits[np.arange(T), pick] = True
    bits[3] = False
    mask = np.packbits(bits, axis=1, bitorder="little").view(np.int32)
    out, tokens = torch.empty_like(x), torch.empty(T, dtype=torch.int32, device=device())
    q4.q4_adjust_logits(out, x, mask=dev(mask))
    q4.q4_sample(tokens, out, torch.rand(T, device=device()))
    torch.cuda.synchronize()
    want = pick.copy()
    want[3] = -1                      # nothing is allowed
    assert tokens.tolist() == want.tolist()
