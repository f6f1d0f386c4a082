"""The entry points for long and drafted decoding check their arguments on the host,
before any CUDA call (no GPU needed), and the binding checks its tensors."""

import ctypes

import pytest

import quantized_weight_q4_gb300 as q4
from quantized_weight_q4_gb300 import _build
from test_serve_abi import BAD_CACHES, GOOD, ODD, cache

ARG, DTYPE, ALIGN, SHAPE = q4.Q4_ERR_ARG, q4.Q4_ERR_DTYPE, q4.Q4_ERR_ALIGN, q4.Q4_ERR_SHAPE


@pytest.fixture(scope="module")
def L():
    _build.build()
    return q4.lib()


def append_at(L, c=None, **over):
    a = dict(cache=ctypes.byref(c or cache()), q_out=GOOD, q_out_dtype=0, q=GOOD, qs=256, k=GOOD, ks=128, v=GOOD,
             vs=128, dtype=0, Hq=4, rope=ctypes.byref(q4.RopeStruct(GOOD, GOOD, 9, 64, 0)), positions=GOOD, qn=None,
             kn=None, eps=1e-6, table=GOOD, stride=4, lens=GOOD, cu=GOOD, B=2, T=3, stream=None)
    a.update(over)
    return L.q4_kv_append_at(*a.values())


def attention(L, c=None, **over):
    a = dict(out=GOOD, out_dtype=1, q=GOOD, q_dtype=1, qs=256, Hq=4, cache=ctypes.byref(c or cache()), table=GOOD,
             stride=4, lens=GOOD, cu=GOOD, B=2, T=3, max_q=2, max_kv=100, total=0, scale=0.1, causal=1, window=0,
             sinks=0, tree=None, words=0, lse=None, ws=None, ws_bytes=0, stream=None)
    a.update(over)
    return L.q4_kv_attention_ex(*a.values())


def weigh(L, c=None, **over):
    a = dict(weight=GOOD, q=GOOD, q_dtype=1, qs=256, Hq=4, lse=GOOD, cache=ctypes.byref(c or cache()), table=GOOD,
             stride=4, lens=GOOD, cu=GOOD, held=None, B=2, T=3, max_q=2, max_kv=100, scale=0.1, causal=1, window=0,
             sinks=0, stream=None)
    a.update(over)
    return L.q4_kv_weigh(*a.values())


def select(L, c=None, **over):
    a = dict(kept=GOOD, width=8, count=GOOD, weight=GOOD, cache=ctypes.byref(c or cache()), table=GOOD, stride=4,
             lens=GOOD, budget=GOOD, B=2, max_kv=100, sinks=0, recent=0, stream=None)
    a.update(over)
    return L.q4_kv_select(*a.values())


def compact(L, c=None, **over):
    a = dict(cache=ctypes.byref(c or cache()), weight=GOOD, table=GOOD, stride=4, to=None, to_stride=0, lens=GOOD,
             first=None, kept=GOOD, kept_heads=2, width=8, count=GOOD, B=2, stream=None)
    a.update(over)
    return L.q4_kv_compact(*a.values())


def adjust(L, **over):
    a = dict(out=GOOD, out_dtype=0, out_stride=100, logits=GOOD + 64, dtype=0, stride=100, T=2, V=100, request=None,
             requests=2, history=GOOD, width=9, history_len=GOOD, prompt=None, rep=GOOD, freq=None, pres=None,
             bias_index=GOOD, bias=GOOD, bias_width=3, mask=GOOD, masks=2, mask_row=None, stream=None)
    a.update(over)
    return L.q4_adjust_logits(*a.values())


@pytest.mark.parametrize("call", [append_at, attention, weigh, select, compact])
def test_bad_caches_and_batches(L, call):
    for over, code in BAD_CACHES:
        assert call(L, cache(**over)) == code, over
    assert call(L, cache=None) == ARG
    for over, code in ((dict(table=None), ARG), (dict(lens=None), ARG), (dict(B=0), ARG), (dict(stride=0), ARG),
                       (dict(B=2049), SHAPE), (dict(table=GOOD + 2), ALIGN), (dict(lens=GOOD + 1), ALIGN)):
        assert call(L, **over) == code, over


def test_append_at(L):
    for over, code in ((dict(rope=None), ARG), (dict(positions=GOOD + 2), ALIGN), (dict(dtype=2), DTYPE),
                       (dict(k=None), ARG), (dict(vs=127), ARG)):
        assert append_at(L, **over) == code, over


def test_attention(L):
    for over, code in ((dict(sinks=-1), ARG), (dict(tree=GOOD), ARG), (dict(tree=GOOD, words=-1), ARG),
                       (dict(tree=GOOD, words=1, causal=0), ARG), (dict(sinks=1 << 31), SHAPE),
                       (dict(tree=GOOD, words=1 << 20), SHAPE), (dict(tree=GOOD + 2, words=1), ALIGN),
                       (dict(lse=GOOD + 1), ALIGN), (dict(out=None), ARG), (dict(Hq=5), SHAPE), (dict(window=-1), ARG),
                       (dict(q_dtype=4), DTYPE), (dict(causal=0, window=5), ARG)):
        assert attention(L, **over) == code, over


def test_weigh(L):
    for over, code in ((dict(weight=None), ARG), (dict(lse=None), ARG), (dict(q=None), ARG), (dict(Hq=0), ARG),
                       (dict(Hq=5), SHAPE), (dict(max_q=0), ARG), (dict(max_kv=0), ARG), (dict(window=-1), ARG),
                       (dict(causal=0, window=5), ARG), (dict(causal=3), ARG), (dict(sinks=-2), ARG),
                       (dict(q_dtype=3), DTYPE), (dict(max_kv=1 << 31), SHAPE), (dict(sinks=1 << 31), SHAPE),
                       (dict(weight=ODD), ALIGN), (dict(lse=GOOD + 2), ALIGN), (dict(held=GOOD + 2), ALIGN),
                       (dict(q=ODD), ALIGN), (dict(qs=255), ARG), (dict(qs=260), ALIGN), (dict(T=0), ARG)):
        assert weigh(L, **over) == code, over


def test_select(L):
    for over, code in ((dict(kept=None), ARG), (dict(count=None), ARG), (dict(weight=None), ARG), (dict(width=0), ARG),
                       (dict(budget=None), ARG), (dict(max_kv=0), ARG), (dict(sinks=-1), ARG), (dict(recent=-1), ARG),
                       (dict(max_kv=1 << 31), SHAPE), (dict(width=1 << 31), SHAPE), (dict(weight=ODD), ALIGN),
                       (dict(kept=GOOD + 2), ALIGN), (dict(count=GOOD + 1), ALIGN)):
        assert select(L, **over) == code, over


def test_compact(L):
    for over, code in ((dict(kept=None), ARG), (dict(count=None), ARG), (dict(width=0), ARG), (dict(kept_heads=3), ARG),
                       (dict(kept_heads=0), ARG), (dict(to=GOOD), ARG), (dict(width=1 << 31), SHAPE),
                       (dict(to=GOOD, to_stride=1 << 28), SHAPE), (dict(weight=ODD), ALIGN), (dict(first=GOOD + 2), ALIGN),
                       (dict(to=GOOD + 2, to_stride=4), ALIGN), (dict(kept=GOOD + 3), ALIGN)):
        assert compact(L, **over) == code, over


def test_adjust(L):
    for over, code in ((dict(out=None), ARG), (dict(logits=None), ARG), (dict(T=0), ARG), (dict(V=0), ARG),
                       (dict(stride=99), ARG), (dict(out_stride=99), ARG), (dict(dtype=7), DTYPE), (dict(out_dtype=2), DTYPE),
                       (dict(history_len=None), ARG), (dict(width=0), ARG), (dict(history=None), ARG), (dict(bias=None), ARG),
                       (dict(bias_index=None), ARG), (dict(bias_width=0), ARG), (dict(masks=0), ARG), (dict(masks=1), ARG),
                       (dict(requests=1), ARG), (dict(requests=0, request=GOOD), ARG), (dict(mask=None, mask_row=GOOD), ARG),
                       (dict(logits=GOOD, out_dtype=1), ARG), (dict(logits=GOOD, out_stride=104), ARG),
                       (dict(V=327673, stride=327673, out_stride=327673), SHAPE), (dict(width=1 << 19), SHAPE),
                       (dict(bias_width=4096), SHAPE), (dict(T=65536, requests=65536, masks=65536), SHAPE),
                       (dict(logits=GOOD + 2), ALIGN), (dict(out=GOOD + 1, out_dtype=1), ALIGN), (dict(mask=GOOD + 2), ALIGN),
                       (dict(history=GOOD + 1), ALIGN), (dict(rep=GOOD + 1), ALIGN)):
        assert adjust(L, **over) == code, over
    none = dict(request=None, history=None, history_len=None, rep=None, bias_index=None, bias=None, mask=None)
    assert adjust(L, **{**none, "request": GOOD}) == ARG
    for name in ("prompt", "rep", "freq", "pres"):
        assert adjust(L, **{**none, name: GOOD}) == ARG      # penalties need a history


def test_the_names_are_the_package_s():
    from quantized_weight_q4_gb300 import serving
    for name in ("q4_kv_weigh", "q4_kv_select", "q4_kv_compact", "q4_adjust_logits"):
        assert getattr(q4, name) is getattr(serving, name) and name in dir(q4)


def test_the_binding_refuses_host_tensors():
    import torch
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)
    f = lambda *n: torch.zeros(*n)
    with pytest.raises((TypeError, ValueError)):
        q4.q4_adjust_logits(f(1, 8), f(1, 8))

    class Held:      # a cache's sizes without its tensors
        pages, heads, page_tokens, dim, ref = 2, 2, 16, 64, 0
    with pytest.raises((TypeError, ValueError)):
        q4.q4_kv_weigh(f(2, 2, 16), f(1, 4, 64), f(1, 4), Held, i(1, 2), i(1), i(2), 1, 8)
    with pytest.raises((TypeError, ValueError)):
        q4.q4_kv_select(i(1, 2, 8), i(1), f(2, 2, 16), Held, i(1, 2), i(1), i(1), 8)
    with pytest.raises(ValueError):
        q4.q4_kv_select(i(1, 3, 8), i(1), f(2, 2, 16), Held, i(1, 2), i(1), i(1), 8)
    with pytest.raises((TypeError, ValueError)):
        q4.q4_kv_compact(Held, i(1, 2), i(1), i(1, 2, 8), i(1))
    with pytest.raises(ValueError):
        q4.q4_kv_compact(Held, i(1, 2), i(1), i(1, 3, 8), i(1))
