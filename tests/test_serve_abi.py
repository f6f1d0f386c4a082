"""The serving entry points check their arguments on the host, before any CUDA
call (no GPU needed), and the binding checks its tensors."""

import ctypes

import pytest

import quantized_weight_q4_gb300 as q4
from quantized_weight_q4_gb300 import _build

vp = ctypes.c_void_p
GOOD, ODD = 0x10000, 0x10004


@pytest.fixture(scope="module")
def L():
    _build.build()
    return q4.lib()


def cache(k=GOOD, pages=4, heads=2, dim=64, page=64):
    return q4.KvCacheStruct(k, GOOD, GOOD, GOOD, pages, heads, dim, page)


BAD_CACHES = [(dict(k=None), q4.Q4_ERR_ARG), (dict(pages=0), q4.Q4_ERR_ARG), (dict(heads=-1), q4.Q4_ERR_ARG),
              (dict(dim=96), q4.Q4_ERR_SHAPE), (dict(page=8), q4.Q4_ERR_SHAPE), (dict(page=48), q4.Q4_ERR_SHAPE),
              (dict(page=512), q4.Q4_ERR_SHAPE), (dict(heads=2000), q4.Q4_ERR_SHAPE),
              (dict(pages=1 << 29, heads=8), q4.Q4_ERR_SHAPE), (dict(k=ODD), q4.Q4_ERR_ALIGN)]


def append(L, c=None, **over):
    a = dict(cache=ctypes.byref(c or cache()), q_out=GOOD, q_out_dtype=0, q=GOOD, qs=256, k=GOOD, ks=128, v=GOOD,
             vs=128, dtype=0, Hq=4, rope=None, qn=None, kn=None, eps=1e-6, table=GOOD, stride=4, lens=GOOD, cu=GOOD,
             B=2, T=3, stream=None)
    a.update(over)
    return L.q4_kv_append(*a.values())


def gather(L, c=None, **over):
    a = dict(k=GOOD, v=GOOD, dtype=0, cache=ctypes.byref(c or cache()), table=GOOD, stride=4, first=GOOD, cu=GOOD,
             B=2, T=3, stream=None)
    a.update(over)
    return L.q4_kv_gather(*a.values())


def attention(L, c=None, **over):
    a = dict(out=GOOD, out_dtype=1, q=GOOD, q_dtype=1, qs=256, Hq=4, cache=ctypes.byref(c or cache()), table=GOOD,
             stride=4, lens=GOOD, cu=GOOD, B=2, T=3, max_q=2, max_kv=100, total=0, scale=0.1, causal=1, window=0,
             ws=None, ws_bytes=0, stream=None)
    a.update(over)
    return L.q4_kv_attention(*a.values())


def sample(L, **over):
    a = dict(tokens=GOOD, probs=None, logits=GOOD, dtype=0, stride=100, T=2, V=100, u=GOOD, t=None, k=None, p=None,
             m=None, stream=None)
    a.update(over)
    return L.q4_sample(*a.values())


@pytest.mark.parametrize("call", [append, gather, attention])
def test_bad_caches_and_batches(L, call):
    for over, code in BAD_CACHES:
        assert call(L, cache(**over)) == code, over
    assert call(L, cache=None) == q4.Q4_ERR_ARG
    for over, code in ((dict(table=None), q4.Q4_ERR_ARG), (dict(cu=None), q4.Q4_ERR_ARG), (dict(B=0), q4.Q4_ERR_ARG),
                       (dict(T=0), q4.Q4_ERR_ARG), (dict(stride=0), q4.Q4_ERR_ARG), (dict(B=2049), q4.Q4_ERR_SHAPE),
                       (dict(T=(1 << 24) + 1), q4.Q4_ERR_SHAPE), (dict(table=GOOD + 2), q4.Q4_ERR_ALIGN)):
        assert call(L, **over) == code, over


def test_append(L):
    rope = lambda **o: ctypes.byref(q4.RopeStruct(*{**dict(cos=GOOD, sin=GOOD, rows=9, dim=64, style=0), **o}.values()))
    for over, code in ((dict(dtype=2), q4.Q4_ERR_DTYPE), (dict(q_out_dtype=7), q4.Q4_ERR_DTYPE),
                       (dict(q=None), q4.Q4_ERR_ARG), (dict(q_out=None), q4.Q4_ERR_ARG), (dict(k=None), q4.Q4_ERR_ARG),
                       (dict(Hq=0), q4.Q4_ERR_ARG), (dict(eps=-1.0), q4.Q4_ERR_ARG), (dict(eps=float("nan")), q4.Q4_ERR_ARG),
                       (dict(q=None, q_out=None, qn=GOOD), q4.Q4_ERR_ARG), (dict(ks=127), q4.Q4_ERR_ARG),
                       (dict(qs=255), q4.Q4_ERR_ARG), (dict(ks=129), q4.Q4_ERR_ALIGN), (dict(v=ODD), q4.Q4_ERR_ALIGN),
                       (dict(dtype=1, vs=132), q4.Q4_ERR_ALIGN), (dict(q_out=ODD), q4.Q4_ERR_ALIGN),
                       (dict(rope=rope(cos=None)), q4.Q4_ERR_ARG), (dict(rope=rope(rows=0)), q4.Q4_ERR_ARG),
                       (dict(rope=rope(dim=128)), q4.Q4_ERR_ARG), (dict(rope=rope(style=2)), q4.Q4_ERR_ARG),
                       (dict(rope=rope(dim=20)), q4.Q4_ERR_SHAPE), (dict(rope=rope(sin=ODD)), q4.Q4_ERR_ALIGN)):
        assert append(L, **over) == code, over


def test_gather(L):
    for over, code in ((dict(k=None), q4.Q4_ERR_ARG), (dict(dtype=3), q4.Q4_ERR_DTYPE), (dict(v=ODD), q4.Q4_ERR_ALIGN)):
        assert gather(L, **over) == code, over


def test_attention(L):
    for over, code in ((dict(out=None), q4.Q4_ERR_ARG), (dict(q=None), q4.Q4_ERR_ARG), (dict(Hq=0), q4.Q4_ERR_ARG),
                       (dict(Hq=5), q4.Q4_ERR_SHAPE), (dict(max_q=0), q4.Q4_ERR_ARG), (dict(max_kv=0), q4.Q4_ERR_ARG),
                       (dict(total=-1), q4.Q4_ERR_ARG), (dict(window=-1), q4.Q4_ERR_ARG),
                       (dict(causal=0, window=5), q4.Q4_ERR_ARG), (dict(causal=2), q4.Q4_ERR_ARG),
                       (dict(q_dtype=4), q4.Q4_ERR_DTYPE), (dict(out_dtype=4), q4.Q4_ERR_DTYPE),
                       (dict(qs=260), q4.Q4_ERR_ALIGN), (dict(out=ODD), q4.Q4_ERR_ALIGN), (dict(ws=ODD), q4.Q4_ERR_ALIGN),
                       (dict(max_kv=1 << 31), q4.Q4_ERR_SHAPE)):
        assert attention(L, **over) == code, over
    assert L.q4_kv_attention_workspace_size(ctypes.byref(cache(dim=96)), 4, 2, 3, 2, 100, 0) == 0
    assert L.q4_kv_attention_workspace_size(ctypes.byref(cache()), 5, 2, 3, 2, 100, 0) == 0


def test_sample(L):
    for over, code in ((dict(tokens=None), q4.Q4_ERR_ARG), (dict(u=None), q4.Q4_ERR_ARG), (dict(T=0), q4.Q4_ERR_ARG),
                       (dict(V=0), q4.Q4_ERR_ARG), (dict(stride=99), q4.Q4_ERR_ARG), (dict(dtype=5), q4.Q4_ERR_DTYPE),
                       (dict(V=327673, stride=327673), q4.Q4_ERR_SHAPE), (dict(logits=GOOD + 2), q4.Q4_ERR_ALIGN),
                       (dict(logits=GOOD + 1, dtype=1), q4.Q4_ERR_ALIGN), (dict(k=GOOD + 1), q4.Q4_ERR_ALIGN)):
        assert sample(L, **over) == code, over


def test_binding_refuses_host_tensors():
    import torch
    i8, f = torch.zeros(2, 2, 16, 64, dtype=torch.int8), torch.zeros(2, 2, 1)
    with pytest.raises(ValueError):
        q4.KVCache(i8, i8, f, f)
    with pytest.raises(TypeError):
        q4.KVCache(i8.float(), i8, f, f)
    with pytest.raises(TypeError):
        q4.KVCache(i8, i8, f[:, :1], f)
    with pytest.raises((TypeError, ValueError)):
        q4.q4_sample(torch.zeros(1, dtype=torch.int32), torch.zeros(1, 8), torch.zeros(1))
