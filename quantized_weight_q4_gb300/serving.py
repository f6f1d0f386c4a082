"""The serving operators beside the matmuls: the paged 8-bit key/value cache,
attention over it, leaving tokens out of it, and logits to tokens (include/q4.h, "Serving").  Reached through the
package's names.

These calls are made once a token and layer, so their checks are kept short:
one attribute at a time, nothing looked up twice.
"""

from __future__ import annotations

import ctypes

import torch

from . import (Q4_BF16, Q4_F32, Q4_KV_BLOCK, Q4_ROPE_HALVES, KvCacheStruct, Q4Error, RopeStruct,
               _require_cuda, lib)

_FLOAT_CODES = {torch.float32: Q4_F32, torch.bfloat16: Q4_BF16}


class KVCache:
    """A paged 8-bit key/value cache over caller tensors (q4_kv_cache): k, v
    int8 [pages, heads, page_tokens, dim], k_scale, v_scale fp32 [pages, heads,
    page_tokens / 16].  KVCache.empty() allocates them.  The object keeps the
    tensors alive."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "struct", "ref", "pages", "heads", "page_tokens",
                 "dim")

    def __init__(self, k, v, k_scale, v_scale):
        shape = pages, heads, page, dim = k.shape
        scales = pages * heads * (page // Q4_KV_BLOCK)
        if k.dtype is not torch.int8 or v.dtype is not torch.int8 or v.shape != shape:
            raise TypeError("k and v are int8 tensors of one shape")
        if (k_scale.dtype is not torch.float32 or v_scale.dtype is not torch.float32
                or k_scale.numel() != scales or v_scale.numel() != scales):
            raise TypeError(f"k_scale and v_scale are fp32 tensors of shape "
                            f"{(pages, heads, page // Q4_KV_BLOCK)}")
        if not (k.is_cuda and v.is_cuda and k_scale.is_cuda and v_scale.is_cuda):
            raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
        if not (k.is_contiguous() and v.is_contiguous() and k_scale.is_contiguous()
                and v_scale.is_contiguous()):
            raise ValueError("all tensors must be contiguous")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.struct = KvCacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                                    v_scale.data_ptr(), pages, heads, dim, page)
        self.ref = ctypes.addressof(self.struct)
        self.pages, self.heads, self.page_tokens, self.dim = pages, heads, page, dim

    @classmethod
    def empty(cls, pages: int, heads: int, dim: int, page_tokens: int = 64, device="cuda"):
        codes = (pages, heads, page_tokens, dim)
        scales = (pages, heads, page_tokens // Q4_KV_BLOCK)
        return cls(*(torch.empty(codes, dtype=torch.int8, device=device) for _ in range(2)),
                   *(torch.empty(scales, dtype=torch.float32, device=device) for _ in range(2)))


def _rows(t, heads, dim):
    """Data pointer and row stride of a [T, heads, dim] view whose rows are dense."""
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if h != heads or d != dim or s2 != 1 or (s1 != dim and heads > 1):
        raise ValueError(f"expected a [T, {heads}, {dim}] tensor with dense rows")
    if not t.is_cuda:
        raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
    return t.data_ptr(), s0 if n > 1 else heads * dim


def _index(name, t, n):
    """Data pointer of a contiguous int32 CUDA tensor of n elements."""
    if t.dtype is not torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} is a contiguous int32 CUDA tensor")
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, not {n}")
    return t.data_ptr()


def _table(t, n):
    """Data pointer and columns of a contiguous int32 CUDA tensor of n rows."""
    if t.dtype is not torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError("page_table is a contiguous int32 CUDA tensor")
    rows, cols = t.shape
    if rows != n:
        raise ValueError(f"page_table has {rows} rows, not {n}")
    return t.data_ptr(), cols


def _words(name, t, n=None):
    """Data pointer and columns of a contiguous int32 CUDA tensor of two dimensions, of n rows."""
    if t.dtype is not torch.int32 or t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} is a contiguous int32 CUDA tensor of two dimensions")
    rows, cols = t.shape
    if n is not None and rows != n:
        raise ValueError(f"{name} has {rows} rows, not {n}")
    return t.data_ptr(), cols


def _floats(name, t, n):
    """Data pointer of a contiguous fp32 CUDA tensor of n elements, or None."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.numel() != n or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} is a contiguous fp32 CUDA tensor of {n} elements")
    return t.data_ptr()


def _out(name, t, n):
    """Data pointer and dtype code of a contiguous fp32 or bf16 CUDA tensor of n elements."""
    code = _FLOAT_CODES.get(t.dtype)
    if code is None or t.numel() != n or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} is a contiguous fp32 or bf16 CUDA tensor of {n} elements")
    return t.data_ptr(), code


def _raw_stream(stream, t):
    """cudaStream_t of a torch stream (default: the current stream of the tensor's device)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device()) or None
    return stream.cuda_stream or None


def q4_kv_append(cache: KVCache, q_out, q, k, v, page_table, kv_len, cu_q, cos=None, sin=None,
                 rope_style: int = Q4_ROPE_HALVES, q_norm=None, k_norm=None, eps: float = 1e-6,
                 stream=None, positions=None) -> None:
    """New tokens' keys and values into the cache, their queries rotated into
    q_out (include/q4.h).  q [T, Hq, dim], k, v [T, heads, dim]: views whose
    rows may be strided; q and q_out may both be None.  cos, sin: fp32
    [positions, rotated dim / 2], or None.  positions: int32 [T], each token's row
    of the tables where that is not its slot (drafted tokens; after an eviction)."""
    T, B, heads, dim = k.shape[0], kv_len.shape[0], cache.heads, cache.dim
    kp, ks = _rows(k, heads, dim)
    vp, vs = _rows(v, heads, dim)
    dtype = _FLOAT_CODES.get(k.dtype)
    if v.shape[0] != T or v.dtype is not k.dtype or dtype is None or (q is None) != (q_out is None):
        raise ValueError("k and v have the same rows and type (fp32 or bf16); q and q_out go together")
    qp, qs, Hq, out, out_dtype = None, 0, 0, None, Q4_F32
    if q is not None:
        Hq = q.shape[1]
        qp, qs = _rows(q, Hq, dim)
        if q.shape[0] != T or q.dtype is not k.dtype:
            raise ValueError("q has the rows and type of k")
        out, out_dtype = _out("q_out", q_out, T * Hq * dim)
    rope = None
    if cos is not None:
        if cos.dim() != 2 or sin is None or sin.shape != cos.shape:
            raise ValueError("cos and sin are two tables of one shape [positions, rotated dim / 2]")
        n, half = cos.shape
        table = RopeStruct(_floats("cos", cos, n * half), _floats("sin", sin, n * half), n, 2 * half,
                           rope_style)
        rope = ctypes.addressof(table)
    pages, cols = _table(page_table, B)
    if positions is not None:
        if rope is None:
            raise ValueError("positions need cos and sin")
        positions = _index("positions", positions, T)
    rc = lib().q4_kv_append_at(
        cache.ref, out, out_dtype, qp, qs, kp, ks, vp, vs, dtype, Hq, rope, positions,
        _floats("q_norm", q_norm, dim), _floats("k_norm", k_norm, dim), eps,
        pages, cols,
        _index("kv_len", kv_len, B), _index("cu_q", cu_q, B + 1), B, T, _raw_stream(stream, k))
    if rc:
        raise Q4Error("q4_kv_append", rc)


def q4_kv_gather(k_out, v_out, cache: KVCache, page_table, first, cu, stream=None) -> None:
    """Cached tokens first[b] .. of each sequence b as numbers into rows
    cu[b] .. cu[b + 1] - 1 of k_out and v_out [T, heads, dim]."""
    B, T = first.shape[0], k_out.shape[0]
    n = T * cache.heads * cache.dim
    kp, dtype = _out("k_out", k_out, n)
    vp, v_dtype = _out("v_out", v_out, n)
    if v_dtype != dtype:
        raise ValueError("k_out and v_out have one type")
    pages, cols = _table(page_table, B)
    rc = lib().q4_kv_gather(
        kp, vp, dtype, cache.ref, pages, cols,
        _index("first", first, B), _index("cu", cu, B + 1), B, T, _raw_stream(stream, k_out))
    if rc:
        raise Q4Error("q4_kv_gather", rc)


def q4_kv_attention(out, q, cache: KVCache, page_table, kv_len, cu_q, max_q: int, max_kv: int,
                    total_kv: int = 0, scale: float | None = None, causal: bool = True,
                    window: int = 0, workspace=None, stream=None, sinks: int = 0, tree=None,
                    lse=None) -> None:
    """Attention of the new tokens' queries q [T, Hq, dim] over the cached
    tokens into out [T, Hq, dim] (include/q4.h).  scale: dim ** -0.5 by default.
    sinks: first tokens that a window leaves visible.  tree: int32 [T, words],
    the bits of the new tokens that each one sees.  lse: fp32 [T, Hq] (out), the
    logarithm of each row's sum of exponentials."""
    T, Hq, dim = q.shape
    B = kv_len.shape[0]
    qp, qs = _rows(q, Hq, cache.dim)
    op, out_dtype = _out("out", out, T * Hq * dim)
    q_dtype = _FLOAT_CODES.get(q.dtype)
    if q_dtype is None:
        raise TypeError(f"unsupported dtype {q.dtype}")
    ws, ws_bytes = None, 0
    if workspace is not None:
        _require_cuda(workspace)
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    pages, cols = _table(page_table, B)
    tree_ptr, words = None, 0
    if tree is not None:
        tree_ptr, words = _words("tree", tree, T)
    rc = lib().q4_kv_attention_ex(
        op, out_dtype, qp, q_dtype, qs, Hq, cache.ref,
        pages, cols,
        _index("kv_len", kv_len, B), _index("cu_q", cu_q, B + 1), B, T, max_q, max_kv, total_kv,
        dim ** -0.5 if scale is None else scale, 1 if causal else 0, window, sinks, tree_ptr, words,
        _floats("lse", lse, T * Hq), ws, ws_bytes, _raw_stream(stream, q))
    if rc:
        raise Q4Error("q4_kv_attention", rc)


def q4_kv_attention_workspace_size(cache: KVCache, Hq: int, B: int, T: int, max_q: int,
                                   max_kv: int, total_kv: int = 0) -> int:
    return lib().q4_kv_attention_workspace_size(cache.ref, Hq, B, T, max_q, max_kv, total_kv)


def q4_kv_weigh(weight, q, lse, cache: KVCache, page_table, kv_len, cu_q, max_q: int, max_kv: int,
                held=None, scale: float | None = None, causal: bool = True, window: int = 0,
                sinks: int = 0, stream=None) -> None:
    """Adds to weight (fp32 [pages, heads, page_tokens], the cache's slots) the
    attention weight that each cached token gets from the queries q [T, Hq, dim],
    with lse [T, Hq] of q4_kv_attention over the same queries.  held: int32 [B],
    tokens whose weight is kept; the others begin at 0 (default: the new ones).
    Sequences that share pages are weighed by calls of their own: a slot's weight
    comes from one sequence of a call (include/q4.h)."""
    T, Hq, dim = q.shape
    B = kv_len.shape[0]
    qp, qs = _rows(q, Hq, cache.dim)
    q_dtype = _FLOAT_CODES.get(q.dtype)
    if q_dtype is None:
        raise TypeError(f"unsupported dtype {q.dtype}")
    pages, cols = _table(page_table, B)
    rc = lib().q4_kv_weigh(
        _weights(weight, cache), qp, q_dtype, qs, Hq, _floats("lse", lse, T * Hq), cache.ref, pages, cols,
        _index("kv_len", kv_len, B), _index("cu_q", cu_q, B + 1),
        None if held is None else _index("held", held, B), B, T, max_q, max_kv,
        dim ** -0.5 if scale is None else scale, 1 if causal else 0, window, sinks, _raw_stream(stream, q))
    if rc:
        raise Q4Error("q4_kv_weigh", rc)


def _weights(weight, cache):
    """Data pointer of a fp32 tensor of the cache's slots, or None."""
    return _floats("weight", weight, cache.pages * cache.heads * cache.page_tokens)


def q4_kv_select(kept, count, weight, cache: KVCache, page_table, kv_len, budget, max_kv: int,
                 sinks: int = 0, recent: int = 0, stream=None) -> None:
    """The tokens that each head keeps of a budget (int32 [B]): the first `sinks`,
    the last `recent` and the heaviest others, ascending, into kept (int32
    [B, heads, width]); how many, into count (int32 [B])."""
    B, heads, width = kept.shape
    if heads != cache.heads:
        raise ValueError(f"kept has {heads} heads, not {cache.heads}")
    pages, cols = _table(page_table, B)
    rc = lib().q4_kv_select(
        _index("kept", kept, B * heads * width), width, _index("count", count, B), _weights(weight, cache),
        cache.ref, pages, cols, _index("kv_len", kv_len, B), _index("budget", budget, B), B, max_kv, sinks,
        recent, _raw_stream(stream, kept))
    if rc:
        raise Q4Error("q4_kv_select", rc)


def q4_kv_compact(cache: KVCache, page_table, kv_len, kept, count, weight=None, first=None, to_table=None,
                  stream=None) -> None:
    """Moves the tokens kept (int32 [B, 1 or heads, width], ascending; count [B] of
    them) to places first[b] .. (default 0) of their sequences, with their weights,
    within page_table or into the pages of to_table (pages that other sequences
    read stay whole there).  Each sequence then has first + count tokens: kv_len is
    the caller's to set."""
    B, heads, width = kept.shape
    if heads not in (1, cache.heads):
        raise ValueError(f"kept has {heads} heads, neither 1 nor {cache.heads}")
    pages, cols = _table(page_table, B)
    to, to_cols = (None, 0) if to_table is None else _table(to_table, B)
    rc = lib().q4_kv_compact(
        cache.ref, _weights(weight, cache), pages, cols, to, to_cols, _index("kv_len", kv_len, B),
        None if first is None else _index("first", first, B), _index("kept", kept, B * heads * width), heads,
        width, _index("count", count, B), B, _raw_stream(stream, kept))
    if rc:
        raise Q4Error("q4_kv_compact", rc)


def _logit_rows(name, t):
    """Data pointer, dtype code and row stride of a [T, V] view whose rows are dense."""
    n, width = t.shape
    s0, s1 = t.stride()
    dtype = _FLOAT_CODES.get(t.dtype)
    if dtype is None or not t.is_cuda or (s1 != 1 and width > 1):
        raise ValueError(f"{name} is a [T, V] fp32 or bf16 CUDA tensor with dense rows")
    return t.data_ptr(), dtype, s0 if n > 1 else width


def q4_adjust_logits(out, logits, history=None, history_len=None, prompt_len=None, repetition=None,
                     presence=None, frequency=None, bias_index=None, bias=None, request=None, mask=None,
                     mask_row=None, stream=None) -> None:
    """Penalties for the tokens of a history (int32 [requests, width]; history_len
    of them, the first prompt_len a prompt), biases (bias_index int32 and bias fp32
    [requests, n]) and a grammar's bits (mask int32 [masks, words]) on logits
    [T, V], into out (which may be logits).  request, mask_row: int32 [T], each
    row's row of these (include/q4.h)."""
    T, V = logits.shape
    op, out_dtype, out_stride = _logit_rows("out", out)
    lp, dtype, stride = _logit_rows("logits", logits)
    if out.shape != logits.shape:
        raise ValueError("out has the shape of logits")
    hp, hw, bp, bw, requests, mp, masks = None, 0, None, 0, 0, None, 0
    if history is not None:
        hp, hw = _words("history", history)
        requests = history.shape[0]
    if bias_index is not None:
        bp, bw = _words("bias_index", bias_index)
        if history is not None and bias_index.shape[0] != requests:
            raise ValueError("history and bias_index have the same rows")
        requests = bias_index.shape[0]
    if mask is not None:
        mp, words = _words("mask", mask)
        masks = mask.shape[0]
        if words != (V + 31) // 32:
            raise ValueError(f"mask has {words} words a row, not {(V + 31) // 32}")
    rc = lib().q4_adjust_logits(
        op, out_dtype, out_stride, lp, dtype, stride, T, V,
        None if request is None else _index("request", request, T), requests, hp, hw,
        None if history_len is None else _index("history_len", history_len, T),
        None if prompt_len is None else _index("prompt_len", prompt_len, T),
        _floats("repetition", repetition, T), _floats("frequency", frequency, T),
        _floats("presence", presence, T), bp,
        None if bias is None else _floats("bias", bias, requests * bw), bw, mp, masks,
        None if mask_row is None else _index("mask_row", mask_row, T), _raw_stream(stream, logits))
    if rc:
        raise Q4Error("q4_adjust_logits", rc)


def q4_sample(tokens, logits, u, temperature=None, top_k=None, top_p=None, min_p=None, probs=None,
              stream=None) -> None:
    """One token a row of logits [T, V] (fp32 or bf16, rows may be strided),
    from the uniform numbers u [T]; settings are [T] tensors or None."""
    T, V = logits.shape
    s0, s1 = logits.stride()
    dtype = _FLOAT_CODES.get(logits.dtype)
    if dtype is None or not logits.is_cuda or (s1 != 1 and V > 1):
        raise ValueError("logits is a [T, V] fp32 or bf16 CUDA tensor with dense rows")
    rc = lib().q4_sample(
        _index("tokens", tokens, T), _floats("probs", probs, T), logits.data_ptr(), dtype,
        s0 if T > 1 else V, T, V, _floats("u", u, T), _floats("temperature", temperature, T),
        None if top_k is None else _index("top_k", top_k, T), _floats("top_p", top_p, T),
        _floats("min_p", min_p, T), _raw_stream(stream, logits))
    if rc:
        raise Q4Error("q4_sample", rc)
