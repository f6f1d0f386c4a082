"""The serving operators beside the matmuls: the paged 8-bit key/value cache,
attention over it, and sampling (include/q4.h, "Serving").  Reached through the
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
                 stream=None) -> None:
    """New tokens' keys and values into the cache, their queries rotated into
    q_out (include/q4.h).  q [T, Hq, dim], k, v [T, heads, dim]: views whose
    rows may be strided; q and q_out may both be None.  cos, sin: fp32
    [positions, rotated dim / 2], or None."""
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
    rc = lib().q4_kv_append(
        cache.ref, out, out_dtype, qp, qs, kp, ks, vp, vs, dtype, Hq, rope,
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
                    window: int = 0, workspace=None, stream=None) -> None:
    """Attention of the new tokens' queries q [T, Hq, dim] over the cached
    tokens into out [T, Hq, dim] (include/q4.h).  scale: dim ** -0.5 by default."""
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
    rc = lib().q4_kv_attention(
        op, out_dtype, qp, q_dtype, qs, Hq, cache.ref,
        pages, cols,
        _index("kv_len", kv_len, B), _index("cu_q", cu_q, B + 1), B, T, max_q, max_kv, total_kv,
        dim ** -0.5 if scale is None else scale, 1 if causal else 0, window, ws, ws_bytes,
        _raw_stream(stream, q))
    if rc:
        raise Q4Error("q4_kv_attention", rc)


def q4_kv_attention_workspace_size(cache: KVCache, Hq: int, B: int, T: int, max_q: int,
                                   max_kv: int, total_kv: int = 0) -> int:
    return lib().q4_kv_attention_workspace_size(cache.ref, Hq, B, T, max_q, max_kv, total_kv)


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
