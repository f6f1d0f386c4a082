"""GB300 (sm_103a) Q4_0 weight-only dequant-matmul and the serving operators
beside it (paged 8-bit key/value cache, attention, sampling): the Python binding.

A thin ctypes layer over the C ABI declared in ``include/q4.h``.  Every
function marshals arguments only (device pointers, sizes, the current torch
stream) and calls the library; all arithmetic runs in the CUDA kernels.
PyTorch provides device memory and streams.

If the compiled library is missing, importing this package raises: there is
no CPU fallback.
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch as _torch

from . import _build

Q4_OK = 0
Q4_ERR_ARG = -1
Q4_ERR_DTYPE = -2
Q4_ERR_ALIGN = -3
Q4_ERR_CUDA = -4
Q4_ERR_WORKSPACE = -5
Q4_ERR_SHAPE = -6
Q4_ERR_DEVICE = -7
Q4_DEVERR_INDEX = 0x1
Q4_DEVERR_TIMEOUT = 0x2
Q4_DEVERR_VALUE = 0x4
Q4_F32 = 0
Q4_BF16 = 1
Q4_LAYOUT_BLOCKS = 0
Q4_LAYOUT_PLANAR = 1
Q4_LAYOUT_Q8_0 = 2
Q4_KV_BLOCK = 16
Q4_ROPE_HALVES = 0
Q4_ROPE_PAIRS = 1

_lock = threading.Lock()
_lib = None

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t
_int = ctypes.c_int


class SeqOp(ctypes.Structure):
    """q4_seq_op of include/q4.h: one matmul of a host-streamed sequence."""
    _fields_ = [("C", ctypes.c_void_p), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("a_dtype", ctypes.c_int), ("c_dtype", ctypes.c_int)]


class GemvOp(ctypes.Structure):
    """q4_gemv_op of include/q4.h: one M = 1 GEMV of a decode sequence."""
    _fields_ = [("C", ctypes.c_void_p), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("a_dtype", ctypes.c_int), ("c_dtype", ctypes.c_int),
                ("ndeps", ctypes.c_int), ("deps", ctypes.c_int * 4), ("slice_rows", ctypes.c_int)]


class KvCacheStruct(ctypes.Structure):
    """q4_kv_cache of include/q4.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("page_tokens", ctypes.c_int64)]


class RopeStruct(ctypes.Structure):
    """q4_rope of include/q4.h."""
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("style", ctypes.c_int)]


# name -> (restype, argtypes), as declared in include/q4.h
SIGNATURES = {
    "q4_matmul": (_int, [_vp, _vp, _vp, _i64, _i64, _i64]),
    "q4_matmul_ex": (_int, [_vp, _int, _vp, _int, _vp, _int, _i64, _i64, _i64, _vp, _sz, _vp]),
    "q4_matmul_workspace_size": (_sz, [_i64, _i64, _i64]),
    "q4_matmul_bf16_tiles": (_int, [_vp, _int, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp]),
    "q4_release_scratch": (_int, []),
    "q4_moe_experts": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64]),
    "q4_moe_experts_ex": (_int, [_vp, _vp, _int, _vp, _vp, _vp, _vp, _vp,
                                 _i64, _i64, _i64, _i64, _i64, _vp, _sz, _vp]),
    "q4_moe_workspace_size": (_sz, [_i64, _i64, _i64, _i64, _i64]),
    "q4_moe_experts_trace": (_int, [_vp, _vp, _int, _vp, _vp, _vp, _vp, _vp,
                                    _i64, _i64, _i64, _i64, _i64, _vp, _sz,
                                    _vp, _vp, _vp, _vp, _vp]),
    "q4_moe_experts_noalloc": (_int, [_vp, _vp, _int, _vp, _vp, _vp, _vp, _vp,
                                      _i64, _i64, _i64, _i64, _i64, _vp]),
    "q4_moe_static_scratch_bytes": (_sz, []),
    "q4_repack": (_int, [_vp, _vp, _i64, _i64, _vp]),
    "q4_unpack": (_int, [_vp, _vp, _i64, _i64, _vp]),
    "q4_planar_qs_offset": (_sz, [_i64, _i64]),
    "q4_planar_bytes": (_sz, [_i64, _i64]),
    "q4_dequant": (_int, [_vp, _vp, _i64, _i64, _vp]),
    "q4_dequant_bf16": (_int, [_vp, _vp, _i64, _i64, _vp]),
    "q4_quantize": (_int, [_vp, _vp, _int, _i64, _i64, _vp]),
    "q4_moe_gate": (_int, [_vp, _vp, _vp, _i64, _i64, _i64, _vp]),
    "q4_moe_block": (_int, [_vp, _vp, _int, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64,
                            _vp, _vp, _vp, _i64, _vp, _sz, _vp]),
    "q4_moe_block_workspace_size": (_sz, [_i64, _i64, _i64, _i64, _i64, _i64]),
    "q4_selftest_wait": (_int, [_i64, _int, _vp]),
    "q4_prefill_units": (_i64, [_i64, _i64, _i64, _int, _vp, _i64]),
    "q4_host_stream_slot_bytes": (_sz, [ctypes.POINTER(SeqOp), _int]),
    "q4_matmul_host_stream": (_int, [ctypes.POINTER(SeqOp), _int, _vp, _sz, _int, _vp, _vp]),
    "q4_gemv_seq_bytes": (_sz, [ctypes.POINTER(GemvOp), _int]),
    "q4_gemv_seq_create": (_int, [ctypes.POINTER(GemvOp), _int, _vp, _sz,
                                  ctypes.POINTER(ctypes.c_void_p)]),
    "q4_gemv_seq_run": (_int, [_vp, _vp]),
    "q4_gemv_seq_destroy": (None, [_vp]),
    "q4_gemv_seq_grid": (_int, [_vp]),
    "q4_kv_append": (_int, [_vp, _vp, _int, _vp, _i64, _vp, _i64, _vp, _i64, _int, _i64, _vp,
                            _vp, _vp, ctypes.c_float, _vp, _i64, _vp, _vp, _i64, _i64, _vp]),
    "q4_kv_gather": (_int, [_vp, _vp, _int, _vp, _vp, _i64, _vp, _vp, _i64, _i64, _vp]),
    "q4_kv_attention": (_int, [_vp, _int, _vp, _int, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64,
                               _i64, _i64, _i64, _i64, ctypes.c_float, _int, _i64, _vp, _sz, _vp]),
    "q4_kv_attention_workspace_size": (_sz, [_vp, _i64, _i64, _i64, _i64, _i64, _i64]),
    "q4_sample": (_int, [_vp, _vp, _vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "q4_get_device_status": (_int, [_vp]),
    "q4_last_device_flags": (ctypes.c_uint, []),
    "q4_status_str": (ctypes.c_char_p, [_int]),
    "q4_version": (_int, []),
}


class Q4Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status} ({status_str(status)})")
        self.status = status


def library_path() -> str:
    return _build.LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded C library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.LIB_PATH
            if not os.path.exists(path):
                raise ImportError(
                    f"{path} is missing: build it with quantized_weight_q4_gb300._build.build() "
                    "(or __graft_entry__.build()); there is no CPU fallback")
            L = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
        return _lib


def status_str(status: int) -> str:
    return lib().q4_status_str(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != Q4_OK:
        raise Q4Error(fn, status)


# ------------------------------------------------------------------ helpers
def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int | None:
    """cudaStream_t of a torch stream (default: torch's current stream)."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream or None


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return Q4_F32
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return Q4_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")


# ------------------------------------------------------------------ entry points
def q4_matmul(C, A, B, M: int, N: int, K: int) -> None:
    """C = A . W (fp32 A and C, legacy default stream), as the C entry point."""
    _require_cuda(C, A, B)
    _check("q4_matmul", lib().q4_matmul(_ptr(C), _ptr(A), _ptr(B), M, N, K))


def q4_matmul_ex(C, A, B, M: int, N: int, K: int, workspace=None, stream=None,
                 b_layout: int = Q4_LAYOUT_BLOCKS) -> None:
    _require_cuda(C, A, B, workspace)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("q4_matmul_ex", lib().q4_matmul_ex(
        _ptr(C), _dtype_code(C), _ptr(A), _dtype_code(A), _ptr(B), b_layout,
        M, N, K, _ptr(workspace), ws_bytes, _stream(stream)))


def q4_matmul_bf16_tiles(C, A, B, M: int, N: int, K: int, workspace=None, stream=None) -> None:
    """C = A . bf16_rn(W) on the tensor cores (bf16 A), whatever K."""
    _require_cuda(C, A, B, workspace)
    if _dtype_code(A) != Q4_BF16:
        raise TypeError("q4_matmul_bf16_tiles takes bf16 activations")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("q4_matmul_bf16_tiles", lib().q4_matmul_bf16_tiles(
        _ptr(C), _dtype_code(C), _ptr(A), _ptr(B), M, N, K, _ptr(workspace), ws_bytes,
        _stream(stream)))


def q4_release_scratch() -> None:
    """Frees the library-owned scratch and workspaces of the current device."""
    _check("q4_release_scratch", lib().q4_release_scratch())


def _seq_ops(ops):
    """ops: list of (C, A, B_host, M, N, K): C and A CUDA tensors, B a pinned CPU tensor."""
    arr = (SeqOp * len(ops))()
    for i, (C, A, B, M, N, K) in enumerate(ops):
        _require_cuda(C, A)
        arr[i] = SeqOp(_ptr(C), _ptr(A), B.data_ptr(), M, N, K, _dtype_code(A), _dtype_code(C))
    return arr


def q4_host_stream_slot_bytes(ops) -> int:
    return lib().q4_host_stream_slot_bytes(_seq_ops(ops), len(ops))


def q4_matmul_host_stream(ops, staging, slots: int, stream=None, copy_stream=None) -> None:
    """Runs ops [(C, A, B_host, M, N, K), ...] in order on `stream`, copying each
    pinned host B into one of `slots` slots of the device buffer `staging` on
    `copy_stream` while earlier matmuls run."""
    _require_cuda(staging)
    arr = _seq_ops(ops)
    nbytes = staging.numel() * staging.element_size()
    _check("q4_matmul_host_stream", lib().q4_matmul_host_stream(
        arr, len(ops), _ptr(staging), nbytes, slots, _stream(stream), _stream(copy_stream)))


def _gemv_ops(ops, slice_rows=0):
    arr = (GemvOp * len(ops))()
    for i, op in enumerate(ops):
        C, A, B, N, K = op[:5]
        deps = list(op[5]) if len(op) > 5 else []
        _require_cuda(C, A, B)
        if len(deps) > 4:
            raise ValueError("at most 4 dependencies per op")
        d = (ctypes.c_int * 4)(*(deps + [0] * (4 - len(deps))))
        arr[i] = GemvOp(_ptr(C), _ptr(A), _ptr(B), N, K, _dtype_code(A), _dtype_code(C),
                        len(deps), d, slice_rows)
    return arr


class GemvSequence:
    """A decode sequence of M = 1 GEMVs run by one persistent launch
    (q4_gemv_seq_*).  ops: list of (C, A, B, N, K) or (C, A, B, N, K, deps),
    CUDA tensors, deps a list of indices of earlier ops whose C must be
    complete before this op reads A.  slice_rows: rows per unit of work for
    every op, a multiple of 64 up to 4096 (0: the library's choice, which
    shortens the units of ops that others wait for and of the sequence's
    last weights).  The tensors are referenced by the
    plan and kept alive with it."""

    def __init__(self, ops, slice_rows: int = 0):
        import torch
        self.ops = list(ops)
        arr = _gemv_ops(self.ops, slice_rows)
        L = lib()
        nbytes = L.q4_gemv_seq_bytes(arr, len(self.ops))
        if nbytes == 0:
            raise Q4Error("q4_gemv_seq_bytes", Q4_ERR_ARG)
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=self.ops[0][0].device)
        plan = ctypes.c_void_p()
        _check("q4_gemv_seq_create", L.q4_gemv_seq_create(arr, len(self.ops), _ptr(self.buf),
                                                          nbytes, ctypes.byref(plan)))
        self.plan = plan

    def run(self, stream=None) -> None:
        _check("q4_gemv_seq_run", lib().q4_gemv_seq_run(self.plan, _stream(stream)))

    @property
    def grid(self) -> int:
        return lib().q4_gemv_seq_grid(self.plan)

    def __del__(self):
        plan = getattr(self, "plan", None)
        if plan is not None and _lib is not None:
            _lib.q4_gemv_seq_destroy(plan)
            self.plan = None


def q4_matmul_workspace_size(M: int, N: int, K: int) -> int:
    return lib().q4_matmul_workspace_size(M, N, K)


def q4_moe_experts(out, x, W_gate, W_up, W_down, topk_idx, topk_w, T: int, E: int, H: int,
                   I: int) -> None:
    _require_cuda(out, x, W_gate, W_up, W_down, topk_idx, topk_w)
    _check("q4_moe_experts", lib().q4_moe_experts(
        _ptr(out), _ptr(x), _ptr(W_gate), _ptr(W_up), _ptr(W_down), _ptr(topk_idx),
        _ptr(topk_w), T, E, H, I))


def q4_moe_experts_ex(out, x, W_gate, W_up, W_down, topk_idx, topk_w, T: int, topk: int, E: int,
                      H: int, I: int, workspace=None, stream=None) -> None:
    _require_cuda(out, x, W_gate, W_up, W_down, topk_idx, topk_w, workspace)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("q4_moe_experts_ex", lib().q4_moe_experts_ex(
        _ptr(out), _ptr(x), _dtype_code(x), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
        _ptr(topk_idx), _ptr(topk_w), T, topk, E, H, I, _ptr(workspace), ws_bytes,
        _stream(stream)))


def q4_moe_experts_trace(out, x, W_gate, W_up, W_down, topk_idx, topk_w, T: int, topk: int,
                         E: int, H: int, I: int, workspace, g, u, h, y, stream=None) -> None:
    """q4_moe_experts_ex that also writes g, u, h [T*topk, I] and y [T*topk, H]."""
    _require_cuda(out, x, W_gate, W_up, W_down, topk_idx, topk_w, workspace, g, u, h, y)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("q4_moe_experts_trace", lib().q4_moe_experts_trace(
        _ptr(out), _ptr(x), _dtype_code(x), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
        _ptr(topk_idx), _ptr(topk_w), T, topk, E, H, I, _ptr(workspace), ws_bytes,
        _ptr(g), _ptr(u), _ptr(h), _ptr(y), _stream(stream)))


def q4_moe_workspace_size(T: int, topk: int, E: int, H: int, I: int) -> int:
    return lib().q4_moe_workspace_size(T, topk, E, H, I)


def q4_moe_experts_noalloc(out, x, W_gate, W_up, W_down, topk_idx, topk_w, T: int, topk: int,
                           E: int, H: int, I: int, stream=None) -> None:
    """Routed experts with the library's built-in scratch: no device memory
    is allocated, for callers that cannot allocate (see include/q4.h)."""
    _require_cuda(out, x, W_gate, W_up, W_down, topk_idx, topk_w)
    _check("q4_moe_experts_noalloc", lib().q4_moe_experts_noalloc(
        _ptr(out), _ptr(x), _dtype_code(x), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
        _ptr(topk_idx), _ptr(topk_w), T, topk, E, H, I, _stream(stream)))


def q4_quantize(B, W, K: int, N: int, stream=None) -> None:
    """Q4_0 blocks of W (fp32 or bf16) into B (uint8 [K, ceil(N/32)*18])."""
    _require_cuda(B, W)
    _check("q4_quantize", lib().q4_quantize(_ptr(B), _ptr(W), _dtype_code(W), K, N,
                                            _stream(stream)))


def q4_moe_gate(topk_idx, topk_w, logits, T: int, E: int, topk: int, stream=None) -> None:
    _require_cuda(topk_idx, topk_w, logits)
    _check("q4_moe_gate", lib().q4_moe_gate(_ptr(topk_idx), _ptr(topk_w), _ptr(logits), T, E,
                                            topk, _stream(stream)))


def q4_moe_block(out, x, logits, W_gate, W_up, W_down, T: int, topk: int, E: int, H: int, I: int,
                 S_gate=None, S_up=None, S_down=None, Is: int = 0, workspace=None,
                 stream=None) -> None:
    """Router + shared expert + routed experts of one MoE block (include/q4.h)."""
    _require_cuda(out, x, logits, W_gate, W_up, W_down, S_gate, S_up, S_down, workspace)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("q4_moe_block", lib().q4_moe_block(
        _ptr(out), _ptr(x), _dtype_code(x), _ptr(logits), _ptr(W_gate), _ptr(W_up),
        _ptr(W_down), T, topk, E, H, I, _ptr(S_gate), _ptr(S_up), _ptr(S_down), Is,
        _ptr(workspace), ws_bytes, _stream(stream)))


def q4_moe_block_workspace_size(T: int, topk: int, E: int, H: int, I: int, Is: int = 0) -> int:
    return lib().q4_moe_block_workspace_size(T, topk, E, H, I, Is)


# ------------------------------------------------------------------ serving
# The serving calls are made once a token and layer, so their checks are kept
# short: one attribute at a time, nothing looked up twice.
_FLOAT_CODES = {_torch.float32: Q4_F32, _torch.bfloat16: Q4_BF16}


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
        if k.dtype is not _torch.int8 or v.dtype is not _torch.int8 or v.shape != shape:
            raise TypeError("k and v are int8 tensors of one shape")
        if (k_scale.dtype is not _torch.float32 or v_scale.dtype is not _torch.float32
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
        torch = _torch
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
    if t.dtype is not _torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} is a contiguous int32 CUDA tensor")
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, not {n}")
    return t.data_ptr()


def _table(t, n):
    """Data pointer and columns of a contiguous int32 CUDA tensor of n rows."""
    if t.dtype is not _torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError("page_table is a contiguous int32 CUDA tensor")
    rows, cols = t.shape
    if rows != n:
        raise ValueError(f"page_table has {rows} rows, not {n}")
    return t.data_ptr(), cols


def _floats(name, t, n):
    """Data pointer of a contiguous fp32 CUDA tensor of n elements, or None."""
    if t is None:
        return None
    if t.dtype is not _torch.float32 or t.numel() != n or not t.is_cuda or not t.is_contiguous():
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
        return _torch._C._cuda_getCurrentRawStream(t.get_device()) or None
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


def q4_moe_static_scratch_bytes() -> int:
    return lib().q4_moe_static_scratch_bytes()


def q4_repack(dst, src, K: int, N: int, stream=None) -> None:
    _require_cuda(dst, src)
    _check("q4_repack", lib().q4_repack(_ptr(dst), _ptr(src), K, N, _stream(stream)))


def q4_unpack(dst, src, K: int, N: int, stream=None) -> None:
    _require_cuda(dst, src)
    _check("q4_unpack", lib().q4_unpack(_ptr(dst), _ptr(src), K, N, _stream(stream)))


def q4_planar_qs_offset(K: int, N: int) -> int:
    return lib().q4_planar_qs_offset(K, N)


def q4_planar_bytes(K: int, N: int) -> int:
    return lib().q4_planar_bytes(K, N)


def q4_dequant(W, B, K: int, N: int, stream=None) -> None:
    _require_cuda(W, B)
    _check("q4_dequant", lib().q4_dequant(_ptr(W), _ptr(B), K, N, _stream(stream)))


def q4_dequant_bf16(W, B, K: int, N: int, stream=None) -> None:
    _require_cuda(W, B)
    _check("q4_dequant_bf16", lib().q4_dequant_bf16(_ptr(W), _ptr(B), K, N, _stream(stream)))


def q4_selftest_wait(limit_ns: int, arrive: bool, stream=None) -> None:
    """One bounded pipeline wait run to its limit (arrive=False) or completed."""
    _check("q4_selftest_wait", lib().q4_selftest_wait(int(limit_ns), 1 if arrive else 0,
                                                      _stream(stream)))


def q4_prefill_units(M: int, N: int, K: int, sms: int):
    """The prefill form's units per CTA for this shape on `sms` SMs (host
    only): an int32 array [units, 9] of (CTA, unit, m0, n0, first K step,
    end K step, role, first helper CTA, helper count)."""
    import numpy as np
    L = lib()
    n = L.q4_prefill_units(M, N, K, sms, None, 0)
    if n < 0:
        raise Q4Error("q4_prefill_units", int(n))
    out = np.zeros((max(n, 1), 9), dtype=np.int32)
    got = L.q4_prefill_units(M, N, K, sms, out.ctypes.data, n)
    if got != n:
        raise Q4Error("q4_prefill_units", int(got))
    return out[:n]


def q4_get_device_status(stream=None) -> int:
    return lib().q4_get_device_status(_stream(stream))


def q4_last_device_flags() -> int:
    return lib().q4_last_device_flags()


def q4_version() -> int:
    return lib().q4_version()
