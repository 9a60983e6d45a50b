"""The decode-step operators in front of the sampler: per-head norm and rotation, the paged key/value
cache and the attention of a batch that shares a long prefix.  Like the rest of the binding these
functions only check tensors and hand pointers and the CUDA stream to the C ABI (``include/tps.h``); the
checking is native code too (``csrc/tps_torch.cpp``), because in Python it takes longer than a decode step's
kernels."""
from __future__ import annotations

import contextlib
import ctypes
import threading

import torch

_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class _NormRope(ctypes.Structure):  # tps_norm_rope
    _fields_ = ([(n, _P) for n in ("q", "k", "out_q", "out_k")]
                + [(n, _I64) for n in ("q_ld", "q_hd", "k_ld", "k_hd", "oq_ld", "oq_hd", "ok_ld", "ok_hd")]
                + [(n, _P) for n in ("q_weight", "k_weight", "positions", "cos_sin", "out_status")]
                + [(n, _I64) for n in ("T", "n_positions")]
                + [(n, _I32) for n in ("n_q_heads", "n_k_heads", "head_dim", "rot_dim", "interleaved", "dtype")]
                + [("eps", ctypes.c_float)])


class _Cache(ctypes.Structure):  # tps_kv_cache
    _fields_ = ([(n, _P) for n in ("k", "v", "k_scale", "v_scale")] + [("n_pages", _I64)]
                + [(n, _I32) for n in ("n_heads", "page_size", "head_dim", "format")])


class _Attention(ctypes.Structure):  # tps_attention
    _fields_ = ([(n, _P) for n in ("q", "out", "out_lse", "prefix_pages", "page_table", "suffix_len", "out_status",
                                   "workspace")]
                + [(n, _I64) for n in ("workspace_bytes", "B", "prefix_len", "table_width", "table_ld")]
                + [("q_len", _I32), ("n_q_heads", _I32), ("scale", ctypes.c_float)])


def declare(lib):
    """The argument and result types of this module's entry points."""
    lib.tps_qk_norm_rope.restype = ctypes.c_int
    lib.tps_qk_norm_rope.argtypes = [_P, _P]
    lib.tps_kv_write.restype = ctypes.c_int
    lib.tps_kv_write.argtypes = [_P, _P, _P, ctypes.c_int, _I64, _I64, _I64, _I64, _I64, _P, _P]
    lib.tps_kv_read.restype = ctypes.c_int
    lib.tps_kv_read.argtypes = [_P, _P, _I64, _P, _P, ctypes.c_int, _P]
    lib.tps_prefix_attention.restype = ctypes.c_int
    lib.tps_prefix_attention.argtypes = [_P, _P, _P]
    lib.tps_prefix_attention_stall_test.restype = ctypes.c_int
    lib.tps_prefix_attention_stall_test.argtypes = [_P, _P, ctypes.c_int, ctypes.c_uint64, _P]
    lib.tps_prefix_attention_workspace.restype = _I64
    lib.tps_prefix_attention_workspace.argtypes = [_P, _P]


_Tensor = torch.Tensor
_ops = None  # the native module once it is bound: other threads read this without the lock
_ops_lock = threading.Lock()


def _torch_ops():
    """The native module that checks tensors and calls the library (csrc/tps_torch.cpp), loaded with it."""
    global _ops
    with _ops_lock:
        if _ops is None:
            from . import load, load_binding
            lib = load()
            ops = load_binding()
            address = lambda f: ctypes.cast(f, ctypes.c_void_p).value
            ops.bind(address(lib.tps_qk_norm_rope), address(lib.tps_kv_write), address(lib.tps_kv_read),
                     address(lib.tps_prefix_attention), _fail, torch.OutOfMemoryError)
            _ops = ops
        return _ops


def _fail(rc, name):
    from . import _ERRORS, load
    extra = f" (cudaError {load().tps_last_cuda_error()})" if rc == 5 else ""
    raise RuntimeError(f"{name} failed: {_ERRORS.get(rc, rc)}{extra}")


def _on(stream, device):
    """Run on `stream`: what the call allocates and launches there goes there."""
    both = contextlib.ExitStack()
    both.enter_context(torch.cuda.device(device))
    both.enter_context(torch.cuda.stream(stream))
    return both


def _cache(cache):
    if not isinstance(cache, KVCache):
        raise ValueError("cache must be a KVCache")
    return cache


def _dense(t, name, shape, dtype, device):
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def qk_norm_rope(q, k, q_weight, k_weight, positions, cos_sin, *, eps: float = 1e-6, interleaved: bool = False,
                 out=None, status=None, stream=None):
    """Root-mean-square norm of each query and key head and the rotation by the token's position, in one
    pass: ``y = x * rsqrt(mean(x^2) + eps) * w`` over a head, then ``(a, b) -> (a cos - b sin,
    b cos + a sin)`` on its first ``cos_sin.shape[1]`` components, in float32, rounded once.

    ``q``: [T, Hq, D], ``k``: [T, Hk, D] CUDA tensors of one dtype (float32 or bfloat16; token and head
    strides are free, so both may be cut out of one projection).  ``q_weight``, ``k_weight``: [D]
    float32, or None.  ``positions``: [T] int32.  ``cos_sin``: [positions, R] float32, cosines then sines
    (R even, at most D; the other components are only normed).  ``interleaved``: pairs are neighbours
    (2i, 2i + 1) rather than (i, i + R/2).  ``out``: a (q, k) pair to write to (the inputs themselves to
    work in place), else new tensors.  ``status``: an int32 [T] tensor that gets 3 for a token whose
    position is not in the table (its outputs are NaN), else 0.  Returns (q, k)."""
    ops = _ops or _torch_ops()
    if stream is not None:
        with _on(stream, q.device):
            return ops.norm(q, k, q_weight, k_weight, positions, cos_sin, eps, interleaved, out, status)
    return ops.norm(q, k, q_weight, k_weight, positions, cos_sin, eps, interleaved, out, status)


class KVCache:
    """A paged key/value cache of one layer: ``k`` and ``v`` [pages, heads, page_size, head_dim], of
    bfloat16 values or of 8-bit codes (float8_e4m3fn, int8) with one bfloat16 scale per (token, head) in
    ``k_scale`` and ``v_scale`` [pages, heads, page_size].  Token slot s lives in page s // page_size at
    row s % page_size.  The tensors belong to the caller; ``KVCache.empty`` makes new ones.  A cache keeps the
    tensors it was made with (the calls hold their addresses): for others make another cache."""

    FORMATS = {"bf16": (0, torch.bfloat16), "fp8": (1, torch.float8_e4m3fn), "int8": (2, torch.int8)}

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if not isinstance(k, torch.Tensor) or not k.is_cuda or k.dim() != 4:
            raise ValueError("k must be a CUDA tensor [pages, heads, page_size, head_dim]")
        self.format = next((f for f, (_, dt) in self.FORMATS.items() if dt == k.dtype), None)
        if self.format is None:
            raise TypeError(f"a cache holds bfloat16, float8_e4m3fn or int8, got {k.dtype}")
        pages, heads, page, D = k.shape
        if page not in (16, 32, 64, 128, 256):
            raise ValueError("page_size must be 16, 32, 64, 128 or 256")
        if D % 16 or not 16 <= D <= 512:
            raise ValueError("head_dim must be a multiple of 16, at most 512")
        if pages < 1 or heads < 1:
            raise ValueError("a cache holds at least one page and one head")
        dev = k.device
        _dense(k, "k", (pages, heads, page, D), k.dtype, dev)
        _dense(v, "v", (pages, heads, page, D), k.dtype, dev)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if self.format == "bf16":
                if t is not None:
                    raise ValueError(f"{name}: a bfloat16 cache has no scales")
            else:
                _dense(t, name, (pages, heads, page), torch.bfloat16, dev)
        self._k, self._v, self._k_scale, self._v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_heads, self.page_size, self.head_dim = pages, heads, page, D
        self.device = k.device
        ptr = lambda t: None if t is None else t.data_ptr()
        self._index = dev.index
        self._bytes = bytes(_Cache(ptr(k), ptr(v), ptr(k_scale), ptr(v_scale), pages, heads, page, D, self.FORMATS[self.format][0]))

    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    k_scale = property(lambda self: self._k_scale)
    v_scale = property(lambda self: self._v_scale)

    @classmethod
    def empty(cls, n_pages: int, n_heads: int, page_size: int, head_dim: int, format: str = "fp8", device="cuda"):
        """A cache with tensors of its own; nothing is stored in it yet (its slots read as zeros)."""
        if format not in cls.FORMATS:
            raise ValueError(f"format must be one of {sorted(cls.FORMATS)}")
        shape = (n_pages, n_heads, page_size, head_dim)
        bits = torch.int16 if format == "bf16" else torch.uint8
        k, v = (torch.zeros(shape, dtype=bits, device=device).view(cls.FORMATS[format][1]) for _ in range(2))
        ks, vs = (None if format == "bf16" else torch.zeros(shape[:3], dtype=torch.bfloat16, device=device)
                  for _ in range(2))
        return cls(k, v, ks, vs)


def kv_write(cache: KVCache, k, v, slots, *, stream=None) -> None:
    """Store T tokens: ``k``, ``v`` [T, heads, head_dim] (float32 or bfloat16, token and head strides
    free) at the slots ``slots`` ([T] int64).  8-bit caches get codes and a scale per (token, head); a
    slot outside the cache is skipped (-1 pads).  Slots of one call must differ from one another."""
    c = _cache(cache)
    ops = _ops or _torch_ops()
    if stream is not None:
        with _on(stream, c.device):
            return ops.write(c._bytes, c._index, k, v, slots)
    return ops.write(c._bytes, c._index, k, v, slots)


def kv_read(cache: KVCache, slots, *, dtype=torch.bfloat16, out=None, stream=None):
    """The stored values of the slots ``slots`` ([T] int64) as (k, v), [T, heads, head_dim] of ``dtype``
    (float32 or bfloat16); a slot outside the cache reads as zeros.  ``out``: a (k, v) pair to write to."""
    c = _cache(cache)
    ops = _ops or _torch_ops()
    if dtype is torch.bfloat16:
        code = 1
    elif dtype is torch.float32:
        code = 0
    else:
        raise TypeError(f"values are read as float32 or bfloat16, not {dtype}")
    if stream is not None:
        with _on(stream, c.device):
            return ops.read(c._bytes, c._index, slots, code, out)
    return ops.read(c._bytes, c._index, slots, code, out)


def prefix_attention(q, cache: KVCache, prefix_pages, prefix_len: int, page_table, suffix_len, *, scale=None,
                     want_lse: bool = False, out=None, status=None, workspace=None, stream=None):
    """Softmax attention of a batch of sequences over ``prefix_len`` tokens that all of them share (in the
    pages ``prefix_pages``, int32) and over each sequence's own tokens (in the pages of its row of
    ``page_table``, [B, W] int32; ``suffix_len``, [B] int32, counts them, the query tokens among them).
    The products with the shared keys and values are computed once for the whole batch.

    ``q``: [B, Hq, D] (decode: one token each) or [B, Tq, Hq, D] bfloat16, contiguous; Hq is a multiple
    of the cache's heads, D 64 or 128.  Query t sees the whole prefix and the first
    ``suffix_len - Tq + 1 + t`` own tokens.  ``scale``: of q.k, by default D ** -0.5.  Returns the
    bfloat16 output of q's shape, or (output, log-sum-exp) with ``want_lse`` (float32, q's shape without
    D).  A query that sees no token yields 0 and -inf.  ``status``: an int32 [B] tensor that gets 3 for a
    sequence with a page outside the cache or a length outside its table (its outputs are NaN), 4 where a
    wait on the GPU ran out for any of its heads (their outputs are NaN), else 0.
    ``workspace``: a uint8 tensor of at least ``prefix_attention_workspace(...)`` bytes to use instead of
    the library's memory pool."""
    c = _cache(cache)
    ops = _ops or _torch_ops()
    if stream is not None:
        with _on(stream, c.device):
            return ops.attention(q, c._bytes, c._index, prefix_pages, prefix_len, page_table, suffix_len, scale, want_lse,
                                 out, status, workspace)
    return ops.attention(q, c._bytes, c._index, prefix_pages, prefix_len, page_table, suffix_len, scale, want_lse, out, status,
                         workspace)


def prefix_attention_workspace(q_shape, cache: KVCache, prefix_len: int, table_width: int) -> int:
    """Bytes of workspace ``prefix_attention`` needs for a query of this shape."""
    B, Hq = q_shape[0], q_shape[-2]
    from . import load
    a = _Attention(B=B, prefix_len=int(prefix_len), table_width=table_width, table_ld=table_width,
                   q_len=q_shape[1] if len(q_shape) == 4 else 1, n_q_heads=Hq, scale=1.0)
    n = load().tps_prefix_attention_workspace(_cache(cache)._bytes, ctypes.byref(a))
    if n < 0:
        raise ValueError("arguments that prefix_attention would refuse")
    return n
