"""The decode-step operators in front of the sampler: per-head norm and rotation, the paged key/value
cache and the attention of a batch that shares a long prefix.  Like the rest of the binding these
functions only check tensors and hand pointers and the CUDA stream to the C ABI (``include/tps.h``)."""
from __future__ import annotations

import contextlib
import ctypes

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
    lib.tps_prefix_attention_workspace.restype = _I64
    lib.tps_prefix_attention_workspace.argtypes = [_P, _P]


_SAME = contextlib.nullcontext()


def _on(dev, stream):
    """The context a call allocates and launches in, and the raw stream.  A call on the current device
    and stream, the usual one, enters nothing: the two context managers cost several microseconds."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev.index)
        return (_SAME if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)), raw
    both = contextlib.ExitStack()
    both.enter_context(torch.cuda.device(dev))
    both.enter_context(torch.cuda.stream(stream))
    return both, stream.cuda_stream


def _lib():
    from . import load
    return load()


def _check(rc, name):
    if rc != 0:
        from . import _ERRORS
        lib = _lib()
        extra = f" (cudaError {lib.tps_last_cuda_error()})" if rc == 5 else ""
        raise RuntimeError(f"{name} failed: {_ERRORS.get(rc, rc)}{extra}")


def _code(dt):
    from . import _dtype_code
    return _dtype_code(dt)


def _index(t, name, shape, dtype, dev, dense=True):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != dev or tuple(t.shape) != shape or (
            dense and not t.is_contiguous()):
        raise ValueError(f"{name} must be a{' contiguous' if dense else ''} {dtype} tensor of shape {shape} on {dev}")
    return t.data_ptr()


def _heads(t, name, dev=None, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name} must be [T, heads, head_dim] with unit stride along head_dim")
    if dev is not None and (t.device != dev or t.dtype != dtype):
        raise ValueError(f"{name} must be a {dtype} tensor on {dev}")
    return t


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
    _heads(q, "q")
    dev, dt = q.device, q.dtype
    _heads(k, "k", dev, dt)
    T, Hq, D = q.shape
    Hk = k.shape[1]
    if k.shape[0] != T or k.shape[2] != D:
        raise ValueError("q and k must hold the same tokens and head size")
    if not isinstance(cos_sin, torch.Tensor) or cos_sin.dim() != 2:
        raise ValueError("cos_sin must be a float32 [positions, R] tensor")
    n_pos, R = cos_sin.shape
    if R % 2 or R > D:
        raise ValueError("cos_sin must hold an even number of columns, at most the head size")
    code = _code(dt)
    ctx, raw = _on(dev, stream)
    with ctx:
        if out is None:
            oq, ok = q.new_empty((T, Hq, D)), k.new_empty((T, Hk, D))
        else:
            oq, ok = _heads(out[0], "out[0]", dev, dt), _heads(out[1], "out[1]", dev, dt)
            if oq.shape != q.shape or ok.shape != k.shape:
                raise ValueError("out must have the shapes of q and k")
        a = _NormRope(q.data_ptr(), k.data_ptr(), oq.data_ptr(), ok.data_ptr(), q.stride(0), q.stride(1), k.stride(0),
                      k.stride(1), oq.stride(0), oq.stride(1), ok.stride(0), ok.stride(1),
                      None if q_weight is None else _index(q_weight, "q_weight", (D,), torch.float32, dev),
                      None if k_weight is None else _index(k_weight, "k_weight", (D,), torch.float32, dev),
                      _index(positions, "positions", (T,), torch.int32, dev),
                      _index(cos_sin, "cos_sin", (n_pos, R), torch.float32, dev),
                      None if status is None else _index(status, "status", (T,), torch.int32, dev),
                      T, n_pos, Hq, Hk, D, R, bool(interleaved), code, eps)
        rc = _lib().tps_qk_norm_rope(ctypes.byref(a), raw)
    _check(rc, "tps_qk_norm_rope")
    return oq, ok


class KVCache:
    """A paged key/value cache of one layer: ``k`` and ``v`` [pages, heads, page_size, head_dim], of
    bfloat16 values or of 8-bit codes (float8_e4m3fn, int8) with one bfloat16 scale per (token, head) in
    ``k_scale`` and ``v_scale`` [pages, heads, page_size].  Token slot s lives in page s // page_size at
    row s % page_size.  The tensors belong to the caller; ``KVCache.empty`` makes new ones."""

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
        _index(k, "k", (pages, heads, page, D), k.dtype, k.device)
        _index(v, "v", (pages, heads, page, D), k.dtype, k.device)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if self.format == "bf16":
                if t is not None:
                    raise ValueError(f"{name}: a bfloat16 cache has no scales")
            else:
                _index(t, name, (pages, heads, page), torch.bfloat16, k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_heads, self.page_size, self.head_dim = pages, heads, page, D
        self.device = k.device
        ptr = lambda t: None if t is None else t.data_ptr()
        self._c = _Cache(ptr(k), ptr(v), ptr(k_scale), ptr(v_scale), pages, heads, page, D, self.FORMATS[self.format][0])

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
    _heads(k, "k", cache.device, k.dtype)
    _heads(v, "v", cache.device, k.dtype)
    T = k.shape[0]
    if k.shape != (T, cache.n_heads, cache.head_dim) or v.shape != k.shape:
        raise ValueError(f"k and v must be [T, {cache.n_heads}, {cache.head_dim}]")
    at = _index(slots, "slots", (T,), torch.int64, cache.device)
    ctx, raw = _on(cache.device, stream)
    with ctx:
        rc = _lib().tps_kv_write(ctypes.byref(cache._c), k.data_ptr(), v.data_ptr(), _code(k.dtype), T, k.stride(0),
                                 k.stride(1), v.stride(0), v.stride(1), at, raw)
    _check(rc, "tps_kv_write")


def kv_read(cache: KVCache, slots, *, dtype=torch.bfloat16, out=None, stream=None):
    """The stored values of the slots ``slots`` ([T] int64) as (k, v), [T, heads, head_dim] of ``dtype``
    (float32 or bfloat16); a slot outside the cache reads as zeros.  ``out``: a (k, v) pair to write to."""
    dev = cache.device
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be an int64 [T] tensor")
    T = slots.shape[0]
    at = _index(slots, "slots", (T,), torch.int64, dev)
    shape = (T, cache.n_heads, cache.head_dim)
    code = _code(dtype)
    ctx, raw = _on(dev, stream)
    with ctx:
        if out is None:
            k, v = torch.empty(shape, dtype=dtype, device=dev), torch.empty(shape, dtype=dtype, device=dev)
        else:
            k, v = out
            _index(k, "out[0]", shape, dtype, dev)
            _index(v, "out[1]", shape, dtype, dev)
        rc = _lib().tps_kv_read(ctypes.byref(cache._c), at, T, k.data_ptr(), v.data_ptr(), code, raw)
    _check(rc, "tps_kv_read")
    return k, v


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
    sequence with a page outside the cache or a length outside its table (its outputs are NaN), else 0.
    ``workspace``: a uint8 tensor of at least ``prefix_attention_workspace(...)`` bytes to use instead of
    the library's memory pool."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dtype != torch.bfloat16 or q.dim() not in (3, 4) or (
            not q.is_contiguous()):
        raise ValueError("q must be a contiguous bfloat16 CUDA tensor [B, heads, D] or [B, tokens, heads, D]")
    dev = q.device
    B, D = q.shape[0], q.shape[-1]
    if dev != cache.device or D != cache.head_dim:
        raise ValueError(f"q must have head size {cache.head_dim} and be on {cache.device}")
    if D not in (64, 128):
        raise ValueError("prefix_attention takes head sizes 64 and 128")
    Hq = q.shape[-2]
    if Hq % cache.n_heads:
        raise ValueError(f"the query heads must be a multiple of the cache's {cache.n_heads} heads")
    prefix_len = int(prefix_len)
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2 or (
            page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be an int32 [B, W] tensor with unit stride along W")
    W = page_table.shape[1]
    if not isinstance(prefix_pages, torch.Tensor) or prefix_pages.dim() != 1 or prefix_len < 0 or (
            prefix_pages.shape[0] * cache.page_size < prefix_len):
        raise ValueError("prefix_pages must be an int32 [n] tensor whose pages hold prefix_len tokens")
    ctx, raw = _on(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty_like(q)
        else:
            _index(out, "out", tuple(q.shape), torch.bfloat16, dev)
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=dev) if want_lse else None
        a = _Attention(q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
                       _index(prefix_pages, "prefix_pages", tuple(prefix_pages.shape), torch.int32, dev),
                       _index(page_table, "page_table", (B, W), torch.int32, dev, dense=False),
                       _index(suffix_len, "suffix_len", (B,), torch.int32, dev),
                       None if status is None else _index(status, "status", (B,), torch.int32, dev),
                       None if workspace is None else workspace.data_ptr(),
                       0 if workspace is None else workspace.numel() * workspace.element_size(),
                       B, prefix_len, W, page_table.stride(0) if B > 1 else W, q.shape[1] if q.dim() == 4 else 1, Hq,
                       D ** -0.5 if scale is None else scale)
        rc = _lib().tps_prefix_attention(ctypes.byref(cache._c), ctypes.byref(a), raw)
    _check(rc, "tps_prefix_attention")
    return (out, lse) if want_lse else out


def prefix_attention_workspace(q_shape, cache: KVCache, prefix_len: int, table_width: int) -> int:
    """Bytes of workspace ``prefix_attention`` needs for a query of this shape."""
    B, Hq = q_shape[0], q_shape[-2]
    a = _Attention(None, None, None, None, None, None, None, None, 0, B, int(prefix_len), table_width, table_width,
                   q_shape[1] if len(q_shape) == 4 else 1, Hq, 1.0)
    n = _lib().tps_prefix_attention_workspace(ctypes.byref(cache._c), ctypes.byref(a))
    if n < 0:
        raise ValueError("arguments that prefix_attention would refuse")
    return n
