"""The decode-step operators in front of the sampler: per-head norm and rotation, the paged key/value
cache and the attention of a batch that shares a long prefix.  Like the rest of the binding these
functions only check tensors and hand pointers and the CUDA stream to the C ABI (``include/tps.h``)."""
from __future__ import annotations

import contextlib
import ctypes
import struct

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


# A call's arguments are packed as the structures above lie in memory (native sizes and alignment):
# several times faster than filling a ctypes structure field by field.
# ("0q" pads the end to their alignment.)
_NORM_LAYOUT, _ATTENTION_LAYOUT = struct.Struct("@4P8q5P2q6if0q"), struct.Struct("@8P5q2if0q")
assert _NORM_LAYOUT.size == ctypes.sizeof(_NormRope) and _ATTENTION_LAYOUT.size == ctypes.sizeof(_Attention)
_pack_norm, _pack_attention = _NORM_LAYOUT.pack, _ATTENTION_LAYOUT.pack

_Tensor = torch.Tensor
_empty = torch.empty  # with a device object: Tensor.new_empty and device strings take twice as long
_fns = None


def _bound():
    """The entry points, once the library is loaded."""
    global _fns
    if _fns is None:
        from . import load
        lib = load()
        _fns = (lib.tps_qk_norm_rope, lib.tps_kv_write, lib.tps_kv_read, lib.tps_prefix_attention,
                lib.tps_prefix_attention_workspace)
    return _fns


def _run(device_index, stream, call, *args):
    """``call(raw stream, *args)`` on the given stream or the current one.  A call on the current device
    and stream, the usual one, enters no context: the two managers cost several microseconds."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device_index)
        if device_index == torch._C._cuda_getDevice():
            return call(raw, *args)
        with torch.cuda.device(device_index):
            return call(raw, *args)
    with torch.cuda.device(device_index), torch.cuda.stream(stream):
        return call(stream.cuda_stream, *args)


def _fail(rc, name):
    from . import _ERRORS, load
    extra = f" (cudaError {load().tps_last_cuda_error()})" if rc == 5 else ""
    raise RuntimeError(f"{name} failed: {_ERRORS.get(rc, rc)}{extra}")


def _code(dt):
    if dt is torch.bfloat16:
        return 1
    if dt is torch.float32:
        return 0
    raise TypeError(f"values must be float32 or bfloat16, got {dt}")


def _dense(t, name, shape, dtype, device_index):
    """The address of a contiguous tensor of this shape, type and device."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != device_index or (
            not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{device_index}")
    return t.data_ptr()


def _heads(t, name, device_index=None, dtype=None):
    """Token and head strides of a [T, heads, head_dim] CUDA tensor."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    st = t.stride()
    if len(st) != 3 or (st[2] != 1 and t.shape[2] > 1):
        raise ValueError(f"{name} must be [T, heads, head_dim] with unit stride along head_dim")
    if dtype is not None and (t.dtype is not dtype or t.get_device() != device_index):
        raise ValueError(f"{name} must be a {dtype} tensor on cuda:{device_index}")
    return st


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
    qs = _heads(q, "q")
    dev, dt = q.get_device(), q.dtype
    ks = _heads(k, "k", dev, dt)
    T, Hq, D = q.shape
    Tk, Hk, Dk = k.shape
    if Tk != T or Dk != D:
        raise ValueError("q and k must hold the same tokens and head size")
    if not isinstance(cos_sin, _Tensor) or cos_sin.dim() != 2:
        raise ValueError("cos_sin must be a float32 [positions, R] tensor")
    n_pos, R = cos_sin.shape
    if R % 2 or R > D:
        raise ValueError("cos_sin must hold an even number of columns, at most the head size")
    if out is not None:
        oqs, oks = _heads(out[0], "out[0]", dev, dt), _heads(out[1], "out[1]", dev, dt)
        if out[0].shape != q.shape or out[1].shape != k.shape:
            raise ValueError("out must have the shapes of q and k")
    else:
        oqs, oks = (Hq * D, D), (Hk * D, D)
    tail = (qs[0], qs[1], ks[0], ks[1], oqs[0], oqs[1], oks[0], oks[1],
            0 if q_weight is None else _dense(q_weight, "q_weight", (D,), torch.float32, dev),
            0 if k_weight is None else _dense(k_weight, "k_weight", (D,), torch.float32, dev),
            _dense(positions, "positions", (T,), torch.int32, dev),
            _dense(cos_sin, "cos_sin", (n_pos, R), torch.float32, dev),
            0 if status is None else _dense(status, "status", (T,), torch.int32, dev),
            T, n_pos, Hq, Hk, D, R, 1 if interleaved else 0, _code(dt), eps)
    return _run(dev, stream, _norm, q, k, out, tail)


def _norm(raw, q, k, out, tail):
    if out is None:
        dt, dev = q.dtype, q.device
        out = _empty(q.shape, dtype=dt, device=dev), _empty(k.shape, dtype=dt, device=dev)
    oq, ok = out
    rc = _bound()[0](_pack_norm(q.data_ptr(), k.data_ptr(), oq.data_ptr(), ok.data_ptr(), *tail), raw)
    if rc:
        _fail(rc, "tps_qk_norm_rope")
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
        dev = k.get_device()
        _dense(k, "k", (pages, heads, page, D), k.dtype, dev)
        _dense(v, "v", (pages, heads, page, D), k.dtype, dev)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if self.format == "bf16":
                if t is not None:
                    raise ValueError(f"{name}: a bfloat16 cache has no scales")
            else:
                _dense(t, name, (pages, heads, page), torch.bfloat16, dev)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_heads, self.page_size, self.head_dim = pages, heads, page, D
        self.device = k.device
        ptr = lambda t: None if t is None else t.data_ptr()
        self._index = dev
        self._bytes = bytes(_Cache(ptr(k), ptr(v), ptr(k_scale), ptr(v_scale), pages, heads, page, D, self.FORMATS[self.format][0]))

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
    dev = cache._index
    dt = k.dtype
    ks, vs = _heads(k, "k", dev, dt), _heads(v, "v", dev, dt)
    T = k.shape[0]
    if k.shape != (T, cache.n_heads, cache.head_dim) or v.shape != k.shape:
        raise ValueError(f"k and v must be [T, {cache.n_heads}, {cache.head_dim}]")
    _run(dev, stream, _write, (cache._bytes, k.data_ptr(), v.data_ptr(), _code(dt), T, ks[0], ks[1], vs[0], vs[1],
                               _dense(slots, "slots", (T,), torch.int64, dev)))


def _write(raw, args):
    rc = _bound()[1](*args, raw)
    if rc:
        _fail(rc, "tps_kv_write")


def kv_read(cache: KVCache, slots, *, dtype=torch.bfloat16, out=None, stream=None):
    """The stored values of the slots ``slots`` ([T] int64) as (k, v), [T, heads, head_dim] of ``dtype``
    (float32 or bfloat16); a slot outside the cache reads as zeros.  ``out``: a (k, v) pair to write to."""
    dev = cache._index
    if not isinstance(slots, _Tensor) or slots.dim() != 1:
        raise ValueError("slots must be an int64 [T] tensor")
    T = slots.shape[0]
    at = _dense(slots, "slots", (T,), torch.int64, dev)
    shape = (T, cache.n_heads, cache.head_dim)
    if out is not None:
        _dense(out[0], "out[0]", shape, dtype, dev)
        _dense(out[1], "out[1]", shape, dtype, dev)
    return _run(dev, stream, _read, cache, at, shape, dtype, _code(dtype), out)


def _read(raw, cache, at, shape, dtype, code, out):
    if out is None:
        dev = cache.device
        out = _empty(shape, dtype=dtype, device=dev), _empty(shape, dtype=dtype, device=dev)
    k, v = out
    rc = _bound()[2](cache._bytes, at, shape[0], k.data_ptr(), v.data_ptr(), code, raw)
    if rc:
        _fail(rc, "tps_kv_read")
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
    if not isinstance(q, _Tensor) or not q.is_cuda or q.dtype is not torch.bfloat16 or q.dim() not in (3, 4) or (
            not q.is_contiguous()):
        raise ValueError("q must be a contiguous bfloat16 CUDA tensor [B, heads, D] or [B, tokens, heads, D]")
    dev, shape = q.get_device(), q.shape
    B, Hq, D = shape[0], shape[-2], shape[-1]
    if dev != cache._index or D != cache.head_dim:
        raise ValueError(f"q must have head size {cache.head_dim} and be on {cache.device}")
    if D not in (64, 128):
        raise ValueError("prefix_attention takes head sizes 64 and 128")
    if Hq % cache.n_heads:
        raise ValueError(f"the query heads must be a multiple of the cache's {cache.n_heads} heads")
    prefix_len = int(prefix_len)
    if not isinstance(page_table, _Tensor) or page_table.dim() != 2 or page_table.shape[0] != B or (
            page_table.dtype is not torch.int32 or page_table.get_device() != dev):
        raise ValueError(f"page_table must be an int32 [{B}, W] tensor on {cache.device}")
    W = page_table.shape[1]
    ts = page_table.stride()
    if W > 1 and ts[1] != 1:
        raise ValueError("page_table must have unit stride along W")
    if not isinstance(prefix_pages, _Tensor) or prefix_pages.dim() != 1 or prefix_len < 0 or (
            prefix_pages.shape[0] * cache.page_size < prefix_len):
        raise ValueError("prefix_pages must be an int32 [n] tensor whose pages hold prefix_len tokens")
    if out is not None:
        _dense(out, "out", shape, torch.bfloat16, dev)
    tail = (_dense(prefix_pages, "prefix_pages", prefix_pages.shape, torch.int32, dev), page_table.data_ptr(),
            _dense(suffix_len, "suffix_len", (B,), torch.int32, dev),
            0 if status is None else _dense(status, "status", (B,), torch.int32, dev),
            0 if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel() * workspace.element_size(),
            B, prefix_len, W, ts[0] if B > 1 else W, shape[1] if len(shape) == 4 else 1, Hq,
            D ** -0.5 if scale is None else scale)
    return _run(dev, stream, _attend, q, cache, out, want_lse, tail)


def _attend(raw, q, cache, out, want_lse, tail):
    if out is None:
        out = _empty(q.shape, dtype=torch.bfloat16, device=q.device)
    lse = _empty(q.shape[:-1], dtype=torch.float32, device=q.device) if want_lse else None
    rc = _bound()[3](cache._bytes, _pack_attention(q.data_ptr(), out.data_ptr(), lse.data_ptr() if want_lse else 0, *tail), raw)
    if rc:
        _fail(rc, "tps_prefix_attention")
    return (out, lse) if want_lse else out


def prefix_attention_workspace(q_shape, cache: KVCache, prefix_len: int, table_width: int) -> int:
    """Bytes of workspace ``prefix_attention`` needs for a query of this shape."""
    B, Hq = q_shape[0], q_shape[-2]
    n = _bound()[4](cache._bytes, _pack_attention(0, 0, 0, 0, 0, 0, 0, 0, 0, B, int(prefix_len), table_width, table_width,
                                                  q_shape[1] if len(q_shape) == 4 else 1, Hq, 1.0))
    if n < 0:
        raise ValueError("arguments that prefix_attention would refuse")
    return n
