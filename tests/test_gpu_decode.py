"""The decode-step operators against their plain 64-bit forms, through the C ABI.

Tolerances.  A bfloat16 result is off by at most half a unit, 2^-8 of its magnitude.
 - Norm and rotation: D float32 terms are summed (relative error up to D 2^-24, halved by the square
   root) and a handful of operations follow, on components no larger than the head's largest: (D/2 + 16) 2^-24
   of that.
 - Cache: codes and scales are exact for bfloat16 input (quotients of two 8-bit significands lie at least 2^-9 of
   a code away from a rounding boundary unless on it); for float32 input a code may be either neighbour
   where the quotient lies within 2^-22 of a boundary.
 - Attention: the weights are rounded to 8 bits (bfloat16) or 11 bits (float16): at most 2^-8 or 2^-11 of
   sum p |v|; the scores' float32 sums are off by at most 2^-18 of the largest sum of |products|, and base-2
   exponentials, the joins of parts and weights below 2^-31 of the largest by less than 2^-14.
"""
import ctypes
import math

import pytest
import torch

import nucleus_token_sampler_gb300 as tps

from . import _decode as plain

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda:0"


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _table(n, R):
    f = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64) / max(1, R // 2))
    return torch.cat([f.cos(), f.sin()], 1).float().to(DEV)


# --------------------------------------------------------------------------------------------- norm
def _check_norm(got, x, w, pos, table, eps, interleaved):
    want = plain.norm_rope(x, w, pos, table, eps, interleaved)
    D = x.shape[-1]
    # a component is at most sqrt(2) times the largest before the rotation
    top = want.abs().amax(-1, keepdim=True) * math.sqrt(2)
    tol = (D / 2 + 16) * 2.0 ** -24 * top + (2.0 ** -8 * want.abs() if x.dtype == torch.bfloat16 else 0)
    assert got.dtype == x.dtype and got.shape == x.shape
    assert ((got.double() - want).abs() <= tol).all(), float(((got.double() - want).abs() - tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hk,D,R,interleaved", [
    (1, 32, 8, 128, 128, False), (7, 32, 8, 128, 64, True), (130, 28, 4, 96, 96, False), (33, 5, 1, 256, 128, False),
    (3, 1, 1, 64, 64, True), (9, 3, 2, 80, 80, False), (5, 2, 1, 80, 32, True), (4, 3, 3, 66, 66, False), (6, 2, 2, 7, 4, True),
    (2, 1, 1, 1, 0, False), (3, 4, 0, 128, 128, False), (3, 0, 4, 128, 128, True), (2, 2, 2, 512, 512, False),
    (2, 1, 1, 1000, 500, False), (1000, 9, 3, 128, 128, False), (2, 300, 1, 16, 16, False)])
def test_norm_rope(dtype, T, Hq, Hk, D, R, interleaved):
    g = _gen(T * 1000 + D)
    qkv = (3 * torch.randn(T, Hq + 2 * Hk + 1, D, generator=g, device=DEV)).to(dtype)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    wq, wk = torch.randn(D, generator=g, device=DEV), torch.randn(D, generator=g, device=DEV)
    table = _table(50, R)
    pos = torch.randint(0, 50, (T,), generator=g, device=DEV).int()
    oq, ok = tps.qk_norm_rope(q, k, wq, wk, pos, table, eps=1e-5, interleaved=interleaved)
    _check_norm(oq, q, wq, pos, table, 1e-5, interleaved)
    _check_norm(ok, k, wk, pos, table, 1e-5, interleaved)


def test_norm_rope_without_weights_unaligned_in_place_and_zero_rows():
    g = _gen(5)
    base = torch.randn(11 * 6 * 128 + 3, generator=g, device=DEV).bfloat16()
    x = base[3:].view(11, 6, 128)  # rows start 6 bytes past a 16-byte boundary
    x[2, 1] = 0
    q, k = x[:, :4], x[:, 4:]
    table, pos = _table(20, 128), torch.arange(11, device=DEV).int()
    keep = x.clone()
    a = tps.qk_norm_rope(q, k, None, None, pos, table)
    _check_norm(a[0], keep[:, :4], None, pos, table, 1e-6, False)
    assert (a[0][2, 1] == 0).all()
    b = tps.qk_norm_rope(q, k, None, None, pos, table, out=(q, k))
    assert b[0] is q and torch.equal(q, a[0]) and torch.equal(k, a[1])
    # heads ahead of tokens in memory
    y = torch.randn(6, 11, 128, generator=g, device=DEV).transpose(0, 1)
    c = tps.qk_norm_rope(y[:, :4], y[:, 4:], None, None, pos, table)
    _check_norm(c[0], y[:, :4], None, pos, table, 1e-6, False)
    # the same in place, on the aligned path
    z = y.contiguous()
    d = tps.qk_norm_rope(z[:, :4], z[:, 4:], None, None, pos, table, out=(z[:, :4], z[:, 4:]))
    assert torch.equal(d[0], c[0]) and torch.equal(d[1], c[1])


@pytest.mark.parametrize("D", [128, 36])
def test_norm_rope_positions_outside_the_table_and_values_that_are_not_finite(D):
    q = torch.randn(5, 2, D, device=DEV)
    q[3, 0, 5] = math.inf
    q[4, 1, 0] = math.nan
    pos = torch.tensor([0, -1, 9, 2, 3], dtype=torch.int32, device=DEV)
    st = torch.full((5,), 77, dtype=torch.int32, device=DEV)
    oq, ok = tps.qk_norm_rope(q, q, None, None, pos, _table(9, D), status=st)
    assert st.tolist() == [0, 3, 3, 0, 0]
    assert torch.isfinite(oq[0]).all() and oq[1].isnan().all() and oq[2].isnan().all()
    assert oq[3, 0].isnan().any() and torch.isfinite(oq[3, 1]).all()
    assert oq[4, 1].isnan().all() and torch.isfinite(oq[4, 0]).all()
    assert torch.equal(oq.view(torch.int32), ok.view(torch.int32))
    assert tps.qk_norm_rope(q[:0], q[:0], None, None, pos[:0], _table(9, D))[0].shape == (0, 2, D)


# -------------------------------------------------------------------------------------------- cache
def _vectors(g, T, H, D, dtype):
    x = torch.randn(T, H, D, generator=g, device=DEV) * torch.exp(2 * torch.randn(T, H, 1, generator=g, device=DEV))
    x[0, 0] = 0
    if T > 2:
        x[1, 0], x[1, 0, D // 2] = 0, 448.0       # the largest code itself
        x[2, 0], x[2, 0, 0] = 2.0 ** -60, 2.0 ** -50  # below the smallest scale
    if T > 4:
        x[3, 0, 1] = 3e38
        x[4, 0] = torch.arange(D, device=DEV) % 8 + 0.5  # ties
        x[4, 0, 0] = 127.0
    return x.to(dtype)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 16, 16), (5, 8, 128, 64), (77, 3, 96, 16), (130, 2, 256, 128), (9, 1, 512, 256),
                                        (6, 5, 80, 32), (3000, 4, 64, 32)])
def test_cache_write_and_read(fmt, dtype, T, H, D, page):
    g = _gen(T + D)
    pages = -(-T // page) + 2
    c = tps.KVCache.empty(pages, H, page, D, fmt, device=DEV)
    k, v = _vectors(g, T, H, D, dtype), _vectors(g, T, 2 * H, D, dtype)[:, H - 1:2 * H - 1]
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:T].contiguous()
    tps.kv_write(c, k, v, slots)
    for x, code, scale in ((k, c.k, c.k_scale), (v, c.v, c.v_scale)):
        at = (slots // page, slice(None), slots % page)
        bits = code.view(torch.int16 if fmt == "bf16" else torch.uint8)[at].view(code.dtype)
        got = bits.double()
        if fmt == "bf16":
            assert torch.equal(got, x.bfloat16().double())
            continue
        s = scale[at].double()
        assert torch.equal(s, plain.scale_of(x, fmt))
        y = x.double() / s.unsqueeze(-1)
        want = plain.nearest(y, fmt)
        if dtype == torch.bfloat16 or fmt == "fp8":
            assert torch.equal(got, want)
        else:
            other = (got != want)
            assert ((got - want).abs()[other] == 1).all() and ((y - y.floor() - 0.5).abs()[other] <= 127 * 2.0 ** -22).all()
    for dt in (torch.bfloat16, torch.float32):
        rk, rv = tps.kv_read(c, slots, dtype=dt)
        K, V = plain.values(c)
        at = (slots // page, slice(None), slots % page)
        assert torch.equal(rk, K[at].float().to(dt)) and torch.equal(rv, V[at].float().to(dt))
    # nothing else was touched
    mask = torch.ones(pages * page, dtype=torch.bool, device=DEV)
    mask[slots] = False
    rest = mask.nonzero().flatten()
    rk, rv = tps.kv_read(c, rest)
    assert (rk == 0).all() and (rv == 0).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
def test_cache_padding_slots_unaligned_input_and_values_that_are_not_finite(fmt):
    g = _gen(3)
    c = tps.KVCache.empty(3, 2, 16, 64, fmt, device=DEV)
    base = torch.randn(6 * 2 * 64 + 1, generator=g, device=DEV).bfloat16()
    k = base[1:].view(6, 2, 64)
    v = torch.randn(2, 6, 64, generator=g, device=DEV).bfloat16().transpose(0, 1)
    k[4, 1, 7] = math.nan
    k[5, 0, 3] = -math.inf
    slots = torch.tensor([-1, 47, 48, 1 << 40, 5, 0], device=DEV)
    tps.kv_write(c, k, v, slots)
    rk, rv = tps.kv_read(c, torch.tensor([47, 5, 0, 48, -5, 3], device=DEV), dtype=torch.float32)
    assert torch.equal(rk[0].double(), plain.stored(k[1], fmt)) and torch.equal(rv[0].double(), plain.stored(v[1], fmt))
    assert torch.equal(rv[1].double(), plain.stored(v[4], fmt)) and torch.equal(rk[1, 0].double(), plain.stored(k[4, 0], fmt))
    assert (rk[3:] == 0).all() and (rv[3:] == 0).all()
    if fmt == "bf16":
        assert rk[1, 1].isnan().sum() == 1 and rk[2, 0].isinf().sum() == 1
    else:  # such a vector reads as NaN as a whole
        assert rk[1, 1].isnan().all() and rk[2, 0].isnan().all() and torch.isfinite(rk[2, 1]).all()
    tps.kv_write(c, k[:0], v[:0], slots[:0])
    assert tps.kv_read(c, slots[:0])[0].shape == (0, 2, 64)


def test_cache_past_four_gigabytes():
    """Rows whose byte offset does not fit 32 bits, written, read and attended to."""
    pages, H, page, D = 37000, 8, 128, 128  # 4.85 GB of codes each
    k, v = (torch.empty((pages, H, page, D), dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((pages, H, page), math.nan, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c = tps.KVCache(k, v, ks, vs)
    g = _gen(8)
    T = 300
    ids = torch.tensor([36999, 2, 35000], device=DEV)
    slots = ids[torch.arange(T, device=DEV) // page] * page + torch.arange(T, device=DEV) % page
    x, y = torch.randn(T, H, D, generator=g, device=DEV).bfloat16(), torch.randn(T, H, D, generator=g, device=DEV).bfloat16()
    tps.kv_write(c, x, y, slots)
    rk, rv = tps.kv_read(c, slots, dtype=torch.float32)
    assert torch.equal(rk.double(), plain.stored(x, "int8")) and torch.equal(rv.double(), plain.stored(y, "int8"))
    q = torch.randn(6, 1, 16, D, generator=g, device=DEV).bfloat16()
    near = [rk.view(T, H, D), rv.view(T, H, D)]
    pad = torch.zeros(384 - T, H, D, device=DEV)
    kv = [torch.cat([t, pad]).view(3, page, H, D).transpose(1, 2).double() for t in near]
    lens = torch.zeros(6, dtype=torch.int32, device=DEV)
    own = torch.zeros(6, 1, dtype=torch.int32, device=DEV)
    _check_attention(tps.prefix_attention(q, c, ids.int(), T, own, lens, want_lse=True), q, kv,
                     torch.arange(3, device=DEV), T, own, lens, D ** -0.5, "int8")
    lens[:] = T
    own = ids.int().expand(6, 3).contiguous()
    local = torch.arange(3, device=DEV).expand(6, 3)
    _check_attention(tps.prefix_attention(q, c, ids.int(), 0, own, lens, want_lse=True), q, kv, ids, 0, local, lens, D ** -0.5,
                     "int8")


# ---------------------------------------------------------------------------------------- attention
def _check_attention(got, q, kv, prefix_pages, prefix_len, page_table, lens, scale, fmt):
    out, lse = got
    want, wl, mag, big = plain.attention(q, kv, prefix_pages, prefix_len, page_table, lens, scale)
    rest = 2.0 ** -18 * big + 2.0 ** -14
    tol = 2.0 ** -8 * want.abs() + ((2.0 ** -8 if fmt == "bf16" else 2.0 ** -11) + rest).unsqueeze(-1) * mag
    err = (out.double() - want).abs()
    assert (err <= tol).all(), (float((err - tol).max()), int((err > tol).sum()), err.numel())
    seen = wl > -math.inf
    assert torch.equal(lse > -math.inf, seen)
    assert ((lse.double() - wl)[seen].abs() <= rest[seen] + 2.0 ** -22 * wl[seen].abs()).all()
    assert (out[~seen] == 0).all()


def _case(g, B, Tq, Hq, Hkv, D, prefix, lens, page, fmt, poison=True, spare=2):
    """A cache that holds the prefix and the sequences' tokens in scattered pages; every row that is no
    token of the call is NaN (or has a NaN scale)."""
    lens = [lens[i % len(lens)] for i in range(B)]
    shared, each = -(-prefix // page), max([1] + [-(-n // page) for n in lens])
    pages = shared + B * each + spare
    c = tps.KVCache.empty(pages, Hkv, page, D, fmt, device=DEV)
    order = torch.randperm(pages, generator=g, device=DEV)
    pp, table = order[:shared].int().contiguous(), order[shared:shared + B * each].int().reshape(B, each).contiguous()
    if poison:
        if fmt == "bf16":
            c.k.fill_(math.nan), c.v.fill_(math.nan)
        else:
            c.k_scale.fill_(math.nan), c.v_scale.fill_(math.nan)
    at = torch.arange(prefix, device=DEV)
    slots = [pp.long()[at // page] * page + at % page]
    for b in range(B):
        at = torch.arange(lens[b], device=DEV)
        slots.append(table[b].long()[at // page] * page + at % page)
    slots = torch.cat(slots)
    n = slots.shape[0]
    k = torch.randn(n, Hkv, D, generator=g, device=DEV) * torch.exp(0.5 * torch.randn(1, Hkv, D, generator=g, device=DEV))
    v = torch.randn(n, Hkv, D, generator=g, device=DEV) * torch.exp(torch.randn(n, Hkv, 1, generator=g, device=DEV))
    tps.kv_write(c, k.bfloat16(), v.bfloat16(), slots)
    q = (1.5 * torch.randn(B, Tq, Hq, D, generator=g, device=DEV)).bfloat16()
    return c, q, pp, table, torch.tensor(lens, dtype=torch.int32, device=DEV)


SHAPES = [  # B, Tq, Hq, Hkv, D, prefix, own lengths, page
    (1, 1, 1, 1, 64, 1, [0], 16),
    (1, 1, 4, 1, 128, 0, [1], 16),
    (2, 1, 8, 8, 128, 17, [0, 33], 16),
    (3, 1, 32, 8, 128, 1000, [0, 1, 40], 16),
    (5, 1, 8, 2, 64, 0, [0, 1, 15, 16, 300], 32),
    (8, 1, 28, 4, 128, 129, [64, 7], 64),
    (4, 5, 20, 4, 64, 333, [5, 6, 2, 0, 70], 32),   # fewer own tokens than queries: some see none
    (4, 3, 12, 4, 128, 0, [3, 1, 0], 16),           # and no prefix: nothing at all
    (16, 1, 8, 1, 128, 640, [20], 128),             # 128 rows of one head
    (33, 1, 8, 1, 128, 1023, [0, 5, 130], 256),     # 264 rows
    (40, 1, 16, 2, 64, 511, [9, 0], 16),            # 320 rows
    (70, 2, 10, 2, 128, 257, [2, 50], 32),          # 700 rows
    (1, 1, 16, 1, 64, 5000, [3], 64),
    (2, 1, 8, 2, 128, 100, [4000, 1], 16),          # a long own part: several CTAs for each sequence
    (1, 40, 6, 1, 64, 200, [40], 16),               # 240 rows of one sequence
    (257, 1, 4, 1, 64, 130, [1, 2, 3], 16),
    (6, 1, 8, 2, 64, 6000, [0, 2500, 100], 32),     # long own parts cut evenly, the prefix shared by 24 rows
    (3, 5, 16, 2, 128, 17000, [5, 2600, 700], 64),  # three row tiles for each sequence, 120 rows
    (12, 1, 32, 4, 128, 900, [0, 3000, 64, 65], 16),
    (5, 1, 4, 4, 64, 0, [0, 0, 4097, 0, 0], 256),
    (2, 1, 8, 8, 128, 2500, [0], 64),               # the prefix walked over by each sequence, nothing of their own
    (30, 1, 4, 2, 64, 100, [5, 0, 17], 16),
    (9, 7, 6, 2, 64, 50, [7, 20], 16),              # 21 rows for each sequence and key head
]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:6])))
def test_attention(fmt, shape):
    B, Tq, Hq, Hkv, D, prefix, lens, page = shape
    g = _gen(B * 100 + prefix)
    c, q, pp, table, n = _case(g, B, Tq, Hq, Hkv, D, prefix, lens, page, fmt)
    st = torch.full((B,), 9, dtype=torch.int32, device=DEV)
    got = tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True, status=st)
    assert (st == 0).all()
    _check_attention(got, q, plain.values(c), pp, prefix, table, n, D ** -0.5, fmt)
    again = tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    if Tq == 1:
        assert torch.equal(tps.prefix_attention(q[:, 0].contiguous(), c, pp, prefix, table, n), got[0][:, 0])


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("B", [2, 48])
def test_attention_to_one_token_and_growing_scores(fmt, B):
    """Scores that rise along the tokens by hundreds of units (every block raises the reference), and a
    token whose score towers over the others."""
    g = _gen(7)
    D, prefix = 128, 700
    c, q, pp, table, n = _case(g, B, 1, 8, 2, D, prefix, [40], 64, fmt)
    at = torch.arange(prefix, device=DEV)
    slots = pp.long()[at // 64] * 64 + at % 64
    u = torch.randn(1, 2, D, generator=g, device=DEV)
    q[:] = (u.repeat_interleave(4, 1) * torch.linspace(0.25, 2, B * 8, device=DEV).view(B, 8, 1)).unsqueeze(1).bfloat16()
    k = (u * (at.view(-1, 1, 1) / 100 - 2)).bfloat16()
    v = torch.randn(prefix, 2, D, generator=g, device=DEV).bfloat16()
    tps.kv_write(c, k, v, slots)
    _check_attention(tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True), q, plain.values(c), pp, prefix, table, n,
                     D ** -0.5, fmt)
    _check_attention(tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True, scale=3.0), q, plain.values(c), pp, prefix,
                     table, n, 3.0, fmt)
    _check_attention(tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True, scale=-0.5), q, plain.values(c), pp, prefix,
                     table, n, -0.5, fmt)


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("B,mag", [(2, 2.0 ** -30), (2, 2.0 ** 20), (40, 2.0 ** -30), (40, 2.0 ** 20)])
def test_attention_queries_outside_float16(fmt, B, mag):
    g = _gen(9)
    c, q, pp, table, n = _case(g, B, 1, 4, 1, 64, 200, [30], 32, fmt)
    q[0] = (q[0].float() * mag).bfloat16()
    q[1, 0, 0] = 0
    kv = plain.values(c)
    scale = 0.125 / max(1.0, mag)
    _check_attention(tps.prefix_attention(q, c, pp, 200, table, n, want_lse=True, scale=scale), q, kv, pp, 200, table, n, scale, fmt)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("B", [3, 40])
def test_attention_bad_pages_lengths_and_values(fmt, B):
    g = _gen(11)
    c, q, pp, table, n = _case(g, B, 1, 8, 1, 128, 300, [40], 16, fmt)
    good = tps.prefix_attention(q, c, pp, 300, table, n)
    table[0, 1] = c.n_pages
    table[1, 2] = -1
    n2 = n.clone()
    n2[1] = 32  # its bad page holds no token that is seen
    n2[2] = table.shape[1] * 16 + 1
    st = torch.empty(B, dtype=torch.int32, device=DEV)
    out, lse = tps.prefix_attention(q, c, pp, 300, table, n2, status=st, want_lse=True)
    assert st[:3].tolist() == [3, 0, 3] and (st[3:] == 0).all()
    assert out[0].isnan().all() and out[2].isnan().all() and torch.isfinite(out[1]).all()
    assert lse[0].isnan().all() and torch.isfinite(lse[1]).all()
    assert torch.equal(out[3:], good[3:])
    n2[0] = -1
    tps.prefix_attention(q, c, pp, 300, table, n2, status=st)
    assert st[:3].tolist() == [3, 0, 3]
    bad = pp.clone()
    bad[5] = c.n_pages + 7
    out = tps.prefix_attention(q, c, bad, 300, table, n, status=st)
    assert (st == 3).all() and out.isnan().all()
    # NaN in one sequence's query and in another's own tokens stay there
    table = torch.arange(table.numel(), device=DEV, dtype=torch.int32).reshape(table.shape)
    c, q, pp, table, n = _case(_gen(11), B, 1, 8, 1, 128, 300, [40], 16, fmt)
    q[1, 0, 3, 5] = math.nan
    s = table[2, 1].long().reshape(1) * 16 + 3
    tps.kv_write(c, torch.full((1, 1, 128), math.nan, device=DEV), torch.zeros(1, 1, 128, device=DEV), s)
    out = tps.prefix_attention(q, c, pp, 300, table, n)
    assert out[1, 0, 3].isnan().all() and out[2].isnan().all()
    keep = torch.ones(B, 1, 8, dtype=torch.bool, device=DEV)
    keep[1, 0, 3] = False
    keep[2] = False
    assert torch.equal(out[keep], good[keep])


def test_attention_table_stride_workspace_stream_and_graph():
    g = _gen(13)
    c, q, pp, table, n = _case(g, 40, 1, 8, 2, 128, 777, [0, 33, 50], 16, "fp8")
    want = tps.prefix_attention(q, c, pp, 777, table, n)
    wide = torch.full((40, table.shape[1] + 5), -9, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    assert torch.equal(tps.prefix_attention(q, c, pp, 777, wide[:, :table.shape[1]], n), want)
    size = tps.prefix_attention_workspace(q.shape, c, 777, table.shape[1])
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    assert torch.equal(tps.prefix_attention(q, c, pp, 777, table, n, workspace=ws), want)
    with pytest.raises(RuntimeError):
        tps.prefix_attention(q, c, pp, 777, table, n, workspace=ws[:size - 1])
    side = torch.cuda.Stream(DEV)
    q2 = torch.empty_like(q)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        q2.copy_(q)
    got = tps.prefix_attention(q2, c, pp, 777, table, n, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        tps.prefix_attention(q, c, pp, 777, table, n, out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert tps.prefix_attention(q[:0].contiguous(), c, pp, 777, table[:0], n[:0]).shape == (0, 1, 8, 128)


def test_attention_does_not_depend_on_the_other_sequences():
    g = _gen(17)
    c, q, pp, table, n = _case(g, 64, 1, 8, 2, 128, 900, [10, 33], 32, "int8")
    want = tps.prefix_attention(q, c, pp, 900, table, n)
    q2 = q.clone()
    q2[:20] = (q2[:20].float() * 1000).bfloat16()
    q2[20:40] = 0
    assert torch.equal(tps.prefix_attention(q2, c, pp, 900, table, n)[40:], want[40:])


def test_no_prefix_equals_all_prefix():
    """The same tokens as one sequence's own and as its prefix give the same answer to rounding."""
    g = _gen(19)
    c, q, pp, table, n = _case(g, 1, 1, 8, 2, 128, 500, [0], 16, "bf16")
    a, la = tps.prefix_attention(q, c, pp, 500, table, n, want_lse=True)
    m = torch.tensor([500], dtype=torch.int32, device=DEV)
    b, lb = tps.prefix_attention(q, c, pp[:0], 0, pp.view(1, -1), m, want_lse=True)
    kv = plain.values(c)
    _check_attention((a, la), q, kv, pp, 500, table, n, 128 ** -0.5, "bf16")
    _check_attention((b, lb), q, kv, pp[:0], 0, pp.view(1, -1), m, 128 ** -0.5, "bf16")


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("B,Hq,Hkv,D,prefix,lens", [
    (12, 32, 4, 128, 900, [0, 3000, 64, 65]),   # the prefix walked over by each sequence, long rings
    (16, 32, 4, 128, 2048, [1000, 3000]), (48, 8, 2, 64, 700, [500]), (400, 32, 8, 128, 300, [150, 20])])
def test_attention_repeats_itself(fmt, B, Hq, Hkv, D, prefix, lens):
    """Bit for bit, over many runs: copies into a ring never overtake the reads of what they replace."""
    c, q, pp, table, n = _case(_gen(77), B, 1, Hq, Hkv, D, prefix, lens, 16, fmt)
    want, lse = tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True)
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(300):
        got, again = tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True)
        differ += (got != want).sum() + (again != lse).sum()
    assert int(differ) == 0


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("B,prefix", [(3, 70), (60, 1500)])
def test_attention_scales_past_the_end_may_be_tiny(fmt, B, prefix):
    """1 / s overflows for a subnormal scale; in a row that is no token it must not reach the sum (0 * inf)."""
    c, q, pp, table, n = _case(_gen(78), B, 1, 8, 2, 128, prefix, [3, 21], 16, fmt)
    want, lse = tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True)
    assert torch.isfinite(want).all() and torch.isfinite(lse).all()
    for s in (c.k_scale, c.v_scale):
        s[torch.isnan(s)] = 1e-39
    got, again = tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True)
    assert torch.equal(got, want) and torch.equal(again, lse)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("B,Tq,Hq,Hkv,D,prefix", [
    (2100, 5, 64, 8, 64, 1), (512, 5, 64, 8, 128, 100), (512, 5, 64, 8, 64, 127), (1024, 1, 64, 8, 128, 100)])
def test_attention_short_prefixes_with_several_items_a_cta(fmt, B, Tq, Hq, Hkv, D, prefix):
    """Every item is one block that ends past the prefix, and each CTA has two or more of them, two in its ring at a time.  All outputs
    are compared for the first and last sequences, whose rows lie in the first and last tiles, and some between."""
    c, q, pp, table, n = _case(_gen(prefix), B, Tq, Hq, Hkv, D, prefix, [Tq, Tq + 3], 16, fmt, spare=20)
    st = torch.full((B,), 9, dtype=torch.int32, device=DEV)
    for _ in range(3):
        out, lse = tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True, status=st)
        assert (st == 0).all() and torch.isfinite(out).all() and torch.isfinite(lse).all()
    some = torch.cat([torch.arange(8), torch.arange(B // 2 - 4, B // 2 + 4), torch.arange(B - 8, B)]).to(DEV)
    _check_attention((out[some], lse[some]), q[some], plain.values(c), pp, prefix, table[some], n[some], D ** -0.5, fmt)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("B,Tq,Hq,Hkv,D,prefix,lens", [
    (40, 1, 24, 3, 128, 1500, [30, 7]),    # the prefix shared, a cluster or a CTA for each sequence
    (40, 1, 24, 3, 64, 0, [30, 700]),      # one launch
    (3, 1, 24, 3, 128, 300, [0, 20]),      # one launch, the prefix walked over by each sequence
    (20, 5, 24, 3, 64, 2000, [4500, 20]),  # the own tokens cut evenly, three row tiles
    (900, 1, 6, 3, 64, 400, [5, 20])])     # a warp for each sequence
def test_attention_status_tells_of_a_wait_that_ran_out_in_any_head(fmt, B, Tq, Hq, Hkv, D, prefix, lens):
    """One head's keys and values never arrive: its outputs are NaN, and the status says so whichever head it is."""
    c, q, pp, table, n = _case(_gen(79), B, Tq, Hq, Hkv, D, prefix, lens, 16, fmt)
    want = tps.prefix_attention(q, c, pp, prefix, table, n)
    lib, G = tps.load(), Hq // Hkv
    size = tps.prefix_attention_workspace(q.shape, c, prefix, table.shape[1])
    ws = torch.zeros(max(size, 1), dtype=torch.uint8, device=DEV)
    for head in range(Hkv):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
        st = torch.full((B,), 9, dtype=torch.int32, device=DEV)
        a = tps.decode._Attention(q.data_ptr(), out.data_ptr(), lse.data_ptr(), pp.data_ptr(), table.data_ptr(), n.data_ptr(),
                                  st.data_ptr(), ws.data_ptr(), size, B, prefix, table.shape[1], table.shape[1], Tq, Hq, D ** -0.5)
        assert lib.tps_prefix_attention_stall_test(c._bytes, ctypes.byref(a), head, 2_000_000,
                                                   torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert (st == 4).all(), (head, st.tolist())
        mine = out[:, :, head * G:(head + 1) * G]
        assert mine.isnan().all() and lse[:, :, head * G:(head + 1) * G].isnan().all()
        good = ~out.isnan().any(-1)
        assert torch.equal(out[good], want[good])
    again = tps.prefix_attention(q, c, pp, prefix, table, n, status=st)
    assert (st == 0).all() and torch.equal(again, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,R,interleaved", [(128, 64, False), (128, 64, True), (96, 32, False), (64, 0, False), (36, 8, True)])
def test_norm_rope_components_that_do_not_turn_keep_to_themselves(dtype, D, R, interleaved):
    """An infinity makes itself NaN and its head's other components 0, as the formula does; only pairs that turn mix."""
    q = torch.randn(4, 2, D, device=DEV).to(dtype)
    q[1, 0, D - 3] = math.inf
    q[2, 1, R] = -math.inf
    w = torch.ones(D, device=DEV)
    w[D - 1] = math.inf
    pos, table = torch.arange(4, device=DEV).int(), _table(9, R)
    for weight in (None, w):
        got, _ = tps.qk_norm_rope(q, q, weight, weight, pos, table, interleaved=interleaved)
        want = plain.norm_rope(q, weight, pos, table, 1e-6, interleaved)
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
        assert (got[1:3][~got[1:3].isnan() & ~got[1:3].isinf()].abs() < 100).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("B,G,prefix,lens", [(64, 4, 900, [10, 33]), (24, 1, 2000, [5]), (600, 4, 500, [3]), (3, 4, 200, [30])])
def test_attention_has_the_same_bits_whatever_its_neighbours_are(fmt, B, G, prefix, lens):
    """Every other sequence gets other queries: its neighbours, rows of the same warps and tiles, keep every bit."""
    c, q, pp, table, n = _case(_gen(80), B, 1, 2 * G, 2, 128, prefix, lens, 32, fmt)
    want, lse = tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True)
    for factor in (30.0, 1000.0, 0.0):
        q2 = q.clone()
        q2[::2] = (q2[::2].float() * factor).bfloat16()
        got, again = tps.prefix_attention(q2, c, pp, prefix, table, n, want_lse=True)
        assert torch.equal(got[1::2], want[1::2]) and torch.equal(again[1::2], lse[1::2])


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("B", [2, 100])
def test_attention_products_below_every_float(fmt, B):
    """Queries near 2^-125 on keys with the smallest scale: the scores are 0, in blocks that end past the prefix too."""
    c, q, pp, table, n = _case(_gen(81), B, 1, 4, 1, 64, 700, [30], 32, fmt)
    c.k_scale[~c.k_scale.isnan()] = 2.0 ** -40
    q[:] = (q.float().clamp(-3, 3) * 2.0 ** -126).bfloat16()
    _check_attention(tps.prefix_attention(q, c, pp, 700, table, n, want_lse=True), q, plain.values(c), pp, 700, table, n, 0.125, fmt)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("B", [2, 100])
@pytest.mark.parametrize("scale,mag", [(0.0, 1.0), (0.0, 2.0 ** 104), (1e-36, 2.0 ** 100)])
def test_attention_with_a_scale_of_nothing(fmt, B, scale, mag):
    """All tokens weigh the same at scale 0, and nearly so where the products are as large as the scale is small."""
    c, q, pp, table, n = _case(_gen(85), B, 1, 4, 1, 64, 700, [30], 32, fmt)
    q[:] = (q.float() * mag).bfloat16()
    _check_attention(tps.prefix_attention(q, c, pp, 700, table, n, want_lse=True, scale=scale), q, plain.values(c), pp, 700, table, n,
                     scale, fmt)


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("B", [2, 40, 200])
@pytest.mark.parametrize("factor", [1.3, 2.0 ** -25, 2.0 ** -50, 2.0 ** 30])
def test_attention_on_a_callers_own_codes_and_scales(fmt, B, factor):
    """Scales that are no powers of two, and scales below and above those kv_write makes of ordinary values: one
    tensor's at a time, so that scores stay ordinary where the values are not."""
    D, prefix = 64, 400
    for name in ("k_scale", "v_scale"):
        c, q, pp, table, n = _case(_gen(84), B, 1, 4, 1, D, prefix, [60], 32, fmt)
        s = getattr(c, name)
        s.copy_((s.float() * factor).bfloat16())
        scale = 0.125 / factor if name == "k_scale" else 0.125
        _check_attention(tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True, scale=scale), q, plain.values(c), pp, prefix,
                         table, n, scale, fmt)


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("B", [2, 40, 200])
@pytest.mark.parametrize("power", [-12, -20, -30])
def test_attention_to_a_token_whose_values_are_far_below_its_neighbours(fmt, B, power):
    """One key takes nearly all the weight, and its values are 2^power of the others'."""
    g = _gen(82)
    D, prefix, page = 128, 300, 16
    c, q, pp, table, n = _case(g, B, 1, 8, 2, D, prefix, [40], page, fmt)
    u = torch.randn(1, 2, D, generator=g, device=DEV)
    q[:] = (u.repeat_interleave(4, 1) * torch.linspace(0.75, 1.5, B * 8, device=DEV).view(B, 8, 1)).unsqueeze(1).bfloat16()
    at = torch.tensor([5, 200], device=DEV)
    slots = pp.long()[at // page] * page + at % page
    k = (torch.tensor([12.0, 11.0], device=DEV).view(2, 1, 1) * u).bfloat16()
    v = (torch.randn(2, 2, D, generator=g, device=DEV) * 2.0 ** power).bfloat16()
    tps.kv_write(c, k, v, slots)
    kv = plain.values(c)
    _check_attention(tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True), q, kv, pp, prefix, table, n, D ** -0.5, fmt)


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("B", [2, 40, 200])
@pytest.mark.parametrize("power", [8, 16, 26])
def test_attention_beside_a_token_whose_keys_are_far_above_its_neighbours(fmt, B, power):
    """A key 2^power times the others', whose score is so low that it takes no weight, costs its neighbours nothing."""
    g = _gen(83)
    D, prefix, page = 128, 300, 16
    c, q, pp, table, n = _case(g, B, 1, 8, 2, D, prefix, [40], page, fmt)
    at = torch.tensor([17], device=DEV)
    slots = pp.long()[at // page] * page + at % page
    u = torch.randn(1, 2, D, generator=g, device=DEV)
    q[:] = (q.float().abs() * u.sign().repeat_interleave(4, 1)).bfloat16()
    tps.kv_write(c, (-u.sign() * 2.0 ** power).bfloat16(), torch.zeros(1, 2, D, device=DEV).bfloat16(), slots)
    kv = plain.values(c)
    out, lse = tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True)
    want, wl, mag, _ = plain.attention(q, kv, pp, prefix, table, n, D ** -0.5)
    kv[0][pp[1].long(), :, 1] = 0
    big = plain.attention(q, kv, pp, prefix, table, n, D ** -0.5)[3]
    rest = 2.0 ** -18 * big + 2.0 ** -14
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -11 + rest).unsqueeze(-1) * mag).all()
    assert ((lse.double() - wl).abs() <= rest + 2.0 ** -22 * wl.abs()).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("B,Tq,Hq,Hkv,D,prefix,lens", [
    (3, 5, 8, 2, 128, 40, [5, 21, 33]), (2, 16, 4, 4, 64, 0, [16, 40]), (40, 3, 8, 1, 64, 2000, [30]),
    (3, 7, 8, 2, 64, 100, [4200, 17]), (900, 2, 4, 2, 64, 100, [20, 5])])
def test_attention_values_that_are_not_finite_stay_with_those_who_see_them(fmt, B, Tq, Hq, Hkv, D, prefix, lens):
    """NaN and infinities in the values of the last own tokens: queries they are hidden from keep every bit, the others get
    what the formula gives."""
    c, q, pp, table, n = _case(_gen(86), B, Tq, Hq, Hkv, D, prefix, lens, 16, fmt)
    b = torch.arange(B, device=DEV)
    slots = lambda back: table[b, (n.long() - back) // 16].long() * 16 + (n.long() - back) % 16
    k = torch.randn(B, Hkv, D, generator=_gen(87), device=DEV).bfloat16()
    v = torch.zeros(2, B, Hkv, D, device=DEV).bfloat16()
    for back in (1, 2):
        tps.kv_write(c, k, v[0], slots(back))
    calm, calm_lse = tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True)
    v[0, :, :, 3] = math.nan
    v[0, :, 0, D - 1] = math.inf
    v[1, :, Hkv - 1, 7] = -math.inf
    for back in (1, 2):
        tps.kv_write(c, k, v[back - 1], slots(back))
    out, lse = tps.prefix_attention(q, c, pp, prefix, table, n, want_lse=True)
    assert torch.equal(out[:, :-2], calm[:, :-2])
    some = slice(0, 4)
    want = plain.attention(q[some], plain.values(c), pp, prefix, table[some], n[some], D ** -0.5)[0]
    got = out[some]
    assert torch.equal(got.isnan(), want.isnan())
    if fmt == "bf16":
        assert torch.equal(got.isposinf(), want.isposinf()) and torch.equal(got.isneginf(), want.isneginf())
        assert torch.equal(lse, calm_lse)
        assert want[:, -1].isnan().any() and want[:, -2:].isinf().any()


def test_flags_that_have_no_truth_value_are_refused():
    """Their exception reaches the caller, and nothing is launched."""
    class Neither:
        def __bool__(self):
            raise KeyError("neither")
    q = torch.randn(3, 2, 64, device=DEV)
    with pytest.raises(KeyError):
        tps.qk_norm_rope(q, q, None, None, torch.arange(3, device=DEV).int(), _table(4, 64), interleaved=Neither())
    c, q, pp, table, n = _case(_gen(88), 2, 1, 4, 1, 64, 20, [3], 16, "bf16")
    with pytest.raises(KeyError):
        tps.prefix_attention(q, c, pp, 20, table, n, want_lse=Neither())
