"""Attention of drafted trees over the paged cache against its plain 64-bit form (tolerances: tests/_serve.py)."""
import ctypes
import math

import pytest
import torch

import nucleus_token_sampler_gb300 as tps
from nucleus_token_sampler_gb300 import decode

from . import _decode, _serve as plain

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda:0"
BF16 = 2.0 ** -8


def _trees(g, B, N):
    """Random trees: bit j of node i where j is i or above it."""
    t = torch.zeros(B, N, dtype=torch.int64, device=DEV)
    for i in range(N):
        bit = 1 << i if i < 63 else -(1 << 63)
        parent = torch.randint(-1, i, (B, 1), generator=g, device=DEV) if i else torch.full((B, 1), -1, device=DEV)
        above = t.gather(1, parent.clamp(min=0)).squeeze(1)
        t[:, i] = torch.where(parent.squeeze(1) >= 0, above, 0) | bit
    return t


def _case(seed, lens, N, Hq, Hk, D, page, fmt, nodes=None, poison=True, spare=3):
    """Arguments of a call: a cache in scattered pages whose rows past each sequence's length are NaN (or have a NaN scale)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    B = len(lens)
    W = max(1, -(-max(lens) // page)) + 1
    pages = B * W + spare
    c = tps.KVCache.empty(pages, Hk, page, D, fmt, device=DEV)
    x = torch.randn(pages * page, Hk, D, generator=g, device=DEV) * torch.exp(0.5 * torch.randn(pages * page, Hk, 1, generator=g, device=DEV))
    tps.kv_write(c, x.bfloat16(), torch.randn(pages * page, Hk, D, generator=g, device=DEV).bfloat16(), torch.arange(pages * page, device=DEV))
    table = torch.randperm(pages, generator=g, device=DEV)[:B * W].int().view(B, W)
    if poison:
        free = torch.ones(pages * page, dtype=torch.bool, device=DEV)
        for b, n in enumerate(lens):
            at = torch.arange(n, device=DEV)
            free[table[b].long()[at // page] * page + at % page] = False
        free = free.view(pages, page)
        for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
            (t if s is None else s).transpose(1, 2)[free] = math.nan
    q = (1.5 * torch.randn(B, N, Hq, D, generator=g, device=DEV)).bfloat16()
    n = None if nodes is None else torch.tensor(nodes, dtype=torch.int32, device=DEV)
    return q, c, table, torch.tensor(lens, dtype=torch.int32, device=DEV), _trees(g, B, N), n


def _want(q, c, table, lens, tree, nodes, scale):
    B, N, Hq, D = q.shape
    Hk, page = c.n_heads, c.page_size
    K, V = _decode.values(c)
    out = [torch.zeros(s, dtype=torch.float64, device=DEV) for s in ((B, N, Hq, D), (B, N, Hq), (B, N, Hq, D), (B, N, Hq))]
    out[1].fill_(-math.inf)
    if c.format != "bf16":
        out.append(torch.zeros_like(out[0]))
    tree = tree.expand(B, N)
    for b in range(B):
        n, L = (N if nodes is None else int(nodes[b])), int(lens[b])
        if n == 0 or L == 0:
            continue
        at = torch.arange(L, device=DEV)
        p = table[b].long()[at // page]
        k, v = (x[p, :, at % page].repeat_interleave(Hq // Hk, 1) for x in (K, V))
        seen = torch.ones(n, L, dtype=torch.bool, device=DEV)
        for j in range(n):
            seen[:, L - n + j] = (tree[b, :n] >> j) & 1 == 1
        s = None if c.format == "bf16" else c.v_scale[p, :, at % page].double().repeat_interleave(Hq // Hk, 1)
        for o, r in zip(out, plain.softmax_rows(q[b, :n].double(), k, v, seen, scale, s)):
            o[b, :n] = r
    return out


def _check(args, scale=None, **kw):
    q, c, table, lens, tree, nodes = args
    st = torch.full((q.shape[0],), 9, dtype=torch.int32, device=DEV)
    out, lse = tps.tree_attention(q, c, table, lens, tree, nodes=nodes, scale=scale, want_lse=True, status=st, **kw)
    assert (st == 0).all()
    plain.check(out, lse, _want(q, c, table, lens, tree, nodes, q.shape[3] ** -0.5 if scale is None else scale), BF16)
    return out, lse


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("N,Hq,Hk,D,page,lens", [
    (1, 1, 1, 64, 16, [1]), (1, 8, 2, 128, 64, [1, 128, 129, 700]), (8, 32, 8, 128, 16, [1000]), (5, 10, 2, 64, 32, [5, 6, 127, 128, 133, 300]),
    (16, 4, 1, 128, 128, [140, 16, 400]), (33, 4, 4, 64, 256, [300, 33]), (64, 8, 8, 128, 16, [64, 65, 127, 128, 129, 191, 192, 1000]),
    (64, 8, 1, 64, 32, [2000, 90]), (7, 64, 1, 128, 16, [77, 1500]), (64, 5, 1, 128, 64, [500]), (3, 6, 2, 64, 16, list(range(3, 300, 7)))])
def test_trees(fmt, N, Hq, Hk, D, page, lens):
    _check(_case(N * Hq, lens, N, Hq, Hk, D, page, fmt))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("N,Hq,Hk,D,page,lens", [(16, 8, 2, 128, 16, [9000, 20, 5000]), (4, 4, 1, 64, 64, [30000]), (12, 32, 8, 64, 32, [300] * 70),
                                                 (1, 4, 2, 128, 16, [40] * 1300)])
def test_lines_cut_over_many_ctas(fmt, N, Hq, Hk, D, page, lens):
    args = _case(len(lens), lens, N, Hq, Hk, D, page, fmt)
    a = _check(args)
    for _ in range(20):
        b = tps.tree_attention(*args[:5], want_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("D", [64, 128])
def test_a_lone_token_has_its_value_as_it_is(D):
    """The rounded weight is divided by itself."""
    q, c, table, lens, tree, _ = _case(12, [3, 1, 130, 70], 1, 6, 2, D, 16, "bf16")
    one = torch.ones_like(lens)
    out = tps.tree_attention(q, c, table, one, tree)
    for b in range(4):
        assert torch.equal(out[b, 0], c.v[table[b, 0], :, 0].repeat_interleave(3, 0))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
def test_padded_batches_and_sequences_without_tokens(fmt):
    nodes = [0, 3, 8, 0, 1, 5, 8, 2]
    args = _case(3, [0, 3, 8, 40, 500, 130, 129, 128], 8, 8, 2, 64, 16, fmt, nodes=nodes)
    out, lse = _check(args)
    for b, n in enumerate(nodes):
        assert (out[b, n:] == 0).all() and (lse[b, n:] == -math.inf).all()
    args[0][:, 3:].fill_(math.nan)  # padding's queries hold anything
    out2, _ = tps.tree_attention(*args[:5], nodes=torch.tensor([0, 3, 3, 0, 1, 3, 3, 2], dtype=torch.int32, device=DEV), want_lse=True)
    assert torch.isfinite(out2).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
def test_masks_that_are_no_trees(fmt):
    """Bits of later nodes and of nodes past the last count as the mask says; rows that see nothing yield 0."""
    q, c, table, lens, tree, _ = _case(4, [6, 6, 140, 133], 6, 4, 2, 128, 16, fmt)
    g = torch.Generator(device=DEV).manual_seed(1)
    wild = torch.randint(-2 ** 62, 2 ** 62, tree.shape, generator=g, device=DEV)
    wild[0, 2], wild[0, 4], wild[2, 1] = 0, -64, 0
    out, lse = _check((q, c, table, lens, wild, None))
    assert (out[0, 2] == 0).all() and (lse[0, 4] == -math.inf).all() and torch.isfinite(lse[2, 1]).all()
    _check((q, c, table, lens, wild, torch.tensor([6, 2, 5, 3], dtype=torch.int32, device=DEV)))
    _check((q, c, table, lens, wild[1].contiguous(), None))  # one for all


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("scale", [0.7, -0.4, 0.0, 1e-32])
def test_scales_and_rising_scores(fmt, scale):
    args = _case(5, [700, 20], 9, 4, 1, 128, 32, fmt, poison=False)
    c = args[1]
    if fmt == "bf16":
        c.k.mul_(torch.linspace(0, 6, 32, device=DEV).bfloat16()[None, None, :, None])
    else:
        c.k_scale.mul_(torch.exp2(torch.arange(-4, 4, device=DEV).repeat(4).float()).bfloat16())
    _check(args, scale=scale)


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("N,Hq,Hk,D,page,lens", [(1, 8, 2, 128, 16, [1, 700, 0, 33]), (4, 8, 2, 64, 32, [300, 4, 0, 17, 90]), (16, 2, 2, 128, 64, [500, 16, 3]),
                                                 (3, 5, 1, 64, 16, list(range(0, 400, 3))), (2, 16, 2, 128, 128, [20000, 3, 9000]), (5, 3, 1, 64, 16, [60] * 1500),
                                                 (8, 2, 1, 64, 256, [5000, 8, 40])])
def test_few_rows_over_eight_bits(fmt, N, Hq, Hk, D, page, lens):
    _few_rows(fmt, N, Hq, Hk, D, page, lens)


# Up to 8 rows: up to 256 pairs of a sequence and a key head, or tables of up to 1,024 tokens.  Up to 16: up to 8 pairs, or at least
# 1,024 with tables of up to 512.
@pytest.mark.parametrize("N,Hq,Hk,D,page,lens", [(1, 8, 2, 128, 16, [1, 700, 0, 33]), (4, 8, 2, 64, 32, [300, 4, 0]), (16, 2, 2, 128, 64, [500, 16, 3]),
                                                 (3, 2, 1, 64, 16, list(range(0, 400, 3))), (2, 16, 2, 128, 128, [20000, 3, 9000]),
                                                 (5, 1, 1, 64, 16, [60] * 250), (8, 1, 1, 128, 256, [5000, 8, 40]), (8, 2, 2, 64, 16, [4100, 3, 777] * 40),
                                                 (2, 12, 3, 128, 32, [1100, 1, 65, 64, 2] * 17), (2, 12, 3, 128, 32, [1100, 1, 65, 64, 2] * 18),
                                                 (2, 8, 2, 128, 16, [60, 2, 33] * 150), (1, 8, 2, 128, 64, [900, 1, 257] * 230), (4, 16, 4, 128, 32, [60, 4, 133] * 120),
                                                 (3, 40, 8, 64, 128, [300, 3, 128] * 44)])
def test_few_rows_in_bfloat16(N, Hq, Hk, D, page, lens):
    _few_rows("bf16", N, Hq, Hk, D, page, lens)


def _few_rows(fmt, N, Hq, Hk, D, page, lens):
    """Trees of few rows go another way: padding, masks that are no trees, pages and lengths that are wrong."""
    nodes = [min(n, (i * 5 + 1) % (N + 1)) for i, n in enumerate(lens)]
    q, c, table, n, tree, k = _case(N + Hq, lens, N, Hq, Hk, D, page, fmt, nodes=nodes)
    out, lse = _check((q, c, table, n, tree, k))
    for b, m in enumerate(nodes):
        assert (out[b, m:] == 0).all() and (lse[b, m:] == -math.inf).all()
    g = torch.Generator(device=DEV).manual_seed(1)
    wild = torch.randint(-2 ** 62, 2 ** 62, tree.shape, generator=g, device=DEV)
    wild[0] = 0
    _check((q, c, table, n, wild, k), scale=-0.2)
    _check((q, c, table, n, wild[-1].contiguous(), k))
    size = tps.tree_attention_workspace(q.shape, c, table.shape[1])
    again = tps.tree_attention(q, c, table, n, tree, nodes=k, workspace=torch.empty(max(size, 1), dtype=torch.uint8, device=DEV))
    assert torch.equal(again, out)
    want, table, n, k = _want(q, c, table, n, tree, k, D ** -0.5), table.clone(), n.clone(), k.clone()
    table[0, 0], n[1], k[2] = c.n_pages, page * table.shape[1] + 1, N + 1
    st = torch.full((len(lens),), 9, dtype=torch.int32, device=DEV)
    out, lse = tps.tree_attention(q, c, table, n, tree, nodes=k, want_lse=True, status=st)
    good = torch.arange(3, len(lens), device=DEV)
    assert st[:3].tolist() == [3 if lens[0] else 0, 3, 3] and (st[3:] == 0).all()
    assert out[1].isnan().all() and out[2].isnan().all() and (not lens[0] or out[0].isnan().all())
    plain.check(out, lse, want, BF16, good)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("N,Hq,Hk,D", [(4, 4, 2, 64), (8, 1, 1, 128), (4, 8, 2, 128), (16, 1, 1, 64)])
@pytest.mark.parametrize("length", [16, 18, 130, 4100])
def test_few_rows_in_bfloat16_hidden_nodes_hold_anything(bad, N, Hq, Hk, D, length):
    q, c, table, lens, tree, _ = _case(13, [length, 300], N, Hq, Hk, D, 16, "bf16")
    base, base_lse = tps.tree_attention(q, c, table, lens, tree, want_lse=True)
    for j in range(N):
        at = length - N + j
        page, row = int(table[0, at // 16]), at % 16
        sees = (tree[0] >> j) & 1 == 1
        for x in (c.k, c.v):
            keep = x[page, :, row, 5::9].clone()
            x[page, :, row, 5::9] = bad
            out, lse = tps.tree_attention(q, c, table, lens, tree, want_lse=True)
            x[page, :, row, 5::9] = keep
            assert torch.equal(out[0, ~sees], base[0, ~sees]) and torch.equal(lse[0, ~sees], base_lse[0, ~sees])
            assert torch.equal(out[1], base[1]) and torch.equal(lse[1], base_lse[1])
            if x is c.v:
                other = torch.ones(D, dtype=torch.bool, device=DEV)
                other[5::9] = False
                assert torch.equal(lse, base_lse) and torch.equal(out[0][..., other], base[0][..., other])
                assert (out[0, sees][..., ~other].isnan() if math.isnan(bad) else out[0, sees][..., ~other] == bad).all()


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("length", [4, 16, 18, 130, 3000])
def test_few_rows_hidden_nodes_hold_anything(fmt, bad, length):
    q, c, table, lens, tree, _ = _case(13, [length, 300], 4, 8, 2, 64, 16, fmt)
    base, base_lse = tps.tree_attention(q, c, table, lens, tree, want_lse=True)
    for j in range(4):
        at = length - 4 + j
        page, row = int(table[0, at // 16]), at % 16
        sees = (tree[0] >> j) & 1 == 1
        for x in (c.k_scale, c.v_scale):
            keep = x[page, :, row].clone()
            x[page, :, row] = bad
            out, lse = tps.tree_attention(q, c, table, lens, tree, want_lse=True)
            x[page, :, row] = keep
            assert torch.equal(out[0, ~sees], base[0, ~sees]) and torch.equal(lse[0, ~sees], base_lse[0, ~sees])
            assert torch.equal(out[1], base[1]) and torch.equal(lse[1], base_lse[1])
            assert x is c.k_scale or (~torch.isfinite(out[0, sees])).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("length", [12, 128, 133, 900])
def test_hidden_nodes_hold_anything(fmt, bad, length):
    """A node that is not seen changes no output, whatever it holds; one that is seen does."""
    N = 12
    q, c, table, lens, tree, _ = _case(6, [length, 300], N, 8, 2, 64, 16, fmt)
    base, base_lse = tps.tree_attention(q, c, table, lens, tree, want_lse=True)
    for j in (0, 5, 11):
        at = length - N + j
        page, row = int(table[0, at // 16]), at % 16
        sees = (tree[0] >> j) & 1 == 1
        for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
            x = t if s is None else s
            keep = x[page, :, row].clone()
            x[page, :, row] = bad
            out, lse = tps.tree_attention(q, c, table, lens, tree, want_lse=True)
            x[page, :, row] = keep
            hidden = ~sees
            if fmt == "bf16":
                assert torch.equal(out[0, hidden], base[0, hidden]) and torch.equal(lse[0, hidden], base_lse[0, hidden])
            else:  # another way through the same sums: each rounding may differ
                tol = 2 * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12)
                scale = base[0, hidden].double().abs().amax(-1, keepdim=True).clamp(min=1)
                assert ((out[0, hidden].double() - base[0, hidden].double()).abs() <= tol * 8 * scale).all()
                assert ((lse[0, hidden] - base_lse[0, hidden]).abs() <= 2.0 ** -12).all()
            assert torch.equal(out[1], base[1]) and torch.equal(lse[1], base_lse[1])
            if (x is c.v or x is c.v_scale) and (fmt == "bf16" or bad != -math.inf):  # a scale below 2^-80 counts as anything up to that
                assert (~torch.isfinite(out[0, sees])).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("lens", [[500, 40, 300, 77, 10, 9, 33, 12], [9000, 40, 3000, 77, 10, 9, 33, 12]])
def test_bad_pages_and_lengths_are_told_and_stay_with_their_sequence(fmt, lens):
    q, c, table, n, tree, _ = _case(7, lens, 8, 4, 2, 128, 16, fmt)
    want = _want(q, c, table, n, tree, None, 128 ** -0.5)
    table, n = table.clone(), n.clone()
    table[0, lens[0] // 32], table[2, 0] = c.n_pages, -1
    table[1, -1] = 2 ** 31 - 1  # not a page of its tokens
    n[4], n[5], n[6] = 7, -3, 16 * table.shape[1] + 1
    st = torch.full((8,), 9, dtype=torch.int32, device=DEV)
    for status in (st, None):
        out, lse = tps.tree_attention(q, c, table, n, tree, want_lse=True, status=status)
        good = torch.tensor([1, 3, 7], device=DEV)
        plain.check(out, lse, want, BF16, good)
        for b in (0, 2, 4, 5, 6):
            assert out[b].isnan().all() and lse[b].isnan().all()
    assert st.tolist() == [3, 0, 3, 0, 3, 3, 3, 0]
    k = torch.tensor([8, 9, 8, 8, 8, 8, 8, -1], dtype=torch.int32, device=DEV)
    out, _ = tps.tree_attention(q, c, table, n, tree, nodes=k, want_lse=True, status=st)
    assert st.tolist() == [3, 3, 3, 0, 3, 3, 3, 3] and out[1].isnan().all() and out[7].isnan().all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("N,Hq,Hk,D", [(2, 4, 2, 64), (12, 8, 2, 128), (64, 8, 2, 64), (64, 10, 2, 128)])
def test_scores_of_great_magnitude(fmt, N, Hq, Hk, D):
    """Scores up to 10^8, over 8-bit caches 10^7 (tests/_serve.py)."""
    q, c, table, lens, tree, _ = _case(16, [700, 64, 130, 30000], N, Hq, Hk, D, 16, fmt, poison=False)
    k, factor = plain.great_keys(16, c.n_pages * 16, Hk, D, 1e8 if fmt == "bf16" else 1e7)
    v = torch.randn(c.n_pages * 16, Hk, D, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).bfloat16()
    tps.kv_write(c, k, v, torch.arange(c.n_pages * 16, device=DEV))
    plain.great_queries(q, factor)
    out, lse = tps.tree_attention(q, c, table, lens, tree, scale=0.125, want_lse=True)
    plain.check_great(out, lse, _want(q, c, table, lens, tree, None, 0.125), fmt != "bf16")


def test_strided_tables_given_outputs_and_workspaces():
    q, c, table, lens, tree, _ = _case(8, [400, 90, 2000], 10, 8, 2, 128, 32, "fp8")
    base = tps.tree_attention(q, c, table, lens, tree)
    wide = torch.full((3, table.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    wide[:, 2:2 + table.shape[1]] = table
    out = torch.empty_like(q)
    size = tps.tree_attention_workspace(q.shape, c, table.shape[1])
    ws = torch.full((size + 256,), 255, dtype=torch.uint8, device=DEV)
    got = tps.tree_attention(q, c, wide[:, 2:2 + table.shape[1]], lens, tree, out=out, workspace=ws[:size])
    assert got is out and torch.equal(out, base) and (ws[size:] == 255).all()
    with pytest.raises(RuntimeError):
        tps.tree_attention(q, c, table, lens, tree, workspace=ws[:size - 256])
    assert tps.tree_attention(q[:0], c, table[:0], lens[:0], tree[:0]).shape == (0, 10, 8, 128)
    none = torch.zeros(2, 0, dtype=torch.int32, device=DEV)
    assert tps.tree_attention(q[:2].contiguous(), c, none, torch.zeros(2, dtype=torch.int32, device=DEV), tree[:2],
                              nodes=torch.zeros(2, dtype=torch.int32, device=DEV)).eq(0).all()


def test_streams_and_graphs():
    args = [_case(9 + i, [700, 30, 256], 6, 8, 2, 64, 16, f) for i, f in enumerate(("bf16", "fp8", "int8"))]
    want = [tps.tree_attention(*a[:5]) for a in args]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [(i, tps.tree_attention(*args[i][:5], stream=streams[(i + j) % 3])) for j in range(9) for i in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in outs)
    graphs, outs = [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(tps.tree_attention(*a[:5]))
        graphs.append(g)
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_cache_past_four_gigabytes():
    pages, H, page, D = 37000, 8, 128, 128
    k, v = (torch.empty((pages, H, page, D), dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((pages, H, page), math.nan, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c = tps.KVCache(k, v, ks, vs)
    g = torch.Generator(device=DEV).manual_seed(8)
    T, ids = 300, torch.tensor([36999, 2, 35000], device=DEV)
    slots = ids[torch.arange(T, device=DEV) // page] * page + torch.arange(T, device=DEV) % page
    x, y = (torch.randn(T, H, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    tps.kv_write(c, x, y, slots)
    near = tps.KVCache.empty(3, H, page, D, "int8", device=DEV)
    tps.kv_write(near, x, y, torch.arange(T, device=DEV))
    q, tree = torch.randn(1, 7, 16, D, generator=g, device=DEV).bfloat16(), _trees(g, 1, 7)
    n = torch.tensor([T], dtype=torch.int32, device=DEV)
    a = tps.tree_attention(q, c, ids.int()[None], n, tree)
    assert torch.equal(a, tps.tree_attention(q, near, torch.arange(3, dtype=torch.int32, device=DEV)[None], n, tree))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("lens", [[500, 40], [60000, 200]])
def test_a_wait_that_runs_out_reaches_the_status(fmt, lens):
    q, c, table, n, tree, _ = _case(10, lens, 4, 4, 2, 64, 16, fmt)
    out, st = torch.zeros_like(q), torch.zeros(2, dtype=torch.int32, device=DEV)
    a = decode._Tree(q=q.data_ptr(), out=out.data_ptr(), page_table=table.data_ptr(), seq_len=n.data_ptr(), tree=tree.data_ptr(),
                     out_status=st.data_ptr(), B=2, table_width=table.shape[1], table_ld=table.shape[1], tree_ld=4, n_nodes=4, n_q_heads=4, scale=0.125)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert tps.load().tps_tree_attention_stall_test(c._bytes, ctypes.byref(a), 1, 20_000_000, stream) == 0
    torch.cuda.synchronize()
    assert st.tolist() == [4, 4] and out[:, :, 2:].isnan().all()
    want = tps.tree_attention(q, c, table, n, tree, status=st)
    assert st.tolist() == [0, 0] and torch.isfinite(want).all()
    fine = ~out.isnan()
    assert torch.equal(out[fine], want[fine])


# Rows of a key head: 48 (two softmax groups take blocks in turn), 256 (two row tiles at once), 320 (three tiles of 128 in turn).
SHAPES = [(12, 8, 2), (64, 8, 2), (64, 10, 2)]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("N,Hq,Hk", SHAPES)
@pytest.mark.parametrize("more", [0, 200])  # cut over many CTAs; whole items of several sequences in each
def test_many_rows_padding_and_masks_that_are_no_trees(fmt, N, Hq, Hk, more):
    lens, nodes = [0, 1, N, N, 40 + N, 500, 128 + N, 129, 256], [0, 1, N, N - 1, 1, N // 2, N, 0, 3 * N // 4]
    lens, nodes = lens + [N + i % 90 for i in range(more)], nodes + [i % (N + 1) for i in range(more)]
    q, c, table, n, tree, k = _case(14, lens, N, Hq, Hk, 64, 32, fmt, nodes=nodes)
    out, lse = _check((q, c, table, n, tree, k))
    for b, m in enumerate(nodes):
        assert (out[b, m:] == 0).all() and (lse[b, m:] == -math.inf).all()
    full = torch.tensor([max(x, N) for x in lens], dtype=torch.int32, device=DEV)
    q2, c2, table2, n2, _, _ = _case(15, full.tolist(), N, Hq, Hk, 128, 16, fmt)
    g = torch.Generator(device=DEV).manual_seed(1)
    wild = torch.randint(-2 ** 62, 2 ** 62, tree.shape, generator=g, device=DEV)
    wild[2, ::3], wild[3], wild[6, 1] = 0, 0, 0  # sequences 2 and 3 are all tree: those rows see nothing
    out, lse = _check((q2, c2, table2, n2, wild, None))
    assert (out[2, ::3] == 0).all() and (lse[3] == -math.inf).all() and torch.isfinite(lse[6, 1]).all()
    few = k.clone()
    few[:4] = torch.tensor([N, 0, 1, N // 3], dtype=torch.int32, device=DEV)
    _check((q2, c2, table2, n2, wild, few), scale=-0.2)
    _check((q2, c2, table2, n2, wild[5].contiguous(), few))
    q2[3, N // 3:] = math.nan  # padding's queries hold anything
    out, _ = tps.tree_attention(q2, c2, table2, n2, wild, nodes=few, want_lse=True)
    assert torch.isfinite(out).all() and (out[3, N // 3:] == 0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,Hq,Hk", SHAPES)
def test_a_lone_token_of_a_large_tree_has_its_value_as_it_is(D, N, Hq, Hk):
    """The rounded weight is divided by itself: on the matrix unit, too."""
    q, c, table, _, tree, _ = _case(12, [200] * 5, N, Hq, Hk, D, 16, "bf16")
    one = torch.ones(5, dtype=torch.int32, device=DEV)
    out, lse = tps.tree_attention(q, c, table, one, tree, nodes=one, want_lse=True)
    none = tps.tree_attention(q, c, table, 130 * one, tree, nodes=0 * one)
    for b in range(5):
        assert torch.equal(out[b, 0], c.v[table[b, 0], :, 0].repeat_interleave(Hq // Hk, 0))
    assert (out[:, 1:] == 0).all() and (lse[:, 1:] == -math.inf).all() and (none == 0).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("N,Hq,Hk", SHAPES)
@pytest.mark.parametrize("lens", [[500, 64, 300, 77, 100, 90, 133, 65], [9000, 64, 3000, 77, 100, 90, 133, 65], [500, 64, 300, 77, 100, 90, 133, 65] + [70] * 300])
def test_bad_pages_and_lengths_beside_large_trees(fmt, N, Hq, Hk, lens):
    q, c, table, n, tree, _ = _case(7, lens, N, Hq, Hk, 128, 32, fmt)
    B = len(lens)
    want = _want(q, c, table, n, tree, None, 128 ** -0.5)
    table, n = table.clone(), n.clone()
    table[0, lens[0] // 32], table[2, 0] = c.n_pages, -1
    table[1, -1] = 2 ** 31 - 1  # not a page of its tokens
    n[4], n[5], n[6] = N - 1, -3, 32 * table.shape[1] + 1
    st, rest = torch.full((B,), 9, dtype=torch.int32, device=DEV), [0] * (B - 8)
    good = torch.tensor([1, 3, *range(7, B)], device=DEV)
    for status in (st, None):
        out, lse = tps.tree_attention(q, c, table, n, tree, want_lse=True, status=status)
        plain.check(out, lse, want, BF16, good)
        for b in (0, 2, 4, 5, 6):
            assert out[b].isnan().all() and lse[b].isnan().all()
    assert st.tolist() == [3, 0, 3, 0, 3, 3, 3, 0] + rest
    k = torch.tensor([N, N + 1, 0, N, 0, 0, 0, -1] + [N] * (B - 8), dtype=torch.int32, device=DEV)
    out, lse = tps.tree_attention(q, c, table, n, tree, nodes=k, want_lse=True, status=st)
    assert st.tolist() == [3, 3, 3, 0, 0, 3, 3, 3] + rest
    plain.check(out, lse, want, BF16, torch.tensor([3, *range(8, B)], device=DEV))
    for b in (0, 1, 2, 5, 6, 7):
        assert out[b].isnan().all() and lse[b].isnan().all()
    assert (out[4] == 0).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("N,Hq,Hk", SHAPES)
@pytest.mark.parametrize("length,more", [(64, 0), (130, 0), (900, 0), (133, 200)])
def test_hidden_nodes_of_large_trees_hold_anything(fmt, bad, N, Hq, Hk, length, more):
    """A node that is not seen changes no output, whatever it holds (in 8 bits beyond its roundings); one that is seen does."""
    q, c, table, lens, tree, _ = _case(6, [length, 300] + [N + i % 50 for i in range(more)], N, Hq, Hk, 64, 16, fmt)
    base, base_lse = tps.tree_attention(q, c, table, lens, tree, want_lse=True)
    want = _want(q, c, table, lens, tree, None, 0.125)
    here = [x[0] for x in want]
    for j in (0, N // 2, N - 1):
        at = length - N + j
        page, row = int(table[0, at // 16]), at % 16
        sees = (tree[0] >> j) & 1 == 1
        hidden = ~sees
        for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
            x = t if s is None else s
            keep = x[page, :, row].clone()
            x[page, :, row] = bad
            out, lse = tps.tree_attention(q, c, table, lens, tree, want_lse=True)
            x[page, :, row] = keep
            if fmt == "bf16":
                assert torch.equal(out[0, hidden], base[0, hidden]) and torch.equal(lse[0, hidden], base_lse[0, hidden])
            else:
                plain.check(out[0], lse[0], here, BF16, hidden)
            assert torch.equal(out[1:], base[1:]) and torch.equal(lse[1:], base_lse[1:])
            if (x is c.v or x is c.v_scale) and (fmt == "bf16" or bad != -math.inf):  # a scale below 2^-80 counts as anything up to that
                assert (~torch.isfinite(out[0, sees])).all()


@pytest.mark.parametrize("fmt,N", [("bf16", 24), ("fp8", 24), ("int8", 24), ("int8", 64)])
def test_large_trees_in_a_cache_past_four_gigabytes(fmt, N):
    H, page, D = 8, 128, 128
    pages = 18500 if fmt == "bf16" else 37000
    dt = tps.KVCache.FORMATS[fmt][1]
    k, v = (torch.empty((pages, H, page, D), dtype=torch.int16 if fmt == "bf16" else torch.int8, device=DEV).view(dt) for _ in range(2))
    ks, vs = (None if fmt == "bf16" else torch.full((pages, H, page), math.nan, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c = tps.KVCache(k, v, ks, vs)
    g = torch.Generator(device=DEV).manual_seed(8)
    T, ids = 300, torch.tensor([pages - 1, 2, pages - 2000], device=DEV)
    slots = ids[torch.arange(T, device=DEV) // page] * page + torch.arange(T, device=DEV) % page
    x, y = (torch.randn(T, H, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    tps.kv_write(c, x, y, slots)
    near = tps.KVCache.empty(3, H, page, D, fmt, device=DEV)
    tps.kv_write(near, x, y, torch.arange(T, device=DEV))
    q, tree = torch.randn(1, N, 32, D, generator=g, device=DEV).bfloat16(), _trees(g, 1, N)
    n = torch.tensor([T], dtype=torch.int32, device=DEV)
    a = tps.tree_attention(q, c, ids.int()[None], n, tree)
    assert torch.isfinite(a).all()
    assert torch.equal(a, tps.tree_attention(q, near, torch.arange(3, dtype=torch.int32, device=DEV)[None], n, tree))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,Hq,Hk", SHAPES)
@pytest.mark.parametrize("lens", [[500, 70], [60000, 200], [64, 700] * 60])
def test_a_wait_that_runs_out_reaches_every_sequence_beside_it(fmt, D, N, Hq, Hk, lens):
    """Of the kernel on the matrix unit.  An output is NaN, and its sequence's status tells, or it is what it is without the stall."""
    q, c, table, n, tree, _ = _case(10, lens, N, Hq, Hk, D, 16, fmt)
    B = len(lens)
    out, lse, st = torch.zeros_like(q), torch.zeros(B, N, Hq, device=DEV), torch.full((B,), 9, dtype=torch.int32, device=DEV)
    a = decode._Tree(q=q.data_ptr(), out=out.data_ptr(), out_lse=lse.data_ptr(), page_table=table.data_ptr(), seq_len=n.data_ptr(), tree=tree.data_ptr(),
                     out_status=st.data_ptr(), B=B, table_width=table.shape[1], table_ld=table.shape[1], tree_ld=N, n_nodes=N, n_q_heads=Hq, scale=D ** -0.5)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    want, want_lse = tps.tree_attention(q, c, table, n, tree, want_lse=True)
    assert torch.isfinite(want).all()
    assert tps.load().tps_tree_attention_stall_test(c._bytes, ctypes.byref(a), 1, 20_000_000, stream) == 0
    torch.cuda.synchronize()
    assert (st == 4).all() and out[:, :, Hq // 2:].isnan().all() and lse[:, :, Hq // 2:].isnan().all()
    fine = ~out.isnan()
    assert torch.equal(fine.all(-1), fine.any(-1)) and torch.equal(fine.all(-1), ~lse.isnan())
    assert torch.equal(out[fine], want[fine]) and torch.equal(lse[fine.all(-1)], want_lse[fine.all(-1)])
    again = tps.tree_attention(q, c, table, n, tree, status=st)
    assert (st == 0).all() and torch.equal(again, want)


def test_refusals():
    q, c, table, lens, tree, _ = _case(11, [100, 20], 4, 4, 2, 64, 16, "bf16")
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    for args in ((q.float(), c, table, lens, tree), (q[:, :, ::2], c, table, lens, tree), (q[0], c, table, lens, tree), (q, None, table, lens, tree),
                 (q, c, table.long(), lens, tree), (q, c, table[:1], lens, tree), (q, c, table.T.contiguous().T, lens, tree), (q, c, table, lens.long(), tree),
                 (q, c, table, one, tree), (q, c, table, lens, tree.int()), (q, c, table, lens, tree[:, :3]), (q, c, table, lens, tree[:1]),
                 (q, c, table, lens, tree.cpu()), (q[:, :, :3].contiguous(), c, table, lens, tree), (q[:, :0], c, table, lens, tree[:, :0]),
                 (torch.zeros(2, 65, 4, 64, dtype=torch.bfloat16, device=DEV), c, table, lens, torch.zeros(2, 65, dtype=torch.int64, device=DEV)),
                 (q[..., :32].contiguous(), c, table, lens, tree), (q.cpu(), c, table, lens, tree), (q, c, table[:1].expand(2, -1), lens, tree)):
        with pytest.raises(ValueError):
            tps.tree_attention(*args)
    for kw in (dict(nodes=one), dict(status=one), dict(out=q.float()), dict(workspace=torch.zeros(4))):
        with pytest.raises(ValueError):
            tps.tree_attention(q, c, table, lens, tree, **kw)
    with pytest.raises(RuntimeError):
        tps.tree_attention(q, c, table, lens, tree, scale=math.inf)
    with pytest.raises(ValueError):
        tps.tree_attention_workspace((2, 65, 4, 64), c, 4)
