"""Attention of packed prompts against its plain 64-bit form (tolerances: tests/_serve.py)."""
import ctypes
import math

import pytest
import torch

import nucleus_token_sampler_gb300 as tps
from nucleus_token_sampler_gb300 import decode

from . import _serve as plain

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda:0"
BF16 = 2.0 ** -8


def _heads(seed, T, Hq, Hk, D, spare=0):
    """q, k, v cut out of one projection of T (+ spare) tokens."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T + spare, Hq + 2 * Hk, D, generator=g, device=DEV).bfloat16()
    x[:, :Hq] *= 2
    return x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]


def _bounds(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu, torch.tensor(cu, dtype=torch.int32, device=DEV)


LENGTHS = [[1], [2], [127], [128], [129], [64, 64], [0, 0, 5], [255, 256, 257], [130, 1, 0, 257], [700, 33], [3, 0, 1000, 2, 500]]


@pytest.mark.parametrize("status", [False, True])
@pytest.mark.parametrize("Hq,Hk,D", [(1, 1, 64), (8, 2, 128), (5, 1, 128), (4, 4, 64), (14, 2, 64), (32, 8, 128)])
def test_prompts(Hq, Hk, D, status):
    for lens in LENGTHS:
        cu, c = _bounds(lens)
        q, k, v = _heads(sum(lens), cu[-1], Hq, Hk, D)
        st = torch.full((len(lens),), 9, dtype=torch.int32, device=DEV) if status else None
        out, lse = tps.prompt_attention(q, k, v, c, want_lse=True, status=st)
        plain.check(out, lse, plain.prompt(q, k, v, zip(cu, cu[1:]), D ** -0.5), BF16)
        assert not status or (st == 0).all()


@pytest.mark.parametrize("lens,Hq,Hk,D", [([4001], 4, 1, 128), ([90] * 200, 8, 2, 128), ([2500, 7, 1900], 3, 1, 64), ([600, 40], 100, 1, 64),
                                          ([300], 128, 1, 128), ([200, 33], 200, 1, 64), ([150], 600, 2, 128),
                                          (list(range(400)), 2, 1, 64), ([1] * 1500, 4, 2, 128)])
def test_many_tiles_and_many_heads_to_a_key_head(lens, Hq, Hk, D):
    cu, c = _bounds(lens)
    q, k, v = _heads(len(lens), cu[-1], Hq, Hk, D)
    out, lse = tps.prompt_attention(q, k, v, c, want_lse=True)
    plain.check(out, lse, plain.prompt(q, k, v, zip(cu, cu[1:]), D ** -0.5), BF16)


@pytest.mark.parametrize("scale", [0.5, -0.3, 0.0, 1e-30, 3.0])
def test_scales(scale):
    cu, c = _bounds([200, 5])
    q, k, v = _heads(1, 205, 4, 2, 64)
    out, lse = tps.prompt_attention(q, k, v, c, scale=scale, want_lse=True)
    plain.check(out, lse, plain.prompt(q, k, v, zip(cu, cu[1:]), scale), BF16)


def test_scores_that_rise_and_fall_along_the_keys():
    """The reference is raised in the first, in a later and in the last block, and by more than float32's exponents hold."""
    cu, c = _bounds([700, 700, 700])
    q, k, v = _heads(2, 2100, 4, 1, 128)
    ramp = torch.linspace(0, 4, 700, device=DEV)
    k = (k.float() * torch.cat([ramp, 4 - ramp, 30 * (ramp > 3.9)])[:, None, None]).bfloat16()
    out, lse = tps.prompt_attention(q, k, v, c, want_lse=True)
    plain.check(out, lse, plain.prompt(q, k, v, zip(cu, cu[1:]), 128 ** -0.5), BF16)


@pytest.mark.parametrize("Hq,Hk,D", [(4, 2, 64), (3, 1, 128)])
def test_scores_of_great_magnitude(Hq, Hk, D):
    """Scores up to 10^8 (tests/_serve.py)."""
    cu, c = _bounds([700, 1, 130, 300])
    q, _, v = (x.contiguous() for x in _heads(13, cu[-1], Hq, Hk, D))
    k, factor = plain.great_keys(13, cu[-1], Hk, D, 1e8)
    plain.great_queries(q, factor)
    out, lse = tps.prompt_attention(q, k, v, c, scale=0.125, want_lse=True)
    plain.check_great(out, lse, plain.prompt(q, k, v, zip(cu, cu[1:]), 0.125), False)


@pytest.mark.parametrize("D", [64, 128])
def test_a_lone_token_has_its_value_as_it_is(D):
    """The rounded weight is divided by itself."""
    cu, c = _bounds([1, 300, 1, 2])
    q, k, v = _heads(11, 304, 6, 2, D)
    out = tps.prompt_attention(q, k, v, c)
    for t in (0, 1, 301, 302):
        assert torch.equal(out[t], v[t].repeat_interleave(3, 0))


def test_strides_out_and_rows_of_no_sequence():
    cu, c = _bounds([100, 0, 140], first=3)
    T = cu[-1] + 9
    q, k, v = _heads(3, T, 6, 2, 64)
    want = plain.prompt(q, k, v, zip(cu, cu[1:]), 0.125)
    mine = slice(cu[0], cu[-1])
    ahead = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # heads ahead of tokens in memory
    wide = torch.zeros(T, 6, 72, dtype=torch.bfloat16, device=DEV)
    wide[..., :64] = q
    for qq, kk, vv in ((q, k, v), (q.contiguous(), k.contiguous(), v.contiguous()), (ahead(q), ahead(k), ahead(v)), (wide[..., :64], k, ahead(v))):
        out = torch.full((T, 6, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        got, lse = tps.prompt_attention(qq, kk, vv, c, want_lse=True, out=out)
        assert got is out
        plain.check(got, lse, want, BF16, mine)
        assert (out[:cu[0]] == 7).all() and (out[cu[-1]:] == 7).all()


@pytest.mark.parametrize("Hq,Hk,D", [(4, 1, 128), (2, 2, 64), (6, 2, 64)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_hidden_tokens_hold_anything(Hq, Hk, D, bad):
    """Later tokens, the next sequence and the rows behind the last one change no bit; a row that sees such a value has it."""
    lens = [150, 300]
    cu, c = _bounds(lens)
    q, k, v = (x.clone() for x in _heads(4, 450, Hq, Hk, D, spare=20))
    base, base_lse = tps.prompt_attention(q, k, v, c, want_lse=True)
    for x in (q, k, v):
        x[450:] = bad
    for j in (0, 1, 149, 150, 151, 277, 449):
        v2 = v.clone()
        v2[j, :, 5] = bad
        out, lse = tps.prompt_attention(q, k, v2, c, want_lse=True)
        sees = torch.arange(450, device=DEV) >= j
        if j < 150:
            sees &= torch.arange(450, device=DEV) < 150
        assert torch.equal(out[:450][~sees], base[:450][~sees]) and torch.equal(lse[:450], base_lse[:450])
        assert (~torch.isfinite(out[:450][sees][..., 5])).all()
        rest = torch.arange(D, device=DEV) != 5
        assert torch.equal(out[:450][..., rest], base[:450][..., rest])
        k2 = k.clone()
        k2[j] = bad
        out, lse = tps.prompt_attention(q, k2, v, c, want_lse=True)
        assert torch.equal(out[:450][~sees], base[:450][~sees]) and torch.equal(lse[:450][~sees], base_lse[:450][~sees])
        q2 = q.clone()
        q2[j] = bad
        out, lse = tps.prompt_attention(q2, k, v, c, want_lse=True)
        other = torch.arange(450, device=DEV) != j
        assert torch.equal(out[:450][other], base[:450][other]) and out[j].isnan().all()


@pytest.mark.parametrize("Hq,Hk,D", [(1, 1, 64), (2, 2, 128)])
def test_values_taken_out_reach_their_rows_ahead_of_many_short_prompts(Hq, Hk, D):
    """Each CTA has a prompt of two query tiles, whose second one sees values that are not finite, and then more prompts of one
    tile than there are marks of such values."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lens = [140 + i % 100 for i in range(sms // Hk)] + [1 + i % 9 for i in range(12 * sms)]
    cu, c = _bounds(lens)
    q, k, v = (x.clone() for x in _heads(12, cu[-1], Hq, Hk, D))
    base, base_lse = tps.prompt_attention(q, k, v, c, want_lse=True)
    sees = torch.zeros(cu[-1], dtype=torch.bool, device=DEV)
    for i in range(sms // Hk):
        at = cu[i] + 128 + i % 11  # the second tile begins at 128
        v[at, :, 3] = math.inf
        sees[at:cu[i + 1]] = True
    rest = torch.arange(D, device=DEV) != 3
    for _ in range(20):
        out, lse = tps.prompt_attention(q, k, v, c, want_lse=True)
        assert (out[sees][..., 3] == math.inf).all() and torch.equal(out[~sees], base[~sees])
        assert torch.equal(out[..., rest], base[..., rest]) and torch.equal(lse, base_lse)


def test_bounds_that_are_not_in_order():
    q, k, v = _heads(5, 300, 4, 2, 64)
    for cu, good in (([0, 100, 50, 60, 200, 300], [1, 0, 0, 0, 1]), ([-1, 5, 10], [0, 1]), ([0, 301], [0]), ([0, 10, 400, 20, 30], [1, 0, 0, 0]),
                     ([200, 100, 250], [0, 0]), ([0, 2 ** 31 - 1, 5], [0, 0]), ([-2 ** 31, 2 ** 31 - 1], [0]), ([300, 300], [1])):
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        st = torch.full((len(good),), 9, dtype=torch.int32, device=DEV)
        pairs = [p for p, ok in zip(zip(cu, cu[1:]), good) if ok]
        want = plain.prompt(q, k, v, pairs, 0.125)
        covered = ~want[1][:, 0].isnan()
        for s in (st, None):
            out = torch.full((300, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
            got, lse = tps.prompt_attention(q, k, v, c, want_lse=True, out=out, status=s)
            plain.check(got, lse, want, BF16, covered)
            assert (out[~covered] == 7).all()
        assert st.tolist() == [0 if ok else 3 for ok in good]


def test_no_tokens_and_no_sequences():
    q, k, v = _heads(6, 4, 2, 1, 64)
    st = torch.full((3,), 9, dtype=torch.int32, device=DEV)
    c = torch.tensor([0, 0, 0, 1], dtype=torch.int32, device=DEV)
    assert tps.prompt_attention(q[:0], k[:0], v[:0], c, status=st).shape == (0, 2, 64)
    assert st.tolist() == [0, 0, 3]
    out = torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    tps.prompt_attention(q, k, v, c[:1], out=out)
    assert (out == 7).all()


def test_repeats_itself_on_other_streams_and_in_graphs():
    cu, c = _bounds([500, 3, 900, 128])
    q, k, v = _heads(7, cu[-1], 8, 2, 128)
    want = tps.prompt_attention(q, k, v, c)
    for _ in range(50):
        assert torch.equal(tps.prompt_attention(q, k, v, c), want)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [tps.prompt_attention(q, k, v, c, stream=s) for s in streams for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(tps.prompt_attention(q, k, v, c))
        graphs.append(g)
    for s, g in zip(streams, graphs):  # both in flight at once
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_rows_past_thirty_two_bits():
    """Elements whose index does not fit 32 bits (7.4 GB of queries, keys and values)."""
    T, n = 600_000, 400
    x = torch.empty(T, 48, 128, dtype=torch.bfloat16, device=DEV)
    x[-n:] = torch.randn(n, 48, 128, generator=torch.Generator(device=DEV).manual_seed(8), device=DEV).bfloat16()
    c = torch.tensor([T - n, T - 150, T], dtype=torch.int32, device=DEV)
    out, lse = tps.prompt_attention(x[:, :32], x[:, 32:40], x[:, 40:], c, want_lse=True)
    near = x[-n:]
    plain.check(out[-n:], lse[-n:], plain.prompt(near[:, :32], near[:, 32:40], near[:, 40:], [(0, n - 150), (n - 150, n)], 128 ** -0.5), BF16)


def test_a_wait_that_runs_out_reaches_the_status():
    cu, c = _bounds([300, 40])
    q, k, v = _heads(9, 340, 4, 2, 64)
    out = torch.zeros(340, 4, 64, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(2, dtype=torch.int32, device=DEV)
    a = decode._Prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), None, c.data_ptr(), st.data_ptr(), 340, 2,
                       q.stride(0), q.stride(1), k.stride(0), k.stride(1), v.stride(0), v.stride(1), 4, 2, 64, 0.125)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert tps.load().tps_prompt_attention_stall_test(ctypes.byref(a), 1, 20_000_000, stream) == 0
    torch.cuda.synchronize()
    assert st.tolist() == [4, 4] and out[:, 2:].isnan().all()
    want = tps.prompt_attention(q, k, v, c, status=st)
    assert st.tolist() == [0, 0]
    fine = ~out[:, :2].isnan()
    assert torch.equal(out[:, :2][fine], want[:, :2][fine])


def test_refusals():
    q, k, v = _heads(10, 8, 4, 2, 64)
    c = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    odd = torch.zeros(8, 4, 68, dtype=torch.bfloat16, device=DEV)[..., :64]
    shifted = torch.zeros(8 * 4 * 64 + 4, dtype=torch.bfloat16, device=DEV)[4:].view(8, 4, 64)
    for args in ((q.float(), k, v, c), (q, k.float(), v, c), (q, k, v[:7], c), (q, k[:, :1], v, c), (q[:, :3], k, v, c), (q, k, v, c.long()),
                 (q, k, v, c.cpu()), (q, k, v, c[:0]), (q[..., :32], k[..., :32], v[..., :32], c), (odd, k, v, c), (shifted, k, v, c),
                 (q.cpu(), k, v, c), (q, k[:1].expand(8, 2, 64), v, c), (q[0], k, v, c), (None, k, v, c), (q, k, v, None)):
        with pytest.raises(ValueError):
            tps.prompt_attention(*args)
    for kw in (dict(out=q), dict(status=torch.zeros(2, dtype=torch.int32, device=DEV)), dict(out=torch.zeros(8, 4, 64, device=DEV))):
        with pytest.raises(ValueError):
            tps.prompt_attention(q, k, v, c, **kw)
    with pytest.raises(RuntimeError):
        tps.prompt_attention(q, k, v, c, scale=math.nan)
