"""Plain 64-bit forms of the operators around the paged cache (whole prompts, drafted trees, pages), for the tests."""
import math

import torch


def softmax_rows(q, k, v, seen, scale, value_scale=None):
    """(output, log-sum-exp, sum of weight * |value|, largest sum of |products|) of the rows q [R, H, D] over the tokens
    k, v [n, H, D] that `seen` [R, n] allows; a row that sees none yields 0 and -inf.  With the scales [n, H] of 8-bit values a
    fifth: how far the float16 weights' rounding may move the output.  A weight p over the row's reference is lifted by 2^7 and
    takes its value's scale s in units of a power of two that is at most 2^8 times the largest weight's scale; the
    largest weight is at least 1/2 of the reference, so that p s is held to 2^-11 of itself or, below float16's normal numbers, to
    2^-25 / (2^7 / 2 / 2^8) = 2^-24 of the largest p s: within the 2^-23 that is documented."""
    z = torch.einsum("rhd,nhd->rhn", q, k) * scale
    z = z.masked_fill(~seen[:, None], -math.inf)
    p = torch.nan_to_num(torch.softmax(z, -1), nan=0.0) if not seen.any(1).all() else torch.softmax(z, -1)
    big = (torch.einsum("rhd,nhd->rhn", q.abs(), k.abs()) * abs(scale)).masked_fill(~seen[:, None], 0)
    out = (torch.einsum("rhn,nhd->rhd", p, v), torch.logsumexp(z, -1), torch.einsum("rhn,nhd->rhd", p, v.abs()),
           big.amax(-1) if k.shape[0] else big.sum(-1))
    if value_scale is None:
        return out
    ps = p * value_scale.T[None]
    off = torch.maximum(2.0 ** -11 * ps, 2.0 ** -23 * ps.amax(-1, keepdim=True)).masked_fill(~seen[:, None], 0)
    return out + (torch.einsum("rhn,nhd->rhd", off, v.abs() / value_scale.unsqueeze(-1)),)


def prompt(q, k, v, bounds, scale):
    """The four results of softmax_rows for packed prompts; rows of no sequence are NaN."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = [torch.full(s, math.nan, dtype=torch.float64, device=q.device) for s in ((T, Hq, D), (T, Hq), (T, Hq, D), (T, Hq))]
    for a, b in bounds:
        if a >= b:
            continue
        seen = torch.ones(b - a, b - a, dtype=torch.bool, device=q.device).tril()
        kk, vv = (x[a:b].double().repeat_interleave(G, 1) for x in (k, v))
        for o, r in zip(out, softmax_rows(q[a:b].double(), kk, vv, seen, scale)):
            o[a:b] = r
    return out


def check(got, lse, want, weights=None, where=None):
    """Tolerances: a bfloat16 result is off by at most 2^-8 of its magnitude.  Weights p (1 + d), |d| <= u = `weights` (bfloat16:
    2^-8), whose sum takes some of them (M) rounded and the others not, yield sum p (1 + d) v / (1 + sum over M of p d), which is
    off by (sum p d v - o sum over M of p d) / (1 + sum over M of p d): at most u / (1 - u) (sum p |v| + |o|).  Or by a fifth element
    of `want`.  Further the scores' float32 sums by at most 2^-18 of the largest sum of
    |products|, and base-2 exponentials, joins of parts and weights below 2^-31 of the largest by less than 2^-14.  The last
    rounding is of the value as computed: with e off before it, |x + e| 2^-8 <= (|x| + e) 2^-8, so e counts 1 + 2^-8 times."""
    out, wl, mag, big = want[:4]
    off = want[4] if len(want) == 5 else weights / (1 - weights) * (mag + out.abs())
    if where is not None:
        got, lse, out, wl, mag, big, off = (x[where] for x in (got, lse, out, wl, mag, big, off))
    rest = 2.0 ** -18 * big + 2.0 ** -14
    tol = 2.0 ** -8 * out.abs() + (1 + 2.0 ** -8) * (off + rest.unsqueeze(-1) * mag)
    err = (got.double() - out).abs()
    assert (err <= tol).all(), (float((err - tol).max()), int((~(err <= tol)).sum()), err.numel())
    seen = wl > -math.inf
    assert torch.equal(lse > -math.inf, seen)
    assert ((lse.double() - wl)[seen].abs() <= rest[seen] + 2.0 ** -22 * wl[seen].abs()).all()
    assert (got[~seen] == 0).all()


def great_keys(seed, n, H, D, most):
    """Keys [n, H, D] whose components are all the same whole number, and the power of two that scores reach `most` with (a scale of 1/8)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randint(128, 256, (n, H, 1), generator=g, device="cuda").bfloat16().expand(n, H, D).contiguous()
    return k, 2.0 ** math.floor(math.log2(most / (D * 255 / 8)))


def great_queries(q, factor):
    """Queries whose components are all the same, of either sign."""
    q.copy_((torch.rand(q.shape[:-1], generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") < 0.5).mul(2).sub(1).mul(factor).unsqueeze(-1))


def check_great(got, lse, want, in_exponent):
    """Products of such queries and keys, and their sums, are exact in float32, and scores of different keys lie so far apart that all
    weight is on the largest ones.  They share it evenly: all are 2^r of the reference with the same r, which is what rounding of
    a score against the reference has left (2^3 at most, in base-2 units below 2^28), and a bfloat16 weight holds 2^r as well as 1.  A value is then
    off by the weights' rounding (`check`) and its own; a logarithm by those of the scale's base-2 form, of the score and of the result:
    at most 2^-22 of it.
    `in_exponent`: the scales of 8-bit values go through the scores, whose float32 sum with their logarithm is rounded to a whole number, from
    2^23 on and below 2^24.  So each of these weights may be off by 2^(1/2) either way, or (1 + d) of what it is, -0.30 < d < 0.42:
    sum p (1 + d) v / sum p (1 + d) is off by sum p d (v - o) / sum p (1 + d), at most 0.42 / 0.70 (sum p |v| + |o|); the
    logarithm by ln 2 / 2, less than the 2^-22 of some 10^7 that it has."""
    out, wl, mag = want[:3]
    u, d = 2.0 ** -8, 0.42 / 0.70 if in_exponent else 0.0
    assert ((got.double() - out).abs() <= u * out.abs() + (1 + u) * ((u / (1 - u) + d) * (mag + out.abs()) + 2.0 ** -14 * mag)).all()
    seen = wl > -math.inf
    assert torch.equal(lse > -math.inf, seen) and ((lse.double() - wl)[seen].abs() <= 2.0 ** -22 * wl[seen].abs()).all()
