"""Plain 64-bit forms of the decode-step operators, for the tests."""
import math

import torch

F8 = torch.float8_e4m3fn


def norm_rope(x, w, pos, table, eps, interleaved):
    x = x.double()
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        y = y * w.double()
    R = table.shape[1]
    ang = table.double()[pos.long()].unsqueeze(1)
    c, s = ang[..., :R // 2], ang[..., R // 2:]
    if interleaved:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:R]
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([r, y[..., R:]], -1)


def scale_of(x, fmt):
    """The scale of each vector, from the definition, in 64 bits."""
    a = x.double().abs().amax(-1)
    tiny = torch.full_like(a, 2.0 ** -40)
    if fmt == "fp8":
        e = torch.floor(torch.log2(torch.maximum(a, tiny * 2.0 ** -20) / 448)) - 1
        for _ in range(3):  # the least e with a <= 448 * 2^e
            e = torch.where(a > 448 * torch.exp2(e), e + 1, e)
        s = torch.maximum(torch.exp2(e), tiny)
    else:
        q = a / 127
        up = q.to(torch.bfloat16)
        bits = up.view(torch.int16)
        s = torch.where(up.double() < q, (bits + 1).view(torch.bfloat16), up).double()
        s = torch.maximum(s, tiny)
    return torch.where(torch.isfinite(a), s, torch.full_like(a, math.nan))


def nearest(y, fmt):
    """The nearest code value of each y, ties to even, in 64 bits."""
    if fmt == "int8":
        return torch.round(y).clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def stored(x, fmt):
    """What a cache of this format holds of x, in 64 bits."""
    if fmt == "bf16":
        return x.bfloat16().double()
    s = scale_of(x, fmt).unsqueeze(-1)
    return nearest(x.double() / s, fmt) * s


def values(cache):
    """Every value of a cache, [pages, heads, page, D] (k, v), in 64 bits."""
    out = []
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        t = t.double()
        out.append(t if s is None else t * s.double().unsqueeze(-1))
    return out


def attention(q, kv, prefix_pages, prefix_len, page_table, suffix_len, scale):
    """(output, log-sum-exp, sum of weight * |value|, largest sum of |products|) of every query."""
    K, V = kv
    B, Tq, Hq, D = q.shape
    Hkv, page = K.shape[1], K.shape[2]
    G = Hq // Hkv
    out = torch.zeros(B, Tq, Hq, D, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    lse = torch.full((B, Tq, Hq), -math.inf, dtype=torch.float64, device=q.device)
    big = torch.zeros_like(lse)
    at = torch.arange(prefix_len, device=q.device)
    pp = prefix_pages.long()[at // page]
    pk, pv = K[pp, :, at % page], V[pp, :, at % page]
    for b in range(B):
        n = int(suffix_len[b])
        at = torch.arange(n, device=q.device)
        sp = page_table[b].long()[at // page] if n else at
        k = torch.cat([pk, K[sp, :, at % page]]) if n else pk
        v = torch.cat([pv, V[sp, :, at % page]]) if n else pv
        for t in range(Tq):
            m = prefix_len + max(0, n - Tq + 1 + t)
            if m == 0:
                continue
            qq = q[b, t].double().reshape(Hkv, G, D)
            z = torch.einsum("hgd,nhd->hgn", qq, k[:m]) * scale
            p = torch.softmax(z, -1)
            out[b, t] = torch.einsum("hgn,nhd->hgd", p, v[:m]).reshape(Hq, D)
            mag[b, t] = torch.einsum("hgn,nhd->hgd", p, v[:m].abs()).reshape(Hq, D)
            lse[b, t] = torch.logsumexp(z, -1).reshape(Hq)
            big[b, t] = (torch.einsum("hgd,nhd->hgn", qq.abs(), k[:m].abs()) * abs(scale)).amax(-1).reshape(Hq)
    return out, lse, mag, big
