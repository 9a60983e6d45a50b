"""The cases the decode-step operators are measured on: the per-head norm with rotation, the quantised
paged key/value cache, and the attention of a batch that shares a long prefix."""
import math

import torch

own = False  # True: the framework's kernels; False: the plain forms below

NORM, CACHE, READ, ATTN = "norm", "cache", "read", "attention"


def listed():
    return [
        # One decode step of eight requests: latency.
        dict(name="norm 8", kind=NORM, T=8, Hq=32, Hkv=8, D=128, rot=128, pairs="half", dtype="bf16", table=4096),
        # A float32 model's decode batch of 1,024 rows, partial rotation of adjacent pairs, a head size off the powers of two.
        dict(name="norm 1024 f32", kind=NORM, T=1024, Hq=16, Hkv=4, D=96, rot=64, pairs="adjacent", dtype="f32", table=32768),
        # A prefill chunk of odd length, heads cut out of one fused projection.
        dict(name="norm 16383", kind=NORM, T=16383, Hq=32, Hkv=8, D=128, rot=128, pairs="half", dtype="bf16", table=32768),
        # A decode step's new tokens of 64 sequences into the cache, and read back.
        dict(name="cache 64 fp8", kind=CACHE, T=64, Hkv=8, D=128, format="fp8", page=64, dtype="bf16"),
        # A prompt's tokens stored as it is prefilled, and read back for the next chunk.
        dict(name="cache 32749 int8", kind=CACHE, T=32749, Hkv=8, D=128, format="int8", page=32, dtype="bf16"),
        # A short context fetched from scattered pages.
        dict(name="read 257 int8", kind=READ, T=257, Hkv=4, D=64, format="int8", page=16, dtype="f32"),
        # A long context fetched from scattered pages.
        dict(name="read 131072 fp8", kind=READ, T=131072, Hkv=8, D=128, format="fp8", page=64, dtype="bf16"),
        # Eight completions of a short prompt that have just begun: latency.
        dict(name="attention 8x1000", kind=ATTN, B=8, Tq=1, Hq=32, Hkv=8, D=128, prefix=1000, suffix=40, page=16,
             format="bf16"),
        # Sixty-four completions of a document that ends inside a page.
        dict(name="attention 64x8191 fp8", kind=ATTN, B=64, Tq=1, Hq=32, Hkv=8, D=128, prefix=8191, suffix=300, page=64,
             format="fp8"),
        # Verification of four draft tokens and one more of each sequence; five query heads to a key head.
        dict(name="attention 48x5x20011 int8", kind=ATTN, B=48, Tq=5, Hq=40, Hkv=8, D=64, prefix=20011, suffix=500,
             page=32, format="int8"),
        # Few sequences whose own text is longer than what they share.
        dict(name="attention 16x2048 own", kind=ATTN, B=16, Tq=1, Hq=32, Hkv=4, D=128, prefix=2048, suffix=16000, page=64,
             format="bf16"),
        # The full decode batch on one long shared context.
        dict(name="attention 1024x16384 fp8", kind=ATTN, B=1024, Tq=1, Hq=32, Hkv=8, D=128, prefix=16384, suffix=256,
             page=64, format="fp8"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice([NORM, CACHE, READ, ATTN, ATTN])
    heads = rng.choice([1, 2, 4, 8])
    if kind == NORM:
        D = rng.choice([64, 96, 128, 256])
        return dict(kind=kind, T=log(1, 8000), Hq=heads * rng.choice([1, 4, 7]), Hkv=heads, D=D,
                    rot=D if rng.random() < 0.5 else D // 2, pairs=rng.choice(["half", "adjacent"]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), table=rng.choice([8192, 65536]))
    fmt, page = rng.choice(["fp8", "int8"]), rng.choice([16, 32, 64, 128])
    if kind in (CACHE, READ):
        return dict(kind=kind, T=log(1, 32000), Hkv=heads, D=rng.choice([64, 96, 128, 256]), format=fmt, page=page,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    B, Tq = log(1, 512), rng.choice([1, 1, 1, 2, 5])
    return dict(kind=kind, B=B, Tq=Tq, Hq=heads * rng.choice([1, 4, 5, 8]), Hkv=heads, D=rng.choice([64, 128]),
                prefix=log(16, 16000), suffix=max(Tq, log(1, max(2, 60000 // B))), page=page,
                format=rng.choice(["bf16", "fp8", "int8"]))


_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
_CODE = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}


def _quantise(x, fmt):
    """Codes and one scale for each vector of x's last axis, in 32 bits."""
    if fmt == "bf16":
        return x.bfloat16(), None
    x = x.float()
    a = x.abs().amax(-1)
    if fmt == "fp8":  # the least power of two that brings the largest magnitude to 448 or below
        m, e = torch.frexp(a)
        s = torch.ldexp(torch.ones_like(a), torch.where(a > 0, e - 9 + (m > 0.875).int(), -40).clamp(min=-40))
        return (x / s.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn), s.bfloat16()
    s = a / 127  # rounded up to bfloat16
    s = ((s.view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32).clamp(min=2.0 ** -40)
    return torch.round(x / s.unsqueeze(-1)).clamp(-127, 127).to(torch.int8), s.bfloat16()


def _values(code, scale):
    return code.float() if scale is None else code.float() * scale.float().unsqueeze(-1)


def _pool(g, pages, c):
    """A paged cache that holds tokens: codes [pages, heads, page, D] and their scales."""
    shape = (pages, c["Hkv"], c["page"], c["D"])
    channel = torch.exp(0.5 * torch.randn(c["Hkv"], 1, c["D"], generator=g, device="cuda"))  # a few channels are large
    pool = []
    for t in range(2):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        pool += _quantise(x * channel.bfloat16() if t == 0 else x, c["format"])
    return dict(zip(("k", "k_scale", "v", "v_scale"), pool))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    kind, D, Hkv = case["kind"], case["D"], case["Hkv"]
    if kind == NORM:
        T, Hq, rot = case["T"], case["Hq"], case["rot"]
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda").mul_(2).to(_TYPE[case["dtype"]])
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        s["wq"], s["wk"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2))
        start = torch.randint(0, max(1, case["table"] - T), (1,), generator=g, device="cuda")
        s["pos"] = ((start + torch.arange(T, device="cuda")) % case["table"]).int()
        f = torch.arange(case["table"], device="cuda").double().unsqueeze(1) * torch.pow(
            torch.tensor(10000.0, device="cuda").double(), -torch.arange(rot // 2, device="cuda").double() * 2 / rot)
        s["table"] = torch.cat([f.cos(), f.sin()], 1).float()
    elif kind in (CACHE, READ):
        T, page = case["T"], case["page"]
        pages = -(-T // page) + 3
        s["pool"] = _pool(g, pages, case)
        order = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(T, device="cuda")
        if kind == CACHE and T <= 1024:  # a decode step: one token here and there
            s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:T].contiguous()
        else:
            s["slots"] = order[at // page] * page + at % page
        if kind == CACHE:
            s["k"] = torch.randn(T, Hkv, D, generator=g, device="cuda").to(_TYPE[case["dtype"]])
            s["v"] = torch.randn(T, 2 * Hkv, D, generator=g, device="cuda").to(_TYPE[case["dtype"]])[:, Hkv:]
    else:
        B, page, P = case["B"], case["page"], case["prefix"]
        shared, each = -(-P // page), max(1, -(-case["suffix"] // page))
        pages = shared + B * each
        s["pool"] = _pool(g, pages, case)
        order = torch.randperm(pages, generator=g, device="cuda").int()
        s["prefix_pages"] = order[:shared].contiguous()
        s["page_table"] = order[shared:].reshape(B, each).contiguous()
        s["suffix_len"] = torch.tensor(_lengths(case), device="cuda", dtype=torch.int32)[
            torch.randperm(B, generator=g, device="cuda")]
        s["q"] = torch.randn(B, case["Tq"], case["Hq"], D, generator=g, device="cuda").mul_(1.5).bfloat16()
    if own and "pool" in s:
        import nucleus_token_sampler_gb300 as tps
        s["cache"] = tps.KVCache(s["pool"]["k"], s["pool"]["v"], s["pool"]["k_scale"], s["pool"]["v_scale"])
    return s


def _lengths(case):
    """Own lengths of the sequences: evenly from the query's tokens alone to the longest (from none where a query is one token)."""
    lo = 0 if case["Tq"] == 1 else case["Tq"]
    return [lo + (case["suffix"] - lo) * i // max(1, case["B"] - 1) if case["B"] > 1 else case["suffix"] for i in range(case["B"])]


def run(state):
    c = state["case"]
    if own:
        import nucleus_token_sampler_gb300 as tps
        if c["kind"] == NORM:
            return tps.qk_norm_rope(state["q"], state["k"], state["wq"], state["wk"], state["pos"], state["table"],
                                    eps=1e-6, interleaved=c["pairs"] == "adjacent")
        if c["kind"] == ATTN:
            return tps.prefix_attention(state["q"], state["cache"], state["prefix_pages"], c["prefix"], state["page_table"],
                                        state["suffix_len"])
        if c["kind"] == CACHE:
            tps.kv_write(state["cache"], state["k"], state["v"], state["slots"])
        return tps.kv_read(state["cache"], state["slots"], dtype=_TYPE[c["dtype"]])
    return {NORM: _norm, CACHE: _cache, READ: _read, ATTN: _attention}[c["kind"]](state, c)


def _norm(s, c):
    at = s["table"][s["pos"].long()].unsqueeze(1)
    cos, sin = at[..., :c["rot"] // 2], at[..., c["rot"] // 2:]

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        r = x[..., :c["rot"]]
        if c["pairs"] == "adjacent":
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :c["rot"] // 2], r[..., c["rot"] // 2:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, x[..., c["rot"]:]], -1).to(_TYPE[c["dtype"]])

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _cache(s, c):
    page, off = s["slots"] // c["page"], s["slots"] % c["page"]
    for name in ("k", "v"):
        code, scale = _quantise(s[name], c["format"])
        s["pool"][name].view(torch.uint8)[page, :, off] = code.view(torch.uint8)
        s["pool"][name + "_scale"][page, :, off] = scale
    return _read(s, c)


def _gather(pool, name, page, off):
    code, scale = pool[name], pool[name + "_scale"]
    if code.dtype == torch.float8_e4m3fn:
        code = code.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn)
    else:
        code = code[page, :, off]
    return _values(code, None if scale is None else scale[page, :, off])


def _read(s, c):
    page, off = s["slots"] // c["page"], s["slots"] % c["page"]
    return tuple(_gather(s["pool"], name, page, off).to(_TYPE[c["dtype"]]) for name in ("k", "v"))


def _attention(s, c):
    B, Tq, Hq, Hkv, D, P, page = (c[n] for n in ("B", "Tq", "Hq", "Hkv", "D", "prefix", "page"))
    G = Hq // Hkv
    at, own_at = torch.arange(P, device="cuda"), torch.arange(c["suffix"], device="cuda")
    pk, pv = (_gather(s["pool"], n, s["prefix_pages"].long()[at // page], at % page) for n in ("k", "v"))  # [P, Hkv, D]
    pages, off = s["page_table"].long()[:, own_at // page], (own_at % page).expand(B, -1)
    sk, sv = (_gather(s["pool"], n, pages, off) for n in ("k", "v"))  # [B, suffix, Hkv, D]
    q = (s["q"].float() / math.sqrt(D)).reshape(B, Tq, Hkv, G, D)
    shared = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(Hkv, -1, D), pk.permute(1, 2, 0))
    shared = shared.reshape(Hkv, B, Tq, G, P)
    each = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(Hkv, B, Tq * G, D), sk.permute(2, 0, 3, 1))
    each = each.reshape(Hkv, B, Tq, G, -1)
    seen = s["suffix_len"].long().reshape(B, 1, 1) - Tq + 1 + torch.arange(Tq, device="cuda").reshape(1, Tq, 1)
    each = each.masked_fill((own_at >= seen).unsqueeze(2), -math.inf)
    top = torch.maximum(shared.amax(-1, keepdim=True), each.amax(-1, keepdim=True))
    shared, each = (shared - top).exp_(), (each - top).exp_()
    total = shared.sum(-1, keepdim=True) + each.sum(-1, keepdim=True)
    o = torch.matmul(shared.reshape(Hkv, -1, P), pv.transpose(0, 1)).reshape(Hkv, B, Tq, G, D)
    o = o + torch.matmul(each.reshape(Hkv, B, Tq * G, -1), sv.permute(2, 0, 1, 3)).reshape(Hkv, B, Tq, G, D)
    return (o / total).permute(1, 2, 0, 3, 4).reshape(B, Tq, Hq, D).bfloat16()


def work(case):
    D, Hkv = case["D"], case["Hkv"]
    if case["kind"] == NORM:
        n, size = case["T"] * (case["Hq"] + Hkv) * D, 4 if case["dtype"] == "f32" else 2
        return dict(bytes=2 * n * size + min(case["T"], case["table"]) * case["rot"] * 4 + 4 * case["T"], flops=8 * n)
    if case["kind"] in (CACHE, READ):
        n, size = 2 * case["T"] * Hkv, 4 if case["dtype"] == "f32" else 2
        return dict(bytes=n * (D + 2) + n * D * size * (2 if case["kind"] == CACHE else 1) + 8 * case["T"], flops=4 * n * D)
    rows, size = case["B"] * case["Tq"], D * 2 if case["format"] == "bf16" else D + 2
    tokens = sum(_lengths(case))
    return dict(bytes=2 * Hkv * (case["prefix"] + tokens) * size + 4 * rows * case["Hq"] * D,
                flops=4 * D * case["Hq"] * case["Tq"] * (case["B"] * case["prefix"] + tokens))


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["kind"] == NORM:
        out = []
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            x = x.double()
            x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
            half = c["rot"] // 2
            i = torch.arange(half, device="cuda")
            i, j = (2 * i, 2 * i + 1) if c["pairs"] == "adjacent" else (i, i + half)
            angle = s["table"].double().index_select(0, s["pos"].long())[:, None, :]
            y = x.clone()
            y[..., i] = x[..., i] * angle[..., :half] - x[..., j] * angle[..., half:]
            y[..., j] = x[..., j] * angle[..., :half] + x[..., i] * angle[..., half:]
            out.append(y)
        return tuple(out)
    if c["kind"] == CACHE:
        out = []
        for x in (s["k"].double(), s["v"].double()):
            a = x.abs().amax(-1, keepdim=True)
            if c["format"] == "fp8":
                unit = torch.exp2(torch.ceil(torch.log2(a / 448)).clamp(min=-40))
                unit = torch.where(a <= 224 * unit, unit / 2, unit)  # where log2 rounded up past a whole number
                y = x / unit
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                out.append(torch.round(y / step) * step * unit)
            else:
                least = torch.exp2(torch.floor(torch.log2((a / 127).clamp(min=2.0 ** -60))) - 7)
                unit = (torch.ceil(a / 127 / least) * least).clamp(min=2.0 ** -40)
                out.append(torch.round(x / unit) * unit)
        return tuple(out)

    def fetch(name, page, off):
        code, scale = s["pool"][name], s["pool"][name + "_scale"]
        bits = code.view(torch.int16 if code.dtype == torch.bfloat16 else torch.uint8)[page, :, off].view(code.dtype)
        return bits.double() if scale is None else bits.double() * scale[page, :, off].double()[..., None]

    if c["kind"] == READ:
        return tuple(fetch(n, s["slots"] // c["page"], s["slots"] % c["page"]) for n in ("k", "v"))
    B, Tq, Hq, Hkv, D, P, page = (c[n] for n in ("B", "Tq", "Hq", "Hkv", "D", "prefix", "page"))
    G = Hq // Hkv
    out = torch.empty(B, Tq, Hq, D, dtype=torch.float64, device="cuda")
    at = torch.arange(P, device="cuda")
    pk, pv = (fetch(n, s["prefix_pages"].long()[at // page], at % page) for n in ("k", "v"))
    lengths = s["suffix_len"].tolist()
    top = torch.empty(B, Tq, Hq, dtype=torch.float64, device="cuda")
    total = torch.empty_like(top)
    q = s["q"].double()
    for h in range(Hkv):  # what all share, a few rows at a time
        mine = slice(h * G, (h + 1) * G)
        for b in range(0, B, 64):
            z = q[b:b + 64, :, mine] @ pk[:, h].T * D ** -0.5
            top[b:b + 64, :, mine] = z.amax(-1)
            e = torch.exp(z - z.amax(-1, keepdim=True))
            total[b:b + 64, :, mine] = e.sum(-1)
            out[b:b + 64, :, mine] = e @ pv[:, h]
    for b in range(B):  # what is each one's own
        n = lengths[b]
        if not n:
            continue
        at = torch.arange(n, device="cuda")
        k, v = (fetch(m, s["page_table"][b].long()[at // page], at % page) for m in ("k", "v"))
        z = torch.einsum("thgd,nhd->thgn", q[b].reshape(Tq, Hkv, G, D), k) * D ** -0.5
        hidden = at > n - Tq + torch.arange(Tq, device="cuda")[:, None]
        z = z.masked_fill(hidden[:, None, None], -math.inf)
        most = torch.maximum(z.amax(-1), top[b].reshape(Tq, Hkv, G))
        e, before = torch.exp(z - most[..., None]), torch.exp(top[b].reshape(Tq, Hkv, G) - most)
        total[b] = (total[b].reshape(Tq, Hkv, G) * before + e.sum(-1)).reshape(Tq, Hq)
        out[b] = (out[b].reshape(Tq, Hkv, G, D) * before[..., None] + torch.einsum("thgn,nhd->thgd", e, v)).reshape(Tq, Hq, D)
    return out / total[..., None]
