"""The cases that the operators around the paged cache are measured on: the attention of whole prompts, packed
one behind another; the attention of drafted token trees over the cache; and the pages and slots that requests
get and give back."""
import math

import torch

own = False  # True: the framework's kernels; False: the plain forms below

PROMPT, TREE, PAGES = "prompt", "tree", "pages"


def listed():
    return [
        # A short question of one user: latency.
        dict(name="prompt 1x300", kind=PROMPT, B=1, low=300, high=300, Hq=32, Hkv=8, D=128),
        # Sixty-four chat turns prefilled together, from one token to 250.
        dict(name="prompt 64x250", kind=PROMPT, B=64, low=1, high=250, Hq=32, Hkv=8, D=128),
        # Ragged prompts of a small model: head size 64, five query heads to a key head.
        dict(name="prompt 24x2011 D64", kind=PROMPT, B=24, low=700, high=2011, Hq=40, Hkv=8, D=64),
        # Four prompts of a model whose query heads all have keys of their own.
        dict(name="prompt 4x4001 mha", kind=PROMPT, B=4, low=2500, high=4001, Hq=16, Hkv=16, D=128),
        # One long document.
        dict(name="prompt 1x16384", kind=PROMPT, B=1, low=16384, high=16384, Hq=32, Hkv=8, D=128),
        # One request's eight drafted tokens after a short text: latency.
        dict(name="tree 1x1000", kind=TREE, B=1, N=8, ragged=False, Hq=32, Hkv=8, D=128, low=1000, high=1000, page=16, format="bf16"),
        # Trees of sixteen for a small batch, in an fp8 cache.
        dict(name="tree 8x4093x16 fp8", kind=TREE, B=8, N=16, ragged=False, Hq=32, Hkv=8, D=128, low=1500, high=4093, page=64,
             format="fp8"),
        # Large trees of a small model on long texts, some of them not full; five query heads to a key head.
        dict(name="tree 32x8111x64 int8", kind=TREE, B=32, N=64, ragged=True, Hq=40, Hkv=8, D=64, low=2000, high=8111, page=32,
             format="int8"),
        # A full batch's trees of five.
        dict(name="tree 256x4000x5 bf16", kind=TREE, B=256, N=5, ragged=True, Hq=32, Hkv=8, D=128, low=500, high=4000, page=16,
             format="bf16"),
        # A decode step of eight requests: one new token each.
        dict(name="pages 8x1", kind=PAGES, B=8, low=1, high=1, held=4000, width=512, page=16),
        # A large batch's drafted tokens, of which some requests have none.
        dict(name="pages 1024x16", kind=PAGES, B=1024, low=0, high=16, held=8000, width=600, page=16),
        # Prompts that are prefilled together get all their pages.
        dict(name="pages 300x6000", kind=PAGES, B=300, low=100, high=6000, held=0, width=128, page=64),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice([PROMPT, PROMPT, TREE, TREE, PAGES])
    heads, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if kind == PROMPT:
        B = log(1, 64)
        high = log(1, 12000 // math.isqrt(B))
        return dict(kind=kind, B=B, low=rng.randint(1, high), high=high, Hq=heads * rng.choice([1, 3, 4, 5, 8]) if heads < 8 else 8 * rng.choice([1, 4]),
                    Hkv=heads, D=D)
    if kind == TREE:
        B, N = log(1, 256), log(1, 64)
        high = max(N, log(N, max(2 * N, min(30000, 600000 // B))))
        return dict(kind=kind, B=B, N=N, ragged=rng.random() < 0.5, Hq=heads * rng.choice([1, 4, 5, 8]), Hkv=heads, D=D,
                    low=rng.randint(N, high), high=high, page=rng.choice([16, 32, 64, 128]), format=rng.choice(["bf16", "fp8", "int8"]))
    B, page, held = log(1, 2000), rng.choice([16, 32, 64]), log(1, 8000)
    high = log(1, max(2, min(6000, 1500000 // B)))
    return dict(kind=kind, B=B, low=rng.randint(0, high), high=high, held=held, width=-(-(held + high) // page) + rng.randint(0, 9), page=page)


_CODE = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}


def _spread(B, low, high):
    """B lengths, evenly from the lowest to the highest."""
    return [low + (high - low) * i // (B - 1) for i in range(B)] if B > 1 else [high]


def _nodes(case):
    """Drafted tokens of each sequence: all N of them, or (ragged) from N / 2 on."""
    return [case["N"] - (i * 7 % (case["N"] // 2 + 1) if case["ragged"] else 0) for i in range(case["B"])]


def _pool(g, pages, c):
    """A paged cache that holds tokens: codes [pages, heads, page, D] and, for 8 bits, a scale for each token and head."""
    shape, pool = (pages, c["Hkv"], c["page"], c["D"]), {}
    channel = torch.exp(0.5 * torch.randn(c["Hkv"], 1, c["D"], generator=g, device="cuda"))  # a few channels are large
    for name in ("k", "v"):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        if name == "k":
            x *= channel.bfloat16()
        scale = None
        if c["format"] != "bf16":
            top = x.abs().amax(-1).float()
            if c["format"] == "fp8":  # a power of two
                scale = torch.exp2(torch.ceil(torch.log2(top / 448)))
                x = (x / scale.bfloat16().unsqueeze(-1)).clamp_(-448, 448).to(torch.float8_e4m3fn)
            else:
                scale = (top * (1.01 / 127)).bfloat16().float()
                x = torch.round(x / scale.bfloat16().unsqueeze(-1)).clamp_(-127, 127).to(torch.int8)
            scale = scale.bfloat16()
        pool[name], pool[name + "_scale"] = x, scale
    return pool


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    s, kind, B = dict(case=case), case["kind"], case["B"]
    shuffled = lambda x: torch.tensor(x)[torch.randperm(B, generator=host)]
    lengths = shuffled(_spread(B, case["low"], case["high"]))
    if kind == PROMPT:
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.long), lengths.cumsum(0)]).int().cuda()
        s["lengths"] = lengths.tolist()
        qkv = torch.randn(int(lengths.sum()), Hq + 2 * Hkv, D, generator=g, device="cuda", dtype=torch.bfloat16)  # one projection's output
        qkv[:, :Hq] *= 1.5
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    elif kind == TREE:
        N, page = case["N"], case["page"]
        each = -(-case["high"] // page)
        pages = B * each
        s["pool"] = _pool(g, pages, case)
        s["table"] = torch.randperm(pages, generator=g, device="cuda").int().view(B, each)
        s["seq_len"] = lengths.int().cuda()
        s["nodes"] = shuffled(_nodes(case)).int().cuda() if case["ragged"] else None
        s["q"] = torch.randn(B, N, case["Hq"], case["D"], generator=g, device="cuda").mul_(1.5).bfloat16()
        s["tree"] = torch.zeros(B, N, dtype=torch.int64, device="cuda")  # bit j of node i: j is i or above it
        for i in range(N):
            bit = 1 << i if i < 63 else -(1 << 63)
            parent = torch.randint(-1, i, (B, 1), generator=g, device="cuda") if i else torch.full((B, 1), -1, device="cuda")
            above = s["tree"].gather(1, parent.clamp(min=0)).squeeze(1)
            s["tree"][:, i] = torch.where(parent.squeeze(1) >= 0, above, 0) | bit
        if own:
            import nucleus_token_sampler_gb300 as tps
            s["cache"] = tps.KVCache(s["pool"]["k"], s["pool"]["v"], s["pool"]["k_scale"], s["pool"]["v_scale"])
    else:
        page, width = case["page"], case["width"]
        held = torch.randint(0, case["held"] + 1, (B,), generator=host)
        has = (held + page - 1) // page
        pages = B * -(-(case["held"] + case["high"]) // page) + 11
        order = torch.randperm(pages, generator=host).int()
        table = torch.full((B, width), -1, dtype=torch.int32)
        table[torch.arange(width) < has[:, None]] = order[:int(has.sum())]
        free = torch.full((pages,), -1, dtype=torch.int32)
        free[:pages - int(has.sum())] = order[int(has.sum()):]
        s["table"], s["free"] = table.cuda(), free.cuda()
        s["count"] = torch.tensor([pages - int(has.sum())], dtype=torch.int32).cuda()
        s["seq_len"], s["keep"], s["new"] = held.int().cuda(), held.int().cuda(), lengths.int().cuda()
        s["tokens"] = int(lengths.sum())
    return s


def run(state):
    s, c = state, state["case"]
    if not own:
        return {PROMPT: _prompt, TREE: _tree, PAGES: _pages}[c["kind"]](s, c)
    import nucleus_token_sampler_gb300 as tps
    if c["kind"] == PROMPT:
        return tps.prompt_attention(s["q"], s["k"], s["v"], s["cu"])
    if c["kind"] == TREE:
        return tps.tree_attention(s["q"], s["cache"], s["table"], s["seq_len"], s["tree"], nodes=s["nodes"])
    # Room for the new tokens, which are then all taken back: drafts that were not accepted.
    slots, positions, cu = tps.kv_extend(s["table"], s["seq_len"], s["new"], s["free"], s["count"], c["page"], s["tokens"])
    tps.kv_trim(s["table"], s["seq_len"], s["keep"], s["free"], s["count"], c["page"])
    return slots, positions, cu, s["table"], s["seq_len"], s["free"], s["count"]


def _prompt(s, c):
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    first = 0
    for n in s["lengths"]:
        rows = slice(first, first + n)
        k, v = s["k"][rows].float().transpose(0, 1), s["v"][rows].float().transpose(0, 1)  # [Hkv, n, D]
        step = max(1, min(n, 2 ** 28 // (Hq * n)))
        for t in range(0, n, step):  # some query tokens at a time: their scores with all keys fit the memory
            q = s["q"][first + t:first + min(n, t + step)].float() / math.sqrt(D)
            m = q.shape[0]
            z = torch.matmul(q.view(m, Hkv, -1, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D), k[:, :t + m].transpose(1, 2))
            z = z.view(Hkv, -1, m, t + m)
            z.masked_fill_(torch.arange(t + m, device="cuda") > t + torch.arange(m, device="cuda")[:, None], -math.inf)
            z = (z - z.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(z.view(Hkv, -1, t + m), v[:, :t + m]).view(Hkv, -1, m, D) / z.sum(-1, keepdim=True)
            out[first + t:first + t + m] = o.permute(2, 0, 1, 3).reshape(m, Hq, D).bfloat16()
        first += n
    return out


def _gather(pool, name, page, off):
    code, scale = pool[name], pool[name + "_scale"]
    if code.dtype == torch.float8_e4m3fn:
        code = code.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn)
    else:
        code = code[page, :, off]
    return code.float() if scale is None else code.float() * scale[page, :, off].float().unsqueeze(-1)


def _tree(s, c):
    B, N, Hq, Hkv, D, page, L = (c[n] for n in ("B", "N", "Hq", "Hkv", "D", "page", "high"))
    at = torch.arange(L, device="cuda")
    n = torch.full((B,), N, device="cuda") if s["nodes"] is None else s["nodes"].long()
    node = at - (s["seq_len"].long() - n)[:, None]  # [B, L]: below 0 the text, then the drafted tokens
    bit = s["tree"][:, :, None] >> node.clamp(0, 63)[:, None] & 1
    seen = (node[:, None] < 0) | ((bit == 1) & (node < n[:, None])[:, None])
    seen &= (torch.arange(N, device="cuda") < n[:, None])[:, :, None]  # [B, N, L]
    out = torch.empty(B, N, Hq, D, dtype=torch.bfloat16, device="cuda")
    step = max(1, min(B, 2 ** 29 // (L * Hkv * max(D, N * Hq // Hkv))))
    for b in range(0, B, step):
        rows = slice(b, b + step)
        k, v = (_gather(s["pool"], x, s["table"][rows].long()[:, at // page], (at % page).expand(s["table"][rows].shape[0], -1))
                for x in ("k", "v"))  # [b, L, Hkv, D]
        q = (s["q"][rows].float() / math.sqrt(D)).view(-1, N, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4)
        z = torch.matmul(q.reshape(q.shape[0], Hkv, -1, D), k.permute(0, 2, 3, 1)).view(*q.shape[:4], L)
        z.masked_fill_(~seen[rows][:, None, :, None], -math.inf)
        z = (z - z.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
        o = torch.matmul(z.view(q.shape[0], Hkv, -1, L), v.transpose(1, 2)).view(q.shape) / z.sum(-1, keepdim=True).clamp(min=1e-30)
        out[rows] = o.permute(0, 2, 1, 3, 4).reshape(-1, N, Hq, D).bfloat16()
    return out


def _pages(s, c):
    page, T, width = c["page"], s["tokens"], c["width"]
    table, length, free = s["table"], s["seq_len"].long(), s["free"]
    # New pages come from the end of the free list, for the first request first.
    new, column = s["new"].long(), torch.arange(width, device="cuda")
    has, to = (length + page - 1) // page, (length + new + page - 1) // page
    before = (to - has).cumsum(0) - (to - has)
    fresh = (column >= has[:, None]) & (column < to[:, None])
    at = s["count"].long() - 1 - (before - has)[:, None] - column
    table.copy_(torch.where(fresh, free[at.clamp(min=0)], table))
    s["count"] -= (to - has).sum().int()
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), new.cumsum(0)])
    which = torch.searchsorted(cu, torch.arange(T, device="cuda"), right=True) - 1
    positions = length[which] + torch.arange(T, device="cuda") - cu[which]
    slots = table[which, positions // page].long() * page + positions % page
    # Pages that are no longer needed go back, the first request's first one last.
    keep = s["keep"].long()
    kept = (keep + page - 1) // page
    back = to - kept
    before = back.cumsum(0) - back
    gone = (column >= kept[:, None]) & (column < to[:, None])
    at = s["count"].long() + back.sum() - 1 - (before - kept)[:, None] - column
    free[at[gone]] = table[gone]
    s["count"] += back.sum().int()
    s["seq_len"].copy_(keep)
    return slots, positions.int(), cu.int(), table, s["seq_len"], free, s["count"]


def work(case):
    B, lengths = case["B"], _spread(case["B"], case["low"], case["high"])
    if case["kind"] == PROMPT:
        T, Hq, Hkv, D = sum(lengths), case["Hq"], case["Hkv"], case["D"]
        return dict(bytes=4 * T * (Hq + Hkv) * D + 4 * (B + 1), flops=2 * D * Hq * sum(n * (n + 1) for n in lengths))
    if case["kind"] == TREE:
        N, Hq, Hkv, D = case["N"], case["Hq"], case["Hkv"], case["D"]
        size, rows = D * 2 if case["format"] == "bf16" else D + 2, B * N * Hq * D
        tokens = sum(lengths)
        nodes = _nodes(case)
        pairs = sum(nodes) * tokens // B  # of a drafted token and one of its sequence: the lengths come in any order
        return dict(bytes=2 * tokens * Hkv * size + 4 * rows + 8 * B * N + 4 * sum(-(-n // case["page"]) for n in lengths),
                    flops=4 * D * Hq * pairs)
    tokens, pages = sum(lengths), sum(-(-n // case["page"]) for n in lengths)
    # Slots and positions; a page is read from the list, put in a table, and goes back; lengths and counts.
    return dict(bytes=12 * tokens + 16 * pages + 24 * B, flops=4 * tokens)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["kind"] == PROMPT:
        Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        cu = s["cu"].tolist()
        for a, b in zip(cu, cu[1:]):
            for h in range(Hq):
                k, v = s["k"][a:b, h * Hkv // Hq].double(), s["v"][a:b, h * Hkv // Hq].double()
                for t in range(a, b, 2048):
                    e = min(b, t + 2048)
                    z = s["q"][t:e, h].double() @ k[:e - a].T * D ** -0.5
                    hidden = torch.ones_like(z, dtype=torch.bool).triu(t - a + 1)
                    out[t:e, h] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v[:e - a]
        return out
    if c["kind"] == TREE:
        B, N, Hq, Hkv, D, page = (c[n] for n in ("B", "N", "Hq", "Hkv", "D", "page"))
        out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device="cuda")
        lengths = s["seq_len"].tolist()
        nodes = [N] * B if s["nodes"] is None else s["nodes"].tolist()

        def fetch(name, b):
            code, scale = s["pool"][name], s["pool"][name + "_scale"]
            ids = s["table"][b].long()
            bits = code.view(torch.int16 if code.dtype == torch.bfloat16 else torch.uint8)[ids].view(code.dtype).double()
            x = bits if scale is None else bits * scale[ids].double()[..., None]
            return x.transpose(1, 2).flatten(0, 1)[:lengths[b]]  # [length, Hkv, D]

        for b in range(B):
            k, v, n = fetch("k", b), fetch("v", b), nodes[b]
            text = lengths[b] - n
            hidden = torch.zeros(n, lengths[b], dtype=torch.bool, device="cuda")
            for j in range(n):
                hidden[:, text + j] = (s["tree"][b, :n] >> j) & 1 == 0
            z = torch.einsum("nhgd,lhd->nhgl", s["q"][b, :n].double().view(n, Hkv, -1, D), k) * D ** -0.5
            z = torch.softmax(z.masked_fill(hidden[:, None, None], -math.inf), -1)
            out[b, :n] = torch.einsum("nhgl,lhd->nhgd", z, v).reshape(n, Hq, D)
        return out
    page = c["page"]
    table, free = s["table"].tolist(), s["free"].tolist()
    count, slots, positions, cu = s["count"].item(), [], [], [0]
    held, new = s["seq_len"].tolist(), s["new"].tolist()
    for b in range(c["B"]):
        for p in range(-(-held[b] // page), -(-(held[b] + new[b]) // page)):
            count -= 1
            table[b][p] = free[count]
        at = torch.arange(held[b], held[b] + new[b])
        slots.append(torch.tensor(table[b])[at // page].long() * page + at % page)
        positions.append(at.int())
        cu.append(cu[-1] + new[b])
    for b in reversed(range(c["B"])):  # what came last goes back first
        for p in reversed(range(-(-held[b] // page), -(-(held[b] + new[b]) // page))):
            free[count] = table[b][p]
            count += 1
    whole = lambda x: torch.tensor(x, dtype=torch.int32)
    return torch.cat(slots), torch.cat(positions), whole(cu), whole(table), whole(held), whole(free), whole([count])
