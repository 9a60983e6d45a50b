"""examples/shared_prompt.py against the same decoder without a cache, in float32.

Tolerance, as the root mean square of the logits' difference over that of the logits: each layer rounds its
normed input, the projections, the attention's weights and output, the gate and the residual to bfloat16, eight
roundings of at most 2^-8 each that add up over the layers at most linearly: 8 * 2^-8 a layer, of which the plain
form does as many of its own (factor 2).  A cache in 8 bits adds, for keys and values each, the format's
rounding: at most 2^-4 (e4m3: half a unit of a 4-bit significand) or 2^-6 (int8: half of 1/127 of the head's
largest component, at most four times the mean one).  A wrong page, position or length leaves a ratio near 1.
"""
import pytest
import torch

from examples import shared_prompt

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def _plain_logits(model, tokens):
    """Logits [n, vocab] of one sequence."""
    H, K, D, n = model.q_heads, model.kv_heads, model.head_dim, tokens.numel()
    norm = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    cos, sin = (t[:n, None] for t in model.cos_sin.chunk(2, 1))

    def rotate(x, w):
        a, b = (norm(x) * w).chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    hidden = torch.ones(n, n, dtype=torch.bool, device=tokens.device).triu(1)
    x = model.embedding[tokens.long()].float()
    for w in model.layers:
        qkv = (norm(x) @ w["qkv"].float()).view(n, H + 2 * K, D)
        q, k, v = rotate(qkv[:, :H], w["q_weight"]), rotate(qkv[:, H:H + K], w["k_weight"]), qkv[:, H + K:]
        k, v = (t.repeat_interleave(H // K, 1) for t in (k, v))
        s = torch.einsum("qhd,khd->hqk", q, k) * D ** -0.5
        p = s.masked_fill(hidden, float("-inf")).softmax(-1)
        x = x + torch.einsum("hqk,khd->qhd", p, v).reshape(n, H * D) @ w["out"].float()
        gate, up = (norm(x) @ w["up"].float()).chunk(2, 1)
        x = x + (torch.nn.functional.silu(gate) * up) @ w["down"].float()
    return norm(x) @ model.head.float()


@pytest.mark.parametrize("format,answers,prompt,page", [
    ("bf16", 5, 300, 16), ("fp8", 5, 300, 16), ("int8", 5, 300, 16), ("bf16", 24, 1000, 32), ("fp8", 3, 1, 64), ("int8", 1, 77, 32)])
def test_shared_prompt_matches_the_plain_decoder(format, answers, prompt, page):
    model = shared_prompt.Decoder(layers=2, vocab=1024, positions=2048, pages=200, page_size=page, format=format)
    tokens = torch.randint(0, 1024, (prompt,), generator=torch.Generator().manual_seed(prompt), dtype=torch.int32).cuda()
    steps, rounds = 20, 2
    tol = 2 * (2 * 8 * 2.0 ** -8 + {"bf16": 0.0, "fp8": 2 * 2.0 ** -4, "int8": 2 * 2.0 ** -6}[format])
    shared = shared_prompt.SharedPrompt(model, answers, steps, prompt + rounds * steps)

    def check(got, want):
        ratio = float((got.float() - want).square().mean().sqrt() / want.square().mean().sqrt())
        assert ratio <= tol, (ratio, tol)

    logits = shared.extend(tokens)
    check(logits[0], _plain_logits(model, tokens)[-1])
    for i in range(rounds):
        seen = []
        chosen, score, after = shared.answer(logits, steps, step=i * steps, on_logits=lambda t, l: seen.append(l))
        assert ((chosen >= 0) & (chosen < 1024)).all() and torch.isfinite(score).all()
        for b in range(answers):
            whole = torch.cat([tokens, chosen[b]])
            check(torch.stack([l[b] for l in seen]), _plain_logits(model, whole)[-steps:])
        best = int(score.argmax())
        shared.keep(best, steps)
        tokens = torch.cat([tokens, chosen[best]])
        logits = after[best:best + 1]
    assert shared.prefix_len == tokens.numel()
