"""Several answers to one prompt: a small decoder with random weights, its key/value cache and the sampler.

    python examples/shared_prompt.py [--format bf16|fp8|int8] [--answers N] [--prompt P] [--tokens T] [--rounds R]

The prompt is cached once, in chunks.  Then N answers are sampled together: each step norms and rotates its queries
and keys (qk_norm_rope), stores the new tokens in pages of each answer's own (kv_write), attends to the shared prompt
and the answer's own tokens (prefix_attention) and draws the next tokens (sample).  After a round the answer with the
largest log-probability is kept: its tokens are moved behind the prompt (kv_read, kv_write), where they are part of
the prefix that the next round's answers share.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nucleus_token_sampler_gb300 as tps  # noqa: E402


def rms(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


def rotation_table(positions, dim, device):
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(dim // 2) / (dim // 2))
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


class Decoder:
    """Weights of a decoder with grouped query heads, and one paged cache per layer."""

    def __init__(self, layers=2, hidden=512, q_heads=8, kv_heads=2, head_dim=64, vocab=4096, positions=4096,
                 pages=512, page_size=32, format="fp8", device="cuda", seed=0):
        g = torch.Generator(device="cpu").manual_seed(seed)
        make = lambda rows, cols: (torch.randn(rows, cols, generator=g) * rows ** -0.5).bfloat16().to(device)
        self.q_heads, self.kv_heads, self.head_dim, self.device = q_heads, kv_heads, head_dim, torch.device(device)
        self.embedding = torch.randn(vocab, hidden, generator=g).bfloat16().to(device)
        self.head = make(hidden, vocab)
        self.layers = [dict(qkv=make(hidden, (q_heads + 2 * kv_heads) * head_dim), out=make(q_heads * head_dim, hidden),
                            up=make(hidden, 2 * hidden), down=make(hidden, hidden),
                            q_weight=(1 + 0.1 * torch.randn(head_dim, generator=g)).to(device),
                            k_weight=(1 + 0.1 * torch.randn(head_dim, generator=g)).to(device)) for _ in range(layers)]
        self.cos_sin = rotation_table(positions, head_dim, device)
        self.caches = [tps.KVCache.empty(pages, kv_heads, page_size, head_dim, format, device) for _ in range(layers)]

    def forward(self, tokens, positions, slots, prefix_pages, prefix_len, page_table, suffix_len):
        """Logits [B, Tq, vocab] of the tokens [B, Tq], which are stored in the slots [B * Tq] of the caches."""
        B, Tq = tokens.shape
        H, K, D = self.q_heads, self.kv_heads, self.head_dim
        x = self.embedding[tokens.reshape(-1).long()]
        for w, cache in zip(self.layers, self.caches):
            qkv = (rms(x) @ w["qkv"]).view(B * Tq, H + 2 * K, D)
            q, k = tps.qk_norm_rope(qkv[:, :H], qkv[:, H:H + K], w["q_weight"], w["k_weight"], positions, self.cos_sin)
            tps.kv_write(cache, k, qkv[:, H + K:], slots)
            o = tps.prefix_attention(q.view(B, Tq, H, D), cache, prefix_pages, prefix_len, page_table, suffix_len)
            x = x + o.view(B * Tq, H * D) @ w["out"]
            gate, up = (rms(x) @ w["up"]).chunk(2, dim=1)
            x = x + (torch.nn.functional.silu(gate) * up) @ w["down"]
        return (rms(x) @ self.head).float().view(B, Tq, -1)


class SharedPrompt:
    """A prefix that grows, and pages for the answers that are sampled after it."""

    def __init__(self, model, answers, answer_tokens, prefix_tokens):
        self.model, self.answers, page = model, answers, model.caches[0].page_size
        own, dev = -(-answer_tokens // page), model.device
        room = -(-prefix_tokens // page)
        assert room + answers * own <= model.caches[0].n_pages, "the cache has too few pages"
        self.page, self.prefix_len = page, 0
        self.prefix_pages = torch.arange(room, dtype=torch.int32, device=dev)
        self.table = (room + torch.arange(answers * own, dtype=torch.int32, device=dev)).view(answers, own)

    def _prefix_slots(self, first, count):
        at = torch.arange(first, first + count, device=self.model.device)
        return self.prefix_pages[at // self.page].long() * self.page + at % self.page

    def extend(self, tokens, chunk=256):
        """Cache more prefix tokens, `chunk` (whole pages) at a time.  Returns the logits after the last one."""
        assert self.prefix_len % self.page == 0 and chunk % self.page == 0
        for part in tokens.split(chunk):
            n, done, dev = part.numel(), self.prefix_len, self.model.device
            table = self.prefix_pages[done // self.page:][None]  # the chunk's own tokens: where the prefix goes on
            logits = self.model.forward(part[None], torch.arange(done, done + n, dtype=torch.int32, device=dev),
                                        self._prefix_slots(done, n), self.prefix_pages, done, table,
                                        torch.full((1,), n, dtype=torch.int32, device=dev))
            self.prefix_len += n
        return logits[:, -1]

    def answer(self, logits, tokens, step, seed=1, temperature=0.8, top_p=0.95, on_logits=None):
        """Sample `tokens` tokens for each answer, the first from `logits` [1, vocab].  Returns the tokens
        [answers, tokens], their summed log-probabilities and the logits after the last token."""
        B, dev = self.answers, self.model.device
        logits = logits.expand(B, -1).contiguous()
        chosen = torch.empty(B, tokens, dtype=torch.int32, device=dev)
        score = torch.zeros(B, device=dev)
        for t in range(tokens):
            r = tps.sample(logits, temperature, 0, top_p, 0.0, seed, step + t, want_logprob=True)
            chosen[:, t] = r["token"]
            score += r["logprob"]
            slots = self.table[:, t // self.page].long() * self.page + t % self.page
            logits = self.model.forward(chosen[:, t:t + 1],
                                        torch.full((B,), self.prefix_len + t, dtype=torch.int32, device=dev), slots,
                                        self.prefix_pages, self.prefix_len, self.table,
                                        torch.full((B,), t + 1, dtype=torch.int32, device=dev))[:, 0]
            if on_logits is not None:
                on_logits(t, logits)
        return chosen, score, logits

    def keep(self, which, tokens):
        """Make the first `tokens` tokens of answer `which` part of the prefix."""
        at = torch.arange(tokens, device=self.model.device)
        own = self.table[which, at // self.page].long() * self.page + at % self.page
        to = self._prefix_slots(self.prefix_len, tokens)
        for cache in self.model.caches:
            k, v = tps.kv_read(cache, own)
            tps.kv_write(cache, k, v, to)
        self.prefix_len += tokens


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--format", choices=sorted(tps.KVCache.FORMATS), default="fp8")
    ap.add_argument("--answers", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--rounds", type=int, default=2)
    a = ap.parse_args()
    model = Decoder(format=a.format)
    prompt = torch.randint(0, model.embedding.shape[0], (a.prompt,), generator=torch.Generator().manual_seed(1),
                           dtype=torch.int32).to(model.device)
    shared = SharedPrompt(model, a.answers, a.tokens, a.prompt + a.rounds * a.tokens)
    logits = shared.extend(prompt)
    for i in range(a.rounds):
        torch.cuda.synchronize()
        start = time.perf_counter()
        chosen, score, after = shared.answer(logits, a.tokens, step=i * a.tokens)
        best = int(score.argmax())
        ms = (time.perf_counter() - start) * 1e3
        print(f"round {i}: {a.answers} answers of {a.tokens} tokens after {shared.prefix_len} shared ones in {ms:.1f} ms; "
              f"kept answer {best} (ln P {float(score[best]):.2f}): {chosen[best, :8].tolist()} ...")
        shared.keep(best, a.tokens)
        logits = after[best:best + 1]


if __name__ == "__main__":
    main()
