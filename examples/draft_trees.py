"""Several requests of their own length, answered with drafted trees: a small decoder with random weights.

    python examples/draft_trees.py [--format bf16|fp8|int8] [--requests N] [--prompt P] [--tokens T]

The prompts are prefilled together, packed one behind another: pages and slots for all of them (kv_extend), norm and
rotation (qk_norm_rope), the cache (kv_write), causal attention (prompt_attention).  Then each step drafts a tree of tokens
for every request: its root is the token that is certain, its other nodes are guesses.  One pass over all nodes
(kv_extend, qk_norm_rope, kv_write, tree_attention, sample) tells the token after each node; the longest chain of guesses
that came true is kept: its keys and values are moved together (kv_read, kv_write), and the rest's room is given back
(kv_trim).  No length is copied to the host to make a page table or a slot.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nucleus_token_sampler_gb300 as tps  # noqa: E402
from examples.shared_prompt import Decoder, rms  # noqa: E402

PARENTS = (-1, 0, 0, 0, 1, 1, 2, 4)  # of a tree's nodes: three guesses for the token after the root, three below those, one below that


def tree_of(parents):
    """Bits of the nodes that each node sees, and its depth."""
    bits, depth = [], []
    for i, p in enumerate(parents):
        bits.append(1 << i | (bits[p] if p >= 0 else 0))
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return bits, depth


class Requests:
    """Requests with pages from one list, and what the model makes of them."""

    def __init__(self, model, prompts, room, parents=PARENTS):
        dev, page, pages = model.device, model.caches[0].page_size, model.caches[0].n_pages
        self.model, self.page, self.parents, B = model, page, parents, len(prompts)
        width = -(-(max(p.numel() for p in prompts) + room + len(parents)) // page)
        self.table = torch.zeros(B, width, dtype=torch.int32, device=dev)
        self.length = torch.zeros(B, dtype=torch.int32, device=dev)
        self.free, self.count = torch.arange(pages, dtype=torch.int32, device=dev), torch.full((1,), pages, dtype=torch.int32, device=dev)
        self.status = torch.zeros(B, dtype=torch.int32, device=dev)
        bits, depth = tree_of(parents)
        self.tree = torch.tensor(bits, dtype=torch.int64, device=dev)
        self.depth = torch.tensor(depth, dtype=torch.int32, device=dev)
        lengths = torch.tensor([p.numel() for p in prompts], dtype=torch.int32, device=dev)
        tokens = torch.cat(prompts).to(dev)
        slots, positions, cu = self.extend(lengths, tokens.numel())
        x = self._layers(tokens, positions, slots, lambda q, k, v, cache: tps.prompt_attention(q, k, v, cu))
        logits = (rms(x[cu[1:].long() - 1]) @ model.head).float()
        self.pending = tps.sample(logits, 0.0, 0, 1.0, 0.0, 0, 0)  # greedy: the next token of each request

    def extend(self, new, tokens):
        out = tps.kv_extend(self.table, self.length, new, self.free, self.count, self.page, tokens, status=self.status)
        if self.status.any():
            raise RuntimeError(f"no room: {self.status.tolist()}")
        return out

    def _layers(self, tokens, positions, slots, attend):
        m = self.model
        H, K, D = m.q_heads, m.kv_heads, m.head_dim
        x = m.embedding[tokens.long()]
        for w, cache in zip(m.layers, m.caches):
            qkv = (rms(x) @ w["qkv"]).view(-1, H + 2 * K, D)
            q, k = tps.qk_norm_rope(qkv[:, :H], qkv[:, H:H + K], w["q_weight"], w["k_weight"], positions, m.cos_sin)
            tps.kv_write(cache, k, qkv[:, H + K:], slots)
            x = x + attend(q, k, qkv[:, H + K:], cache).view(-1, H * D) @ w["out"]
            gate, up = (rms(x) @ w["up"]).chunk(2, dim=1)
            x = x + (torch.nn.functional.silu(gate) * up) @ w["down"]
        return x

    def step(self, guesses):
        """One tree for each request, its nodes behind the root being `guesses` [B, N - 1].  Returns the tokens that are
        now certain, a list for each request, and the logits [B, N, vocab] after each node."""
        B, N = len(self.table), len(self.parents)
        before = self.length.clone()
        nodes = torch.cat([self.pending[:, None], guesses], 1)
        slots, _, _ = self.extend(torch.full_like(before, N), B * N)
        positions = (before[:, None] + self.depth).flatten()

        def attend(q, k, v, cache):
            return tps.tree_attention(q.view(B, N, *q.shape[1:]), cache, self.table, self.length, self.tree)
        x = self._layers(nodes.flatten(), positions, slots, attend)
        logits = (rms(x) @ self.model.head).float()
        after = tps.sample(logits, 0.0, 0, 1.0, 0.0, 0, 0).view(B, N)
        chains, kept, ahead = [], [], after.tolist()
        for b, row in enumerate(nodes.tolist()):
            chain, node = [0], 0
            while True:
                node = next((i for i in range(N) if self.parents[i] == node and row[i] == ahead[b][node]), None)
                if node is None:
                    break
                chain.append(node)
            chains.append(chain)
            kept.append([row[i] for i in chain])
        # The chains' tokens move to where the trees began; what lies behind them is given back.
        dev = self.model.device
        own = slots.view(B, N)
        source = torch.cat([own[b, torch.tensor(c, device=dev)] for b, c in enumerate(chains)])
        target = torch.cat([own[b, :len(c)] for b, c in enumerate(chains)])
        for cache in self.model.caches:
            k, v = tps.kv_read(cache, source)
            tps.kv_write(cache, k, v, target)
        count = torch.tensor([len(c) for c in chains], dtype=torch.int32, device=dev)
        tps.kv_trim(self.table, self.length, before + count, self.free, self.count, self.page)
        self.pending = torch.stack([after[b, c[-1]] for b, c in enumerate(chains)])
        return kept, logits.view(B, N, -1)

    def end(self):
        """All requests are answered: every page goes back."""
        tps.kv_trim(self.table, self.length, torch.zeros_like(self.length), self.free, self.count, self.page)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--format", choices=sorted(tps.KVCache.FORMATS), default="fp8")
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--tokens", type=int, default=32)
    a = ap.parse_args()
    model = Decoder(format=a.format, vocab=32, pages=1024)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 32, (1 + a.prompt * (i + 1) // a.requests,), generator=g, dtype=torch.int32) for i in range(a.requests)]
    requests, answers, steps = Requests(model, prompts, a.tokens), [[] for _ in prompts], 0
    torch.cuda.synchronize()
    start = time.perf_counter()
    while min(map(len, answers)) < a.tokens and max(map(len, answers)) + len(PARENTS) < a.tokens + 64:
        guesses = torch.randint(0, 32, (a.requests, len(PARENTS) - 1), generator=g, dtype=torch.int32).to(model.device)
        for answer, kept in zip(answers, requests.step(guesses)[0]):
            answer += kept
        steps += 1
    ms = (time.perf_counter() - start) * 1e3
    print(f"{a.requests} requests, {sum(map(len, answers))} tokens in {steps} steps, {ms:.1f} ms; the first: {answers[0][:12]} ...")
    requests.end()


if __name__ == "__main__":
    main()
