"""examples/draft_trees.py against the same decoder without a cache, in float32: packed prompts, trees, kept chains and pages
together.  Tolerance: that of tests/test_gpu_example.py, whose plain decoder and derivation it shares."""
import pytest
import torch

from examples import draft_trees, shared_prompt

from .test_gpu_example import _plain_logits

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("format", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("lengths,page", [([1, 77, 300, 16], 16), ([130, 64], 64)])
def test_draft_trees_match_the_plain_decoder(format, lengths, page):
    vocab, steps = 24, 5
    model = shared_prompt.Decoder(layers=2, vocab=vocab, positions=1024, pages=100, page_size=page, format=format)
    g = torch.Generator().manual_seed(len(lengths))
    prompts = [torch.randint(0, vocab, (n,), generator=g, dtype=torch.int32).cuda() for n in lengths]
    tol = 2 * (2 * 8 * 2.0 ** -8 + {"bf16": 0.0, "fp8": 2 * 2.0 ** -4, "int8": 2 * 2.0 ** -6}[format])
    r = draft_trees.Requests(model, prompts, steps * len(draft_trees.PARENTS))
    texts, N = [p.clone() for p in prompts], len(draft_trees.PARENTS)
    bits, _ = draft_trees.tree_of(draft_trees.PARENTS)
    for step in range(steps):
        root = r.pending.clone()
        guesses = torch.randint(0, vocab, (len(lengths), N - 1), generator=g, dtype=torch.int32).cuda()
        for b in range(len(lengths)):  # some guesses that come true
            if step % 2:
                guesses[b, step % 3] = _plain_logits(model, torch.cat([texts[b], root[b:b + 1]]))[-1].argmax()
        nodes = torch.cat([root[:, None], guesses], 1)
        kept, logits = r.step(guesses)
        for b, text in enumerate(texts):
            for i in range(N):
                above = [j for j in range(N) if bits[i] >> j & 1]
                want = _plain_logits(model, torch.cat([text, nodes[b, above]]))[-1]
                ratio = float((logits[b, i] - want).square().mean().sqrt() / want.square().mean().sqrt())
                assert ratio <= tol, (step, b, i, ratio, tol)
            assert kept[b][0] == int(root[b])
            texts[b] = torch.cat([text, torch.tensor(kept[b], dtype=torch.int32, device="cuda")])
        assert r.length.tolist() == [t.numel() for t in texts]
        assert int(r.count) == 100 - sum(-(-t.numel() // page) for t in texts)
    used = {int(p) for b, t in enumerate(texts) for p in r.table[b, :-(-t.numel() // page)]}
    free = {int(p) for p in r.free[:int(r.count)]}
    assert used | free == set(range(100)) and not used & free
    r.end()
    assert int(r.count) == 100 and sorted(r.free.tolist()) == list(range(100)) and r.length.tolist() == [0] * len(lengths)


def test_a_step_without_room_is_told():
    model = shared_prompt.Decoder(layers=1, vocab=24, positions=256, pages=3, page_size=16, format="bf16")
    r = draft_trees.Requests(model, [torch.zeros(40, dtype=torch.int32)], 64)
    with pytest.raises(RuntimeError, match="no room"):
        r.step(torch.zeros(1, len(draft_trees.PARENTS) - 1, dtype=torch.int32, device="cuda"))
        r.step(torch.zeros(1, len(draft_trees.PARENTS) - 1, dtype=torch.int32, device="cuda"))
