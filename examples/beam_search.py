"""Beam search on a small language model with random weights.

    python examples/beam_search.py [--items 4] [--beams 4] [--steps 16] [--vocab 8000] ...

The [V, K] matrix, in TP shards, is both the embedding and the LM head; between them is one
attention layer, in plain torch, with a cache of keys and values. A step runs the operators
as a server would: the lookup, the norms before the attention and (with the residual's
addition) before the head, the head with its gather (of up to 16 rows), the selection of the
next tokens, and the reordering of the cache and of the tokens so far by the beams that were
selected. Prints every item's hypotheses, best first.
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tp_vocab_logits_gb300 import hg  # noqa: E402


def search(items=4, beams=4, steps=16, vocab=8000, hidden=512, heads=8, tp=4, seed=0, end=1,
           watch=None):
    """Hypotheses [items, beams, steps] and their totals [items, beams]. watch, if given, is
    called with what every operator was given and left, by name."""
    cols = -(-vocab // (128 * tp)) * 128  # the fused head's tiles are whole
    rows, width = items * beams, hidden // heads
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = torch.bfloat16

    def normal(shape, std):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    matrix = normal((tp * cols, hidden), 2.0 / math.sqrt(hidden))
    shards = list(matrix.split(cols))
    qkv, proj = (normal((hidden, n * hidden), 1.0 / math.sqrt(hidden)) for n in (3, 1))
    gains = [1 + normal((hidden,), 0.1) for _ in range(2)]

    words = hg.hg_vocab_create(tp, cols, hidden, rows, vocab=vocab, ops=("embed",))
    norm = hg.hg_norm_create(hidden, rows)
    head = hg.hg_create(tp, cols, rows, [rows])
    beam = hg.hg_beam_create(items, beams, vocab, beams)

    x, a, b = (torch.empty((rows, hidden), device="cuda", dtype=dtype) for _ in range(3))
    logits = [torch.empty((rows, tp * cols), device="cuda", dtype=dtype) for _ in range(tp)]
    cache = torch.zeros((2, rows, heads, steps, width), device="cuda", dtype=dtype)
    history = torch.zeros((rows, steps), device="cuda", dtype=torch.int32)
    tokens, parents = (torch.zeros((items, beams), device="cuda", dtype=torch.int64)
                       for _ in range(2))
    # All beams of an item start alike: one of them is searched.
    scores, picked = (torch.full((items, beams), -math.inf, device="cuda") for _ in range(2))
    scores[:, 0] = 0
    finished, done = (torch.zeros((items, beams), device="cuda", dtype=torch.bool)
                      for _ in range(2))
    tokens.copy_(torch.arange(2, items + 2, device="cuda")[:, None] % vocab)
    for step in range(steps):
        hg.hg_vocab_embed(words, tokens.view(-1), shards, x, scale=math.sqrt(hidden) / 20)
        hg.hg_norm_rows(norm, x, gains[0], a)
        q, k, v = (a @ qkv).view(rows, 3, heads, width).unbind(1)
        cache[0, :, :, step], cache[1, :, :, step] = k, v
        filled = cache[:, :, :, :step + 1]
        weight = torch.softmax((filled[0] @ q.unsqueeze(-1)).float() / math.sqrt(width), 2)
        mixed = (filled[1] * weight.to(dtype)).sum(2).view(rows, hidden)
        layer = mixed @ proj
        hg.hg_norm_rows(norm, layer, gains[1], b, residual=x)
        hg.hg_gather_fused(head, [b] * tp, shards, logits)
        hg.hg_beam_select(beam, logits[0][:, :vocab], scores, tokens, parents, picked,
                          finished=finished if end >= 0 else None, end=end, picked_finished=done)
        if watch:
            watch("norm", x, gains[0], a, None)
            watch("norm", layer, gains[1], b, x)
            watch("head", b, matrix, logits)
            watch("select", logits[0][:, :vocab], scores, tokens, parents, picked, finished, done)
            watch("before", parents, filled, history)
        hg.hg_beam_reorder(beam, parents, [(filled, 1), history])
        if watch:
            watch("after", parents, filled, history)
        history[:, step] = tokens.view(-1)
        scores, picked, finished, done = picked, scores, done, finished
    torch.cuda.synchronize()
    for h in (words, norm, head, beam):
        h.close()
    return history.view(items, beams, steps), scores


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("items", 4), ("beams", 4), ("steps", 16), ("vocab", 8000),
                        ("hidden", 512), ("heads", 8), ("tp", 4), ("seed", 0), ("end", 1)):
        ap.add_argument(f"--{name}", type=int, default=value)
    hypotheses, totals = search(**vars(ap.parse_args()))
    for i, (item, total) in enumerate(zip(hypotheses.tolist(), totals.tolist())):
        for tokens, value in zip(item, total):
            print(f"item {i}  {value:9.4f}  {' '.join(map(str, tokens))}")


if __name__ == "__main__":
    main()
