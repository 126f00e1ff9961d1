"""Training steps of a small language model whose two ends are one matrix.

    python examples/tied_vocab_step.py [--steps 30] [--vocab 8192] [--hidden 512] ...

The [V, K] matrix lies in TP shards, as hg_gather_fused takes it, and is both
the embedding and the LM head. Between them stands one residual layer, in plain
torch. A step runs the four vocabulary operators as a trainer would: the lookup,
the loss (a mean over the unmasked targets), its gradient written to the
gradient shards, and the lookup's gradient added to the same shards. With --norm
the residual's addition is the norm's before the head, and its gradient the one of
both of its terms. Prints the loss of every step.
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tp_vocab_logits_gb300 import hg  # noqa: E402


def batch(vocab: int, rows: int, masked: float, gen: torch.Generator):
    """Tokens and the next tokens of a fixed successor rule, some of them masked."""
    tokens = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    targets = (tokens * 5 + 3) % vocab
    hide = torch.rand(rows, generator=gen, device="cuda") < masked
    return tokens, torch.where(hide, -100, targets)


def train(steps=30, vocab=8192, hidden=512, rows=2048, tp=4, masked=0.1, lr=0.03,
          seed=0, log=print, norm=False) -> list:
    cols = -(-vocab // tp)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = torch.bfloat16

    def normal(shape, std):
        return (torch.randn(shape, generator=gen, device="cuda") * std)

    # fp32 masters, their bf16 copies and gradients; the shards are views.
    master = {"matrix": normal((tp * cols, hidden), 0.02),
              "layer": normal((hidden, hidden), 1.0 / math.sqrt(hidden))}
    if norm:
        master["gain"] = torch.ones(hidden, device="cuda")
    weight = {k: v.to(dtype) for k, v in master.items()}
    grad = {k: torch.empty_like(v) for k, v in weight.items()}
    shards, grad_shards = (list(t["matrix"].split(cols)) for t in (weight, grad))
    moments = {k: [torch.zeros_like(v), torch.zeros_like(v)] for k, v in master.items()}

    h = hg.hg_vocab_create(tp, cols, hidden, rows, vocab=vocab, dtype=dtype)
    x = torch.empty((rows, hidden), device="cuda", dtype=dtype)
    y, dy, dx = (torch.empty_like(x) for _ in range(3))
    loss, lse = (torch.empty(rows, device="cuda") for _ in range(2))
    if norm:
        hn = hg.hg_norm_create(hidden, rows, dtype=dtype)
        s, rstd = torch.empty_like(x), torch.empty_like(loss)
    scale = math.sqrt(hidden)
    data = [batch(vocab, rows, masked, gen) for _ in range(4)]
    losses = []
    for step in range(steps):
        tokens, targets = data[step % len(data)]
        # Forward: embedding, a residual layer, the loss.
        hg.hg_vocab_embed(h, tokens, shards, x, scale=scale)
        a = torch.tanh(x @ weight["layer"])
        if norm:
            hg.hg_norm_rows(hn, a, weight["gain"], y, residual=x, sum_out=s, rstd=rstd)
        else:
            torch.add(x, a, out=y)
        hg.hg_vocab_loss(h, y, shards, targets, loss, lse)
        count = (targets >= 0).sum().clamp(min=1)
        mean = loss.sum() / count
        # Backward: the head's gradient is written, the embedding's added to it.
        up = torch.where(targets >= 0, 1.0 / count, 0.0)
        hg.hg_vocab_loss_grad(h, y, shards, targets, lse, up, dy, grad_shards)
        if norm:
            hg.hg_norm_rows_grad(hn, s, weight["gain"], rstd, dy, dy, grad["gain"])
        da = dy * (1 - a * a)
        torch.matmul(x.t(), da, out=grad["layer"])
        torch.add(dy, da @ weight["layer"].t(), out=dx)
        hg.hg_vocab_embed_grad(h, tokens, dx, grad_shards, scale=scale, accumulate=True)
        # Adam on the masters.
        for k, w in master.items():
            m, v = moments[k]
            g = grad[k].float()
            m.lerp_(g, 0.1)
            v.lerp_(g * g, 0.05)
            mh, vh = m / (1 - 0.9 ** (step + 1)), v / (1 - 0.95 ** (step + 1))
            w.addcdiv_(mh, vh.sqrt().add_(1e-8), value=-lr * 0.1)
            weight[k].copy_(w)
        losses.append(mean.item())
        if log:
            log(f"step {step:3d}  loss {losses[-1]:.4f}")
    hg.hg_vocab_sync(h)
    h.close()
    if norm:
        hn.close()
    return losses


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("steps", 30), ("vocab", 8192), ("hidden", 512), ("rows", 2048),
                        ("tp", 4), ("seed", 0)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--masked", type=float, default=0.1)
    ap.add_argument("--lr", type=float, default=0.03)
    ap.add_argument("--norm", action="store_true")
    train(**vars(ap.parse_args()))


if __name__ == "__main__":
    main()
