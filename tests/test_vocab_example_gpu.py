"""The vocabulary operators together, as a trainer uses them: the example's
training steps, against the same steps differentiated by torch."""

import math
import os
import sys

import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tp_vocab_logits_gb300 import _build
    _build.build()


def test_example_learns():
    import tied_vocab_step
    losses = tied_vocab_step.train(steps=24, vocab=1000, hidden=256, rows=600, tp=3, log=None)
    assert all(math.isfinite(x) for x in losses)
    # Four fixed batches of a deterministic rule: memorised from ln(1000) on.
    assert losses[0] > 5.0 and losses[-1] < 0.5 * losses[0]


def test_tied_gradient_matches_autograd():
    """One step's gradient of the tied matrix, through lookup and loss, against
    64-bit autograd. The head's gradient is rounded to bf16, then the
    lookup's is added and rounded again; the hidden gradient in between is
    rounded too: three roundings of 2^-8 of the sum of the terms' magnitudes,
    taken twice for the products' own d (2^-8 each term)."""
    from tp_vocab_logits_gb300 import hg
    gen = torch.Generator(device="cuda").manual_seed(3)
    tp, cols, vocab, K, N, scale = 2, 400, 797, 128, 300, 4.0
    whole = (torch.randn(tp * cols, K, generator=gen, device="cuda") * 0.05).to(torch.bfloat16)
    tokens = torch.randint(0, vocab, (N,), generator=gen, device="cuda")
    targets = torch.randint(0, vocab, (N,), generator=gen, device="cuda")
    targets[::7] = -100
    shards = list(whole.split(cols))
    h = hg.hg_vocab_create(tp, cols, K, N, vocab=vocab)
    x = torch.empty(N, K, device="cuda", dtype=torch.bfloat16)
    loss, lse = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    hg.hg_vocab_embed(h, tokens, shards, x, scale=scale)
    hg.hg_vocab_loss(h, x, shards, targets, loss, lse)
    up = torch.where(targets >= 0, 1.0 / (targets >= 0).sum(), 0.0)
    dx, gw = torch.empty_like(x), torch.empty_like(whole)
    gws = list(gw.split(cols))
    hg.hg_vocab_loss_grad(h, x, shards, targets, lse, up, dx, gws)
    hg.hg_vocab_embed_grad(h, tokens, dx, gws, scale=scale, accumulate=True)

    w = whole.double().requires_grad_()
    y = F.embedding(tokens, w) * scale
    y = y + (x.double() - y).detach()  # the lookup's own rounding, as the head saw it
    want = F.cross_entropy(y @ w[:vocab].t(), targets, ignore_index=-100)
    want.backward()
    mean = (loss.double() * up.double()).sum()
    assert abs(mean.item() - want.item()) <= 2.0 ** -18 * want.item()
    p = torch.softmax(y.detach() @ w[:vocab].detach().t(), 1)
    on = targets >= 0
    p[on, targets[on]] -= 1
    d = (p * up.double()[:, None]).abs()
    head = d.t() @ y.detach().abs()
    dxa = d @ w[:vocab].detach().abs()
    look = torch.zeros_like(whole, dtype=torch.float64).index_add_(0, tokens, dxa * scale)
    head = torch.cat([head, torch.zeros(tp * cols - vocab, K, device="cuda",
                                        dtype=torch.float64)])
    err = (gw.double() - w.grad).abs()
    assert bool((err <= 2 * 3 * 2.0 ** -8 * (head + look) + 1e-12).all())
    h.close()
