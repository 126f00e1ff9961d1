"""The vocabulary operators over seeded random sizes, types, masks, strides and
pieces, against the 64-bit forms and bounds of test_vocab_gpu.py."""

import random

import pytest
import torch

from tp_vocab_logits_gb300 import hg

from test_vocab_gpu import (_built, bf16, check_embed_grad, check_loss, fp16, fp32,  # noqa: F401
                            gen_of, grad_inputs, grad_want, ids_of, loss_inputs, normal, run_loss,
                            table_of, within)

pytestmark = pytest.mark.gpu


def log_int(r, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** r.random())))


@pytest.mark.parametrize("seed", range(48))
def test_loss_and_gradient(seed):
    r = random.Random(seed)
    tp = r.choice([1, 1, 2, 3, 5, 8, 16, 32])
    W = log_int(r, 1, 4000 // tp + 60)
    vocab = tp * W - (r.randint(0, tp * W - 1) if r.random() < 0.3 else 0)
    K = 8 * log_int(r, 1, 160)
    N = log_int(r, 1, 900)
    dtype = r.choice([bf16, fp16])
    masked = r.choice([0.0, 0.3, 0.95])
    scale = r.choice([1.0, 0.5, -0.8])
    whole, shards, hidden, tgt = loss_inputs(tp, W, vocab, K, N, dtype, masked, seed)
    tgt = tgt if r.random() < 0.5 else tgt.int()
    extra = 8 * r.randint(0, 3)  # hidden and its gradient as columns of a wider matrix
    wide = torch.zeros((N, K + extra), device="cuda", dtype=dtype)
    wide[:, extra:] = hidden
    hidden = wide[:, extra:]
    h = hg.hg_vocab_create(tp, W, K, N + r.randint(0, 300), vocab=vocab, dtype=dtype,
                           ops=("loss", "loss_grad"), piece_bytes=r.choice([0, 0, 1, 1 << 20]))
    loss, lse = run_loss(h, hidden, shards, tgt, scale)
    check_loss(loss, lse, whole, hidden, tgt, vocab, scale)
    g = grad_inputs(tgt, seed)
    gwide = torch.full_like(wide, 7.0)
    gh, gw = gwide[:, extra:], torch.full_like(whole, 7.0)
    hg.hg_vocab_loss_grad(h, hidden, shards, tgt, lse, g, gh, list(gw.split(W)),
                          logit_scale=scale)
    hg.hg_vocab_sync(h)
    want = grad_want(whole, hidden, tgt, vocab, scale, lse, g)
    within(gh, want[0], want[1], "grad_hidden")
    within(gw, want[2], want[3], "grad_weight")
    assert bool((gwide[:, :extra] == 7).all())
    h.close()


@pytest.mark.parametrize("seed", range(48))
def test_embedding_and_gradient(seed):
    r = random.Random(1000 + seed)
    tp = r.choice([1, 2, 3, 8, 32])
    W = log_int(r, 1, 9000 // tp + 10)
    vocab = tp * W - (r.randint(0, tp * W - 1) if r.random() < 0.3 else 0)
    K = log_int(r, 1, 1500)
    N = log_int(r, 1, 12000)
    dtype = r.choice([bf16, fp16, fp32])
    scale = r.choice([1.0, 2.3])
    g = gen_of(seed)
    whole, shards = table_of(g, tp, W, K, dtype)
    tok = ids_of(g, N, vocab, r.choice([0.0, 0.4]), r.choice([torch.int32, torch.int64]))
    if r.random() < 0.4:  # few tokens, many times
        tok = torch.where(tok >= 0, tok % max(1, vocab // 50), tok)
    wide = torch.full((N, K + r.randint(0, 9)), 5.0, device="cuda", dtype=dtype)
    rows = wide[:, :K]
    h = hg.hg_vocab_create(tp, W, K, N, vocab=vocab, dtype=dtype, ops=("embed", "embed_grad"))
    hg.hg_vocab_embed(h, tok, shards, rows, scale=scale)
    want = (whole[tok.clamp(min=0).long()].float() * scale).to(dtype)
    assert torch.equal(rows, torch.where((tok >= 0)[:, None], want, torch.zeros_like(want)))
    assert bool((wide[:, K:] == 5).all())
    rows.copy_(normal(g, (N, K), 1.0, dtype))
    for accumulate in (False, True):
        old = whole.clone()
        hg.hg_vocab_embed_grad(h, tok, rows, shards, scale=scale, accumulate=accumulate)
        check_embed_grad(whole, tok, rows, vocab, scale, old if accumulate else None)
    h.close()
