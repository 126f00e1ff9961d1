"""The loss and its gradient at sizes beyond the other tests': rows of many row tiles
and groups of them, pieces cut by the default budget, rows that are sure of their
target and logits in the thousands. 64-bit forms and bounds of test_vocab_gpu.py."""

import pytest
import torch

from tp_vocab_logits_gb300 import hg

from test_vocab_gpu import (_built, bf16, check_loss, fp16, gen_of, grad_inputs,  # noqa: F401
                            grad_want, loss_inputs, normal, run_loss, within)

pytestmark = pytest.mark.gpu


def check_grad(h, whole, shards, hidden, tgt, vocab, scale, lse, up):
    gh, gw = torch.full_like(hidden, 9.0), torch.full_like(whole, 9.0)
    hg.hg_vocab_loss_grad(h, hidden, shards, tgt, lse, up, gh,
                          list(gw.split(shards[0].shape[0])), logit_scale=scale)
    hg.hg_vocab_sync(h)
    want = grad_want(whole, hidden, tgt, vocab, scale, lse, up)
    within(gh, want[0], want[1], "grad_hidden")
    within(gw, want[2], want[3], "grad_weight")


@pytest.mark.parametrize("tp,W,vocab,K,N,dtype,masked,piece", [
    (3, 1000, 2990, 328, 2304, bf16, 0.0, 0),      # nine row tiles: a group and one
    (3, 1000, 2990, 328, 4500, fp16, 0.1, 0),
    (2, 1500, 3000, 72, 4097, bf16, 0.0, 1 << 23),  # several pieces, several groups
    (8, 1200, 9601, 64, 33000, bf16, 0.05, 0),     # pieces cut by the default 512 MB
    (1, 2000, 2000, 1544, 2500, fp16, 0.4, 0),     # sums over K and rows in segments
])
def test_many_rows(tp, W, vocab, K, N, dtype, masked, piece):
    vocab = min(vocab, tp * W)
    whole, shards, hidden, tgt = loss_inputs(tp, W, vocab, K, N, dtype, masked, N)
    h = hg.hg_vocab_create(tp, W, K, N, vocab=vocab, dtype=dtype, ops=("loss", "loss_grad"),
                           piece_bytes=piece)
    loss, lse = run_loss(h, hidden, shards, tgt, 0.7)
    check_loss(loss, lse, whole, hidden, tgt, vocab, 0.7)
    check_grad(h, whole, shards, hidden, tgt, vocab, 0.7, lse, grad_inputs(tgt, N))
    h.close()


@pytest.mark.parametrize("N", [3, 64, 65, 150, 300])
@pytest.mark.parametrize("K", [64, 1160])
@pytest.mark.parametrize("dtype", [bf16, fp16])
def test_gradient_of_sure_rows(N, K, dtype):
    """Row i points along the weights of its target, with a strength from nothing to
    logits in the thousands, so that p - 1 cancels more and more; every third row is
    as sure of a wrong column."""
    W = 300
    g = gen_of(N + K)
    whole = normal(g, (W, K), 1.0, dtype)
    tgt = torch.randint(0, W, (N,), generator=g, device="cuda")
    strength = torch.linspace(0, 2000 / K, N, device="cuda")
    at = torch.where(torch.arange(N, device="cuda") % 3 == 2, (tgt + 7) % W, tgt)
    hidden = (whole[at].float() * strength[:, None]
              + 0.05 * normal(g, (N, K), 1.0, torch.float32)).to(dtype)
    h = hg.hg_vocab_create(1, W, K, N, dtype=dtype, ops=("loss", "loss_grad"))
    loss, lse = run_loss(h, hidden, [whole], tgt, 1.0)
    check_loss(loss, lse, whole, hidden, tgt, W, 1.0)
    assert lse.max().item() > 1000
    check_grad(h, whole, [whole], hidden, tgt, W, 1.0, lse, grad_inputs(tgt, N))
    h.close()
