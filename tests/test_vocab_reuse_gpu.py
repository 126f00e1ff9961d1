"""One handle for calls of every size up to its own, in an order in which what a large
call left in the workspace, NaN among it, is there when a small one comes. 64-bit
forms and bounds of test_vocab_gpu.py."""

import math

import pytest
import torch

from tp_vocab_logits_gb300 import hg

from test_vocab_gpu import (_built, bf16, check_embed_grad, check_loss, fp16, fp32,  # noqa: F401
                            gen_of, grad_inputs, ids_of, loss_inputs, normal, run_loss)
from test_vocab_large_gpu import check_grad

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tp,W,vocab,K,dtype,masked,piece", [
    (2, 900, 1790, 72, bf16, 0.1, 0),
    (5, 333, 1665, 1160, fp16, 0.3, 1),  # pieces of 256 columns
])
def test_loss_and_gradient(tp, W, vocab, K, dtype, masked, piece):
    most = 3000
    whole, shards, hidden, tgt = loss_inputs(tp, W, vocab, K, most, dtype, masked, most)
    h = hg.hg_vocab_create(tp, W, K, most, vocab=vocab, dtype=dtype, ops=("loss", "loss_grad"),
                           piece_bytes=piece)
    bad, gh, gw = hidden.clone(), torch.empty_like(hidden), torch.empty_like(whole)
    bad[(tgt >= 0).nonzero()[0, 0]] = math.nan

    def spoil():
        _, lse = run_loss(h, bad, shards, tgt, 1.0)
        hg.hg_vocab_loss_grad(h, bad, shards, tgt, lse, grad_inputs(tgt, 1), gh,
                              list(gw.split(W)))
        assert bool(torch.isnan(gh).any()) and bool(torch.isnan(gw).any())

    spoil()
    for N in (1, most, 16, 17, 64, 65, 128, 129, 256, 257, 600, 1025, 2049, 63, most):
        x, t = hidden[:N], tgt[:N]
        loss, lse = run_loss(h, x, shards, t, 1.0)
        check_loss(loss, lse, whole, x, t, vocab, 1.0)
        check_grad(h, whole, shards, x, t, vocab, 1.0, lse, grad_inputs(t, N))
        if N == 257:
            spoil()
    h.close()


@pytest.mark.parametrize("K,dtype", [(1500, bf16), (301, fp32)])
def test_lookup_gradient(K, dtype):
    """Row counts around every change of sort and of the rows of a run."""
    tp, W, most = 2, 1500, 30000
    g = gen_of(K)
    whole = torch.empty((tp * W, K), device="cuda", dtype=dtype)
    shards = list(whole.split(W))
    tok = ids_of(g, most, tp * W, 0.1)
    tok[:most // 3] = 7
    tok = tok[torch.randperm(most, generator=g, device="cuda")]
    grad = normal(g, (most, K), 1.0, dtype)
    h = hg.hg_vocab_create(tp, W, K, most, dtype=dtype, ops=("embed_grad",))
    hg.hg_vocab_embed_grad(h, tok, torch.full_like(grad, math.nan), shards)
    for N in (1, most, 16, 17, 2048, 2049, 6432, 6433, 6464, 6465, 25888, 25889, 25920, 25921, 9):
        hg.hg_vocab_embed_grad(h, tok[:N], grad[:N], shards, scale=0.9)
        check_embed_grad(whole, tok[:N], grad[:N], tp * W, 0.9)
    h.close()
