"""A call of the vocabulary operators with another device current than the handle's
is refused on the host, before any device work."""

import ctypes

import pytest
import torch

from tp_vocab_logits_gb300 import _build, hg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


def test_calls_refuse_another_current_device():
    """One GPU is enough: the handle's record of its device, the first word of the
    structure, is set to the next one, so that the current device is another."""
    tp, W, K, N = 2, 40, 64, 5
    h = hg.hg_vocab_create(tp, W, K, N)
    device = ctypes.c_int.from_address(h.ptr)
    assert device.value == torch.cuda.current_device()
    whole = torch.full((tp * W, K), 3.0, device="cuda", dtype=torch.bfloat16)
    shards = list(whole.split(W))
    rows = torch.full((N, K), 5.0, device="cuda", dtype=torch.bfloat16)
    ids = torch.arange(N, device="cuda")
    loss, lse, up = (torch.full((N,), 7.0, device="cuda") for _ in range(3))
    grad, grad_whole = torch.full_like(rows, 9.0), torch.full_like(whole, 9.0)
    grads = list(grad_whole.split(W))
    none = torch.empty((0, K), device="cuda", dtype=torch.bfloat16)
    calls = [lambda: hg.hg_vocab_embed(h, ids, shards, grad),
             lambda: hg.hg_vocab_embed(h, ids[:0], shards, none),
             lambda: hg.hg_vocab_embed_grad(h, ids, rows, grads),
             lambda: hg.hg_vocab_embed_grad(h, ids[:0], none, grads, accumulate=True),
             lambda: hg.hg_vocab_loss(h, rows, shards, ids, loss, lse),
             lambda: hg.hg_vocab_loss_grad(h, rows, shards, ids, lse, up, grad, grads),
             lambda: hg.hg_vocab_sync(h)]
    device.value += 1
    try:
        for call in calls:
            with pytest.raises(hg.HGError) as e:
                call()
            assert e.value.status == hg.HG_ERR_ARG
    finally:
        device.value -= 1
    torch.cuda.synchronize()
    assert bool((grad == 9).all()) and bool((grad_whole == 9).all())
    assert bool((loss == 7).all()) and bool((lse == 7).all())
    for call in calls:  # and served again
        call()
    assert bool((loss != 7).all())
    h.close()
