"""A gather with another device current than the handle's is refused on the host,
before any device work, and leaves handle and outputs as they were."""

import ctypes

import pytest
import torch

from tp_vocab_logits_gb300 import _build, hg, synth

from helpers import assert_mailboxes_armed, empty_outs, rewrite_concat

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


@pytest.mark.parametrize("device_parity", [False, True])
def test_gathers_refuse_another_current_device(device_parity):
    """One GPU is enough: the handle's record of its device, the first word of the
    structure, is set to the next one, so that the current device is another."""
    tp, W, M, K = 2, 1024, 2, 256
    h = hg.hg_create(tp, W, M, device_parity=device_parity)
    device = ctypes.c_int.from_address(h.ptr)
    assert device.value == torch.cuda.current_device()
    bits = synth.shards(5, tp, M, W, scale=3.0, sent_frac=0.01, zero_frac=0.01, negzero_frac=0.01,
                        set_index=0, device="cuda")
    shards = [bits[r] for r in range(tp)]
    outs = empty_outs(tp, M, tp * W)
    before = [o.clone() for o in outs]
    hidden = [torch.zeros((M, K), dtype=torch.bfloat16, device="cuda") for _ in range(tp)]
    weight = [torch.zeros((W, K), dtype=torch.bfloat16, device="cuda") for _ in range(tp)]
    stats = hg.new_row_stats(M)
    call = hg.GatherCall(h, shards, outs, M)
    calls = [lambda: hg.hg_gather(h, shards, outs, M), call,
             lambda: hg.hg_gather_stats(h, shards, outs, stats, M),
             lambda: hg.hg_gather_fused(h, hidden, weight, outs, M),
             lambda: hg.hg_rearm(h)]
    parity = hg.hg_parity(h)
    device.value += 1
    try:
        for refused in calls:
            with pytest.raises(hg.HGError) as e:
                refused()
            assert e.value.status == hg.HG_ERR_ARG
    finally:
        device.value -= 1
    torch.cuda.synchronize()
    hg.hg_sync(h)
    assert hg.hg_parity(h) == parity and not bool(stats.any())
    assert all(torch.equal(o, b) for o, b in zip(outs, before))
    assert_mailboxes_armed(h, hg)
    call()  # and served again
    hg.hg_sync(h)
    want = rewrite_concat(shards)
    assert all(torch.equal(o.view(torch.int32), want) for o in outs)
    h.close()
