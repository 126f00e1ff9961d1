"""Selection among logits that no bound tells apart, which finds the n-th best bit by bit: over
the bits of the value, then over as many as the vocabulary has, of the token."""

import math

import pytest
import torch

from test_beam_gpu import Call, _built, check_select, exact_lse, gen_of  # noqa: F401
from tp_vocab_logits_gb300 import hg

pytestmark = pytest.mark.gpu

bf16, fp16, fp32 = torch.bfloat16, torch.float16, torch.float32


# Vocabularies of an odd number of bits and of an even one; more candidates than are ranked.
@pytest.mark.parametrize("items,beams,V,picks", [
    (2, 3, 4097, 8), (2, 3, 8191, 8), (1, 4, 8192, 16), (1, 4, 32000, 8), (3, 2, 16384, 5),
    (2, 5, 32767, 128), (1, 4, 100277, 8), (2, 2, 128256, 4), (1, 3, 65536, 1), (1, 1, 131071, 7),
    (1, 2, 262144, 4), (1, 64, 5000, 128), (200, 2, 6000, 4), (1, 2, 163840, 16)])
@pytest.mark.parametrize("dtype", [bf16, fp32])
def test_alike_logits(items, beams, V, picks, dtype):
    """One value: the lower beam, then the lower token. Two values: the larger one's few tokens,
    then the lowest of the rest. Values that differ in their last bit alone."""
    rows = items * beams
    h = hg.hg_beam_create(items, beams, V, picks, dtype=dtype)
    scores = torch.zeros((items, beams), device="cuda")
    lse = torch.full((rows,), math.log(V), device="cuda")
    want = [(k % V, k // V) for k in range(picks)]
    for value in (0.0, -3.5):
        logits = torch.full((rows, V), value, device="cuda", dtype=dtype)
        for given in (lse, None):
            call = Call(h, logits, scores, given)
            if given is not None or value == 0:
                assert all([r[:2] for r in call.rows(i)] == want for i in range(items))
            else:
                # V equal terms of an exponential that is rounded: the logsumexps of equal rows
                # are sums in another order where the rows lie or are dealt out otherwise, so
                # they differ by up to LSE_ERROR and put the beams in any order. Of each beam
                # it is the lowest tokens still.
                check_select(call, exact=False)
                for i in range(items):
                    by_beam = {}
                    for token, beam, _ in call.rows(i):
                        by_beam.setdefault(beam, []).append(token)
                    assert all(t == list(range(len(t))) for t in by_beam.values())
            before = [t.clone() for t in (call.tokens, call.parents, call.picked)]
            for _ in range(3):
                call.run()
            for a, b in zip(before, (call.tokens, call.parents, call.picked)):
                assert torch.equal(a, b)
    g = gen_of(V)
    logits = torch.ones((rows, V), device="cuda", dtype=dtype)
    logits[:, torch.randint(0, V, (3,), generator=g, device="cuda")] = 1.5
    check_select(Call(h, logits, scores, lse), exact=True)
    least = torch.finfo(dtype).eps
    logits = 1 + least * torch.randint(0, 2, (rows, V), generator=g, device="cuda").to(dtype)
    check_select(Call(h, logits, scores, lse), exact=True)
    h.close()


@pytest.mark.parametrize("V", [500, 32000, 163840])
@pytest.mark.parametrize("dtype", [bf16, fp32])
@pytest.mark.parametrize("out", [-1e9, -1e20, -math.inf])
def test_one_live_beam(V, dtype, out):
    """A search's first step: the other beams are out by a score far below, or of -inf."""
    items, beams, picks = 3, 4, 8
    g = gen_of(V)
    logits = torch.randn((items * beams, V), generator=g, device="cuda").mul_(2.5).to(dtype)
    scores = torch.full((items, beams), out, device="cuda")
    scores[:, 0] = 0
    h = hg.hg_beam_create(items, beams, V, picks, dtype=dtype)
    call = Call(h, logits, scores, exact_lse(logits).float())
    check_select(call, exact=True)
    assert all(r[1] == 0 for i in range(items) for r in call.rows(i))
    h.close()
