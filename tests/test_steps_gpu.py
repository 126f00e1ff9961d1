"""The norm and the beam search with the operators beside them, as they are used: a
decoding step, captured and replayed too, and a training step; on other streams, by two
handles at once, and with another device current."""

import ctypes
import math
import os
import sys

import numpy as np
import pytest
import torch
import torch.nn.functional as F

from test_beam_gpu import totals, want_picks, want_states
from test_norm_gpu import check_norm
from tp_vocab_logits_gb300 import hg

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
bf16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tp_vocab_logits_gb300 import _build
    _build.build()


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, std=1.0, dtype=bf16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


# ---- decoding ----------------------------------------------------------------------


@pytest.mark.parametrize("items,beams,steps,vocab,hidden,heads,tp,end", [
    (4, 4, 9, 1000, 256, 4, 4, 1), (1, 2, 5, 129, 64, 1, 1, 0), (2, 8, 6, 3001, 128, 2, 2, 7),
    (3, 5, 4, 600, 192, 3, 3, -1), (1, 1, 3, 200, 64, 2, 1, 3)])
def test_beam_search_example(items, beams, steps, vocab, hidden, heads, tp, end):
    """Every call of a search, each on what it was given. The head's bf16 logits: the
    product's rounding, 2^-8, and its fp32 sums. The totals' order is the picks' own; where
    two are as close as the logsumexp's error, 2^-14, either may come first."""
    import beam_search
    paths = [[[] for _ in range(beams)] for _ in range(items)]
    kept, calls = {}, []

    def watch(name, *t):
        calls.append(name)
        if name == "norm":
            x, gain, out, residual = t
            s = x if residual is None else (x.float() + residual.float()).to(bf16)
            check_norm(s, gain, 1e-6, None, out)
        elif name == "head":
            b, matrix, logits = t
            want = b.double() @ matrix.double().t()
            terms = b.double().abs() @ matrix.double().abs().t()
            bound = 2.0 ** -8 * want.abs() + (hidden + 8) * 2.0 ** -24 * terms
            for one in logits:
                assert bool(((one.double() - want).abs() <= bound).all())
        elif name == "select":
            logits, scores, tokens, parents, picked, finished, done = t
            total = totals(logits, torch.logsumexp(logits.double(), 1), scores,
                           finished if end >= 0 else None, end)
            want = want_picks(total, logits, items, beams, beams)
            new = []
            for i in range(items):
                for k in range(beams):
                    token, parent = tokens[i, k].item(), parents[i, k].item()
                    value = total[i * beams + parent, token].item()
                    assert abs(picked[i, k].item() - value) <= 2.0 ** -14 + 2.0 ** -23 * abs(value)
                    assert abs(value - want[i][k][2]) <= 2.0 ** -13
                    over = end >= 0 and (token == end or bool(finished[i, parent]))
                    assert bool(done[i, k]) == over
                new.append([paths[i][parents[i, k]] + [tokens[i, k].item()] for k in range(beams)])
            paths[:] = new
        elif name == "before":
            parents, filled, history = t
            kept["want"] = want_states([(filled, 1), (history, 0)], parents)
        else:
            _, filled, history = t
            assert torch.equal(filled, kept["want"][0]) and torch.equal(history, kept["want"][1])

    hypotheses, scores = beam_search.search(items, beams, steps, vocab, hidden, heads, tp, end=end,
                                            watch=watch)
    assert calls.count("norm") == 2 * steps and calls.count("after") == steps
    assert hypotheses.tolist() == paths
    assert bool((scores[:, :-1] >= scores[:, 1:]).all()) and bool(torch.isfinite(scores).all())


class Decoder:
    """A step with all buffers its own, on fixed hidden states: lookup, norm, head in torch,
    gather with statistics, selection, reordering of a cache."""

    def __init__(self, seed, items=3, beams=4, vocab=1024, hidden=256, tp=2, length=6):
        g = gen_of(seed)
        self.rows, self.tp = items * beams, tp
        self.matrix = normal(g, (vocab, hidden), 0.2)
        self.shards = list(self.matrix.split(vocab // tp))
        self.gain, self.residual = normal(g, (hidden,)), normal(g, (self.rows, hidden))
        self.words = hg.hg_vocab_create(tp, vocab // tp, hidden, self.rows)
        self.norm = hg.hg_norm_create(hidden, self.rows)
        self.head = hg.hg_create(tp, vocab // tp, self.rows, device_parity=True)
        self.beam = hg.hg_beam_create(items, beams, vocab, beams)
        self.x, self.b, self.s = (torch.empty_like(self.residual) for _ in range(3))
        self.part = [torch.empty((self.rows, vocab // tp), device="cuda", dtype=bf16)
                     for _ in range(tp)]
        self.logits = [torch.empty((self.rows, vocab), device="cuda", dtype=bf16)
                       for _ in range(tp)]
        self.stats = hg.new_row_stats(self.rows)
        self.cache0 = normal(g, (2, self.rows, 3, length, 16))
        self.cache = self.cache0.clone()
        self.tokens = torch.empty((items, beams), device="cuda", dtype=torch.int64)
        self.parents = torch.empty_like(self.tokens)
        self.scores, self.picked = (torch.empty((items, beams), device="cuda") for _ in range(2))
        self.restart()

    def restart(self):
        self.tokens.copy_(torch.arange(self.rows, device="cuda").view(self.tokens.shape) * 7)
        self.scores.fill_(-math.inf)
        self.scores[:, 0] = 0
        self.cache.copy_(self.cache0)

    def step(self, gather=True):
        hg.hg_vocab_embed(self.words, self.tokens.view(-1), self.shards, self.x)
        hg.hg_norm_rows(self.norm, self.x, self.gain, self.b, residual=self.residual,
                        sum_out=self.s)
        for part, shard in zip(self.part, self.shards):
            torch.matmul(self.b, shard.t(), out=part)
        lse = None
        if gather:
            hg.hg_gather_stats(self.head, self.part, self.logits, self.stats)
            lse = hg.unpack_row_stats(self.stats)["logsumexp"]
        else:
            torch.cat(self.part, 1, out=self.logits[0])
        hg.hg_beam_select(self.beam, self.logits[0], self.scores, self.tokens, self.parents,
                          self.picked, lse=lse)
        hg.hg_beam_reorder(self.beam, self.parents, [(self.cache, 1)])
        self.scores.copy_(self.picked)

    def state(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.tokens, self.parents, self.scores, self.cache, self.s,
                                    self.b, self.logits[0])]

    def run(self, gather=True):
        self.restart()
        for _ in range(4):
            self.step(gather)
        return self.state()

    def capture(self):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph

    def close(self):
        torch.cuda.synchronize()
        hg.hg_sync(self.head)
        for h in (self.words, self.norm, self.head, self.beam):
            h.close()


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_step_of_the_statistics():
    """The first step's picks from the gather's own logsumexp: the best of one beam."""
    d = Decoder(1)
    d.restart()
    d.step()
    logits, lse = d.logits[0], hg.unpack_row_stats(d.stats)["logsumexp"]
    scores = torch.full_like(d.scores, -math.inf)
    scores[:, 0] = 0
    items, beams = scores.shape
    want = want_picks(totals(logits, lse, scores, None, -1), logits, items, beams, beams)
    for i in range(items):
        got = list(zip(d.tokens[i].tolist(), d.parents[i].tolist(), d.picked[i].tolist()))
        assert got == [(t, p, np.float32(v)) for t, p, v in want[i]]
    # All beams go on from the first.
    first = d.cache0.view(2, items, beams, 3, 6, 16)[:, :, :1].expand(-1, -1, beams, -1, -1, -1)
    assert torch.equal(d.cache.view(first.shape), first)
    d.close()


def test_a_captured_step():
    """Replayed step by step, between eager steps, and after another handle's graph."""
    d, other = Decoder(2), Decoder(3)
    want, want_other = d.run(), other.run()
    graph, graph_other = d.capture(), other.capture()
    for _ in range(2):
        d.restart()
        other.restart()
        for _ in range(4):
            graph.replay()
            graph_other.replay()
        assert same(d.state(), want) and same(other.state(), want_other)
    d.restart()
    for step in range(4):
        graph.replay() if step % 2 else d.step()
    assert same(d.state(), want)
    d.close()
    other.close()


def test_other_streams():
    """Two decoders at once (but for the gathers, whose CTAs wait for one another), each on a
    stream of its own; the current stream counts, and one that is given."""
    d, other = Decoder(4), Decoder(5)
    want, want_other = d.run(gather=False), other.run(gather=False)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for one, s in zip((d, other), streams):
        one.restart()
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for one, s in zip((d, other), streams):
            with torch.cuda.stream(s):
                one.step(gather=False)
    assert same(d.state(), want) and same(other.state(), want_other)
    # Given by name, behind work that its inputs wait for.
    s = streams[0]
    x = torch.zeros_like(d.x)
    out, more = torch.empty_like(x), torch.empty_like(x)
    scores, picked = torch.full_like(d.scores, -math.inf), torch.empty_like(d.picked)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        x.copy_(d.residual)
        scores[:, 0] = 0
        d.cache.copy_(d.cache0)
    hg.hg_norm_rows(d.norm, x, d.gain, out, stream=s)
    hg.hg_beam_select(d.beam, d.logits[0], scores, d.tokens, d.parents, picked, stream=s)
    hg.hg_beam_reorder(d.beam, d.parents, [(d.cache, 1)], stream=s)
    torch.cuda.synchronize()
    hg.hg_norm_rows(d.norm, d.residual, d.gain, more)
    assert torch.equal(out, more) and bool((d.parents == 0).all())
    assert bool(torch.isfinite(picked).all())
    assert torch.equal(d.cache, want_states([(d.cache0, 1)], d.parents)[0])
    d.close()
    other.close()


def test_calls_of_one_handle_that_overlap():
    """Those that need no workspace, on two streams at once."""
    g = gen_of(6)
    h, hb = hg.hg_norm_create(1024, 4000), hg.hg_beam_create(4, 8, 100, 8)
    x, gain = normal(g, (2, 4000, 1024)), normal(g, (1024,))
    out, want = torch.empty_like(x), torch.empty_like(x)
    state = normal(g, (2, 32, 5000))
    parents = torch.randint(0, 8, (2, 4, 8), generator=g, device="cuda")
    moved = [want_states([(state[k], 0)], parents[k])[0] for k in range(2)]
    for k in range(2):
        hg.hg_norm_rows(h, x[k], gain, want[k])
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        for k in range(2):
            hg.hg_norm_rows(h, x[k], gain, out[k], stream=streams[k])
    for k in range(2):
        hg.hg_beam_reorder(hb, parents[k], [state[k]], stream=streams[k])
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.equal(state[k], moved[k]) for k in range(2))
    h.close()
    hb.close()


@pytest.mark.parametrize("states", [1, 33, 256])
def test_many_states_in_a_captured_call(states):
    """More states than a launch takes, of many layouts, captured and replayed."""
    g = gen_of(states)
    hb = hg.hg_beam_create(2, 3, 100, 3)
    parents = torch.tensor([[2, 0, 0], [1, 1, 7]], device="cuda")
    kept = [(normal(g, (6, 3 + k % 5, 16)), 0) if k % 2 else (normal(g, (2, 6, 40))[:, :, :31], 1)
            for k in range(states)]
    first = [t.clone() for t, _ in kept]
    want = want_states(kept, parents)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hg.hg_beam_reorder(hb, parents, kept)
    assert same([t for t, _ in kept], first)
    graph.replay()
    torch.cuda.synchronize()
    assert same([t for t, _ in kept], want)
    hb.close()


# ---- training ----------------------------------------------------------------------


def norm_in_64_bits(s, gain, eps):
    return s * torch.rsqrt((s * s).mean(1, keepdim=True) + eps) * gain


def test_gradients_through_lookup_norm_and_loss():
    """One step's gradients of the tied matrix and of the norm's gain against 64-bit
    autograd, with the forward pass's own roundings on both sides. Roundings of the
    gradients, 2^-8 each of the terms' magnitudes: the products' own d and the head's
    gradient of its input (2), the norm's gradient (1), the matrix's, written and added to
    (2); all others are fp32. Six of them are allowed."""
    g = gen_of(3)
    tp, cols, vocab, K, N, scale, eps = 2, 400, 797, 128, 300, 4.0, 1e-5
    whole, gain = normal(g, (tp * cols, K), 0.05), normal(g, (K,), 0.2) + 1
    residual, more = normal(g, (N, K)), normal(g, (N, K), 0.001)
    tokens = torch.randint(0, vocab, (N,), generator=g, device="cuda")
    targets = torch.randint(0, vocab, (N,), generator=g, device="cuda")
    targets[::7] = -100
    shards = list(whole.split(cols))
    h, hn = hg.hg_vocab_create(tp, cols, K, N, vocab=vocab), hg.hg_norm_create(K, N)
    x, s, y, dy, dx = (torch.empty((N, K), device="cuda", dtype=bf16) for _ in range(5))
    loss, lse, rstd = (torch.empty(N, device="cuda") for _ in range(3))
    up = torch.where(targets >= 0, 1.0 / (targets >= 0).sum(), 0.0)
    gw, gg = torch.empty_like(whole), torch.empty_like(gain)
    gws = list(gw.split(cols))

    def step():
        hg.hg_vocab_embed(h, tokens, shards, x, scale=scale)
        hg.hg_norm_rows(hn, x, gain, y, residual=residual, sum_out=s, rstd=rstd, eps=eps)
        hg.hg_vocab_loss(h, y, shards, targets, loss, lse)
        hg.hg_vocab_loss_grad(h, y, shards, targets, lse, up, dy, gws)
        hg.hg_norm_rows_grad(hn, s, gain, rstd, dy, dx, gg, grad_sum=more)
        hg.hg_vocab_embed_grad(h, tokens, dx, gws, scale=scale, accumulate=True)

    step()
    w, gain64 = whole.double().requires_grad_(), gain.double().requires_grad_()
    e = F.embedding(tokens, w) * scale + residual.double()
    e = e + (s.double() - e).detach()
    n = norm_in_64_bits(e, gain64, eps)
    n = n + (y.double() - n).detach()
    want = F.cross_entropy(n @ w[:vocab].t(), targets, ignore_index=-100)
    (want + (e * more.double()).sum()).backward()
    mean = (loss.double() * up.double()).sum()
    assert abs(mean.item() - want.item()) <= 2.0 ** -18 * want.item()

    w64, n64, s64 = whole.double()[:vocab], y.double(), s.double()
    p = torch.softmax(n64 @ w64.t(), 1)
    on = targets >= 0
    p[on, targets[on]] -= 1
    d = (p * up.double()[:, None]).abs()
    head = torch.cat([d.t() @ n64.abs(), torch.zeros(tp * cols - vocab, K, device="cuda",
                                                     dtype=torch.float64)])
    dn = d @ w64.abs()
    r = torch.rsqrt((s64 * s64).mean(1, keepdim=True) + eps)
    dg = dn * gain.double().abs()
    ds = r * dg + s64.abs() * r ** 3 * (dg * s64.abs()).mean(1, keepdim=True) + more.double().abs()
    look = torch.zeros_like(w, dtype=torch.float64).index_add_(0, tokens, ds * scale)
    assert bool(((gw.double() - w.grad).abs() <= 6 * 2.0 ** -8 * (head + look) + 1e-12).all())
    terms = (dn * s64.abs() * r).sum(0)
    assert bool(((gg.double() - gain64.grad).abs() <= 6 * 2.0 ** -8 * terms + 1e-12).all())

    # Captured, it leaves the same bits.
    want_bits = [t.clone() for t in (gw, gg, dx, loss)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        for t in (gw, gg, dx, loss, y, s, dy):
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert same((gw, gg, dx, loss), want_bits)
    h.close()
    hn.close()


def test_training_example_with_the_norm():
    import tied_vocab_step
    losses = tied_vocab_step.train(steps=4, vocab=1000, hidden=256, rows=600, tp=3, log=None,
                                   norm=True)
    assert len(losses) == 4 and all(math.isfinite(x) for x in losses)


# ---- devices -----------------------------------------------------------------------


def test_calls_refuse_another_current_device():
    """One GPU is enough: the handle's record of its device, the first word of the
    structure, is set to the next one, so that the current device is another."""
    hn, hb = hg.hg_norm_create(64, 3), hg.hg_beam_create(2, 2, 50, 2)
    x = torch.ones((3, 64), device="cuda", dtype=bf16)
    gain, out = x[0].clone(), torch.full_like(x, 5.0)
    grad, rstd = torch.full_like(gain, 5.0), torch.ones(3, device="cuda")
    logits, scores = torch.ones((4, 50), device="cuda", dtype=bf16), torch.ones((2, 2), device="cuda")
    tokens, parents = (torch.full((2, 2), 1, device="cuda") for _ in range(2))
    picked = torch.full((2, 2), 5.0, device="cuda")
    state = torch.arange(4, device="cuda")
    calls = [(hn, lambda: hg.hg_norm_rows(hn, x, gain, out)),
             (hn, lambda: hg.hg_norm_rows(hn, x[:0], gain, out[:0])),
             (hn, lambda: hg.hg_norm_rows_grad(hn, x, gain, rstd, x, out, grad)),
             (hb, lambda: hg.hg_beam_reorder(hb, parents, [state])),
             (hb, lambda: hg.hg_beam_select(hb, logits, scores, tokens, parents, picked))]
    for h, call in calls:
        device = ctypes.c_int.from_address(h.ptr)
        assert device.value == torch.cuda.current_device()
        device.value += 1
        try:
            with pytest.raises(hg.HGError) as e:
                call()
            assert e.value.status == hg.HG_ERR_ARG
        finally:
            device.value -= 1
    torch.cuda.synchronize()
    assert bool((out == 5).all()) and bool((grad == 5).all()) and bool((picked == 5).all())
    assert state.tolist() == [0, 1, 2, 3] and bool((tokens == 1).all())
    for _, call in calls:  # and served again
        call()
    assert bool((out != 5).all()) and bool((grad != 5).all()) and bool((picked != 5).all())
    assert state.tolist() == [1, 1, 3, 3]
    hn.close()
    hb.close()


def test_refusals_of_overlaps():
    hb = hg.hg_beam_create(2, 2, 50, 2)
    logits, scores = torch.ones((4, 50), device="cuda", dtype=bf16), torch.ones((2, 2), device="cuda")
    ids, state = torch.zeros((2, 2), device="cuda", dtype=torch.int64), torch.arange(4, device="cuda")
    for call in (lambda: hg.hg_beam_select(hb, logits, scores, ids, ids.clone(), scores),
                 lambda: hg.hg_beam_select(hb, logits, scores, ids, ids, scores.clone()),
                 lambda: hg.hg_beam_reorder(hb, ids, [state, (state, 0)])):
        with pytest.raises(hg.HGError) as e:
            call()
        assert e.value.status == hg.HG_ERR_ARG
    torch.cuda.synchronize()
    assert bool((scores == 1).all()) and state.tolist() == [0, 1, 2, 3]
    hg.hg_beam_reorder(hb, ids, [state, (state[:0].view(0, 4), 1)])
    assert state.tolist() == [0, 0, 2, 2]
    hb.close()
