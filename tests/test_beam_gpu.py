"""A beam search's selection and reordering against plain forms.

With the logsumexp given, totals are the same 64-bit sums on both sides: picks are equal,
one by one. Where it is computed here it is off by the exponentials' 2^-21 and by sums
of fp32 terms, chains of at most 700 additions: e = 2^-14 covers both; the picks then have
to be the largest totals up to e, in order up to e.
"""

import math
import random

import numpy as np
import pytest
import torch

from tp_vocab_logits_gb300 import hg

pytestmark = pytest.mark.gpu

bf16, fp16, fp32 = torch.bfloat16, torch.float16, torch.float32
INF = math.inf
LSE_ERROR = 2.0 ** -14


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tp_vocab_logits_gb300 import _build
    _build.build()


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def exact_lse(logits):
    """Rows with NaN or +inf give NaN."""
    z = logits.double()
    lse = torch.logsumexp(z, 1)
    return torch.where(torch.isnan(z).any(1) | (z == INF).any(1), math.nan, lse)


def totals(logits, lse, scores, finished, end):
    """[rows, vocab] totals in 64 bits, NaN and -inf alike -inf."""
    z = logits.double()
    t = scores.double().view(-1, 1) + (z - lse.double().view(-1, 1))
    if finished is not None:
        on = finished.view(-1).bool()
        t[on] = -INF
        t[on, end] = scores.double().view(-1)[on]
    return torch.where(t.float() > -INF, t, -INF)


def want_picks(total, logits, items, beams, picks):
    """(token, parent, total) of every item, by total, beam, logit, token."""
    V = total.shape[1]
    t, z = total.view(items, -1).cpu().numpy(), logits.double().view(items, -1).cpu().numpy()
    z = np.nan_to_num(z, nan=-INF, posinf=INF, neginf=-INF)
    out = []
    for i in range(items):
        at = np.nonzero(t[i] > -INF)[0]
        if len(at) > 4 * picks + 100:  # enough to hold every tie of the last pick
            least = np.partition(t[i][at], len(at) - picks)[len(at) - picks]
            at = at[t[i][at] >= least]
        order = np.lexsort((at % V, -z[i][at], at // V, -t[i][at]))[:picks]
        rows = [(int(a % V), int(a // V), float(t[i][a])) for a in at[order]]
        out.append(rows + [(-1, -1, -INF)] * (picks - len(rows)))
    return out


class Call:
    def __init__(self, h, logits, scores, lse=None, finished=None, end=-1, ids=torch.int64):
        items = scores.shape[0]
        self.tokens = torch.full((items, h.picks), 99, device="cuda", dtype=ids)
        self.parents = torch.full_like(self.tokens, 99)
        self.picked = torch.full((items, h.picks), 99.0, device="cuda")
        self.done = torch.full((items, h.picks), 9, device="cuda", dtype=torch.uint8)
        self.args = (h, logits, scores, self.tokens, self.parents, self.picked, lse, finished, end,
                     self.done)
        self.run()

    def run(self):
        hg.hg_beam_select(*self.args)

    def rows(self, i):
        return list(zip(self.tokens[i].tolist(), self.parents[i].tolist(),
                        self.picked[i].tolist()))


def check_select(call, exact):
    h, logits, scores, _, _, _, lse, finished, end, _ = call.args
    items, beams = scores.shape
    base = lse if lse is not None else exact_lse(logits)
    total = totals(logits, base, scores, finished, end)
    want = want_picks(total, logits, items, beams, h.picks)
    grid = total.view(items, beams, -1)
    for i in range(items):
        got = call.rows(i)
        if exact:
            assert [g[:2] for g in got] == [w[:2] for w in want[i]], f"item {i}"
            assert [g[2] for g in got] == [np.float32(w[2]) for w in want[i]], f"item {i}"
        there = [g for g in got if g[0] >= 0]
        assert len(there) == sum(w[0] >= 0 for w in want[i])
        assert len({g[:2] for g in there}) == len(there)
        assert got[len(there):] == [(-1, -1, -INF)] * (len(got) - len(there))
        e = LSE_ERROR
        for k, (token, parent, value) in enumerate(there):
            t = grid[i, parent, token].item()
            if math.isinf(t):
                assert value == t
                continue
            assert abs(t - value) <= e + 2.0 ** -23 * abs(t)
            if not math.isinf(want[i][k][2]):
                assert abs(t - want[i][k][2]) <= 2 * e
        done = [(t == end and end >= 0) or (finished is not None and bool(finished[i, p]))
                for t, p, _ in there]
        assert call.done[i].tolist() == [int(d) for d in done] + [0] * (len(got) - len(there))


def inputs(g, items, beams, V, dtype, pad=0, off=0, std=2.5):
    rows = items * beams
    buf = torch.full((rows * (V + pad) + off,), 50.0, device="cuda").to(dtype)
    logits = buf[off:].view(rows, V + pad)[:, :V]
    logits.copy_(normal(g, (rows, V), std, dtype))
    return logits, -10.0 * torch.rand((items, beams), generator=g, device="cuda")


SELECT = [
    # items, beams, vocab, picks, dtype, pad, offset
    (1, 1, 1, 1, bf16, 0, 0), (1, 2, 3, 6, fp32, 0, 0), (2, 3, 7, 5, fp16, 1, 1),
    (3, 4, 100, 8, bf16, 0, 0), (5, 1, 513, 1, bf16, 7, 0), (1, 4, 4096, 8, bf16, 0, 0),
    (2, 5, 4097, 10, fp16, 0, 3), (7, 5, 9999, 5, fp32, 1, 0), (1, 64, 1000, 128, bf16, 0, 0),
    (2, 64, 2049, 64, fp32, 0, 0), (1, 4, 163840, 8, bf16, 0, 0), (3, 8, 163840, 16, bf16, 0, 8),
    (40, 8, 5000, 16, bf16, 0, 0), (1, 1, 163840, 128, fp16, 0, 0), (2, 3, 50001, 6, bf16, 0, 1),
    (1, 32, 32001, 64, fp32, 3, 0), (300, 2, 333, 4, fp16, 0, 0), (1, 1, 1000000, 5, fp32, 0, 0),
]


@pytest.mark.parametrize("items,beams,V,picks,dtype,pad,off", SELECT)
@pytest.mark.parametrize("given", [True, False])
def test_select(items, beams, V, picks, dtype, pad, off, given):
    g = gen_of(items * 100 + V)
    logits, scores = inputs(g, items, beams, V, dtype, pad, off)
    rows = torch.zeros((items * beams, 4), device="cuda")
    rows[:, 3] = exact_lse(logits)
    h = hg.hg_beam_create(items + 1, beams, V, picks, dtype=dtype)
    call = Call(h, logits, scores, rows[:, 3] if given else None, None, V // 2,
                torch.int64 if given else torch.int32)
    check_select(call, exact=given)
    before = [t.clone() for t in (call.tokens, call.parents, call.picked, call.done)]
    call.run()
    after = (call.tokens, call.parents, call.picked, call.done)
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    h.close()


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("V,dtype", [(300, bf16), (5001, fp16), (40000, fp32), (163840, bf16)])
def test_select_masks(V, dtype, given):
    """Tokens ruled out, whole rows of them, dead and finished beams, the first step of a
    search (one live beam), items with fewer candidates than picks, and none."""
    g = gen_of(V)
    items, beams, picks = 9, 4, 8
    logits, scores = inputs(g, items, beams, V, dtype)
    z = logits.view(items, beams, V)
    z.masked_fill_(torch.rand(z.shape, generator=g, device="cuda") < 0.9, -INF)
    z[0, 2] = -INF                       # a row that has nothing left
    z[1] = -INF                          # an item
    z[2] = -INF
    z[2, 1, V - 1], z[2, 3, 0] = 1.0, 2.0  # two candidates
    scores[3, 1:] = -INF                 # the first step
    scores[4] = -INF                     # dead beams only
    scores[5, 0] = math.nan
    finished = torch.zeros((items, beams), device="cuda", dtype=torch.bool)
    finished[5:, 1] = True
    finished[6] = True                   # all: four candidates
    finished[0, 2] = True                # its row has nothing left, but it goes on
    scores[7, 1] = -INF                  # finished and dead
    lse = exact_lse(logits) if given else None
    lse = None if lse is None else lse.float()
    h = hg.hg_beam_create(items, beams, V, picks, dtype=dtype)
    end = V // 3
    for fin in (None, finished):
        call = Call(h, logits, scores, lse, fin, end)
        check_select(call, exact=given)
    assert call.rows(1) == [(-1, -1, -INF)] * picks
    assert [r[0] for r in call.rows(6)] == [end] * 4 + [-1] * 4
    h.close()


@pytest.mark.parametrize("V,picks", [(100, 8), (9000, 5), (163840, 128)])
@pytest.mark.parametrize("dtype", [bf16, fp32])
def test_select_ties(V, picks, dtype):
    """Equal logits: the lower beam, then the lower token, however many there are."""
    beams = 3
    picks = min(picks, 128)
    h = hg.hg_beam_create(2, beams, V, picks, dtype=dtype)
    logits = torch.zeros((2 * beams, V), device="cuda", dtype=dtype)
    scores = torch.zeros((2, beams), device="cuda")
    lse = torch.full((2 * beams,), math.log(V), device="cuda")
    logits[3:, ::2] = -0.0               # equal to zero too
    for given in (lse, None):
        call = Call(h, logits, scores, given)
        want = [(k % V, k // V) for k in range(picks)]
        assert [r[:2] for r in call.rows(0)] == want
        assert [r[:2] for r in call.rows(1)] == want
    # A few larger ones late in each row, then the tie.
    logits[:, V - 3:] = 1.0
    scores[:, 1] = 0.5
    check_select(Call(h, logits, scores, lse), exact=True)
    # Values of few kinds.
    g = gen_of(V)
    logits.copy_(torch.randint(0, 3, logits.shape, generator=g, device="cuda"))
    check_select(Call(h, logits, scores, lse), exact=True)
    # All in order: the best come last, or first.
    ramp = torch.arange(V, device="cuda").float() / V
    for line in (ramp, ramp.flip(0)):
        logits.copy_(line.to(dtype))
        check_select(Call(h, logits, scores, lse), exact=True)
    h.close()


@pytest.mark.parametrize("items,beams,V,picks", [
    (2, 1, 1000, 128), (1, 64, 20000, 128), (3, 5, 700, 40), (1, 33, 40000, 33), (2, 16, 9000, 16),
    (200, 2, 5000, 8), (160, 1, 3000, 128)])
@pytest.mark.parametrize("order", ["sorted", "by lane", "one beam", "far apart"])
def test_select_uneven_logits(items, beams, V, picks, order):
    """Where the best are not spread over rows and beams: in the order of the tokens, or of
    their place among a warp's lanes; all of one beam; beams a few units apart."""
    g = gen_of(V + picks)
    rows = items * beams
    noise = torch.rand((rows, V), generator=g, device="cuda")
    token = torch.arange(V, device="cuda").float()
    scores = torch.rand((items, beams), generator=g, device="cuda") * 0.01
    if order == "sorted":
        z = -2.0 * torch.log(token + 3) + noise * 0.01
    elif order == "by lane":
        z = -(token // 8 % 32) + noise
    else:
        z = noise * 6 - 3
        step = 30.0 if order == "one beam" else 1.5
        scores = scores - step * torch.arange(beams, device="cuda").flip(0)
    for dtype in (bf16, fp32):
        logits = z.to(dtype)
        h = hg.hg_beam_create(items, beams, V, picks, dtype=dtype)
        lse = exact_lse(logits).float()
        check_select(Call(h, logits, scores, lse=lse), True)
        h.close()


def test_select_special_logits():
    """NaN is no candidate where the logsumexp is given, and takes its row out where it
    is not; +inf likewise, but a candidate before all others in the first case."""
    V, beams = 5000, 3
    g = gen_of(2)
    logits, scores = inputs(g, 2, beams, V, fp32)
    logits[0, ::7] = math.nan
    logits[4, 1234] = INF
    logits[5, :] = math.nan
    lse = torch.full((6,), 10.0, device="cuda")
    h = hg.hg_beam_create(2, beams, V, 6, dtype=fp32)
    call = Call(h, logits, scores, lse)
    check_select(call, exact=True)
    assert call.rows(1)[0] == (1234, 1, INF)
    call = Call(h, logits, scores)
    check_select(call, exact=False)
    assert all(r[1] in (1, 2) for r in call.rows(0))
    assert all(r[1] == 0 for r in call.rows(1))
    # Logits as large as their type has them, and of one value only.
    big = torch.full((6, V), torch.finfo(fp32).min, device="cuda")
    big[:, 17] = torch.finfo(fp32).max
    call = Call(h, big, scores)
    assert sorted(call.rows(0)[:3]) == sorted(
        (17, b, scores[0, b].item()) for b in range(3))
    # Totals that no candidate of fp32 can have.
    low = torch.full((2, beams), -3e38, device="cuda")
    big[:, 17], big[:, 18] = 0.0, -3e38
    call = Call(h, big, low, torch.zeros(6, device="cuda"))
    assert [r[:2] for r in call.rows(0)] == [(17, 0), (17, 1), (17, 2)] + [(-1, -1)] * 3
    h.close()


def test_logsumexp_of_wide_rows():
    """picked - score - logit is the logsumexp: rows whose maximum moves from slice to
    slice, and long flat ones."""
    V = 163840
    ramp = torch.linspace(-40, 40, V, device="cuda")
    rows = torch.stack([ramp, ramp.flip(0), torch.zeros_like(ramp), ramp.sin() * 3,
                        torch.full_like(ramp, -5e4), ramp.abs() * 50])
    for dtype in (bf16, fp16, fp32):
        logits = rows.to(dtype).contiguous()
        h = hg.hg_beam_create(6, 1, V, 1, dtype=dtype)
        call = Call(h, logits, torch.zeros((6, 1), device="cuda"))
        best = logits.double().amax(1)
        want = best - torch.logsumexp(logits.double(), 1)
        assert ((call.picked[:, 0].double() - want).abs() <= LSE_ERROR).all()
        h.close()


@pytest.mark.parametrize("seed", range(40))
def test_select_random(seed):
    r = random.Random(seed)
    beams = r.choice([1, 2, 3, 4, 5, 8, 16, 33, 64])
    V = max(2, round(math.exp(r.uniform(0, math.log(60000)))))
    picks = min(128, beams * V, r.choice([1, beams, 2 * beams, r.randint(1, 128)]))
    items = max(1, min(40, round(math.exp(r.uniform(0, 4))), 3000000 // (beams * V)))
    dtype = r.choice([bf16, fp16, fp32])
    g = gen_of(seed)
    logits, scores = inputs(g, items, beams, V, dtype, r.choice([0, 0, 1, 8]), r.choice([0, 0, 1]),
                            r.choice([0.1, 2.5, 10.0]))
    if r.random() < 0.5:
        logits.masked_fill_(torch.rand(logits.shape, generator=g, device="cuda")
                            < r.choice([0.3, 0.999]), -INF)
    scores.masked_fill_(torch.rand(scores.shape, generator=g, device="cuda") < 0.1, -INF)
    fin = torch.rand(scores.shape, generator=g, device="cuda") < 0.2 if r.random() < 0.5 else None
    lse = exact_lse(logits).float() if r.random() < 0.6 else None
    h = hg.hg_beam_create(items + r.choice([0, 5, 200]), beams, V, picks, dtype=dtype)
    check_select(Call(h, logits, scores, lse, fin, r.randint(0, V - 1),
                      r.choice([torch.int32, torch.int64])), exact=lse is not None)
    h.close()


def test_select_beyond_32_bits():
    """Rows that start beyond 2^31 elements."""
    V, ld = 20000, (1 << 30) + 1
    buf = torch.empty(3 * ld + V, device="cuda", dtype=bf16)
    logits = torch.as_strided(buf, (4, V), (ld, 1))
    g = gen_of(4)
    logits.copy_(normal(g, (4, V), 2.0, bf16))
    scores = torch.zeros((2, 2), device="cuda")
    h = hg.hg_beam_create(2, 2, V, 4)
    check_select(Call(h, logits, scores, exact_lse(logits).float()), exact=True)
    check_select(Call(h, logits, scores), exact=False)
    h.close()


def test_one_handle_for_every_number_of_items():
    g = gen_of(8)
    V, beams = 30000, 4
    logits, scores = inputs(g, 60, beams, V, bf16)
    lse = exact_lse(logits).float()
    h = hg.hg_beam_create(60, beams, V, 8)
    for items in (1, 60, 2, 37, 9, 38, 5, 60, 1):
        r = items * beams
        check_select(Call(h, logits[:r], scores[:items], lse[:r]), exact=True)
    none = scores[:0]
    hg.hg_beam_select(h, logits[:0], none, torch.empty((0, 8), device="cuda", dtype=torch.int64),
                      torch.empty((0, 8), device="cuda", dtype=torch.int64),
                      torch.empty((0, 8), device="cuda"))
    h.close()


# ---- reordering --------------------------------------------------------------------


def want_states(states, parents):
    items, beams = parents.shape
    row = torch.arange(items * beams, device="cuda").view(items, beams)
    ok = (parents >= 0) & (parents < beams)
    source = torch.where(ok, row[:, :1] + parents, row).view(-1).long()
    return [t.index_select(d, source) for t, d in states]


def some_parents(g, items, beams, dead=0.1, dtype=torch.int64):
    p = torch.randint(0, beams, (items, beams), generator=g, device="cuda")
    out = torch.rand((items, beams), generator=g, device="cuda") < dead
    odd = torch.tensor([-1, beams, 1000000, -7], device="cuda")
    return torch.where(out, odd[p % 4], p).to(dtype)


def bits(t):
    return t.contiguous().view(torch.uint8)


def check_reorder(h, parents, states):
    want = want_states(states, parents)
    hg.hg_beam_reorder(h, parents, states)
    for (t, _), w in zip(states, want):
        assert torch.equal(bits(t), bits(w))


def handle(items, beams):
    return hg.hg_beam_create(items, beams, 100, 1)


def random_of(g, shape, dtype):
    """Any bits: NaN and the like are moved as they are."""
    n = math.prod(shape) * dtype.itemsize
    b = torch.randint(0, 256, (max(n, 1),), generator=g, device="cuda", dtype=torch.uint8)
    if dtype == torch.bool:
        return b[:n].bool().view(shape)
    return b[:n].view(dtype).view(shape)


@pytest.mark.parametrize("items,beams", [(1, 1), (1, 2), (3, 4), (2, 7), (5, 8), (1, 33), (2, 64)])
def test_reorder_layouts(items, beams):
    g = gen_of(items * 10 + beams)
    rows = items * beams
    h = handle(items, beams)
    states = [
        (random_of(g, (rows,), torch.int32), 0),
        (random_of(g, (rows, 1), torch.uint8), 0),
        (random_of(g, (rows, 129), bf16), 0),
        (random_of(g, (3, rows, 5, 40, 64), bf16)[..., :17, :], 1),
        (random_of(g, (rows, 2, 3, 20, 33), fp16)[..., :7, :], 0),
        (random_of(g, (2, rows, 1000), torch.int64)[..., :999], 1),
        (random_of(g, (50, rows), torch.int64), 1),
        (random_of(g, (rows, 3, 4), torch.float64), 0),
        (random_of(g, (rows, 77), torch.bool), 0),
        (random_of(g, (rows, 70, 2), torch.int8)[..., 0], 0),
        (random_of(g, (rows, 4, 0), fp32), 0),
    ]
    for ids in (torch.int64, torch.int32):
        for dead in (0.0, 0.3):
            check_reorder(h, some_parents(g, items, beams, dead, ids), states)
    # Nobody moves; everybody takes one beam; a rotation; a swap of the ends.
    own = torch.arange(beams, device="cuda").expand(items, beams).contiguous()
    for p in (own, torch.zeros_like(own), torch.full_like(own, beams - 1), own.roll(1, 1),
              own.flip(1).contiguous()):
        check_reorder(h, p, states)
    h.close()


def test_reorder_leaves_the_rest():
    """What lies between, before and behind the filled part of a cache."""
    g = gen_of(3)
    h = handle(4, 3)
    whole = random_of(g, (2, 15, 6, 50, 24), bf16)
    before = whole.clone()
    part = whole[:, 2:14, 1:5, 10:31]
    parents = some_parents(g, 4, 3, 0.0)
    want = want_states([(part, 1)], parents)[0]
    hg.hg_beam_reorder(h, parents, [(part, 1)])
    assert torch.equal(bits(part), bits(want))
    part.copy_(before[:, 2:14, 1:5, 10:31])
    assert torch.equal(bits(whole), bits(before))
    h.close()


def test_reorder_interleaved_states():
    """Keys and values in one buffer, and more states than one launch takes."""
    g = gen_of(6)
    h = handle(3, 5)
    both = random_of(g, (4, 2, 15, 3, 16, 32), bf16)
    check_reorder(h, some_parents(g, 3, 5), [(both[:, 0], 1), (both[:, 1], 1)])
    many = [(random_of(g, (15, 1 + 7 * k), (bf16, torch.uint8, torch.int64)[k % 3]), 0)
            for k in range(hg.HG_MAX_STATES)]
    check_reorder(h, some_parents(g, 3, 5), many)
    hg.hg_beam_reorder(h, some_parents(g, 3, 5), [])
    hg.hg_beam_reorder(h, some_parents(g, 0, 5), [torch.empty((0, 4), device="cuda")])
    h.close()


@pytest.mark.parametrize("seed", range(30))
def test_reorder_random(seed):
    r = random.Random(seed)
    g = gen_of(seed)
    beams, items = r.choice([1, 2, 3, 4, 8, 13, 32, 64]), r.randint(1, 12)
    rows = items * beams
    states = []
    for _ in range(r.randint(1, 5)):
        dtype = r.choice([bf16, fp32, torch.int64, torch.uint8])
        front = [r.randint(1, 4) for _ in range(r.randint(0, 2))]
        shape = (*front, rows, r.randint(1, 5), r.randint(1, 60), r.randint(1, 140))
        off = r.choice([0, 0, 1, 8])
        flat = random_of(g, (math.prod(shape) + off,), dtype)
        t = flat[off:].view(shape)
        t = t[..., :r.randint(1, shape[-2]), :]
        if r.random() < 0.3:
            t = t[..., :r.randint(1, shape[-1])]
            t = t[..., 0, :] if r.random() < 0.5 else t[..., :1, :]
        states.append((t, len(front)))
    h = handle(items + 2, beams)
    check_reorder(h, some_parents(g, items, beams, 0.2), states)
    h.close()


def test_reorder_beyond_32_bits():
    """A state of 6 GB whose rows and runs pass 2^32 bytes."""
    g = gen_of(1)
    h = handle(1, 2)
    big = torch.zeros((2, 3 << 30), device="cuda", dtype=torch.uint8)
    big[1, ::4097] = 7
    big[1, -5:] = torch.tensor([1, 2, 3, 4, 5], device="cuda", dtype=torch.uint8)
    big[0, 11] = 9
    want = big.flip(0)
    hg.hg_beam_reorder(h, torch.tensor([[1, 0]], device="cuda"), [big])
    assert torch.equal(big, want)
    odd = big[:, 1:-2]  # no alignment
    want = odd.flip(0)
    hg.hg_beam_reorder(h, torch.tensor([[1, 0]], device="cuda"), [odd])
    assert torch.equal(odd, want)
    h.close()


def test_refusals_on_a_device():
    h = hg.hg_beam_create(1, 2, 50, 3)
    z = torch.zeros((4, 50), device="cuda", dtype=bf16)
    ids, f = torch.full((2, 3), 7, device="cuda"), torch.full((2, 3), 7.0, device="cuda")
    with pytest.raises(hg.HGError) as e:
        hg.hg_beam_select(h, z, torch.zeros((2, 2), device="cuda"), ids, ids.clone(), f)
    assert e.value.status == hg.HG_ERR_ROWS
    with pytest.raises(hg.HGError) as e:
        hg.hg_beam_reorder(h, torch.zeros((2, 2), device="cuda", dtype=torch.int64), [z])
    assert e.value.status == hg.HG_ERR_ROWS
    one = torch.zeros((1, 2), device="cuda")
    with pytest.raises(hg.HGError) as e:  # finished, but no token to go on with
        hg.hg_beam_select(h, z[:2], one, ids[:1], ids[:1].clone(), f[:1], finished=one.bool())
    assert e.value.status == hg.HG_ERR_ARG
    with pytest.raises(hg.HGError) as e:  # rows of one address
        hg.hg_beam_reorder(h, one.long(), [z[:1].expand(2, 50)])
    assert e.value.status == hg.HG_ERR_ARG
    assert bool((ids == 7).all()) and bool((f == 7).all())
    h.close()
