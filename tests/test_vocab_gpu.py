"""The vocabulary operators against plain 64-bit forms.

Tolerances. u is the unit roundoff of the matrix's type (2^-8 bf16, 2^-11 fp16,
2^-24 fp32), tiny half its smallest subnormal.

- embed: the lookup rounds one fp32 product: equal to torch bit for bit.
- embed_grad: m terms summed in fp32 and rounded once:
  u |y| + m 2^-24 sum |terms| + tiny.
- loss: a logit's error dz is that of K fp32 additions, taken as a random walk
  of 2^-23 steps at eight deviations, 8 sqrt(K) 2^-23 max_v sum_k |x w|; loss
  and logsumexp are within 2 dz + 2^-20 (1 + |lse|) (exponentials to 2^-22, a
  sum of up to a few hundred partial sums).
- loss_grad: every term's d is off by its rounding, u |d|, and by the error of
  its exponential, e p with e = 2 dz + 2^-20 (1 + |lse|); the sum over it by
  a random walk as above; the result is rounded once:
  u |y| + (u + s) (|d| |M|) + e (p |M|) + tiny', s = 8 sqrt(terms) 2^-23.
  In fp16, d is scaled so that its largest factor is 2^14: the floor of its
  subnormals, 2^-25 / 2^13 of the largest factor at most, is tiny'.
"""

import math

import pytest
import torch

from tp_vocab_logits_gb300 import hg

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
bf16, fp16, fp32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tp_vocab_logits_gb300 import _build
    _build.build()


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def ids_of(g, n, vocab, masked=0.0, dtype=torch.int64):
    t = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    hide = torch.rand(n, generator=g, device="cuda") < masked
    return torch.where(hide, -100, t).to(dtype)


# ---- embedding -----------------------------------------------------------------

EMBED = [
    # tp, W, vocab, K, N, dtype, id type
    (1, 7, 7, 1, 1, bf16, torch.int64),
    (2, 50, 100, 64, 33, bf16, torch.int32),
    (3, 41, 120, 1001, 200, fp32, torch.int64),     # odd width: element accesses
    (3, 41, 120, 1001, 200, bf16, torch.int64),
    (4, 1000, 3999, 1032, 517, fp16, torch.int64),
    (8, 300, 2400, 7168, 129, bf16, torch.int32),
    (2, 600, 1200, 128, 70000, fp16, torch.int64),  # more rows than one pass of the grid
]


def table_of(g, tp, W, K, dtype):
    whole = normal(g, (tp * W, K), 1.0, dtype)
    return whole, list(whole.split(W))


@pytest.mark.parametrize("tp,W,vocab,K,N,dtype,idt", EMBED)
@pytest.mark.parametrize("scale", [1.0, 1.7])
def test_embed(tp, W, vocab, K, N, dtype, idt, scale):
    g = gen_of(N + K)
    whole, shards = table_of(g, tp, W, K, dtype)
    tok = ids_of(g, N, vocab, 0.2, idt)
    tok[0] = vocab - 1
    if N > 2:
        tok[1], tok[2] = vocab, 2 ** 31 - 1  # outside: zeros
    h = hg.hg_vocab_create(tp, W, K, N, vocab=vocab, dtype=dtype, ops=("embed",))
    out = torch.full((N, K), 3.0, device="cuda", dtype=dtype)
    hg.hg_vocab_embed(h, tok, shards, out, scale=scale)
    inside = ((tok >= 0) & (tok < vocab))[:, None]
    rows = whole[torch.where(inside[:, 0], tok, 0).long()]
    want = torch.where(inside, (rows.float() * scale).to(dtype), torch.zeros_like(rows))
    assert torch.equal(out, want)
    h.close()


def test_embed_strided_out_and_special_values():
    g = gen_of(1)
    whole, shards = table_of(g, 2, 16, 24, bf16)
    whole[3, :4] = torch.tensor([math.nan, math.inf, -math.inf, -0.0], device="cuda")
    tok = torch.tensor([3, -1, 31, 3], device="cuda")
    h = hg.hg_vocab_create(2, 16, 24, 4, dtype=bf16, ops=("embed",))
    for width, off in [(24, 0), (32, 8), (29, 3)]:  # the last: no 16-byte alignment
        big = torch.full((4, width + off), 5.0, device="cuda", dtype=bf16)
        out = big[:, off:off + 24]
        hg.hg_vocab_embed(h, tok, shards, out)
        want = whole[tok.clamp(min=0)].clone()
        want[1] = 0
        assert torch.equal(out.contiguous().view(torch.int16), want.view(torch.int16))
        assert bool((big[:, :off] == 5).all()) and bool((big[:, off + 24:] == 5).all())
    h.close()


def embed_grad_want(tok, grad, vocab, rows, scale, old=None):
    """(value, sum of |terms|, terms) of every table row in 64 bits."""
    inside = (tok >= 0) & (tok < vocab)
    ids, gr = tok[inside].long(), grad[inside].double() * scale
    val = torch.zeros((rows, grad.shape[1]), dtype=torch.float64, device="cuda")
    mag, cnt = torch.zeros_like(val), torch.zeros(rows, dtype=torch.float64, device="cuda")
    val.index_add_(0, ids, gr)
    mag.index_add_(0, ids, gr.abs())
    cnt.index_add_(0, ids, torch.ones_like(ids, dtype=torch.float64))
    if old is not None:
        val += old.double()
        mag += old.double().abs()
    return val, mag, cnt[:, None] + 2


def check_embed_grad(got, tok, grad, vocab, scale, old=None):
    dtype = got.dtype
    val, mag, terms = embed_grad_want(tok, grad, vocab, got.shape[0], scale, old)
    bound = U[dtype] * val.abs() + terms * 2.0 ** -24 * mag + TINY[dtype]
    err = (got.double() - val).abs()
    assert bool((err <= bound).all()), f"worst {(err / bound.clamp(min=1e-300)).max().item():.3g}"


@pytest.mark.parametrize("tp,W,vocab,K,N,dtype,idt", EMBED)
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad(tp, W, vocab, K, N, dtype, idt, accumulate):
    g = gen_of(N * 3 + K)
    whole, shards = table_of(g, tp, W, K, dtype)
    old = whole.clone()
    grad = normal(g, (N, K), 1.0, dtype)
    tok = ids_of(g, N, vocab, 0.2, idt)
    tok[N // 2] = vocab - 1
    h = hg.hg_vocab_create(tp, W, K, N, vocab=vocab, dtype=dtype, ops=("embed_grad",))
    hg.hg_vocab_embed_grad(h, tok, grad, shards, scale=1.3, accumulate=accumulate)
    check_embed_grad(whole, tok, grad, vocab, 1.3, old if accumulate else None)
    if accumulate:  # rows without tokens are not touched
        free = torch.ones(tp * W, dtype=torch.bool, device="cuda")
        free[tok[(tok >= 0) & (tok < vocab)].long()] = False
        assert torch.equal(whole[free].view(torch.uint8), old[free].view(torch.uint8))
    h.close()


@pytest.mark.parametrize("kind", ["one", "two", "zipf", "none", "ordered", "lengths"])
@pytest.mark.parametrize("N", [1, 31, 32, 33, 64, 5000])
def test_embed_grad_runs(kind, N):
    """Runs of equal tokens inside chunks, across their ends and over many."""
    g = gen_of(N)
    W, K, dtype = 4097, 40, bf16
    r = torch.arange(N, device="cuda")
    tok = {"one": torch.full((N,), 4096, device="cuda"),
           "two": r % 2 * 4000,
           "zipf": (torch.rand(N, generator=g, device="cuda") ** 8 * W).long(),
           "none": torch.full((N,), -1, device="cuda"),
           "ordered": r % W,
           "lengths": ((8 * r + 1).double().sqrt() - 1).div(2).floor().long() % W}[kind]
    tok = tok[torch.randperm(N, generator=g, device="cuda")]
    grad = normal(g, (N, K), 1.0, dtype)
    whole, shards = table_of(g, 1, W, K, dtype)
    h = hg.hg_vocab_create(1, W, K, N, dtype=dtype, ops=("embed_grad",))
    hg.hg_vocab_embed_grad(h, tok, grad, shards)
    check_embed_grad(whole, tok, grad, W, 1.0)
    again = torch.full_like(whole, math.nan)
    hg.hg_vocab_embed_grad(h, tok, grad, list(again.split(W)))
    assert torch.equal(whole, again)  # the same bits, whatever was there
    h.close()


@pytest.mark.parametrize("vocab_bits", [1, 9, 10, 11, 20, 21])
def test_embed_grad_digit_counts(vocab_bits):
    """One, two and three passes of the sort, at their edges."""
    g = gen_of(vocab_bits)
    W = (1 << vocab_bits) - 1
    tok = ids_of(g, 3000, W, 0.1)
    tok[:2] = torch.tensor([0, W - 1], device="cuda")
    grad = normal(g, (3000, 8), 1.0, fp32)
    out = torch.empty((W, 8), device="cuda")
    h = hg.hg_vocab_create(1, W, 8, 3000, dtype=fp32, ops=("embed_grad",))
    hg.hg_vocab_embed_grad(h, tok, grad, [out])
    check_embed_grad(out, tok, grad, W, 1.0)
    h.close()


def test_embed_grad_is_the_lookups_adjoint():
    """<grad_table, D> = <grad_out, lookup(D)> for any D: the derivative of a
    linear map, by differences of any size. Values on a grid that fp32 sums
    exactly, so both sides are equal."""
    g = gen_of(5)
    W, K, N = 37, 96, 700
    D = torch.randint(-8, 9, (2 * W, K), generator=g, device="cuda").float()
    grad = torch.randint(-8, 9, (N, K), generator=g, device="cuda").float()
    tok = ids_of(g, N, 2 * W, 0.3)
    h = hg.hg_vocab_create(2, W, K, N, dtype=fp32, ops=("embed", "embed_grad"))
    out, gt = torch.empty_like(grad), torch.empty_like(D)
    hg.hg_vocab_embed(h, tok, list(D.split(W)), out, scale=2.0)
    hg.hg_vocab_embed_grad(h, tok, grad, list(gt.split(W)), scale=2.0)
    assert (gt.double() * D.double()).sum().item() == (grad.double() * out.double()).sum().item()
    h.close()


def test_embed_empty_calls():
    h = hg.hg_vocab_create(2, 8, 16, 4, dtype=bf16, ops=("embed", "embed_grad"))
    whole = torch.ones((16, 16), device="cuda", dtype=bf16)
    tok = torch.empty(0, dtype=torch.int64, device="cuda")
    rows = torch.empty((0, 16), device="cuda", dtype=bf16)
    hg.hg_vocab_embed(h, tok, list(whole.split(8)), rows)
    hg.hg_vocab_embed_grad(h, tok, rows, list(whole.split(8)), accumulate=True)
    assert bool((whole == 1).all())
    hg.hg_vocab_embed_grad(h, tok, rows, list(whole.split(8)))
    assert bool((whole == 0).all())
    h.close()


def test_embed_offsets_beyond_32_bits():
    """A table and a token matrix of more than 2^31 elements each."""
    W, K, N = 300000, 8192, 280000
    table = torch.zeros((W, K), device="cuda", dtype=bf16)
    mark = torch.arange(8192, device="cuda").remainder(251).to(bf16)
    table[W - 1] = mark
    tok = torch.full((N,), -1, device="cuda")
    tok[N - 1] = W - 1
    h = hg.hg_vocab_create(1, W, K, N, dtype=bf16, ops=("embed", "embed_grad"))
    out = torch.ones((N, K), device="cuda", dtype=bf16)
    hg.hg_vocab_embed(h, tok, [table], out)
    assert torch.equal(out[N - 1], mark) and not bool(out[:N - 1].any())
    hg.hg_vocab_embed_grad(h, tok, out, [table], accumulate=True)
    assert torch.equal(table[W - 1], mark + mark) and not bool(table[:W - 1].any())
    h.close()


@pytest.mark.parametrize("dtype", [bf16, fp16, fp32])
@pytest.mark.parametrize("K,pad,off", [
    (706, 0, 0),    # rows aligned to 4 bytes
    (706, 2, 0), (705, 1, 0),  # odd width in an even row distance
    (704, 3, 0),    # whole vectors in rows that are not aligned
    (704, 8, 1),    # an unaligned start
    (2, 0, 0), (1, 0, 0),
])
def test_embed_widths_and_alignments(dtype, K, pad, off):
    g = gen_of(K + pad + off)
    N, W, vocab = 37, 20, 39
    tok = ids_of(g, N, vocab, 0.1)
    whole, shards = table_of(g, 2, W, K, dtype)
    big = torch.zeros((N, K + pad + off), device="cuda", dtype=dtype)
    rows = big[:, off:off + K]
    h = hg.hg_vocab_create(2, W, K, N, vocab=vocab, dtype=dtype, ops=("embed", "embed_grad"))
    hg.hg_vocab_embed(h, tok, shards, rows, scale=0.7)
    want = torch.where((tok >= 0)[:, None], (whole[tok.clamp(min=0)].float() * 0.7).to(dtype),
                       torch.zeros((), device="cuda", dtype=dtype))
    assert torch.equal(rows.contiguous(), want)
    rows.copy_(normal(g, (N, K), 1.0, dtype))
    for accumulate in (True, False):
        old = whole.clone()
        hg.hg_vocab_embed_grad(h, tok, rows, shards, scale=1.1, accumulate=accumulate)
        check_embed_grad(whole, tok, rows, vocab, 1.1, old if accumulate else None)
    h.close()


@pytest.mark.parametrize("vocab", [2 ** 21 - 1, 2 ** 21 - 2, 1000])
@pytest.mark.parametrize("N", [9, 16, 17, 2047, 2048, 2049])
def test_embed_grad_between_the_sorts(N, vocab):
    """Token counts at which the sort and the chunks change, with vocabularies
    on both sides of what one word holds."""
    g = gen_of(N)
    tok = ids_of(g, N, vocab, 0.1)
    tok[: N // 3] = vocab - 1
    tok = tok[torch.randperm(N, generator=g, device="cuda")]
    grad = normal(g, (N, 12), 1.0, fp32)
    out = torch.empty((vocab, 12), device="cuda")
    h = hg.hg_vocab_create(1, vocab, 12, N, dtype=fp32, ops=("embed_grad",))
    hg.hg_vocab_embed_grad(h, tok, grad, [out])
    check_embed_grad(out, tok, grad, vocab, 1.0)
    h.close()


# ---- loss ----------------------------------------------------------------------

LOSS = [
    # tp, W, vocab, K, N, dtype, masked, scale
    (1, 1, 1, 8, 1, bf16, 0.0, 1.0),           # one class: loss 0
    (1, 300, 300, 64, 1, bf16, 0.0, 1.0),
    (2, 64, 127, 72, 5, fp16, 0.0, 0.7),       # K short of a block, one pad column
    (3, 257, 700, 200, 128, bf16, 0.3, 1.0),   # pad of the last shard, tiles short
    (3, 257, 500, 200, 129, bf16, 0.3, -1.3),  # a shard without any real column
    (1, 5000, 5000, 1032, 300, fp16, 0.5, 1.0),
    (4, 2048, 8192, 512, 1000, bf16, 0.1, 1.0),
    (2, 20480, 40957, 1024, 16, bf16, 0.0, 2.0),
    (8, 640, 5120, 7168, 257, bf16, 0.9, 1.0),
    (1, 999, 999, 136, 64, bf16, 0.2, 1.0),    # the most rows with d in two terms
    (1, 999, 999, 136, 65, bf16, 0.2, 1.0),    # and one more
    (2, 700, 1390, 520, 256, fp16, 0.0, 1.0),  # hidden as it lies, one pair of tiles
    (16, 90, 1431, 264, 600, bf16, 0.4, 0.5),  # many narrow shards
]


def loss_inputs(tp, W, vocab, K, N, dtype, masked, seed):
    g = gen_of(seed)
    whole = normal(g, (tp * W, K), 0.05, dtype)
    whole[vocab:] = math.nan  # padding: whatever it holds takes no part
    hidden = normal(g, (N, K), 1.0, dtype)
    tgt = ids_of(g, N, vocab, masked)
    tgt[0] = vocab - 1 if masked < 0.5 else tgt[0]
    hidden[tgt < 0] = math.inf  # a masked row's hidden state has no effect
    if N > 1:
        hidden[tgt < 0, ::2] = math.nan
    return whole, list(whole.split(W)), hidden, tgt


def loss_want(whole, hidden, tgt, vocab, scale):
    """64-bit logits, logsumexp, loss and the bound of the module's docstring."""
    on = (tgt >= 0).nonzero()[:, 0]
    X, M = hidden[on].double(), whole[:vocab].double()
    z = X @ M.t() * scale
    lse = torch.logsumexp(z, 1)
    loss = lse - z.gather(1, tgt[on].long()[:, None])[:, 0]
    K = hidden.shape[1]
    dz = 8 * math.sqrt(K) * 2.0 ** -23 * abs(scale) * (X.abs() @ M.abs().t()).amax(1)
    return on, z, lse, loss, 2 * dz + 2.0 ** -20 * (1 + lse.abs())


def run_loss(h, hidden, shards, tgt, scale, stream=None):
    N = hidden.shape[0]
    loss = torch.full((N,), 77.0, device="cuda")
    lse = torch.full((N,), 77.0, device="cuda")
    hg.hg_vocab_loss(h, hidden, shards, tgt, loss, lse, logit_scale=scale, stream=stream)
    return loss, lse


def check_loss(loss, lse, whole, hidden, tgt, vocab, scale):
    on, _, want_lse, want_loss, bound = loss_want(whole, hidden, tgt, vocab, scale)
    off = tgt < 0
    assert not bool(loss[off].any()) and not bool(lse[off].any())
    for got, want in ((loss, want_loss), (lse, want_lse)):
        err = (got[on].double() - want).abs()
        assert bool((err <= bound).all()), f"worst {(err / bound).max().item():.3g} of the bound"


@pytest.mark.parametrize("tp,W,vocab,K,N,dtype,masked,scale", LOSS)
def test_loss(tp, W, vocab, K, N, dtype, masked, scale):
    whole, shards, hidden, tgt = loss_inputs(tp, W, vocab, K, N, dtype, masked, N + K)
    h = hg.hg_vocab_create(tp, W, K, N, vocab=vocab, dtype=dtype, ops=("loss",))
    loss, lse = run_loss(h, hidden, shards, tgt, scale)
    hg.hg_vocab_sync(h)
    check_loss(loss, lse, whole, hidden, tgt, vocab, scale)
    h.close()


def grad_want(whole, hidden, tgt, vocab, scale, lse, grad_loss):
    """64-bit gradients and their bounds."""
    dtype = whole.dtype
    on, z, _, _, e = loss_want(whole, hidden, tgt, vocab, scale)
    X, M = hidden[on].double(), whole[:vocab].double()
    gs = grad_loss[on].double() * scale
    p = torch.exp(z - lse[on].double()[:, None]) * gs.abs()[:, None]
    d = torch.exp(z - lse[on].double()[:, None])
    d[torch.arange(len(on), device="cuda"), tgt[on].long()] -= 1
    d *= gs[:, None]
    u = U[dtype]
    floor = 2.0 ** -25 / 2.0 ** 13 * gs.abs().max().item() if dtype == fp16 and len(on) else 0.0
    pe = p * e[:, None] + floor

    def both(a, b, m, terms):
        s = 8 * math.sqrt(max(1, terms)) * 2.0 ** -23
        y = a @ m
        return y, u * y.abs() + (u + s) * (a.abs() @ m.abs()) + b @ m.abs() + TINY[dtype]

    gh = torch.zeros(hidden.shape, dtype=torch.float64, device="cuda")
    gh_bound = torch.zeros_like(gh)
    gh[on], gh_bound[on] = both(d, pe, M, vocab)
    gw = torch.zeros(whole.shape, dtype=torch.float64, device="cuda")
    gw_bound = torch.zeros_like(gw)
    gw[:vocab], gw_bound[:vocab] = both(d.t(), pe.t(), X, len(on))
    return gh, gh_bound, gw, gw_bound


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    ok = err <= bound
    assert bool(ok.all()), (f"{what}: {int((~ok).sum())} outside, worst "
                            f"{(err / bound.clamp(min=1e-300)).max().item():.3g} of the bound")


def grad_inputs(tgt, seed):
    g = gen_of(seed)
    return (torch.rand(tgt.shape[0], generator=g, device="cuda") - 0.2) / tgt.shape[0]


@pytest.mark.parametrize("tp,W,vocab,K,N,dtype,masked,scale", LOSS)
@pytest.mark.parametrize("piece", [0, 1])  # 1: pieces of 256 columns per shard
def test_loss_grad(tp, W, vocab, K, N, dtype, masked, scale, piece):
    whole, shards, hidden, tgt = loss_inputs(tp, W, vocab, K, N, dtype, masked, N + K)
    h = hg.hg_vocab_create(tp, W, K, N, vocab=vocab, dtype=dtype, ops=("loss", "loss_grad"),
                           piece_bytes=piece)
    _, lse = run_loss(h, hidden, shards, tgt, scale)
    g = grad_inputs(tgt, N)
    gh = torch.full_like(hidden, 9.0)
    gw = torch.full_like(whole, 9.0)
    hg.hg_vocab_loss_grad(h, hidden, shards, tgt, lse, g, gh, list(gw.split(W)),
                          logit_scale=scale)
    hg.hg_vocab_sync(h)
    want = grad_want(whole, hidden, tgt, vocab, scale, lse, g)
    within(gh, want[0], want[1], "grad_hidden")
    within(gw, want[2], want[3], "grad_weight")
    # The same bits again; each gradient alone is the same.
    gh2, gw2 = torch.full_like(gh, math.nan), torch.full_like(gw, math.nan)
    hg.hg_vocab_loss_grad(h, hidden, shards, tgt, lse, g, gh2, None, logit_scale=scale)
    hg.hg_vocab_loss_grad(h, hidden, shards, tgt, lse, g, None, list(gw2.split(W)),
                          logit_scale=scale)
    assert torch.equal(gh, gh2) and torch.equal(gw, gw2)
    # Added to what is there: one rounding of the gradient, one of the sum.
    acc = torch.full_like(gw, 0.5)
    hg.hg_vocab_loss_grad(h, hidden, shards, tgt, lse, g, None, list(acc.split(W)),
                          logit_scale=scale, accumulate=True)
    assert torch.equal(acc, (gw.float() + 0.5).to(dtype))
    h.close()


def test_loss_grad_by_differences():
    """Directional differences of the loss itself along signs in hidden and in
    the weights. Inputs lie on a grid on which x +- h is exact in bf16. h = 1/16:
    the difference's truncation is h^2 / 6 of a third cumulant of the logits'
    change along the direction (at most (sum |w|)^3 / 8, in fact far below),
    the gradients' roundings 2^-8 of sum |terms|; a 2 % bound holds both."""
    g = gen_of(11)
    W, K, N, hstep = 700, 64, 40, 1.0 / 16
    hidden = (torch.randint(-8, 9, (N, K), generator=g, device="cuda") / 8).to(bf16)
    whole = (torch.randint(-8, 9, (2 * W, K), generator=g, device="cuda") / 16).to(bf16)
    tgt = ids_of(g, N, 2 * W)
    up = torch.rand(N, generator=g, device="cuda") + 0.5
    h = hg.hg_vocab_create(2, W, K, N, dtype=bf16, ops=("loss", "loss_grad"))

    def total(x, w):
        return (run_loss(h, x, list(w.split(W)), tgt, 1.0)[0].double() * up.double()).sum().item()

    _, lse = run_loss(h, hidden, list(whole.split(W)), tgt, 1.0)
    gh, gw = torch.empty_like(hidden), torch.empty_like(whole)
    hg.hg_vocab_loss_grad(h, hidden, list(whole.split(W)), tgt, lse, up, gh, list(gw.split(W)))
    for grad, which in ((gh, 0), (gw, 1)):
        step = grad.float().sign() * hstep  # along the gradient's own signs: no cancellation
        plus = [hidden, whole]
        minus = [hidden, whole]
        at = plus[which]
        plus[which] = (at.float() + step).to(bf16)
        minus[which] = (at.float() - step).to(bf16)
        assert torch.equal(plus[which].float() - at.float(), step)
        if which == 1:  # every weight at once moves the logits far: a smaller part of them
            keep = torch.zeros_like(step)
            keep[tgt[0]] = step[tgt[0]]
            step = keep
            plus[1] = (at.float() + step).to(bf16)
            minus[1] = (at.float() - step).to(bf16)
        else:  # one row's few elements
            keep = torch.zeros_like(step)
            keep[:, :4] = step[:, :4]
            step = keep
            plus[0] = (at.float() + step).to(bf16)
            minus[0] = (at.float() - step).to(bf16)
        diff = (total(*plus) - total(*minus)) / 2
        want = (grad.double() * step.double()).sum().item()
        assert abs(diff - want) <= 0.02 * abs(want), (which, diff, want)
    h.close()


def test_loss_all_masked_and_empty():
    W, K = 300, 64
    for N in (3, 200):
        whole, shards, hidden, _ = loss_inputs(2, W, 2 * W, K, N, bf16, 0.0, N)
        hidden[:] = math.nan
        tgt = torch.full((N,), -1, device="cuda")
        h = hg.hg_vocab_create(2, W, K, N, dtype=bf16, ops=("loss", "loss_grad"))
        loss, lse = run_loss(h, hidden, shards, tgt, 1.0)
        assert not bool(loss.any()) and not bool(lse.any())
        gh, gw = torch.ones_like(hidden), torch.ones_like(whole)
        up = torch.ones(N, device="cuda")
        hg.hg_vocab_loss_grad(h, hidden, shards, tgt, lse, up, gh, list(gw.split(W)))
        assert not bool(gh.any()) and not bool(gw.any())
        none = torch.empty((0, K), device="cuda", dtype=bf16)
        gw.fill_(1)
        hg.hg_vocab_loss(h, none, shards, tgt[:0], loss[:0], lse[:0])
        hg.hg_vocab_loss_grad(h, none, shards, tgt[:0], lse[:0], up[:0], none, list(gw.split(W)),
                              accumulate=True)
        assert bool((gw == 1).all())
        hg.hg_vocab_loss_grad(h, none, shards, tgt[:0], lse[:0], up[:0], none, list(gw.split(W)))
        assert not bool(gw.any())
        hg.hg_vocab_sync(h)
        h.close()


@pytest.mark.parametrize("N", [4, 200])
def test_loss_target_outside_the_vocabulary(N):
    """A target >= vocab: a NaN loss beside the others' own, and no gradient."""
    W, K = 300, 64
    whole, shards, hidden, tgt = loss_inputs(2, W, 599, K, N, bf16, 0.0, N)
    tgt[1], tgt[3] = 599, 2 ** 40
    h = hg.hg_vocab_create(2, W, K, N, vocab=599, dtype=bf16, ops=("loss", "loss_grad"))
    loss, lse = run_loss(h, hidden, shards, tgt, 1.0)
    assert torch.isnan(loss).nonzero()[:, 0].tolist() == [1, 3]
    masked = torch.where(tgt >= 599, -1, tgt)
    clean = hidden.clone()
    clean[[1, 3]] = 0
    check_loss(torch.nan_to_num(loss), torch.where(masked < 0, 0.0, lse), whole, clean, masked,
               599, 1.0)
    gh, gw = torch.ones_like(hidden), torch.ones_like(whole)
    gh2, gw2 = torch.ones_like(hidden), torch.ones_like(whole)
    up = torch.ones(N, device="cuda")
    hg.hg_vocab_loss_grad(h, hidden, shards, tgt, lse, up, gh, list(gw.split(W)))
    hg.hg_vocab_loss_grad(h, hidden, shards, masked, lse, up, gh2, list(gw2.split(W)))
    assert torch.equal(gh, gh2) and torch.equal(gw, gw2) and not bool(gh[[1, 3]].any())
    h.close()


@pytest.mark.parametrize("N", [3, 150])
def test_loss_extreme_logits(N):
    """Logits in the thousands, a certain target (loss near 0), a NaN and an
    infinite row that stay in their rows."""
    W, K = 300, 64
    g = gen_of(N)
    whole = normal(g, (W, K), 1.0, bf16)
    hidden = normal(g, (N, K), 1.0, bf16)
    hidden[0] = (whole[7].float() * 64).to(bf16)  # z[7] is thousands above the rest
    tgt = torch.full((N,), 7, device="cuda")
    h = hg.hg_vocab_create(1, W, K, N, dtype=bf16, ops=("loss",))
    loss, lse = run_loss(h, hidden, [whole], tgt, 1.0)
    assert loss[0].item() == 0.0 and bool(torch.isfinite(loss).all())
    check_loss(loss, lse, whole, hidden, tgt, W, 1.0)
    bad = hidden.clone()
    bad[1, 5] = math.nan
    bad[2, 6] = math.inf
    got, _ = run_loss(h, bad, [whole], tgt, 1.0)
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[1:3] = False
    assert bool(torch.isnan(got[1])) and not bool(torch.isfinite(got[2]))
    assert torch.equal(got[rest], loss[rest])
    h.close()


@pytest.mark.parametrize("N", [24, 300])
def test_loss_strided_rows_int32_and_streams(N):
    """Hidden states and gradients as columns of wider matrices, int32 targets,
    a stream of the caller's, and a captured graph: the same bits."""
    W, K, dtype = 500, 72, fp16
    whole, shards, hidden, tgt = loss_inputs(2, W, 999, K, N, dtype, 0.2, N)
    h = hg.hg_vocab_create(2, W, K, N, vocab=999, dtype=dtype, ops=("loss", "loss_grad"))
    loss, lse = run_loss(h, hidden, shards, tgt, 0.5)
    up = grad_inputs(tgt, 3)
    gh, gw = torch.empty_like(hidden), torch.empty_like(whole)
    hg.hg_vocab_loss_grad(h, hidden, shards, tgt, lse, up, gh, list(gw.split(W)), logit_scale=0.5)
    wide = torch.full((N, K + 24), math.nan, device="cuda", dtype=dtype)
    wide[:, 16:16 + K] = hidden
    gwide = torch.full((N, K + 40), 4.0, device="cuda", dtype=dtype)
    gw2, tgt32 = torch.empty_like(whole), tgt.int()
    loss2, lse2 = torch.empty_like(loss), torch.empty_like(lse)
    torch.cuda.synchronize()

    def calls(s):
        hg.hg_vocab_loss(h, wide[:, 16:16 + K], shards, tgt32, loss2, lse2, logit_scale=0.5,
                         stream=s)
        hg.hg_vocab_loss_grad(h, wide[:, 16:16 + K], shards, tgt32, lse2, up, gwide[:, 8:8 + K],
                              list(gw2.split(W)), logit_scale=0.5, stream=s)

    def same():
        torch.cuda.synchronize()
        assert torch.equal(loss, loss2) and torch.equal(lse, lse2) and torch.equal(gw, gw2)
        assert torch.equal(gwide[:, 8:8 + K], gh)
        assert bool((gwide[:, :8] == 4).all()) and bool((gwide[:, 8 + K:] == 4).all())

    s = torch.cuda.Stream()
    calls(s)
    same()
    loss2.zero_(), lse2.zero_(), gw2.zero_(), gwide[:, 8:8 + K].zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        calls(s)
    graph.replay()
    same()
    h.close()


def test_loss_weights_beyond_32_bits():
    """More than 2^31 weight elements in one shard; the last columns matter."""
    W, K, N = 270000, 8192, 4
    whole = torch.zeros((W, K), device="cuda", dtype=bf16)
    hidden = torch.ones((N, K), device="cuda", dtype=bf16)
    whole[W - 1] = 2.0 ** -10  # z = 8 in the last column, 0 elsewhere
    tgt = torch.tensor([W - 1, 0, W - 1, -1], device="cuda")
    h = hg.hg_vocab_create(1, W, K, N, dtype=bf16, ops=("loss", "loss_grad"))
    loss, lse = run_loss(h, hidden, [whole], tgt, 1.0)
    want = math.log(W - 1 + math.exp(8.0))
    for i, z in enumerate([8.0, 0.0, 8.0]):
        assert abs(loss[i].item() - (want - z)) <= 2.0 ** -20 * (1 + want)
    gw = torch.empty_like(whole)
    hg.hg_vocab_loss_grad(h, hidden, [whole], tgt, lse, torch.ones(N, device="cuda"), None, [gw])
    p = math.exp(8.0 - want)
    assert abs(gw[W - 1, K - 1].item() - (3 * p - 2)) <= 2 * 2.0 ** -8 * 2
    q = 3 * math.exp(-want)
    assert abs(gw[W - 2, 5].item() - q) <= 2 * 2.0 ** -8 * q
    h.close()


def test_refusals():
    K, W, N = 64, 32, 8
    h = hg.hg_vocab_create(2, W, K, N, dtype=bf16, ops=("embed", "loss", "loss_grad"))
    whole = torch.zeros((2 * W, K), device="cuda", dtype=bf16)
    shards = list(whole.split(W))
    x = torch.zeros((N, K), device="cuda", dtype=bf16)
    t = torch.zeros(N, dtype=torch.int64, device="cuda")
    f = torch.zeros(N, device="cuda")
    with pytest.raises(hg.HGError, match="hg_vocab_embed_grad"):  # not created for it
        hg.hg_vocab_embed_grad(h, t, x, shards)
    big = torch.zeros((N + 1, K), device="cuda", dtype=bf16)
    with pytest.raises(hg.HGError) as e:  # more rows than the handle's
        hg.hg_vocab_loss(h, big, shards, torch.zeros(N + 1, dtype=torch.int64, device="cuda"),
                         torch.zeros(N + 1, device="cuda"), torch.zeros(N + 1, device="cuda"))
    assert e.value.status == hg.HG_ERR_ROWS
    with pytest.raises(hg.HGError) as e:  # neither gradient wanted
        hg.hg_vocab_loss_grad(h, x, shards, t, f, f, None, None)
    assert e.value.status == hg.HG_ERR_ARG
    wide = torch.zeros((N, K + 8), device="cuda", dtype=bf16)
    with pytest.raises(hg.HGError):  # 16-byte alignment of hidden
        hg.hg_vocab_loss(h, wide[:, 1:1 + K], shards, t, f, f.clone())
    odd = torch.zeros((N, K + 4), device="cuda", dtype=bf16)
    with pytest.raises(hg.HGError):  # row distance a multiple of 8
        hg.hg_vocab_loss(h, odd[:, :K], shards, t, f, f.clone())
    with pytest.raises(ValueError, match="shards"):
        hg.hg_vocab_loss(h, x, shards[:1], t, f, f.clone())
    with pytest.raises(ValueError, match="need CUDA tensors"):
        hg.hg_vocab_loss(h, x, [s.half() for s in shards], t, f, f.clone())
    with pytest.raises(ValueError, match="contiguous rows"):
        hg.hg_vocab_embed(h, t, shards, torch.zeros((K, N), device="cuda", dtype=bf16).t())
    with pytest.raises(ValueError, match="loss"):
        hg.hg_vocab_loss(h, x, shards, t, f.double(), f)
    hg.hg_vocab_sync(h)
    h.close()
