"""The sums of the loss's gradient where the tensor core's own accumulation would
show: it drops the low bits of every step's sum, always downwards, so that long
sums of one sign end up too small. Random signs hide that."""

import pytest
import torch

from tp_vocab_logits_gb300 import hg

from test_vocab_gpu import U, _built, bf16, fp16, gen_of, run_loss  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,dtype", [
    (16, 7168, bf16), (16, 7168, fp16), (64, 1032, fp16), (1, 7168, fp16),
    (80, 7168, fp16),   # one CTA, d in one term
    (200, 7168, fp16),  # pairs
    (200, 1032, fp16),
])
def test_gradient_has_the_losss_own_logits(N, K, dtype):
    """Logits of about 0.005 K, all products positive. Over a row, d sums to
    g (sum of p - 1), and p to 1 if the gradient's logits are those whose
    logsumexp the loss returned: a column of ones in the weights shows the sum in
    grad_hidden. Bound, for g = 1: the logsumexp's and the exponentials' roundings,
    2^-20 (1 + lse), as the loss's own tests have it; 16 addends of each of the
    V / 16 steps cut at 2^-24 of the running sum on average, half of the final one;
    above 64 rows, where d is rounded once, u of the target's term and 8 standard
    deviations of V terms of 1 / V."""
    V = 512
    g = gen_of(N + K)
    weight = (0.005 + 0.01 * torch.rand(V, K, generator=g, device="cuda")).to(dtype)
    weight[:, 0] = 1
    hidden = torch.rand(N, K, generator=g, device="cuda").to(dtype)
    hidden[:, 0] = 0
    tgt = torch.randint(0, V, (N,), generator=g, device="cuda")
    h = hg.hg_vocab_create(1, V, K, N, dtype=dtype, ops=("loss", "loss_grad"))
    _, lse = run_loss(h, hidden, [weight], tgt, 1.0)
    gh = torch.empty_like(hidden)
    hg.hg_vocab_loss_grad(h, hidden, [weight], tgt, lse, torch.ones(N, device="cuda"), gh, None)
    hg.hg_vocab_sync(h)
    bound = 2.0 ** -20 * (1 + lse.double()) + V / 16 * 16 * 2.0 ** -24 / 2
    if N > 64:
        bound += U[dtype] * (1 + 8 / V ** 0.5)
    worst = (gh[:, 0].double().abs() / bound).max().item()
    assert worst <= 1, f"{worst:.3g} of the bound"
    h.close()


def spread_inputs(g, N, V, K):
    """Positive weights and hidden states whose softmaxes spread over a factor of
    several; column 0, every row's target, has no weights, so that the gradients are
    sums of positive terms."""
    weight = (0.1 * torch.rand(V, K, generator=g, device="cuda")).to(fp16)
    weight[0] = 0
    hidden = torch.rand(N, K, generator=g, device="cuda").to(fp16)
    return weight, hidden, torch.zeros(N, dtype=torch.int64, device="cuda")


# What a mean error over many sums may be: a segment of 64 steps loses 16 addends'
# 2^-24 of the running sum at each, half of the final one on average; the segments
# are joined by rounding additions. The logits (4 steps, up to 6.4) the same way, in
# the exponent. The results' own roundings, u each in [-1, 1], to six deviations.
def mean_bound(count):
    steps = 64 * 16 * 2.0 ** -24 / 2
    return steps + 6.4 * 4 * 16 * 2.0 ** -24 / 2 + 6 * U[fp16] / count ** 0.5


def mean_error(got, want):
    return ((got.double() - want) / want).mean().abs().item()


def test_hidden_gradient_does_not_drift():
    """A sum over 65536 columns of one piece, which rows that fill one round of
    tiles leave in one part."""
    N, V, K = 256 * 76, 65536, 64
    weight, hidden, tgt = spread_inputs(gen_of(1), N, V, K)
    h = hg.hg_vocab_create(1, V, K, N, dtype=fp16, ops=("loss", "loss_grad"), piece_bytes=4 << 30)
    _, lse = run_loss(h, hidden, [weight], tgt, 1.0)
    gh = torch.empty_like(hidden)
    hg.hg_vocab_loss_grad(h, hidden, [weight], tgt, lse, torch.ones(N, device="cuda"), gh, None)
    hg.hg_vocab_sync(h)
    rows = torch.arange(0, N, 101, device="cuda")
    p = torch.exp(hidden[rows].double() @ weight.double().t() - lse[rows].double()[:, None])
    want = p @ weight.double()
    assert mean_error(gh[rows], want) <= mean_bound(want.numel())
    h.close()


@pytest.mark.parametrize("N", [65536, 5000])
def test_weight_gradient_does_not_drift(N):
    """A sum over many rows."""
    V, K = 512, 64
    weight, hidden, tgt = spread_inputs(gen_of(N), N, V, K)
    h = hg.hg_vocab_create(1, V, K, N, dtype=fp16, ops=("loss", "loss_grad"))
    _, lse = run_loss(h, hidden, [weight], tgt, 1.0)
    gw = torch.empty_like(weight)
    hg.hg_vocab_loss_grad(h, hidden, [weight], tgt, lse, torch.full((N,), 1 / N, device="cuda"),
                          None, [gw])
    hg.hg_vocab_sync(h)
    X = hidden.double()
    p = torch.exp(X @ weight.double().t() - lse.double()[:, None])
    want = (p.t() @ X / N)[1:]
    assert mean_error(gw[1:], want) <= mean_bound(want.numel())
    h.close()
