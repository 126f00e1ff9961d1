"""Up to 64 rows the loss's gradient keeps d as two rounded terms: beyond the rounding of
the results, only u^2 of each term is lost.

Inputs on which one rounding of d shows: logits that the tensor cores sum exactly
(x multiples of 1/4, w = 1 + multiples of 1/128), weights near 1 so that the sum over
the vocabulary, whose d add up to zero, cancels, and pairs of equal rows with nearly
opposite upstream gradients so that the sum over the rows does. Bound of an element:

  u |y| + (u^2 + 2^-21 + terms 2^-23) (|d| |M|) + e (p |M|) + floor + tiny

with the final rounding, d's two terms, the scalings' and the sum's roundings, the
exponential's error e = 2^-20 (1 + |lse|), and the floor of fp16's subnormals where
the largest factor is scaled to 2^14 (2^-25 / 2^13 of it at most)."""

import pytest
import torch

from tp_vocab_logits_gb300 import hg

from test_vocab_gpu import TINY, U, _built, bf16, fp16, gen_of, run_loss  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [bf16, fp16])
@pytest.mark.parametrize("N", [1, 2, 16, 33, 63, 64])
@pytest.mark.parametrize("tp,W,vocab", [(1, 24, 24), (3, 100, 291)])
def test_d_in_two_terms(tp, W, vocab, N, dtype):
    K = 32
    g = gen_of(N + W)

    def grid(shape, most, step):
        return torch.randint(-most, most + 1, shape, generator=g, device="cuda") * step

    whole = (1 + grid((tp * W, K), 16, 1 / 128)).to(dtype)
    hidden = grid((N, K), 8, 1 / 4).to(dtype)
    tgt = torch.randint(0, vocab, (N,), generator=g, device="cuda")
    up = 1 + torch.rand(N, generator=g, device="cuda") / 32
    hidden[1::2] = hidden[0:N - 1:2]
    tgt[1::2] = tgt[0:N - 1:2]
    up[1::2] *= -1
    h = hg.hg_vocab_create(tp, W, K, N, vocab=vocab, dtype=dtype, ops=("loss", "loss_grad"))
    _, lse = run_loss(h, hidden, list(whole.split(W)), tgt, 1.0)
    gh, gw = torch.empty_like(hidden), torch.empty_like(whole)
    hg.hg_vocab_loss_grad(h, hidden, list(whole.split(W)), tgt, lse, up, gh, list(gw.split(W)))
    hg.hg_vocab_sync(h)

    X, M = hidden.double(), whole[:vocab].double()
    z = X @ M.t()
    p = torch.exp(z - lse.double()[:, None]) * up.double().abs()[:, None]
    d = torch.exp(z - lse.double()[:, None])
    d[torch.arange(N, device="cuda"), tgt] -= 1
    d *= up.double()[:, None]
    most = up.abs().max().item()
    floor = 2.0 ** -25 / 2.0 ** 13 * most if dtype == fp16 else 0.0
    pe = p * (2.0 ** -20 * (1 + lse.double().abs()))[:, None] + floor
    u = U[dtype]
    # d rounded once, with the factor that the operator scales it by.
    factor = (2.0 ** 14 if dtype == fp16 else 1.0) / most
    once = (d * factor).to(dtype).double() / factor
    for got, a, e, a1, m, terms in ((gh, d, pe, once, M, vocab),
                                    (gw[:vocab], d.t(), pe.t(), once.t(), X, N)):
        y = a @ m
        bound = u * y.abs() + (u * u + 2.0 ** -21 + terms * 2.0 ** -23) * (a.abs() @ m.abs()) \
            + e @ m.abs() + TINY[dtype]
        err = (got.double() - y).abs()
        assert bool((err <= bound).all()), f"worst {(err / bound).max().item():.3g} of the bound"
        lost = ((a1 @ m).to(dtype).double() - y).abs()
        assert not bool((lost <= bound).all()), "the bound does not tell one term from two"
    h.close()
