"""The norm's gradient of rows whose scale is far from one.

Errors as in tests/test_norm_gpu.py: with w = s * rstd, whose squares have a mean of one, and
d = grad_out * gain, grad_x = rstd * d - w * (rstd * mean(d * w)) + grad_sum takes at most four
roundings of each term, and nothing between leaves the range of d, w and the result. Where the
result is below 2^-126, fp32 rounds to multiples of 2^-149: the factor rstd * mean(d * w) is off
by up to 2^-150, which w multiplies, and each of the two sums by as much, which TINY holds.
"""

import pytest
import torch

from test_norm_gpu import (TINY, U, _built, check, check_grad, gen_of, grad_want,  # noqa: F401
                           normal)
from tp_vocab_logits_gb300 import hg

pytestmark = pytest.mark.gpu

bf16, fp16, fp32 = torch.bfloat16, torch.float16, torch.float32


# Few rows, a row a group, streamed, 4- and 2-byte accesses, rows that are read again.
@pytest.mark.parametrize("N,K", [(1, 64), (5, 1000), (64, 1001), (100, 1000), (100, 333),
                                 (400, 1000), (400, 1002), (400, 1001), (3, 20001), (70, 20001)])
@pytest.mark.parametrize("dtype", [bf16, fp32])
@pytest.mark.parametrize("scale", [1e-17, 1e-14, 1e15])
def test_gradient_of_far_scales(N, K, dtype, scale):
    """Squares and sums are far from the ends of fp32; rstd^3, or grad_out * s, is not."""
    g = gen_of(N + K)
    s, gain = normal(g, (N, K), 2 * scale, dtype), normal(g, (K,), 0.2, dtype) + 1
    rstd = (1 / s.double().square().mean(1).sqrt()).float()
    h = hg.hg_norm_create(K, N, dtype=dtype)
    gx, gg = torch.empty_like(s), torch.empty_like(gain)
    for up_scale in (1.0, 1e-25):
        up = normal(g, (N, K), 0.5 * up_scale, dtype)
        more = normal(g, (N, K), 0.5 * up_scale / scale, dtype)
        for grad_sum in (None, more):
            hg.hg_norm_rows_grad(h, s, gain, rstd, up, gx, gg, grad_sum=grad_sum)
            want, err, _, _ = grad_want(s, gain, rstd, up, grad_sum)
            err = err * 1.01 + (s.double() * rstd.double()[:, None]).abs() * 2.0 ** -150
            check(gx, want, U[dtype] * want.abs() + err + TINY[dtype], "grad_x")
            check_grad(s, gain, rstd, up, None, None, gg)
        hg.hg_norm_rows_grad(h, s, gain, rstd, up, None, gg)
        check_grad(s, gain, rstd, up, None, None, gg)
    h.close()
