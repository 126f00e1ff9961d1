"""grad_gain is the same sum, bit by bit, whether grad_x is wanted, and over grad_out or grad_sum."""

import pytest
import torch

from test_norm_gpu import _built, check_grad, gen_of, grad_inputs, normal  # noqa: F401
from tp_vocab_logits_gb300 import hg

pytestmark = pytest.mark.gpu

bf16, fp16, fp32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("N", [1, 5, 16, 64, 65, 400])
@pytest.mark.parametrize("K,dtype", [(8, bf16), (130, fp16), (1000, bf16), (1001, fp32),
                                     (7168, bf16), (16384, fp16), (20001, bf16)])
def test_order_of_grad_gain(N, K, dtype):
    g = gen_of(N + K)
    s, gain, rstd, up, more = grad_inputs(g, N, K, dtype)
    h = hg.hg_norm_create(K, N, dtype=dtype)
    old = normal(g, (K,), 1.0, dtype)
    for accumulate in (False, True):
        made = []
        for over in ("apart", "none", "grad_out", "grad_sum"):
            a, b, gg = up.clone(), more.clone(), old.clone()
            gx = {"apart": torch.empty_like(s), "none": None, "grad_out": a, "grad_sum": b}[over]
            hg.hg_norm_rows_grad(h, s, gain, rstd, a, gx, gg, grad_sum=b, accumulate=accumulate)
            check_grad(s, gain, rstd, up, more, gx, gg, old if accumulate else None)
            made.append((gg, gx))
        for gg, gx in made[1:]:
            assert torch.equal(gg, made[0][0])
            assert gx is None or torch.equal(gx, made[0][1])
    h.close()
