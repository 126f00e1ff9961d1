"""The norm of rows and its gradient against plain 64-bit forms.

Tolerances. u is the unit roundoff of the type (2^-8 bf16, 2^-11 fp16, 2^-24 fp32),
tiny half its smallest subnormal, t = 2^-24. A sum of n fp32 terms in any order whose
chains are at most c additions long is off by c t of the sum of its magnitudes; over a
row the chains are at most c = K / 256 + 96 long (a thread's own terms, at most
64 where it holds them in registers, then trees).

- sum_out: one fp32 addition, rounded: equal to torch bit for bit.
- rstd: half the relative error of the mean of squares, (c + 2) t / 2, and 2^-22 of
  the reciprocal root.
- out: |y| times (u + the error of rstd + 2 t), and tiny.
- scales: the same without u, and 2 t for the division.
- 8 bits: out * scale is off by half a step of e4m3, 2^-4 of the value or 2^-10 of the
  scale, and by the errors of y and the scale.
- grad_x: |terms| times 4 t + the inner sum's (c + 6) t, and u of the result.
- grad_gain: (n + 4) t of the terms' magnitudes, n = min(N, N / 152 + 320) additions,
  and u of the result.
"""

import math

import pytest
import torch

from tp_vocab_logits_gb300 import hg

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
T = 2.0 ** -24
bf16, fp16, fp32 = torch.bfloat16, torch.float16, torch.float32
e4m3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tp_vocab_logits_gb300 import _build
    _build.build()


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def padded(g, n, K, dtype, pad=0, off=0, std=1.0):
    """[n, K] of normal values, K + pad apart, off elements into their buffer."""
    buf = torch.full((n * (K + pad) + off,), 3.0, device="cuda").to(dtype)
    view = buf[off:].view(n, K + pad)[:, :K]
    view.copy_(normal(g, (n, K), std, dtype))
    return view


def chains(K):
    return K / 256 + 96


def check(got, want, bound, what):
    err = (got.double() - want).abs()
    worst = (err / bound.clamp(min=1e-300)).max().item() if err.numel() else 0.0
    assert bool((err <= bound).all()), f"{what}: {worst:.3g} of the bound"


def check_norm(s, gain, eps, rstd, out, scales=None):
    """rstd, out (and scales) of the norm of the rows s."""
    dtype, K = s.dtype, s.shape[1]
    v = s.double()
    want_r = 1.0 / ((v * v).sum(1) / K + eps).sqrt()
    e = (chains(K) + 2) * T / 2 + 2.0 ** -22
    if rstd is not None:
        check(rstd, want_r, e * want_r, "rstd")
    y = v * want_r[:, None] * gain.double()
    e += 2 * T
    if scales is None:
        check(out, y, (U[dtype] + e) * y.abs() * (1 + 2.0 ** -7) + TINY[dtype], "out")
        return
    blocks = scales.shape[1]
    width = 128 if blocks > 1 else K
    most = torch.stack([p.abs().amax(1) for p in y.split(width, 1)], 1)
    want = (most / 448).clamp(min=2.0 ** -126)
    want = torch.where(most == 0, 1.0, want)
    check(scales, want, (e + 2 * T) * want, "scales")
    per = scales.double().repeat_interleave(width, 1)[:, :K]
    q = out.double()
    assert q.abs().max().item() <= 448.0
    check(q * per, y, torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * per) + 4 * e * y.abs(),
          "out in 8 bits")


# Widths around what a warp, a CTA and an access hold; strides and offsets that leave 16, 4
# or an element's bytes of alignment; rows from one on.
SHAPES = [
    # N, K, dtype, pad, offset
    (1, 1, bf16, 0, 0), (3, 2, fp32, 1, 0), (5, 7, fp16, 0, 1), (2, 8, bf16, 0, 0),
    (7, 31, bf16, 1, 0), (9, 64, bf16, 0, 0), (4, 128, fp16, 0, 0), (33, 129, fp32, 3, 1),
    (6, 250, bf16, 6, 2), (17, 256, fp32, 0, 0), (5, 1001, fp16, 0, 0), (300, 1001, fp32, 0, 0),
    (11, 1024, bf16, 8, 0), (2, 1032, bf16, 0, 0), (3, 2050, fp16, 0, 0), (40, 2056, fp32, 4, 4),
    (1, 7168, bf16, 0, 0), (200, 7168, bf16, 0, 0), (3, 7168, fp16, 2, 0), (3, 7167, bf16, 0, 0),
    (1, 7168, fp32, 0, 0), (2, 9001, bf16, 0, 0), (3, 16384, fp16, 0, 0), (2, 20000, bf16, 2, 1),
    (1, 40000, fp32, 0, 0), (2, 70001, bf16, 0, 0), (1, 140000, bf16, 0, 0),
    # more rows than SMs, where they are streamed or share a CTA
    (400, 64, bf16, 0, 0), (1000, 256, fp16, 8, 0), (600, 512, fp32, 0, 0), (330, 4096, bf16, 0, 0),
    (700, 3000, fp16, 0, 0), (160, 16384, bf16, 0, 0), (200, 2050, bf16, 0, 0),
    (500, 101, bf16, 0, 0), (3000, 40, bf16, 0, 0), (170, 8192, fp32, 0, 0),
]


@pytest.mark.parametrize("N,K,dtype,pad,off", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(N, K, dtype, pad, off, residual):
    g = gen_of(N * 7 + K)
    x = padded(g, N, K, dtype, pad, off)
    res = padded(g, N, K, dtype, pad, 0, 2.0) if residual else None
    gain = normal(g, (K,), 0.2, dtype) + 1
    total, out = padded(g, N, K, dtype, 2 * pad), padded(g, N, K, dtype, pad, off)
    rstd = torch.empty(N, device="cuda")
    h = hg.hg_norm_create(K, N + 1, dtype=dtype)
    hg.hg_norm_rows(h, x, gain, out, residual=res, sum_out=total, rstd=rstd, eps=1e-5)
    s = (x.float() + res.float()).to(dtype) if residual else x
    assert torch.equal(total, s)
    check_norm(s, gain, 1e-5, rstd, out)
    # The optional outputs change nothing.
    alone = torch.empty((N, K), device="cuda", dtype=dtype)
    hg.hg_norm_rows(h, x, gain, alone, residual=res, eps=1e-5)
    check_norm(s, gain, 1e-5, None, alone)
    h.close()


@pytest.mark.parametrize("N,K,dtype,pad,off", SHAPES)
@pytest.mark.parametrize("block", [0, 128])
def test_norm_in_8_bits(N, K, dtype, pad, off, block):
    g = gen_of(N * 5 + K)
    x, res = padded(g, N, K, dtype, pad, off), padded(g, N, K, dtype, pad, 0, 0.5)
    gain = normal(g, (K,), 0.5, dtype)
    if N > 2:
        x[1], res[1] = 0, 0           # a row of zeros
        x[2, :min(K, 128)] = 0        # and a block of them
        res[2, :min(K, 128)] = 0
    out = torch.zeros(N * (K + pad) + off, device="cuda", dtype=torch.uint8).view(e4m3)
    out = out[off:].view(N, K + pad)[:, :K]
    total, rstd = torch.empty((N, K), device="cuda", dtype=dtype), torch.empty(N, device="cuda")
    scales = torch.full((N, -(-K // 128) if block else 1), 9.0, device="cuda")
    h = hg.hg_norm_create(K, N, dtype=dtype)
    hg.hg_norm_rows(h, x, gain, out, residual=res, sum_out=total, rstd=rstd, scales=scales)
    s = (x.float() + res.float()).to(dtype)
    assert torch.equal(total, s)
    check_norm(s, gain, 1e-6, rstd, out, scales)
    if N > 2:
        assert bool((scales[1] == 1).all()) and bool((out[1].float() == 0).all())
    h.close()


def test_small_scales():
    """Values below 448 * 2^-126: the scale stays there, and nothing overflows."""
    K = 256
    x = torch.full((2, K), 1.0, device="cuda")
    x[1, :128] = 2.0 ** -140
    gain = torch.full((K,), 2.0 ** -124, device="cuda")
    gain[128:] = 1.0
    h = hg.hg_norm_create(K, 2, dtype=fp32)
    out, scales = torch.empty((2, K), device="cuda", dtype=e4m3), torch.empty((2, 2), device="cuda")
    hg.hg_norm_rows(h, x, gain, out, scales=scales, eps=0.0)
    assert scales[0, 0].item() == 2.0 ** -126
    assert bool((out[0, :128].float() == 4.0).all()) and bool((out[1, :128].float() == 0).all())
    h.close()


@pytest.mark.parametrize("K", [1000, 1001, 7168, 20001])
def test_norm_in_place(K):
    """sum_out over the residual and out over x, as a decoder's residual stream has them;
    sum_out over x and out over the residual."""
    g = gen_of(K)
    for dtype in (bf16, fp32):
        x, res = normal(g, (9, K), 1.0, dtype), normal(g, (9, K), 2.0, dtype)
        gain = normal(g, (K,), 0.2, dtype) + 1
        h = hg.hg_norm_create(K, 9, dtype=dtype)
        s = (x.float() + res.float()).to(dtype)
        for swap in (False, True):
            a, b = x.clone(), res.clone()
            total, out = (a, b) if swap else (b, a)
            hg.hg_norm_rows(h, a, gain, out, residual=b, sum_out=total)
            assert torch.equal(total, s)
            check_norm(s, gain, 1e-6, None, out)
        a = x.clone()
        hg.hg_norm_rows(h, a, gain, a, residual=res)
        check_norm(s, gain, 1e-6, None, a)
        h.close()


def test_what_lies_beside_the_rows_stays():
    g = gen_of(1)
    for K, pad, off in [(64, 8, 8), (65, 3, 1), (7168, 16, 0), (999, 1, 0)]:
        h = hg.hg_norm_create(K, 5, dtype=bf16)
        x, gain = padded(g, 5, K, bf16, pad, off), normal(g, (K,), 1.0, bf16)
        bufs = [torch.full((7 * (K + pad) + off,), 3.0, device="cuda", dtype=bf16)
                for _ in range(3)]
        total, out, gx = (b[off:].view(7, K + pad)[:, :K] for b in bufs)
        rstd, gg = torch.full((7,), 3.0, device="cuda"), torch.full((K + 2,), 3.0, device="cuda",
                                                                    dtype=bf16)
        hg.hg_norm_rows(h, x, gain, out[1:6], sum_out=total[1:6], rstd=rstd[1:6])
        hg.hg_norm_rows_grad(h, total[1:6], gain, rstd[1:6], out[1:6], gx[1:6], gg[1:-1])
        for b in bufs:
            m = torch.zeros_like(b, dtype=torch.bool)
            m[off:].view(7, K + pad)[1:6, :K] = True
            assert bool((b[~m] == 3).all()) and bool((b[m] != 3).any())
        assert rstd[0].item() == 3 and rstd[6].item() == 3
        assert gg[0].item() == 3 and gg[-1].item() == 3
        h.close()


def test_special_values():
    """NaN stays in its row; a row with an infinity is zeros and NaN; zeros stay zeros."""
    K = 300
    x = torch.ones((5, K), device="cuda", dtype=bf16)
    x[0, 7], x[1, 8], x[2] = math.nan, math.inf, 0
    x[3, 5] = -0.0
    gain = torch.ones(K, device="cuda", dtype=bf16)
    h = hg.hg_norm_create(K, 5)
    out, rstd = torch.empty_like(x), torch.empty(5, device="cuda")
    hg.hg_norm_rows(h, x, gain, out, rstd=rstd)
    assert bool(torch.isnan(out[0]).all()) and math.isnan(rstd[0].item())
    assert bool(torch.isnan(out[1, 8])) and bool((out[1, 9:] == 0).all())
    assert bool((out[2] == 0).all())
    assert bool(torch.isfinite(out[3:]).all())
    assert torch.signbit(out[3, 5]).item()
    q, scales = torch.empty((5, K), device="cuda", dtype=e4m3), torch.empty((5, 3), device="cuda")
    hg.hg_norm_rows(h, x, gain, q, scales=scales)
    assert bool(torch.isnan(q[0].float()).all())
    assert bool((q[2].float() == 0).all()) and bool((scales[2] == 1).all())
    assert bool(torch.isfinite(q[3:].float()).all())
    h.close()


def grad_want(s, gain, rstd, up, more):
    """grad_x, grad_gain, and the magnitudes that their errors go by, in 64 bits."""
    v, r, u, w = s.double(), rstd.double()[:, None], up.double(), gain.double()
    K = s.shape[1]
    d = u * w
    inner = (d * v).sum(1, keepdim=True) / K
    gx = r * d - v * r ** 3 * inner
    mag = (r * d).abs() + (v * r ** 3 * inner).abs()
    if more is not None:
        gx, mag = gx + more.double(), mag + more.double().abs()
    spread = v.abs() * r ** 3 * (d * v).abs().sum(1, keepdim=True) / K
    terms = u * v * r
    return gx, 4 * T * mag + (chains(K) + 6) * T * spread, terms.sum(0), terms.abs().sum(0)


def check_grad(s, gain, rstd, up, more, grad_x, grad_gain, old=None):
    dtype, N = s.dtype, s.shape[0]
    gx, err, gg, mag = grad_want(s, gain, rstd, up, more)
    if grad_x is not None:
        check(grad_x, gx, U[dtype] * gx.abs() + err * 1.01 + TINY[dtype], "grad_x")
    if grad_gain is not None:
        if old is not None:
            gg, mag = gg + old.double(), mag + old.double().abs()
        n = min(N, N / 152 + 320) + 4
        check(grad_gain, gg, U[dtype] * gg.abs() + n * T * mag * 1.01 + TINY[dtype], "grad_gain")


def grad_inputs(g, N, K, dtype, pad=0, off=0):
    s = padded(g, N, K, dtype, pad, off, 2.0)
    gain = normal(g, (K,), 0.2, dtype) + 1
    rstd = torch.rsqrt(s.float().square().mean(1) + 1e-6)
    up = padded(g, N, K, dtype, 0, off, 0.5)
    more = padded(g, N, K, dtype, 2 * pad, 0, 0.5)
    return s, gain, rstd, up, more


@pytest.mark.parametrize("N,K,dtype,pad,off", SHAPES + [
    (4000, 64, bf16, 0, 0), (5000, 33, fp32, 0, 0), (1500, 1000, fp16, 0, 0),
    (700, 7168, bf16, 0, 0), (2000, 513, bf16, 1, 0), (64, 7168, bf16, 0, 0),
    (65, 1000, bf16, 0, 0), (152, 96, fp32, 0, 0), (153, 96, fp32, 0, 0), (64, 333, fp16, 0, 0),
    (320, 512, bf16, 0, 0), (2500, 1024, fp16, 0, 0), (900, 14336, bf16, 0, 0),
    (400, 5002, bf16, 0, 0), (400, 12000, fp16, 2, 0), (1000, 2048, fp32, 0, 0)])
@pytest.mark.parametrize("residual", [False, True])
def test_gradient(N, K, dtype, pad, off, residual):
    g = gen_of(N * 3 + K)
    s, gain, rstd, up, more = grad_inputs(g, N, K, dtype, pad, off)
    more = more if residual else None
    gx, gg = padded(g, N, K, dtype, pad, off), torch.full((K,), 9.0, device="cuda", dtype=dtype)
    h = hg.hg_norm_create(K, N, dtype=dtype)
    hg.hg_norm_rows_grad(h, s, gain, rstd, up, gx, gg, grad_sum=more)
    check_grad(s, gain, rstd, up, more, gx, gg)
    # Each gradient alone, the second added to what is there; twice the same bits.
    alone, old = torch.empty_like(gx), normal(g, (K,), 1.0, dtype)
    hg.hg_norm_rows_grad(h, s, gain, rstd, up, alone, None, grad_sum=more)
    check_grad(s, gain, rstd, up, more, alone, None)
    add = old.clone()
    hg.hg_norm_rows_grad(h, s, gain, rstd, up, None, add, accumulate=True)
    check_grad(s, gain, rstd, up, more, None, add, old)
    again, twice = torch.empty_like(gx), torch.empty_like(gg)
    hg.hg_norm_rows_grad(h, s, gain, rstd, up, again, twice, grad_sum=more)
    assert torch.equal(again, gx) and torch.equal(twice, gg)
    h.close()


@pytest.mark.parametrize("K", [1000, 1001, 7168, 20001])
def test_gradient_in_place(K):
    g = gen_of(K)
    s, gain, rstd, up, more = grad_inputs(g, 21, K, bf16)
    h = hg.hg_norm_create(K, 21)
    for over in ("up", "more"):
        a, b, gg = up.clone(), more.clone(), torch.empty(K, device="cuda", dtype=bf16)
        gx = a if over == "up" else b
        hg.hg_norm_rows_grad(h, s, gain, rstd, a, gx, gg, grad_sum=b)
        check_grad(s, gain, rstd, up, more, gx, gg)
    h.close()


@pytest.mark.parametrize("K", [40, 41, 7168, 16384, 50000])
def test_gradient_of_no_rows(K):
    h = hg.hg_norm_create(K, 4)
    none = torch.empty((0, K), device="cuda", dtype=bf16)
    gain, gg = (torch.ones(K, device="cuda", dtype=bf16) for _ in range(2))
    rstd = torch.empty(0, device="cuda")
    hg.hg_norm_rows(h, none, gain, none.clone())
    hg.hg_norm_rows_grad(h, none, gain, rstd, none, none.clone(), gg, accumulate=True)
    assert bool((gg == 1).all())
    hg.hg_norm_rows_grad(h, none, gain, rstd, none, none.clone(), gg)
    assert bool((gg == 0).all())
    h.close()


def test_gradient_against_differences():
    """The change of a scalar of both outputs along random directions, in 64 bits from
    fp32 outputs: central differences with a step of 2^-6, whose own error is of its
    square, about 2^-12 times third derivatives of the order of the first."""
    g = gen_of(5)
    N, K = 6, 96
    x, res = normal(g, (N, K), 1.0, fp32), normal(g, (N, K), 1.0, fp32)
    gain, up, more = normal(g, (K,), 0.3, fp32) + 1, normal(g, (N, K), 1.0, fp32), \
        normal(g, (N, K), 1.0, fp32)
    h = hg.hg_norm_create(K, N, dtype=fp32)

    def forward(x, gain):
        s, out, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(N, device="cuda")
        hg.hg_norm_rows(h, x, gain, out, residual=res, sum_out=s, rstd=rstd)
        return s, rstd, (out.double() * up.double()).sum() + (s.double() * more.double()).sum()

    s, rstd, _ = forward(x, gain)
    gx, gg = torch.empty_like(x), torch.empty_like(gain)
    hg.hg_norm_rows_grad(h, s, gain, rstd, up, gx, gg, grad_sum=more)
    step = 2.0 ** -6
    for _ in range(5):
        dx, dg = normal(g, (N, K), 1.0, fp32), normal(g, (K,), 1.0, fp32)
        for a, b, want in [(dx, 0.0, (gx.double() * dx.double()).sum()),
                           (0.0, dg, (gg.double() * dg.double()).sum())]:
            hi = forward(x + step * a, gain + step * b)[2]
            lo = forward(x - step * a, gain - step * b)[2]
            got = (hi - lo) / (2 * step)
            size = gx.double().norm() * dx.double().norm() if a is dx else \
                gg.double().norm() * dg.double().norm()
            assert abs((got - want).item()) <= 2.0 ** -9 * size.item()
    h.close()


def test_refusals_on_a_device():
    h = hg.hg_norm_create(64, 2)
    x = torch.ones((3, 64), device="cuda", dtype=bf16)
    gain, out = x[0].clone(), torch.full_like(x, 5.0)
    with pytest.raises(hg.HGError) as e:
        hg.hg_norm_rows(h, x, gain, out)
    assert e.value.status == hg.HG_ERR_ROWS
    rstd = torch.ones(3, device="cuda")
    with pytest.raises(hg.HGError) as e:
        hg.hg_norm_rows_grad(h, x, gain, rstd, x, out, None)
    assert e.value.status == hg.HG_ERR_ROWS
    for call in (lambda: hg.hg_norm_rows(h, x[:2], gain, out[:2], sum_out=out[:2]),
                 lambda: hg.hg_norm_rows(h, x[:2], gain, out[:2], eps=-1.0),
                 lambda: hg.hg_norm_rows_grad(h, x[:2], gain, rstd[:2], out[:2], None, None)):
        with pytest.raises(hg.HGError) as e:
            call()
        assert e.value.status == hg.HG_ERR_ARG
    torch.cuda.synchronize()
    assert bool((out == 5).all())
    h.close()
    with pytest.raises(hg.HGError):  # a closed handle
        hg.hg_norm_rows(h, x[:2], gain, out[:2])


def test_rows_beyond_32_bits():
    """Row offsets beyond 2^31 elements and 2^32 bytes."""
    K, ld = 1024, (1 << 30) + 8
    buf = torch.empty(2 * ld + K, device="cuda", dtype=bf16)
    g = gen_of(9)
    x = torch.as_strided(buf, (3, K), (ld, 1))
    x.copy_(normal(g, (3, K), 1.0, bf16))
    want = x.clone()
    h = hg.hg_norm_create(K, 3)
    gain, rstd = normal(g, (K,), 1.0, bf16), torch.empty(3, device="cuda")
    near = torch.empty((3, K), device="cuda", dtype=bf16)
    hg.hg_norm_rows(h, x, gain, near, rstd=rstd)
    check_norm(want, gain, 1e-6, rstd, near)
    hg.hg_norm_rows(h, want, gain, x)
    assert torch.equal(x, near)
    gg, gx = torch.empty(K, device="cuda", dtype=bf16), torch.empty_like(near)
    hg.hg_norm_rows_grad(h, want, gain, rstd, near, x, gg)
    hg.hg_norm_rows_grad(h, want, gain, rstd, near, gx, gg)
    assert torch.equal(x, gx)
    h.close()
