"""Rows far from zero: what a mean loses in its fp32 sum and rounding reaches neither
the norm nor its deviation.

Allowances (layer_util's U and chain). A first mean m0 is off by at most
e = (chain + 2) U mean|x|. Each x - m0 is off by U of itself, so the mean of the differences by
(chain + 4) U (mean|x - m| + e) (dm); their mean square by (chain + 4) U (var + e^2), of
which the square of their mean takes off e^2 with 4 U more: (chain + 8) U (var + e^2) (dv).
rstd is off by half of dv rstd^2, relative, and 4 steps; y by dm rstd, by 4 U for the steps of
(x - m0) rstd and of the shift, whose magnitudes add up to h + 2 e rstd, and by half a step of its type.
"""
import numpy as np
import pytest
import torch

import dense_gemm_04_amd as dg
from layer_util import BF16, F32, STEP, U, chain, norm_allow, norm_ref, worst
from ops_util import f64, gen

pytestmark = pytest.mark.gpu

# Widths of every kernel: 16 lanes, a wave, 4 and 16 waves to a row (few and many rows), and the general one.
COLS = [3, 60, 100, 700, 1024, 4096, 5000, 9000, 20000, 40000, 50001, 65536, 70001]


def check(x, dtype, eps):
    rows, cols = x.shape
    y = torch.empty(rows, cols, dtype=dtype, device="cuda")
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dg.layernorm(x.cuda(), y, None, None, eps, mean, rstd)
    x = f64(x)
    want, m, r = norm_ref(x, None, None, eps)
    d = np.abs(x - m[:, None])
    e = (chain(cols) + 2) * U * np.abs(x).mean(1)
    dm = (chain(cols) + 4) * U * (d.mean(1) + e)
    rel = (chain(cols) + 8) * U * ((d * d).mean(1) + e * e) * r * r / 2 + 4 * U
    h = d * r[:, None]
    ay = (dm * r)[:, None] + h * rel[:, None] + 4 * U * (h + 2 * (e * r)[:, None]) + (STEP[dtype] + U) * np.abs(want)
    assert worst(y, want, ay) <= 1
    assert worst(rstd, r, r * rel) <= 1
    assert worst(mean, m, dm + 2 * U * np.abs(m)) <= 1


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_far_from_zero(cols, dtype):
    g = gen(cols)
    for far, wide in ((4096.0, 1.0), (-1e5, 3.0)):
        for rows in (6, 600 if cols <= 9000 else 7):
            print(f"norm of {rows} x {cols} {dtype} around {far}", flush=True)
            check((torch.randn(rows, cols, generator=g) * wide + far).to(dtype), dtype, 1e-6)


@pytest.mark.parametrize("cols", COLS)
def test_constant_rows_far_from_zero(cols):
    """Their norm is 0, up to what the sums of equal differences leave of one."""
    value = torch.tensor([4096.3, -10000.7, 1e6 / 3, 0.1, 77777.7])
    check(value[:, None].expand(5, cols).contiguous(), F32, 1e-5)


@pytest.mark.parametrize("cols", [3, 60, 700, 4096, 70001])
def test_rows_past_the_range_of_their_sums(cols):
    """Finite values whose sums are not: NaN, or a deviation that counts as infinite."""
    x = torch.randn(4, cols, generator=gen(1)).abs() + 1
    x[0] *= 1e30
    x[1] = x[1] * 1e30 + 1e33
    x[2] = 3e38
    b = torch.randn(cols, generator=gen(2)).cuda()
    y, rstd = torch.empty(4, cols, device="cuda"), torch.empty(4, device="cuda")
    dg.layernorm(x.cuda(), y, None, b, 1e-5, None, rstd)
    for i in range(3):
        assert bool(y[i].isnan().all()) or torch.equal(y[i], b) and float(rstd[i]) == 0
    assert bool(y[3].isfinite().all())


@pytest.mark.parametrize("cols", [49152, 49153, 57344, 60007, 65536])
def test_rows_whose_weight_comes_late(cols):
    """The widest rows of one workgroup, whose weight and bias are read after the sums; in place the same bits."""
    g = gen(cols)
    x, w, b = ((torch.randn(*s, generator=g) * 2 + 1).to(BF16).cuda() for s in ((5, cols), (cols,), (cols,)))
    y = torch.empty_like(x)
    for ww, bb in ((w, b), (None, b), (w, None), (None, None)):
        dg.layernorm(x, y, ww, bb)
        args = f64(x), None if ww is None else f64(w), None if bb is None else f64(b), 1e-5
        assert worst(y, norm_ref(*args)[0], norm_allow(*args, BF16)[0]) <= 1
    dg.layernorm(x, x)
    assert torch.equal(x, y)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_means_of_exact_sums(cols, dtype):
    """Multiples of 2^-7 up to 1: every partial sum is below 2^24 of them, so exact, and the mean is a
    quotient off by a step, however near zero it lies."""
    for rows in (5, 600 if cols <= 9000 else 7):
        x = (torch.randint(-128, 129, (rows, cols), generator=gen(cols)) / 128).to(dtype)
        mean = torch.empty(rows, device="cuda")
        dg.layernorm(x.cuda(), torch.empty_like(x, device="cuda"), None, None, 1e-5, mean)
        want = f64(x).mean(1)
        assert worst(mean, want, 2 * U * np.abs(want)) <= 1
