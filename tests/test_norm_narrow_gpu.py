"""The norm's gradients in weight and bias of rows shorter than a vector: many rows, whose
terms of one sign would drift in a long fp32 sum.

Allowances: h = (x - mean) rstd carries 2 steps (2 U) and the sums are exact beside it,
so dweight is off by 2 U of the sum of |dY h| and a step of itself, dbias by a step of itself;
beta's term adds one of each. One U more of each for 64-bit sums and products of steps.
"""
import numpy as np
import pytest
import torch

import dense_gemm_04_amd as dg
from layer_util import BF16, F32, U, norm_grad_allow, norm_grad_ref, worst
from ops_util import f64, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 31, 32, 33, 1023, 1024, 1025, 5000, 262144, 300001, (1 << 20) + 7])
@pytest.mark.parametrize("cols,dtype", [(1, BF16), (3, BF16), (5, BF16), (7, BF16), (1, F32), (2, F32), (3, F32)])
def test_many_short_rows(rows, cols, dtype):
    print(f"norm gradients {rows} x {cols} {dtype}", flush=True)
    g = gen(rows + cols)
    x = torch.randn(rows, cols, generator=g).to(dtype)
    dy = (0.1 + torch.rand(rows, cols, generator=g)).to(dtype)
    w = torch.randn(cols, generator=g).to(dtype)
    mean, rstd = torch.randn(rows, generator=g) - 3, 0.5 + torch.rand(rows, generator=g)
    start = torch.randn(2, cols, generator=g)
    ws = torch.full((dg.gemm_layernorm_grad_workspace_size(rows, cols) + 256,), 0xff, dtype=torch.uint8, device="cuda")
    args = f64(x), f64(w), f64(mean), f64(rstd), f64(dy), None
    dx, dw, db = norm_grad_ref(*args)
    terms = np.abs(f64(dy) * (f64(x) - f64(mean)[:, None]) * f64(rstd)[:, None])
    for beta, wants in ((0.0, (True, True)), (0.5, (True, False)), (-2.0, (False, True))):
        out = torch.full((2, cols + 1), 7.0, device="cuda")
        out[:, :cols] = start.cuda() if beta else float("nan")
        dxv = torch.empty(rows, cols, dtype=dtype, device="cuda")
        dg.layernorm_grad(x.cuda(), dy.cuda(), dxv, mean.cuda(), rstd.cuda(), w.cuda(), None,
                          out[0, :cols] if wants[0] else None, out[1, :cols] if wants[1] else None, beta, ws[:-256])
        torch.cuda.synchronize()
        assert bool((ws[-256:] == 0xff).all()) and bool((out[:, cols] == 7).all())
        assert worst(dxv, dx, norm_grad_allow(*args, dtype)[0]) <= 1
        for i, (want, allow) in enumerate(((dw, 3 * U * terms.sum(0)), (db, 0.0))):
            want = want + (beta * f64(start[i]) if beta else 0.0)
            allow = allow + 2 * U * np.abs(want) + (2 * U * np.abs(beta * f64(start[i])) if beta else 0.0)
            if wants[i]:
                assert worst(out[i, :cols], want, allow) <= 1
            else:
                assert torch.equal(out[i, :cols].cpu(), start[i])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_wide_rows_sum_alike(dtype):
    """Rows longer than the fused kernels take: the same sums."""
    rows, cols = 900, 33000
    print(f"norm gradients {rows} x {cols} {dtype}", flush=True)
    g = gen(1)
    x, dy = torch.randn(rows, cols, generator=g).to(dtype), (0.1 + torch.rand(rows, cols, generator=g)).to(dtype)
    mean, rstd = torch.randn(rows, generator=g) - 3, 0.5 + torch.rand(rows, generator=g)
    ws = torch.empty(dg.gemm_layernorm_grad_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    dxv = torch.empty(rows, cols, dtype=dtype, device="cuda")
    out = torch.empty(2, cols, device="cuda")
    dg.layernorm_grad(x.cuda(), dy.cuda(), dxv, mean.cuda(), rstd.cuda(), None, None, out[0], out[1], 0.0, ws)
    h = (f64(x) - f64(mean)[:, None]) * f64(rstd)[:, None]
    dw, db = (f64(dy) * h).sum(0), f64(dy).sum(0)
    assert worst(out[0], dw, 3 * U * np.abs(f64(dy) * h).sum(0) + 2 * U * np.abs(dw)) <= 1
    assert worst(out[1], db, 2 * U * np.abs(db)) <= 1
