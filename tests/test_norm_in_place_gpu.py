"""The norm's gradients with dX in the place of dY or of R: the same bits as beside
them, at widths where lanes of several waves share a row's last values."""
import pytest
import torch

import dense_gemm_04_amd as dg
from layer_util import BF16, F32
from ops_util import gen
from test_norm_gpu import note, place

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [1025, 1500, 2056, 3001, 4104, 6001, 8200, 9999, 12301, 16380, 16392, 20491, 24601, 28702])
def test_norm_grad_in_place(cols, dtype):
    note(f"norm gradient in place {cols} {dtype}")
    g = gen(cols)
    for rows, odd in ((3, 0), (700, 1)):
        x, dy, r = (torch.randn(rows, cols, generator=g).to(dtype) for _ in range(3))
        w = torch.randn(cols, generator=g).to(dtype).cuda()
        mean, rstd = x.double().mean(1).float().cuda(), (1 / x.double().std(1)).float().cuda()
        ld = cols + odd if odd else -(-cols // 8) * 8
        at = lambda t: place(t, dtype, ld, odd)[1]
        xv = at(x)
        ws = torch.empty(dg.gemm_layernorm_grad_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")

        def grads(dyv, rv, dxv):
            dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
            dg.layernorm_grad(xv, dyv, dxv, mean, rstd, w, rv, dw, db, 0.0, ws)
            return dxv, dw, db

        beside = grads(at(dy), at(r), at(torch.zeros_like(x)))
        dyv, rv = at(dy), at(r)
        for got in (grads(dyv, at(r), dyv), grads(at(dy), rv, rv)):
            assert all(torch.equal(a, b) for a, b in zip(got, beside))
        beside = grads(at(dy), None, at(torch.zeros_like(x)))
        dyv = at(dy)
        assert all(torch.equal(a, b) for a, b in zip(grads(dyv, None, dyv), beside))
