"""GPU tests of the 8-bit product's precision below bf16's last bit, of its
calls' bits, and of the quantiser's longest walk over rows.

C is bf16, so one call shows its fp32 sum only to 2^-9. A second call on the
first one's result C1 with beta = -1 leaves the sum less C1, of at most 2^-8 of it,
rounded to 2^-8 of that: C1 + C2 holds the sum to 2^-16 at worst and, roundings
being spread evenly, to about 2^-18.

Tolerance, root-mean-square of the error over that of C. The instruction aligns
the 8 products of a group to the largest, m: the 7 others lose less than 2^-13 m
each, 2^-13 m / sqrt(3) root-mean-square where the losses are spread evenly, and
sqrt(7 / 3) 2^-13 m together where their signs are not alike. m^2 is at most the
sum of the group's squares, which is the mean square of the group's sum for
products of independent signs; so the errors are within sqrt(7 / 3) 2^-13 < 2^-12.3 of
a group's sum, and of the sum of all groups. Accumulating blocks in fp32 and the
two roundings to bf16 add less than 2^-16 to that, far inside the step from
2^-12.39 to 2^-12.3."""
import pytest
import torch

import dense_gemm_04_amd as dg
from gpu_util import note
from ops_util import f64, fp8_ref, gen, nearest_e4m3, quantize_ref
from test_fp8_gpu import operands, run_fp8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("size", [(16, 2048, 4000), (120, 1000, 4100), (509, 4096, 4000), (1500, 1500, 2000), (2880, 4090, 1040),
                                  (4090, 4003, 1040)])
def test_sums_below_the_last_bit_of_bf16(size, b_rows):
    M, N, K = size
    note(f"fp8 precision {size} b_rows {b_rows}")
    up, ldc = -(-K // 16) * 16, -(-N // 8) * 8
    cpu, views = operands(M, N, K, b_rows, K + M, lda=up, ldb=up)
    first = run_fp8(views, M, N, K, b_rows, ldc=ldc)
    assert torch.equal(first, run_fp8(views, M, N, K, b_rows, ldc=ldc))         # the same bits again
    rest = run_fp8(views, M, N, K, b_rows, 1.0, -1.0, first, ldc=ldc)
    rows = torch.arange(0, M, M // 200 | 1)
    want, _ = fp8_ref(f64(cpu[0].view(torch.uint8)[rows]), f64(cpu[1][:, rows]), f64(cpu[2]), f64(cpu[3]), b_rows)
    off = f64(first[rows.cuda()]) + f64(rest[rows.cuda()]) - want
    rms = float(((off ** 2).mean() / (want ** 2).mean()) ** 0.5)
    print(f"{size} b_rows {b_rows}: {rms:.2e}")
    assert rms <= 2.0 ** -12.3


@pytest.mark.parametrize("op", [dg.OP_N, dg.OP_T])
def test_quantize_more_rows_than_a_grid_holds(op):
    """Past 65535 rows a workgroup walks several of them."""
    rows, cols = 66000, 130
    x = torch.randn(rows, cols, generator=gen(3)).to(torch.bfloat16)
    r, k = (cols, rows) if op == dg.OP_T else (rows, cols)
    q = torch.empty(r, k, dtype=torch.uint8, device="cuda")
    s = torch.empty(-(-k // 128), r, device="cuda")
    dg.quantize_fp8(x.cuda(), q, s, op, 1)
    torch.cuda.synchronize()
    v, scales = quantize_ref(f64(x.t() if op == dg.OP_T else x), 1)
    assert (s.cpu().numpy() == scales).all()
    assert (f64(q) == nearest_e4m3(v)).all()
