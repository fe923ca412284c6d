"""GPU tests of the 8-bit product on its two largest tile sizes, which rounds of
resident workgroups choose between: 256 x 256 in full rounds, 192 x 256 where
those would leave a round partly empty."""
import pytest
import torch

import dense_gemm_04_amd as dg
from gpu_util import note
from ops_util import close, f64, fp8_ref, gen
from test_fp8_gpu import INSTRUCTION, ld_of, operands, run_fp8

pytestmark = pytest.mark.gpu

SIZES = [(4090, 4003, 400), (8100, 4001, 272), (4096, 4096, 128),         # 256 x 256
         (2880, 4096, 400), (2881, 4099, 300), (1536, 8192, 272), (5000, 4504, 129)]


@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("size", SIZES)
def test_product(size, b_rows):
    M, N, K = size
    note(f"fp8 {size} b_rows {b_rows}")
    up = -(-K // 16) * 16
    cpu, views = operands(M, N, K, b_rows, M + K, lda=up + 16, ldb=up)
    g = gen(N)
    c0, bias = torch.randn(M, N, generator=g).to(torch.bfloat16), torch.randn(N, generator=g).to(torch.bfloat16)
    ref = [f64(t) for t in cpu]
    for alpha, beta, act, with_bias in ((1.0, 0.0, dg.ACT_NONE, False), (0.5, -0.5, dg.ACT_GELU_TANH, True)):
        c = run_fp8(views, M, N, K, b_rows, alpha, beta, c0.cuda() if beta else None, bias if with_bias else None, act,
                    ldc=-(-N // 4) * 4)
        want, d = fp8_ref(*ref, b_rows, alpha, beta, f64(c0), f64(bias) if with_bias else None, act)
        assert close(c, want, d, -(-K // 128), instruction=INSTRUCTION) <= 1


@pytest.mark.parametrize("check", ["poison", "sync"])
@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("size", [(8100, 4001, 272), (2881, 4099, 300), (5000, 4504, 400)])
def test_lds_checking_builds_agree(size, b_rows, check):
    M, N, K = size
    note(f"fp8 {check} {size} {b_rows}")
    up = -(-K // 16) * 16
    _, (a, sa, b, sb) = operands(M, N, K, b_rows, 9, lda=up, ldb=up)
    out = [torch.full((M, -(-N // 4) * 4), float("nan"), dtype=torch.bfloat16, device="cuda")[:, :N] for _ in range(2)]
    for handle, c in zip((dg.load(), dg.load_check_build(check)), out):
        assert handle.gemm_fp8(M, N, K, 1.0, a.data_ptr(), ld_of(a), sa.data_ptr(), ld_of(sa), b.data_ptr(), ld_of(b),
                               sb.data_ptr(), ld_of(sb), b_rows, 0.0, c.data_ptr(), c.stride(0), None, 0,
                               None) == dg.GEMM_OK
        torch.cuda.synchronize()
    assert torch.equal(*out)
