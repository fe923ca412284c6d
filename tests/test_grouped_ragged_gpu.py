"""GPU tests of grouped products whose rows of C do not end on 16 bytes: the
vector that crosses the last column leaves by elements, with C read before it."""
import pytest
import torch

import dense_gemm_04_amd as dg
from gpu_util import note
from ops_util import close, f64, gen, grouped_ref, wgrad_ref
from test_grouped_gpu import normal, offsets_of, run_grouped, run_wgrad

pytestmark = pytest.mark.gpu

# Groups of a few rows up to many large tiles; every remainder of N by 8.
SIZES = [([30, 0, 41, 60], 65, 72), ([30, 90, 41], 203, 136), ([150, 0, 333], 514, 80), ([1500, 1100], 1027, 200),
         ([700, 900, 1300], 516, 264), ([5000, 0, 6100, 2], 1061, 136), ([9000, 7300], 1014, 72), ([260, 500], 263, 1000)]


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("lengths,N,K", SIZES)
def test_rows(lengths, N, K, tb):
    note(f"grouped ragged {lengths} {N} {K} {tb}")
    g, E, M = gen(N), len(lengths), sum(lengths) + 3
    A, B = normal(g, M, K), normal(g, E, *((N, K) if tb else (K, N)))
    off, C0 = offsets_of(lengths), normal(g, M, N)
    scale, bias = torch.rand(M, generator=g) + 0.5, normal(g, E, N)
    c = run_grouped(A, B, tb, off, C0, True, 0.5, -0.5, scale, bias, dg.ACT_RELU)
    want, d = grouped_ref(f64(A), f64(B), tb, off, f64(C0), 0.5, -0.5, f64(scale), f64(bias), dg.ACT_RELU)
    assert close(c, want, d, K) <= 1


# The tile sizes of gradients follow the matrices' size and the rows per group.
GRADIENTS = [([30, 0, 41, 60], 65, 72), ([200, 0, 100], 203, 136), ([150, 0, 333, 1], 1027, 1032), ([2000, 1700], 2051, 2056),
             ([600, 900], 4101, 1544), ([9000, 7300], 262, 264)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lengths,N,K", GRADIENTS)
def test_gradients(lengths, N, K, dtype):
    note(f"wgrad ragged {lengths} {N} {K} {dtype}")
    g, M = gen(K), sum(lengths)
    X, dY, off = normal(g, M, K), normal(g, M, N), offsets_of(lengths)
    dW0 = torch.randn(len(lengths), K, N, generator=g).to(dtype)
    dw = run_wgrad(X, dY, off, dtype, True, 0.5, -0.25, dW0)
    want, d = wgrad_ref(f64(X), f64(dY), off, 0.5, -0.25, f64(dW0))
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    assert close(dw, want, d, max(lengths) + 1, step) <= 1


# Few enough tiles that 192 rows to a tile make one round, 256 rows a worse one.
@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("N,K", [(4091, 200), (4096, 328), (4093, 72)])
def test_tiles_of_192_rows(N, K, tb):
    note(f"grouped 192 {N} {K} {tb}")
    lengths = [1300, 0, 1250]
    g, E, M = gen(N + K), len(lengths), sum(lengths) + 3
    A, B = normal(g, M, K), normal(g, E, *((N, K) if tb else (K, N)))
    off, C0 = offsets_of(lengths), normal(g, M, N)
    c = run_grouped(A, B, tb, off, C0)
    want, d = grouped_ref(f64(A), f64(B), tb, off, f64(C0))
    assert close(c, want, d, K) <= 1
    scale, bias = torch.rand(M, generator=g) + 0.5, normal(g, E, N)
    c = run_grouped(A, B, tb, off, C0, True, 0.5, -0.5, scale, bias, dg.ACT_RELU)
    want, d = grouped_ref(f64(A), f64(B), tb, off, f64(C0), 0.5, -0.5, f64(scale), f64(bias), dg.ACT_RELU)
    assert close(c, want, d, K) <= 1


@pytest.mark.parametrize("check", ["poison", "sync"])
def test_tiles_of_192_rows_in_the_lds_checking_builds(check):
    M, E, N, K, g = 2550, 2, 4096, 264, gen(9)
    x = normal(g, M, K).cuda()
    offs = torch.tensor([0, 1300, M], dtype=torch.int32, device="cuda")
    for tb in (False, True):
        w = normal(g, E, *((N, K) if tb else (K, N))).cuda()
        out = []
        for handle in (dg.load(), dg.load_check_build(check)):
            y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
            assert handle.gemm_bf16_grouped(int(tb), E, M, N, K, 1.0, x.data_ptr(), K, w.data_ptr(), w.stride(1),
                                            w.stride(0), 0.0, y.data_ptr(), N, offs.data_ptr(), None, None, 0, 0,
                                            None) == dg.GEMM_OK
            torch.cuda.synchronize()
            out.append(y)
        assert torch.equal(*out)
