"""Refusals and host-only paths of the 8-bit and grouped entry points: no HIP
call is made, so they are checked without a GPU."""
import pytest
import torch

import dense_gemm_04_amd as dg
from ops_util import nearest_e4m3, quantize_ref

BAD = dg.GEMM_ERR_INVALID_VALUE
P = 0x10000            # suitably aligned addresses that validation never follows


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(dg.LIB_PATH):
        from dense_gemm_04_amd import build
        build.build()
    return dg.load()


def reaches_the_device(st):
    return st == (dg.GEMM_OK if torch.cuda.is_available() else dg.GEMM_ERR_UNSUPPORTED_DEVICE)


def quant(op=0, br=1, rows=300, cols=200, X=P, ldx=200, Q=P, ldq=None, S=P, lds=None, fn="bf16"):
    r, k = (cols, rows) if op == 1 else (rows, cols)
    ldq = k if ldq is None else ldq
    lds = -(-r // max(br, 1)) if lds is None else lds
    call = dg.gemm_fp8_quantize_bf16 if fn == "bf16" else dg.gemm_fp8_quantize_f32
    return call(op, br, rows, cols, X, ldx, Q, ldq, S, lds)


def test_quantize_refusals():
    for fn in ("bf16", "f32"):
        for bad in (dict(op=2), dict(op=-1), dict(br=0), dict(br=64), dict(rows=-1), dict(cols=-1, ldq=1),
                    dict(rows=1 << 31), dict(ldx=199), dict(ldq=199), dict(op=1, ldq=299), dict(lds=299),
                    dict(br=128, lds=2), dict(X=None), dict(Q=None), dict(S=None), dict(X=P + 1), dict(S=P + 2),
                    dict(rows=1 << 30, ldx=1 << 40, lds=1 << 30), dict(lds=1 << 62)):
            assert quant(fn=fn, **bad) == BAD, bad
    assert quant(fn="f32", X=P + 2) == BAD
    assert quant(rows=0, X=None, Q=None, S=None, lds=1) == dg.GEMM_OK
    assert quant(cols=0, X=None, Q=None, S=None, ldx=1, ldq=1) == dg.GEMM_OK
    if not torch.cuda.is_available():
        assert quant() == quant(fn="f32") == dg.GEMM_ERR_UNSUPPORTED_DEVICE


def fp8(M=300, N=200, K=400, alpha=1.0, A=P, lda=400, SA=P, ldsa=300, B=P, ldb=400, SB=P, ldsb=2, br=128, beta=0.0,
        C=P, ldc=200, bias=None, act=0):
    return dg.gemm_fp8(M, N, K, alpha, A, lda, SA, ldsa, B, ldb, SB, ldsb, br, beta, C, ldc, bias, act)


def test_product_refusals():
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(M=1 << 31), dict(lda=399), dict(ldb=399), dict(ldc=199),
                dict(ldsa=299), dict(ldsb=1), dict(br=1, ldsb=199), dict(br=2), dict(br=0), dict(A=None), dict(B=None),
                dict(SA=None), dict(SB=None), dict(C=None), dict(C=P + 1), dict(SA=P + 1), dict(SB=P + 2),
                dict(bias=P + 1), dict(act=3), dict(act=-1), dict(ldc=1 << 58), dict(lda=1 << 58), dict(ldsa=1 << 60)):
        assert fp8(**bad) == BAD, bad
    assert fp8(M=0, A=None, SA=None, C=None) == dg.GEMM_OK
    assert fp8(N=0, B=None, SB=None, C=None) == dg.GEMM_OK
    # No product and beta == 1: nothing to do; otherwise only C is needed.
    assert fp8(alpha=0.0, beta=1.0, A=None, B=None, SA=None, SB=None) == dg.GEMM_OK
    if not torch.cuda.is_available():
        assert fp8() == dg.GEMM_ERR_UNSUPPORTED_DEVICE
        assert fp8(alpha=0.0, A=None, B=None, SA=None, SB=None) == dg.GEMM_ERR_UNSUPPORTED_DEVICE
        assert fp8(K=0, A=None, B=None, SA=None, SB=None) == dg.GEMM_ERR_UNSUPPORTED_DEVICE
        assert fp8(A=P + 1, B=P + 3, lda=401, ldb=403) == dg.GEMM_ERR_UNSUPPORTED_DEVICE


def grouped(opb=0, groups=4, M=300, N=200, K=400, alpha=1.0, A=P, lda=400, B=P, ldb=400, strideb=80000, beta=0.0, C=P,
            ldc=200, offsets=P, scale=None, bias=None, stridebias=200, act=0):
    return dg.gemm_bf16_grouped(opb, groups, M, N, K, alpha, A, lda, B, ldb, strideb, beta, C, ldc, offsets, scale, bias,
                                stridebias, act)


def test_grouped_refusals():
    for bad in (dict(opb=2), dict(groups=-1), dict(groups=1 << 31), dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=399),
                dict(ldb=199), dict(opb=1, ldb=399), dict(ldc=199), dict(strideb=-1), dict(A=None), dict(B=None),
                dict(C=None), dict(offsets=None), dict(offsets=P + 2), dict(A=P + 1), dict(B=P + 1), dict(C=P + 1),
                dict(scale=P + 2), dict(bias=P + 1), dict(bias=P, stridebias=-1), dict(act=7),
                dict(strideb=1 << 60), dict(bias=P, stridebias=1 << 60), dict(lda=1 << 58)):
        assert grouped(**bad) == BAD, bad
    assert grouped(groups=0, A=None, B=None, C=None, offsets=None) == dg.GEMM_OK
    assert grouped(M=0, A=None, B=None, C=None, offsets=None) == dg.GEMM_OK
    assert grouped(N=0, B=None, C=None, offsets=None) == dg.GEMM_OK
    assert grouped(alpha=0.0, beta=1.0, A=None, B=None, C=None, offsets=None) == dg.GEMM_OK
    if not torch.cuda.is_available():
        assert grouped() == dg.GEMM_ERR_UNSUPPORTED_DEVICE
        assert grouped(groups=1, strideb=-7) == dg.GEMM_ERR_UNSUPPORTED_DEVICE      # not read
        assert grouped(strideb=0) == dg.GEMM_ERR_UNSUPPORTED_DEVICE                 # one shared matrix


def wgrad(groups=4, M=300, N=200, K=400, alpha=1.0, X=P, ldx=400, dY=P, lddy=200, beta=0.0, dW=P, lddw=200,
          stridedw=80000, offsets=P, fn=None):
    fn = fn or dg.gemm_bf16_grouped_wgrad
    return fn(groups, M, N, K, alpha, X, ldx, dY, lddy, beta, dW, lddw, stridedw, offsets)


def test_wgrad_refusals():
    for fn in (dg.gemm_bf16_grouped_wgrad, dg.gemm_bf16_grouped_wgrad_f32):
        for bad in (dict(groups=-1), dict(M=-1), dict(N=-1), dict(K=-1), dict(ldx=399), dict(lddy=199), dict(lddw=199),
                    dict(stridedw=79999), dict(X=None), dict(dY=None), dict(dW=None), dict(offsets=None), dict(X=P + 1),
                    dict(dY=P + 1), dict(dW=P + 1), dict(offsets=P + 1), dict(stridedw=1 << 60), dict(lddw=1 << 58)):
            assert wgrad(fn=fn, **bad) == BAD, bad
        for empty in (dict(groups=0), dict(N=0, lddy=1), dict(K=0, ldx=1)):
            assert wgrad(fn=fn, X=None, dY=None, dW=None, offsets=None, **empty) == dg.GEMM_OK
        assert wgrad(fn=fn, M=0, beta=1.0, X=None, dY=None, dW=None, offsets=None) == dg.GEMM_OK
    assert wgrad(fn=dg.gemm_bf16_grouped_wgrad_f32, dW=P + 2) == BAD
    if not torch.cuda.is_available():
        assert wgrad() == dg.GEMM_ERR_UNSUPPORTED_DEVICE
        assert wgrad(M=0, X=None, dY=None) == dg.GEMM_ERR_UNSUPPORTED_DEVICE        # dW <- beta dW
        assert wgrad(groups=1, stridedw=0) == dg.GEMM_ERR_UNSUPPORTED_DEVICE        # not read


def test_conveniences_refuse_host_tensors():
    x, b = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.uint8)
    s, o = torch.zeros(1, 4), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: dg.quantize_fp8(x, b, s), lambda: dg.matmul_fp8(b, s, b, s, x),
                 lambda: dg.matmul_bf16_grouped(x, x.view(1, 4, 8), x, o), lambda: dg.grouped_wgrad(x, x, x.view(1, 4, 8), o)):
        with pytest.raises(TypeError):
            call()


def test_the_tests_own_rounding():
    """The 64-bit reference against torch's conversion, on values and ties."""
    v = torch.cat([torch.linspace(-448, 448, 20001), torch.tensor([0.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])]).double()
    want = v.float().to(torch.float8_e4m3fn).float().double().numpy()
    import numpy as np
    np.testing.assert_array_equal(nearest_e4m3(v.float().double().numpy()), want)
    _, s = quantize_ref(np.array([[0.0, 448.0]]), 1)
    assert s[0, 0] == 1.0


def test_group_counts_past_the_kernels_counters_are_refused():
    for groups in ((1 << 31) - 64, (1 << 31) - 1):
        assert grouped(groups=groups, strideb=0) == BAD
        assert wgrad(groups=groups) == BAD
