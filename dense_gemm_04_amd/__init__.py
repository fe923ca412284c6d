"""Python binding of libdense_gemm_04_amd.so (argument marshalling only).

The functions carry the C names and arguments of ``include/gemm.h``: raw
device pointers (ints), sizes, leading dimensions and a stream handle (int,
0 = null stream). All arithmetic runs in the HIP kernels of the library; if
the library is missing or cannot be loaded, every call raises.

``matmul_f32`` / ``matmul_bf16``, ``quantize_fp8`` / ``matmul_fp8`` and
``matmul_bf16_grouped`` / ``grouped_wgrad`` are conveniences that take torch CUDA
tensors (row-major, unit column stride), pass their pointers, strides and
torch's current stream, and raise ``GemmError`` on a non-zero status.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libdense_gemm_04_amd.so")

GEMM_OK = 0
GEMM_ERR_INVALID_VALUE = 1
GEMM_ERR_UNSUPPORTED_DEVICE = 2
GEMM_ERR_LAUNCH = 3
GEMM_ERR_SCRATCH_LIMIT = 4
# Size of the static scratch behind gemm_bf16_ws_noalloc (per GPU).
NOALLOC_SCRATCH_BYTES = (32 << 20) + (64 << 10)

VARIANT_AUTO = 0
VARIANT_MFMA = 1
VARIANT_GENERAL = 2
VARIANT_VALU = 3
VARIANT_SKINNY = 4
VARIANT_SMALL = 5
VARIANT_NAMES = {0: "auto", 1: "mfma", 2: "general", 3: "valu", 4: "skinny", 5: "small"}

ACT_NONE = 0
ACT_RELU = 1
ACT_GELU_TANH = 2
ACT_NAMES = {0: "none", 1: "relu", 2: "gelu_tanh"}

OP_N = 0
OP_T = 1

EXPORTS = ("gemm_f32", "gemm_bf16", "gemm_f32_ex", "gemm_bf16_ex", "gemm_bf16_ws",
           "gemm_bf16_workspace_size", "gemm_bf16_ws_noalloc", "gemm_f32_ws", "gemm_f32_workspace_size",
           "gemm_f32_bias_act", "gemm_bf16_bias_act", "gemm_f32_op", "gemm_bf16_op",
           "gemm_f32_scaled", "gemm_bf16_scaled", "gemm_fp8_quantize_bf16",
           "gemm_fp8_quantize_f32", "gemm_fp8", "gemm_bf16_grouped", "gemm_bf16_grouped_wgrad",
           "gemm_bf16_grouped_wgrad_f32", "gemm_plan",
           "gemm_status_string")

_lib = None


class GemmError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(f"GEMM failed with status {status}: {gemm_status_string(status)}")


def load() -> ctypes.CDLL:
    """Load the native library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        _lib = _bind(LIB_PATH)
    return _lib


def load_check_build(check: str) -> ctypes.CDLL:
    """One of the LDS-checking builds ("poison" or "sync"; see build.py), as
    a separate library handle with the same C functions, for the tests that
    compare it with the normal build."""
    if check not in ("poison", "sync"):
        raise ValueError(check)
    return _bind(os.path.join(PKG, f"libdense_gemm_04_amd_{check}.so"))


def _bind(path: str) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    i64, f32, vp, ci = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int
    base = [i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp]
    for name in ("gemm_f32", "gemm_bf16"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ci, base
    lib.gemm_bf16_ws_noalloc.restype, lib.gemm_bf16_ws_noalloc.argtypes = ci, base
    for name in ("gemm_f32_ex", "gemm_bf16_ex"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ci, base + [ci]
    for name in ("gemm_bf16_ws", "gemm_f32_ws"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ci, base[:11] + [vp, ctypes.c_size_t, vp]
    for name in ("gemm_f32_bias_act", "gemm_bf16_bias_act"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ci, base[:11] + [vp, ci, vp, ctypes.c_size_t, vp]
    for name in ("gemm_f32_op", "gemm_bf16_op"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ci, [ci, ci] + base[:11] + [vp, ci, vp, ctypes.c_size_t, vp]
    for name in ("gemm_f32_scaled", "gemm_bf16_scaled"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ci, [ci, ci] + base[:11] + [vp, vp, vp, ci, vp, ctypes.c_size_t,
                                                              vp]
    for name in ("gemm_bf16_workspace_size", "gemm_f32_workspace_size"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ctypes.c_size_t, [i64, i64, i64]
    for name in ("gemm_fp8_quantize_bf16", "gemm_fp8_quantize_f32"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ci, [ci, ci, i64, i64, vp, i64, vp, i64, vp, i64, vp]
    lib.gemm_fp8.restype = ci
    lib.gemm_fp8.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, vp, i64, vp, i64, ci, f32, vp,
                             i64, vp, ci, vp]
    lib.gemm_bf16_grouped.restype = ci
    lib.gemm_bf16_grouped.argtypes = [ci, i64, i64, i64, i64, f32, vp, i64, vp, i64, i64, f32, vp,
                                      i64, vp, vp, vp, i64, ci, vp]
    for name in ("gemm_bf16_grouped_wgrad", "gemm_bf16_grouped_wgrad_f32"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ci, [i64, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, i64,
                                       vp, vp]
    lib.gemm_plan.restype = ci
    lib.gemm_plan.argtypes = [ci, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, ci]
    lib.gemm_status_string.restype = ctypes.c_char_p
    lib.gemm_status_string.argtypes = [ci]
    return lib


def gemm_f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().gemm_f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_bf16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().gemm_bf16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_f32_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0, variant=0) -> int:
    return load().gemm_f32_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream, variant)


def gemm_bf16_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0, variant=0) -> int:
    return load().gemm_bf16_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream, variant)


def gemm_bf16_ws(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, workspace, workspace_bytes,
                 stream=0) -> int:
    return load().gemm_bf16_ws(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, workspace,
                               workspace_bytes, stream)


def gemm_bf16_ws_noalloc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().gemm_bf16_ws_noalloc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_bf16_workspace_size(M, N, K) -> int:
    return load().gemm_bf16_workspace_size(M, N, K)


def gemm_f32_ws(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, workspace, workspace_bytes,
                stream=0) -> int:
    return load().gemm_f32_ws(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, workspace,
                              workspace_bytes, stream)


def gemm_f32_workspace_size(M, N, K) -> int:
    return load().gemm_f32_workspace_size(M, N, K)


def gemm_f32_bias_act(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act, workspace=0,
                      workspace_bytes=0, stream=0) -> int:
    return load().gemm_f32_bias_act(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act,
                                    workspace, workspace_bytes, stream)


def gemm_bf16_bias_act(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act, workspace=0,
                       workspace_bytes=0, stream=0) -> int:
    return load().gemm_bf16_bias_act(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act,
                                     workspace, workspace_bytes, stream)


def gemm_f32_op(opa, opb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias=None, act=0,
                workspace=None, workspace_bytes=0, stream=0) -> int:
    return load().gemm_f32_op(opa, opb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act,
                              workspace, workspace_bytes, stream)


def gemm_bf16_op(opa, opb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias=None, act=0,
                 workspace=None, workspace_bytes=0, stream=0) -> int:
    return load().gemm_bf16_op(opa, opb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act,
                               workspace, workspace_bytes, stream)


def gemm_f32_scaled(opa, opb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, row_scale=None,
                    col_scale=None, bias=None, act=0, workspace=None, workspace_bytes=0,
                    stream=0) -> int:
    return load().gemm_f32_scaled(opa, opb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                                  row_scale, col_scale, bias, act, workspace, workspace_bytes,
                                  stream)


def gemm_bf16_scaled(opa, opb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, row_scale=None,
                     col_scale=None, bias=None, act=0, workspace=None, workspace_bytes=0,
                     stream=0) -> int:
    return load().gemm_bf16_scaled(opa, opb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                                   row_scale, col_scale, bias, act, workspace, workspace_bytes,
                                   stream)


def gemm_fp8_quantize_bf16(op, block_rows, rows, cols, X, ldx, Q, ldq, S, lds, stream=0) -> int:
    return load().gemm_fp8_quantize_bf16(op, block_rows, rows, cols, X, ldx, Q, ldq, S, lds, stream)


def gemm_fp8_quantize_f32(op, block_rows, rows, cols, X, ldx, Q, ldq, S, lds, stream=0) -> int:
    return load().gemm_fp8_quantize_f32(op, block_rows, rows, cols, X, ldx, Q, ldq, S, lds, stream)


def gemm_fp8(M, N, K, alpha, A, lda, SA, ldsa, B, ldb, SB, ldsb, b_block_rows, beta, C, ldc,
             bias=None, act=0, stream=0) -> int:
    return load().gemm_fp8(M, N, K, alpha, A, lda, SA, ldsa, B, ldb, SB, ldsb, b_block_rows, beta,
                           C, ldc, bias, act, stream)


def gemm_bf16_grouped(opb, groups, M, N, K, alpha, A, lda, B, ldb, strideb, beta, C, ldc, offsets,
                      row_scale=None, bias=None, stridebias=0, act=0, stream=0) -> int:
    return load().gemm_bf16_grouped(opb, groups, M, N, K, alpha, A, lda, B, ldb, strideb, beta, C,
                                    ldc, offsets, row_scale, bias, stridebias, act, stream)


def gemm_bf16_grouped_wgrad(groups, M, N, K, alpha, X, ldx, dY, lddy, beta, dW, lddw, stridedw,
                            offsets, stream=0) -> int:
    return load().gemm_bf16_grouped_wgrad(groups, M, N, K, alpha, X, ldx, dY, lddy, beta, dW, lddw,
                                          stridedw, offsets, stream)


def gemm_bf16_grouped_wgrad_f32(groups, M, N, K, alpha, X, ldx, dY, lddy, beta, dW, lddw, stridedw,
                                offsets, stream=0) -> int:
    return load().gemm_bf16_grouped_wgrad_f32(groups, M, N, K, alpha, X, ldx, dY, lddy, beta, dW,
                                              lddw, stridedw, offsets, stream)


def gemm_plan(elem_bytes, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, variant=0) -> int:
    return load().gemm_plan(elem_bytes, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, variant)


def gemm_status_string(status: int) -> str:
    return load().gemm_status_string(status).decode()


# ---- torch-tensor conveniences (pointers, strides and stream only) ----------

def _ld(t, rows_of: int, cols: int) -> int:
    if t.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError("expected unit column stride (row-major)")
    return max(t.stride(0) if rows_of > 1 else cols, cols, 1)


def _stream_handle(stream) -> int:
    if stream is not None:
        return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
    import torch
    return int(torch.cuda.current_stream().cuda_stream)


def _matmul(kind: str, A, B, C, alpha: float, beta: float, variant: int, stream) -> None:
    import torch
    want = torch.float32 if kind == "f32" else torch.bfloat16
    for name, t in (("A", A), ("B", B), ("C", C)):
        if t.dtype != want or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor of dtype {want}")
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, C {tuple(C.shape)}")
    lda, ldb, ldc = _ld(A, M, K), _ld(B, K, N), _ld(C, M, N)
    fn = gemm_f32_ex if kind == "f32" else gemm_bf16_ex
    st = fn(M, N, K, float(alpha), A.data_ptr(), lda, B.data_ptr(), ldb, float(beta),
            C.data_ptr(), ldc, _stream_handle(stream), int(variant))
    if st != GEMM_OK:
        raise GemmError(st)


def matmul_f32(A, B, C, alpha: float = 1.0, beta: float = 0.0, variant: int = VARIANT_AUTO,
               stream=None) -> None:
    """C <- alpha * A @ B + beta * C for fp32 CUDA tensors (in place on C)."""
    _matmul("f32", A, B, C, alpha, beta, variant, stream)


def matmul_bf16(A, B, C, alpha: float = 1.0, beta: float = 0.0, variant: int = VARIANT_AUTO,
                stream=None) -> None:
    """C <- alpha * A @ B + beta * C for bf16 CUDA tensors (fp32 accumulation)."""
    _matmul("bf16", A, B, C, alpha, beta, variant, stream)


def _want(name: str, t, dtypes, dim: int, shape=None) -> None:
    """Check one operand: a tensor of one of `dtypes` on the current GPU, with
    `dim` dimensions, the last with unit stride, and the given shape (None
    entries are free)."""
    import torch
    if not t.is_cuda or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a CUDA tensor of dtype {' or '.join(map(str, dtypes))}")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    if t.dim() != dim or (shape is not None and
                          any(w is not None and w != s for w, s in zip(shape, t.shape))):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: expected unit stride in the last dimension")
    if dim >= 2 and t.shape[-2] > 1 and t.stride(-2) < t.shape[-1]:
        raise ValueError(f"{name}: its rows overlap")


def _ld2(t) -> int:
    """Leading dimension of the matrix in t's last two dimensions."""
    return max(t.stride(-2) if t.shape[-2] > 1 else t.shape[-1], t.shape[-1], 1)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(status: int) -> None:
    if status != GEMM_OK:
        raise GemmError(status)


def quantize_fp8(X, Q, S, op: int = OP_N, block_rows: int = 1, stream=None) -> None:
    """Quantise a bf16 or fp32 matrix (op OP_T: its transpose) into e4m3 values
    Q (uint8 or float8_e4m3fn) and fp32 scales S, ceil(k / 128) x
    ceil(rows / block_rows) for a Q of rows x k."""
    import torch
    _want("X", X, (torch.bfloat16, torch.float32), 2)
    rows, cols = X.shape
    r, k = (cols, rows) if op == OP_T else (rows, cols)
    _want("Q", Q, (torch.uint8, torch.float8_e4m3fn), 2, (r, k))
    _want("S", S, (torch.float32,), 2, (-(-k // 128), -(-r // max(int(block_rows), 1))))
    fn = gemm_fp8_quantize_bf16 if X.dtype == torch.bfloat16 else gemm_fp8_quantize_f32
    _check(fn(int(op), int(block_rows), rows, cols, X.data_ptr(), _ld2(X), Q.data_ptr(), _ld2(Q),
              S.data_ptr(), _ld2(S), _stream_handle(stream)))


def matmul_fp8(A, SA, B, SB, C, alpha: float = 1.0, beta: float = 0.0, b_block_rows: int = 128,
               bias=None, act: int = ACT_NONE, stream=None) -> None:
    """C <- act(alpha * (A SA) (B SB)^T + bias) + beta * C: A (M x K) and B
    (N x K) in e4m3 with their scales, as quantize_fp8 makes them (A with
    block_rows 1, B with b_block_rows), C in bf16."""
    import torch
    e4m3 = (torch.uint8, torch.float8_e4m3fn)
    _want("A", A, e4m3, 2)
    M, K = A.shape
    _want("B", B, e4m3, 2, (None, K))
    N, nk = B.shape[0], -(-K // 128)
    _want("SA", SA, (torch.float32,), 2, (nk, M))
    _want("SB", SB, (torch.float32,), 2, (nk, -(-N // max(int(b_block_rows), 1))))
    _want("C", C, (torch.bfloat16,), 2, (M, N))
    if bias is not None:
        _want("bias", bias, (torch.bfloat16,), 1, (N,))
    _check(gemm_fp8(M, N, K, float(alpha), A.data_ptr(), _ld2(A), SA.data_ptr(), _ld2(SA),
                    B.data_ptr(), _ld2(B), SB.data_ptr(), _ld2(SB), int(b_block_rows), float(beta),
                    C.data_ptr(), _ld2(C), _ptr(bias), int(act), _stream_handle(stream)))


def matmul_bf16_grouped(A, B, C, offsets, opb: int = OP_N, alpha: float = 1.0, beta: float = 0.0,
                        row_scale=None, bias=None, act: int = ACT_NONE, stream=None) -> None:
    """Rows offsets[e] .. offsets[e + 1] - 1 of A (M x K) times B[e] (K x N, or
    with opb OP_T its transpose, B[e] N x K) into the same rows of C (M x N),
    with optional row scales (M, fp32) and biases (groups x N)."""
    import torch
    bf16 = (torch.bfloat16,)
    _want("A", A, bf16, 2)
    M, K = A.shape
    _want("B", B, bf16, 3, (None, None, K) if opb == OP_T else (None, K, None))
    E, N = B.shape[0], B.shape[1] if opb == OP_T else B.shape[2]
    _want("C", C, bf16, 2, (M, N))
    _want("offsets", offsets, (torch.int32,), 1, (E + 1,))
    if row_scale is not None:
        _want("row_scale", row_scale, (torch.float32,), 1, (M,))
    if bias is not None:
        _want("bias", bias, bf16, 2, (E, N))
    _check(gemm_bf16_grouped(int(opb), E, M, N, K, float(alpha), A.data_ptr(), _ld2(A), B.data_ptr(),
                             _ld2(B), B.stride(0), float(beta), C.data_ptr(), _ld2(C),
                             offsets.data_ptr(), _ptr(row_scale), _ptr(bias),
                             0 if bias is None else bias.stride(0), int(act),
                             _stream_handle(stream)))


def grouped_wgrad(X, dY, dW, offsets, alpha: float = 1.0, beta: float = 0.0, stream=None) -> None:
    """dW[e] <- alpha * X_e^T dY_e + beta * dW[e] over the rows of each group:
    X (M x K) and dY (M x N) in bf16, dW (groups x K x N) in bf16 or fp32."""
    import torch
    _want("X", X, (torch.bfloat16,), 2)
    M, K = X.shape
    _want("dY", dY, (torch.bfloat16,), 2, (M, None))
    N = dY.shape[1]
    _want("dW", dW, (torch.bfloat16, torch.float32), 3, (None, K, N))
    E = dW.shape[0]
    _want("offsets", offsets, (torch.int32,), 1, (E + 1,))
    fn = gemm_bf16_grouped_wgrad if dW.dtype == torch.bfloat16 else gemm_bf16_grouped_wgrad_f32
    _check(fn(E, M, N, K, float(alpha), X.data_ptr(), _ld2(X), dY.data_ptr(), _ld2(dY), float(beta),
              dW.data_ptr(), _ld2(dW), dW.stride(0), offsets.data_ptr(), _stream_handle(stream)))
