"""Python binding of libdense_gemm_04_amd.so (argument marshalling only).

The functions carry the C names and arguments of ``include/gemm.h``: raw
device pointers (ints), sizes, leading dimensions and a stream handle (int,
0 = null stream). All arithmetic runs in the HIP kernels of the library; if
the library is missing or cannot be loaded, every call raises.

``matmul_f32`` / ``matmul_bf16``, ``quantize_fp8`` / ``matmul_fp8`` and
``matmul_bf16_grouped`` / ``grouped_wgrad``, and ``layernorm``, ``dropout`` and the
``moe_*`` calls with their gradients, are conveniences that take torch CUDA
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
           "gemm_bf16_grouped_wgrad_f32", "gemm_layernorm_bf16", "gemm_layernorm_f32",
           "gemm_layernorm_grad_workspace_size", "gemm_layernorm_grad_bf16",
           "gemm_layernorm_grad_f32", "gemm_dropout_bf16", "gemm_dropout_f32",
           "gemm_moe_route_workspace_size", "gemm_moe_route_bf16", "gemm_moe_route_f32",
           "gemm_moe_route_grad_bf16", "gemm_moe_route_grad_f32", "gemm_moe_gather_bf16",
           "gemm_moe_combine_bf16", "gemm_moe_combine_grad_bf16", "gemm_plan",
           "gemm_status_string")

# Limits of the router (experts) and of a token's choices (k).
MOE_MAX_EXPERTS = 1024
MOE_MAX_K = 16

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
    for name in ("gemm_layernorm_bf16", "gemm_layernorm_f32"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ci, [i64, i64, f32, vp, i64, vp, vp, vp, i64, vp, vp, vp]
    for name in ("gemm_layernorm_grad_bf16", "gemm_layernorm_grad_f32"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ci, [i64, i64, vp, i64, vp, vp, vp, vp, i64, vp, i64, vp, i64, f32,
                                       vp, vp, vp, ctypes.c_size_t, vp]
    for name in ("gemm_dropout_bf16", "gemm_dropout_f32"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ci, [i64, i64, f32, vp, vp, i64, vp, i64, vp, i64, vp]
    for name in ("gemm_moe_route_bf16", "gemm_moe_route_f32"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ci, [i64, i64, ci, ci, vp, i64, vp, vp, vp, vp, vp, vp, vp,
                                       ctypes.c_size_t, vp]
    for name in ("gemm_moe_route_grad_bf16", "gemm_moe_route_grad_f32"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ci, [i64, i64, ci, ci, vp, i64, vp, vp, vp, vp, vp, i64, vp]
    lib.gemm_layernorm_grad_workspace_size.restype = ctypes.c_size_t
    lib.gemm_layernorm_grad_workspace_size.argtypes = [i64, i64]
    lib.gemm_moe_route_workspace_size.restype = ctypes.c_size_t
    lib.gemm_moe_route_workspace_size.argtypes = [i64, i64, ci]
    lib.gemm_moe_gather_bf16.restype = ci
    lib.gemm_moe_gather_bf16.argtypes = [i64, ci, i64, i64, vp, i64, vp, vp, i64, vp]
    lib.gemm_moe_combine_bf16.restype = ci
    lib.gemm_moe_combine_bf16.argtypes = [i64, ci, i64, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp]
    lib.gemm_moe_combine_grad_bf16.restype = ci
    lib.gemm_moe_combine_grad_bf16.argtypes = [i64, ci, i64, i64, vp, i64, vp, i64, vp, vp, vp, i64,
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


def gemm_layernorm_bf16(rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean=None, rstd=None,
                        stream=0) -> int:
    return load().gemm_layernorm_bf16(rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean, rstd,
                                      stream)


def gemm_layernorm_f32(rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean=None, rstd=None,
                       stream=0) -> int:
    return load().gemm_layernorm_f32(rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean, rstd,
                                     stream)


def gemm_layernorm_grad_workspace_size(rows, cols) -> int:
    return load().gemm_layernorm_grad_workspace_size(rows, cols)


def gemm_layernorm_grad_bf16(rows, cols, X, ldx, weight, mean, rstd, dY, lddy, R, ldr, dX, lddx,
                             beta, dweight, dbias, workspace, workspace_bytes, stream=0) -> int:
    return load().gemm_layernorm_grad_bf16(rows, cols, X, ldx, weight, mean, rstd, dY, lddy, R, ldr,
                                           dX, lddx, beta, dweight, dbias, workspace,
                                           workspace_bytes, stream)


def gemm_layernorm_grad_f32(rows, cols, X, ldx, weight, mean, rstd, dY, lddy, R, ldr, dX, lddx,
                            beta, dweight, dbias, workspace, workspace_bytes, stream=0) -> int:
    return load().gemm_layernorm_grad_f32(rows, cols, X, ldx, weight, mean, rstd, dY, lddy, R, ldr,
                                          dX, lddx, beta, dweight, dbias, workspace,
                                          workspace_bytes, stream)


def gemm_dropout_bf16(rows, cols, p, rng, X, ldx, R, ldr, Y, ldy, stream=0) -> int:
    return load().gemm_dropout_bf16(rows, cols, p, rng, X, ldx, R, ldr, Y, ldy, stream)


def gemm_dropout_f32(rows, cols, p, rng, X, ldx, R, ldr, Y, ldy, stream=0) -> int:
    return load().gemm_dropout_f32(rows, cols, p, rng, X, ldx, R, ldr, Y, ldy, stream)


def gemm_moe_route_workspace_size(tokens, experts, k) -> int:
    return load().gemm_moe_route_workspace_size(tokens, experts, k)


def gemm_moe_route_bf16(tokens, experts, k, renormalize, logits, ldl, gates, choice, slots, offsets,
                        counts, loss, workspace, workspace_bytes, stream=0) -> int:
    return load().gemm_moe_route_bf16(tokens, experts, k, renormalize, logits, ldl, gates, choice,
                                      slots, offsets, counts, loss, workspace, workspace_bytes,
                                      stream)


def gemm_moe_route_f32(tokens, experts, k, renormalize, logits, ldl, gates, choice, slots, offsets,
                       counts, loss, workspace, workspace_bytes, stream=0) -> int:
    return load().gemm_moe_route_f32(tokens, experts, k, renormalize, logits, ldl, gates, choice,
                                     slots, offsets, counts, loss, workspace, workspace_bytes,
                                     stream)


def gemm_moe_route_grad_bf16(tokens, experts, k, renormalize, logits, ldl, choice, counts, dgates,
                             dloss, dlogits, lddl, stream=0) -> int:
    return load().gemm_moe_route_grad_bf16(tokens, experts, k, renormalize, logits, ldl, choice,
                                           counts, dgates, dloss, dlogits, lddl, stream)


def gemm_moe_route_grad_f32(tokens, experts, k, renormalize, logits, ldl, choice, counts, dgates,
                            dloss, dlogits, lddl, stream=0) -> int:
    return load().gemm_moe_route_grad_f32(tokens, experts, k, renormalize, logits, ldl, choice,
                                          counts, dgates, dloss, dlogits, lddl, stream)


def gemm_moe_gather_bf16(tokens, k, cols, rows, X, ldx, slots, Y, ldy, stream=0) -> int:
    return load().gemm_moe_gather_bf16(tokens, k, cols, rows, X, ldx, slots, Y, ldy, stream)


def gemm_moe_combine_bf16(tokens, k, cols, rows, Y, ldy, slots, gates, R, ldr, C, ldc,
                          stream=0) -> int:
    return load().gemm_moe_combine_bf16(tokens, k, cols, rows, Y, ldy, slots, gates, R, ldr, C, ldc,
                                        stream)


def gemm_moe_combine_grad_bf16(tokens, k, cols, rows, dC, lddc, Y, ldy, slots, gates, dY, lddy,
                               dgates, stream=0) -> int:
    return load().gemm_moe_combine_grad_bf16(tokens, k, cols, rows, dC, lddc, Y, ldy, slots, gates,
                                             dY, lddy, dgates, stream)


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


def _flat(name: str, t, dtypes, shape) -> None:
    """Check an operand that is held without gaps."""
    _want(name, t, dtypes, len(shape), shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _like(name: str, t, X) -> None:
    _want(name, t, (X.dtype,), 2, tuple(X.shape))


def _row_ld(t) -> int:
    return 0 if t is None else _ld2(t)


def layernorm(X, Y, weight=None, bias=None, eps: float = 1e-5, mean=None, rstd=None,
              stream=None) -> None:
    """Y <- (X - mean) rstd weight + bias for each row of X (bf16 or fp32;
    weight and bias of its type). mean and rstd (fp32, one a row) receive what
    layernorm_grad takes. Y may be X."""
    import torch
    _want("X", X, (torch.bfloat16, torch.float32), 2)
    _like("Y", Y, X)
    rows, cols = X.shape
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _want(name, t, (X.dtype,), 1, (cols,))
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is not None:
            _want(name, t, (torch.float32,), 1, (rows,))
    fn = gemm_layernorm_bf16 if X.dtype == torch.bfloat16 else gemm_layernorm_f32
    _check(fn(rows, cols, float(eps), X.data_ptr(), _ld2(X), _ptr(weight), _ptr(bias), Y.data_ptr(),
              _ld2(Y), _ptr(mean), _ptr(rstd), _stream_handle(stream)))


def layernorm_grad(X, dY, dX, mean, rstd, weight=None, R=None, dweight=None, dbias=None,
                   beta: float = 0.0, workspace=None, stream=None) -> None:
    """dX <- R + the norm's gradient; dweight, dbias (fp32) <- beta times
    themselves + their gradients, which needs a workspace (uint8, of
    gemm_layernorm_grad_workspace_size(rows, cols) values). dX may be dY or R."""
    import torch
    _want("X", X, (torch.bfloat16, torch.float32), 2)
    rows, cols = X.shape
    for name, t in (("dY", dY), ("dX", dX), ("R", R)):
        if t is not None:
            _like(name, t, X)
    for name, t in (("mean", mean), ("rstd", rstd)):
        _want(name, t, (torch.float32,), 1, (rows,))
    if weight is not None:
        _want("weight", weight, (X.dtype,), 1, (cols,))
    for name, t in (("dweight", dweight), ("dbias", dbias)):
        if t is not None:
            _want(name, t, (torch.float32,), 1, (cols,))
    if workspace is not None:
        _want("workspace", workspace, (torch.uint8,), 1)
    fn = gemm_layernorm_grad_bf16 if X.dtype == torch.bfloat16 else gemm_layernorm_grad_f32
    _check(fn(rows, cols, X.data_ptr(), _ld2(X), _ptr(weight), mean.data_ptr(), rstd.data_ptr(),
              dY.data_ptr(), _ld2(dY), _ptr(R), _row_ld(R), dX.data_ptr(), _ld2(dX), float(beta),
              _ptr(dweight), _ptr(dbias), _ptr(workspace),
              0 if workspace is None else workspace.numel(), _stream_handle(stream)))


def dropout(X, Y, p: float, rng, R=None, stream=None) -> None:
    """Y <- R + X dropped with probability p and the rest scaled by
    1 / (1 - p). rng: 2 int64 values on the GPU, the seed and an offset that
    the caller steps from draw to draw. The gradient is the same call on dY
    with the same rng. Y may be X or R."""
    import torch
    _want("X", X, (torch.bfloat16, torch.float32), 2)
    _like("Y", Y, X)
    if R is not None:
        _like("R", R, X)
    _want("rng", rng, (torch.int64, torch.uint64), 1, (2,))
    rows, cols = X.shape
    fn = gemm_dropout_bf16 if X.dtype == torch.bfloat16 else gemm_dropout_f32
    _check(fn(rows, cols, float(p), rng.data_ptr(), X.data_ptr(), _ld2(X), _ptr(R), _row_ld(R),
              Y.data_ptr(), _ld2(Y), _stream_handle(stream)))


def moe_route(logits, gates, choice, slots, offsets, counts, workspace, loss=None,
              renormalize: bool = True, stream=None) -> None:
    """The k experts of every token (logits: tokens x experts, bf16 or fp32),
    their gates, each choice's row among the rows sorted by expert, the
    experts' offsets there, their counts (and after them the tokens with a
    choice) and the balance loss. gates (fp32), choice and slots (int32) are
    tokens x k, offsets and counts experts + 1, workspace
    gemm_moe_route_workspace_size(tokens, experts, k) values of uint8."""
    import torch
    _want("logits", logits, (torch.bfloat16, torch.float32), 2)
    T, E = logits.shape
    _want("gates", gates, (torch.float32,), 2, (T, None))
    k = gates.shape[1]
    _flat("gates", gates, (torch.float32,), (T, k))
    for name, t, shape in (("choice", choice, (T, k)), ("slots", slots, (T, k)),
                           ("offsets", offsets, (E + 1,)), ("counts", counts, (E + 1,))):
        _flat(name, t, (torch.int32,), shape)
    _want("workspace", workspace, (torch.uint8,), 1)
    if loss is not None:
        _want("loss", loss, (torch.float32,), 1, (1,))
    fn = gemm_moe_route_bf16 if logits.dtype == torch.bfloat16 else gemm_moe_route_f32
    _check(fn(T, E, k, int(bool(renormalize)), logits.data_ptr(), _ld2(logits), gates.data_ptr(),
              choice.data_ptr(), slots.data_ptr(), offsets.data_ptr(), counts.data_ptr(), _ptr(loss),
              workspace.data_ptr(), workspace.numel(), _stream_handle(stream)))


def moe_route_grad(logits, choice, counts, dlogits, dgates=None, dloss=None,
                   renormalize: bool = True, stream=None) -> None:
    """dlogits <- the gradient of moe_route's gates and loss in its logits.
    dgates: tokens x k, dloss: one value, both fp32, or None for zero."""
    import torch
    _want("logits", logits, (torch.bfloat16, torch.float32), 2)
    T, E = logits.shape
    _like("dlogits", dlogits, logits)
    _want("choice", choice, (torch.int32,), 2, (T, None))
    k = choice.shape[1]
    _flat("choice", choice, (torch.int32,), (T, k))
    _flat("counts", counts, (torch.int32,), (E + 1,))
    if dgates is not None:
        _flat("dgates", dgates, (torch.float32,), (T, k))
    if dloss is not None:
        _want("dloss", dloss, (torch.float32,), 1, (1,))
    fn = gemm_moe_route_grad_bf16 if logits.dtype == torch.bfloat16 else gemm_moe_route_grad_f32
    _check(fn(T, E, k, int(bool(renormalize)), logits.data_ptr(), _ld2(logits), choice.data_ptr(),
              counts.data_ptr(), _ptr(dgates), _ptr(dloss), dlogits.data_ptr(), _ld2(dlogits),
              _stream_handle(stream)))


def _slots_of(slots, T: int) -> int:
    import torch
    _want("slots", slots, (torch.int32,), 2, (T, None))
    _flat("slots", slots, (torch.int32,), tuple(slots.shape))
    return slots.shape[1]


def moe_gather(X, slots, Y, stream=None) -> None:
    """Row slots[t, j] of Y <- row t of X, both bf16 (Y in the experts' order,
    what matmul_bf16_grouped takes)."""
    import torch
    bf16 = (torch.bfloat16,)
    _want("X", X, bf16, 2)
    T, cols = X.shape
    k = _slots_of(slots, T)
    _want("Y", Y, bf16, 2, (None, cols))
    _check(gemm_moe_gather_bf16(T, k, cols, Y.shape[0], X.data_ptr(), _ld2(X), slots.data_ptr(),
                                Y.data_ptr(), _ld2(Y), _stream_handle(stream)))


def moe_combine(Y, slots, C, gates=None, R=None, stream=None) -> None:
    """Row t of C <- row t of R + the sum over j of gates[t, j] (1 without
    gates: moe_gather's gradient) times row slots[t, j] of Y. C may be R."""
    import torch
    bf16 = (torch.bfloat16,)
    _want("C", C, bf16, 2)
    T, cols = C.shape
    k = _slots_of(slots, T)
    _want("Y", Y, bf16, 2, (None, cols))
    if gates is not None:
        _flat("gates", gates, (torch.float32,), (T, k))
    if R is not None:
        _like("R", R, C)
    _check(gemm_moe_combine_bf16(T, k, cols, Y.shape[0], Y.data_ptr(), _ld2(Y), slots.data_ptr(),
                                 _ptr(gates), _ptr(R), _row_ld(R), C.data_ptr(), _ld2(C),
                                 _stream_handle(stream)))


def moe_combine_grad(dC, slots, dY, Y=None, gates=None, dgates=None, stream=None) -> None:
    """moe_combine's gradients: row slots[t, j] of dY <- gates[t, j] times row t
    of dC, and dgates[t, j] <- the product of row t of dC and row slots[t, j] of
    Y (Y is needed for dgates alone). dY may be Y."""
    import torch
    bf16 = (torch.bfloat16,)
    _want("dC", dC, bf16, 2)
    T, cols = dC.shape
    k = _slots_of(slots, T)
    _want("dY", dY, bf16, 2, (None, cols))
    if dgates is not None:
        if Y is None:
            raise ValueError("dgates need Y")
        _want("Y", Y, bf16, 2, (dY.shape[0], cols))
        _flat("dgates", dgates, (torch.float32,), (T, k))
    if gates is not None:
        _flat("gates", gates, (torch.float32,), (T, k))
    _check(gemm_moe_combine_grad_bf16(T, k, cols, dY.shape[0], dC.data_ptr(), _ld2(dC),
                                      _ptr(Y) if dgates is not None else None,
                                      _row_ld(Y) if dgates is not None else 0, slots.data_ptr(),
                                      _ptr(gates), dY.data_ptr(), _ld2(dY), _ptr(dgates),
                                      _stream_handle(stream)))
