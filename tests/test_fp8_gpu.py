"""GPU tests of the e4m3 quantiser and the block-scaled product against plain
64-bit forms (ops_util), at the sizes, layouts, alignments and values where
they can go wrong."""
import numpy as np
import pytest
import torch

import dense_gemm_04_amd as dg
from gpu_util import note
from ops_util import (E4M3, close, f64, fp8_ref, gen, nearest_e4m3, put, quantize_ref, rows_of)

pytestmark = pytest.mark.gpu
INSTRUCTION = 2.0 ** -10


def quantize(x, op, block_rows, ldx=None, ldq=None, lds=None, offset=0):
    """One call; x: a CPU matrix. Returns (Q, S) as CUDA views and the whole
    buffers behind them, filled with ones in every bit beforehand."""
    rows, cols = x.shape
    r, k = (cols, rows) if op == dg.OP_T else (rows, cols)
    _, xv = rows_of(rows, cols, x.dtype, ldx, offset)
    put(xv, x)
    qbuf, q = rows_of(r, k, torch.uint8, ldq, offset)
    sbuf, s = rows_of(-(-k // 128), -(-r // block_rows), torch.float32, lds, offset)
    call = dg.gemm_fp8_quantize_bf16 if x.dtype == torch.bfloat16 else dg.gemm_fp8_quantize_f32
    st = call(op, block_rows, rows, cols, xv.data_ptr(), ldx or max(cols, 1), q.data_ptr(), ldq or max(k, 1),
              s.data_ptr(), lds or max(s.shape[1], 1))
    torch.cuda.synchronize()
    assert st == dg.GEMM_OK
    return q, s, qbuf, sbuf


def check_quantized(x, q, s, op, block_rows):
    want = f64(x.t() if op == dg.OP_T else x)
    v, scales = quantize_ref(want, block_rows)
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    got = f64(q)
    if x.dtype == torch.bfloat16:
        np.testing.assert_array_equal(got, nearest_e4m3(v))
    else:
        # fp32 input: the quotient is within 2^-23 of itself before it is
        # rounded, and 0.875 x within half of the smallest subnormal, 2^-150, of
        # a top of at least 448 * 2^-126 that is 512 / 448 as large.
        off = 2.0 ** -23 * np.abs(v) + 2.0 ** -150 * 512 / (448 * 2.0 ** -126)
        lo, hi = nearest_e4m3(np.clip(v - off, -448, 448)), nearest_e4m3(np.clip(v + off, -448, 448))
        assert np.all((got == lo) | (got == hi))


SIZES = [(1, 1), (1, 128), (3, 129), (130, 127), (128, 128), (257, 300), (16, 4104), (1000, 64), (300, 1031)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("op", [dg.OP_N, dg.OP_T])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("size", SIZES)
def test_quantize(size, block_rows, op, dtype):
    rows, cols = size
    note(f"quantize {size} op {op} block_rows {block_rows} {dtype}")
    g = gen(rows * 7 + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(1, cols, generator=g))
    x = x.to(dtype)
    q, s, _, _ = quantize(x, op, block_rows)
    check_quantized(x, q, s, op, block_rows)
    # 16-byte rows: the wide accesses.
    k = rows if op == dg.OP_T else cols
    ldx, ldq, lds = -(-cols // 8) * 8 + 8, -(-k // 16) * 16 + 16, s.shape[1] + 3
    q2, s2, qbuf, sbuf = quantize(x, op, block_rows, ldx, ldq, lds)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    # Nothing past a row's end is written.
    whole = qbuf[:q2.shape[0] * ldq].view(q2.shape[0], ldq)
    assert bool((whole[:, k:] == 0xff).all()) and bool((qbuf[q2.shape[0] * ldq:] == 0xff).all())
    assert bool(sbuf[:s2.shape[0] * lds].view(s2.shape[0], lds)[:, s2.shape[1]:].isnan().all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("op", [dg.OP_N, dg.OP_T])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_odd_base_and_strides(block_rows, op, dtype):
    x = torch.randn(131, 203, generator=gen(5)).to(dtype)
    k = 131 if op == dg.OP_T else 203
    q, s, _, _ = quantize(x, op, block_rows, 207, k + 2, 205, offset=1)
    check_quantized(x, q, s, op, block_rows)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("op", [dg.OP_N, dg.OP_T])
def test_quantize_extremes(op, dtype):
    """Zero blocks, blocks of subnormal and of the largest values, signed zeros."""
    x = torch.randn(6, 256, generator=gen(9))
    x[0] = 0
    x[1] *= 2.0 ** -130
    x[2] = torch.where(x[2] > 0, 3.3895313892515355e38, -1.7e38)
    x[3, :128] = 2.0 ** -133
    x[4] = -0.0
    x[5, 1:] *= 2.0 ** -60
    x = x.to(dtype)
    x = x.t().contiguous() if op == dg.OP_T else x
    q, s, _, _ = quantize(x, op, 1)
    check_quantized(x, q, s, op, 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("op", [dg.OP_N, dg.OP_T])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_marks_blocks_that_are_not_finite(block_rows, op, dtype):
    x = torch.randn(300, 300, generator=gen(11))
    x[5, 7], x[140, 250], x[299, 299] = float("inf"), float("nan"), float("-inf")
    x = x.to(dtype)
    q, s, _, _ = quantize(x.t().contiguous() if op == dg.OP_T else x, op, block_rows)
    bad = torch.zeros(3, 300, dtype=torch.bool)
    bad[0, 5] = bad[1, 140] = bad[2, 299] = True
    if block_rows == 128:
        bad = torch.stack([bad[:, i:i + 128].any(1) for i in range(0, 300, 128)], 1)
    assert torch.equal(s.cpu().isnan(), bad)
    each = bad.repeat_interleave(block_rows, 1)[:, :300].repeat_interleave(128, 0)[:300].t()
    assert bool((q.cpu()[each] == 0).all())
    clean = torch.where(each, torch.zeros(()), x.float()).to(dtype)
    v, _ = quantize_ref(f64(clean), block_rows)
    got, want = f64(q), nearest_e4m3(v)
    keep = ~each.numpy()
    if dtype == torch.bfloat16:
        np.testing.assert_array_equal(got[keep], want[keep])
    else:
        assert np.mean(got[keep] != want[keep]) < 1e-3


# ---- the product ----------------------------------------------------------------

def operands(M, N, K, b_rows, seed, lda=None, ldb=None, ldsa=None, ldsb=None, offset=0, kind="normal"):
    """Quantised operands (CPU reference values and CUDA views whose buffers hold
    NaN everywhere else)."""
    g = gen(seed)
    def one(rows, per):
        if kind == "bytes":
            q = torch.randint(0, 256, (rows, K), generator=g, dtype=torch.uint8)
            q[(q & 0x7f) == 0x7f] = 0x38
            s = torch.exp(torch.randn(-(-K // 128), -(-rows // per), generator=g))
            return q.view(E4M3), s
        if kind == "ints":
            q = torch.randint(-4, 5, (rows, K), generator=g).float().to(E4M3)
            s = torch.exp2(torch.randint(-2, 3, (-(-K // 128), -(-rows // per)), generator=g).float())
            return q, s
        x = torch.randn(rows, K, generator=g) * torch.exp(torch.randn(1, K, generator=g))
        v, s = quantize_ref(x.double().numpy(), per)
        return torch.from_numpy(nearest_e4m3(v)).float().to(E4M3), torch.from_numpy(np.ascontiguousarray(s))
    qa, sa = one(M, 1)
    qb, sb = one(N, b_rows)
    views = [put(rows_of(r, c, dt, ld, off)[1], v.view(torch.uint8) if dt == torch.uint8 else v)
             for r, c, dt, ld, off, v in ((M, K, torch.uint8, lda, offset, qa), (sa.shape[0], M, torch.float32, ldsa, offset, sa),
                                          (N, K, torch.uint8, ldb, offset, qb), (sb.shape[0], sb.shape[1], torch.float32, ldsb, offset, sb))]
    return (qa, sa, qb, sb), views


def ld_of(v):
    return max(v.stride(0), v.shape[1], 1)


def run_fp8(views, M, N, K, b_rows, alpha=1.0, beta=0.0, c0=None, bias=None, act=0, ldc=None, offset=0):
    a, sa, b, sb = views
    buf, c = rows_of(M, N, torch.bfloat16, ldc, offset)
    if c0 is not None:
        c.copy_(c0)
    before = buf.clone()
    bd = None if bias is None else bias.cuda()
    st = dg.gemm_fp8(M, N, K, alpha, a.data_ptr(), ld_of(a), sa.data_ptr(), ld_of(sa), b.data_ptr(), ld_of(b),
                     sb.data_ptr(), ld_of(sb), b_rows, beta, c.data_ptr(), ldc or max(N, 1),
                     None if bd is None else bd.data_ptr(), act)
    torch.cuda.synchronize()
    assert st == dg.GEMM_OK
    # Only C's own elements were written.
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[offset:offset + M * (ldc or max(N, 1))].view(M, -1)[:, :N] = False
    assert torch.equal(buf[mask].view(torch.int16), before[mask].view(torch.int16))
    return c


# M, N, K: single rows, ragged edges of every dimension, few and many tiles.
PRODUCTS = [(1, 1, 1), (1, 256, 128), (1, 4096, 1000), (7, 300, 129), (16, 512, 512), (17, 1024, 640), (33, 250, 384),
            (64, 2048, 256), (65, 640, 200), (100, 130, 127), (128, 128, 128), (130, 514, 1000), (257, 300, 260),
            (300, 1031, 400), (512, 768, 1152), (1000, 1500, 272), (2100, 1290, 144)]


@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("size", PRODUCTS)
def test_product(size, aligned, b_rows):
    M, N, K = size
    note(f"fp8 {size} b_rows {b_rows} aligned {aligned}")
    up = lambda v, s: -(-v // s) * s
    kw = dict(lda=up(K, 16) + 16, ldb=up(K, 16), ldsa=M + 5, ldsb=N + 3) if aligned else dict(lda=K + 3, ldb=K + 1, offset=1)
    cpu, views = operands(M, N, K, b_rows, 31 * M + N + K, **kw)
    c = run_fp8(views, M, N, K, b_rows, ldc=up(N, 8) + 8 if aligned else N + 1, offset=0 if aligned else 1)
    want, d = fp8_ref(f64(cpu[0]), f64(cpu[1]), f64(cpu[2]), f64(cpu[3]), b_rows)
    assert close(c, want, d, -(-K // 128), instruction=INSTRUCTION) <= 1


@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("size", [(5, 96, 300), (40, 512, 256), (300, 520, 400)])
@pytest.mark.parametrize("act,beta", [(dg.ACT_NONE, 1.0), (dg.ACT_RELU, 0.0), (dg.ACT_GELU_TANH, -0.5)])
def test_product_epilogue(act, beta, size, b_rows):
    M, N, K = size
    cpu, views = operands(M, N, K, b_rows, 3, lda=-(-K // 16) * 16, ldb=-(-K // 16) * 16)
    g = gen(4)
    c0 = torch.randn(M, N, generator=g).to(torch.bfloat16)
    bias = torch.randn(N, generator=g).to(torch.bfloat16)
    c = run_fp8(views, M, N, K, b_rows, 0.25, beta, c0.cuda() if beta else None, bias, act)
    want, d = fp8_ref(f64(cpu[0]), f64(cpu[1]), f64(cpu[2]), f64(cpu[3]), b_rows, 0.25, beta, f64(c0), f64(bias), act)
    assert close(c, want, d, -(-K // 128), instruction=INSTRUCTION) <= 1


@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("size", [(9, 200, 500), (120, 260, 1040), (600, 700, 384)])
def test_product_of_small_integers_is_exact(size, b_rows):
    """Products and sums of small integers with power-of-two scales are exact in
    fp32 whatever the order, so C is their one rounding to bf16."""
    M, N, K = size
    cpu, views = operands(M, N, K, b_rows, 77, lda=-(-K // 16) * 16, ldb=-(-K // 16) * 16, kind="ints")
    c = run_fp8(views, M, N, K, b_rows)
    want, _ = fp8_ref(f64(cpu[0]), f64(cpu[1]), f64(cpu[2]), f64(cpu[3]), b_rows)
    assert torch.equal(c.cpu(), torch.from_numpy(want).float().to(torch.bfloat16))


@pytest.mark.parametrize("size", [(12, 140, 700), (270, 390, 512)])
def test_product_of_any_bytes(size):
    M, N, K = size
    cpu, views = operands(M, N, K, 128, 15, lda=-(-K // 16) * 16, ldb=-(-K // 16) * 16, kind="bytes")
    c = run_fp8(views, M, N, K, 128)
    want, d = fp8_ref(f64(cpu[0]), f64(cpu[1]), f64(cpu[2]), f64(cpu[3]), 128)
    assert close(c, want, d, -(-K // 128), instruction=INSTRUCTION) <= 1


@pytest.mark.parametrize("size", [(16, 256, 512), (300, 512, 512)])
def test_nan_stays_in_its_rows_and_columns(size):
    M, N, K = size
    cpu, views = operands(M, N, K, 1, 21)
    clean = run_fp8(views, M, N, K, 1)
    views[1][2, 3] = float("nan")           # a scale of A's row 3
    views[2][17, 200] = 0x7f                # a byte of B's row 17
    c = run_fp8(views, M, N, K, 1).cpu()
    nan = c.isnan()
    assert bool(nan[3].all()) and bool(nan[:, 17].all())
    nan[3], nan[:, 17] = False, False
    assert not bool(nan.any())
    keep = torch.ones(M, N, dtype=torch.bool)
    keep[3], keep[:, 17] = False, False
    assert torch.equal(c[keep], clean.cpu()[keep])


def test_product_free_calls():
    cpu, views = operands(40, 96, 128, 128, 8)
    c0 = torch.randn(40, 96, generator=gen(1)).to(torch.bfloat16)
    bias = torch.randn(96, generator=gen(2)).to(torch.bfloat16)
    c = run_fp8(views, 40, 96, 128, 128, 0.0, 0.5, c0.cuda(), bias, dg.ACT_RELU)
    want = np.maximum(f64(bias), 0) + 0.5 * f64(c0)
    assert close(c, want, np.abs(want) + np.abs(f64(c0)), 2) <= 1
    _, c = rows_of(40, 96, torch.bfloat16)
    assert dg.gemm_fp8(40, 96, 0, 1.0, None, 1, None, 40, None, 1, None, 1, 128, 0.0, c.data_ptr(), 96) == dg.GEMM_OK
    torch.cuda.synchronize()
    assert bool((c == 0).all())


@pytest.mark.parametrize("size", [(4, 512, 512), (200, 1000, 1024), (1024, 2048, 256)])
def test_same_bits_on_streams_and_in_a_graph(size):
    """Two calls at once on two streams, and a captured call replayed with eager
    work in between, give the eager call's bits."""
    M, N, K = size
    _, views = operands(M, N, K, 128, 6)
    want = run_fp8(views, M, N, K, 128)
    a, sa, b, sb = views
    outs = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for o, st in zip(outs, streams):
        dg.matmul_fp8(a, sa, b, sb, o, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.matmul_fp8(a, sa, b, sb, outs[2])
    for _ in range(4):
        outs[2].fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[2], want)


def test_layer_forward_and_gradients():
    """y = x W^T, dX = dY W, dW = dY^T X in 8 bits, each operand quantised along
    the dimension its product sums over; every result is held to the product of
    the dequantised operands, and the whole to what 8 bits keep of the input."""
    T, O, I = 300, 520, 400
    g = gen(40)
    x = torch.randn(T, I, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(O, I, generator=g) / 20).to(torch.bfloat16).cuda()
    dy = torch.randn(T, O, generator=g).to(torch.bfloat16).cuda()

    def quant(m, op, per):
        r, k = (m.shape[1], m.shape[0]) if op == dg.OP_T else tuple(m.shape)
        q = rows_of(r, k, torch.uint8, -(-k // 16) * 16)[1]
        s = torch.empty(-(-k // 128), -(-r // per), device="cuda")
        dg.quantize_fp8(m, q, s, op, per)
        return q, s

    for (p, op_p), (q, op_q), per, exact in (((x, dg.OP_N), (w, dg.OP_N), 128, lambda: f64(x) @ f64(w).T),
                                             ((dy, dg.OP_N), (w, dg.OP_T), 128, lambda: f64(dy) @ f64(w)),
                                             ((dy, dg.OP_T), (x, dg.OP_T), 1, lambda: f64(dy).T @ f64(x))):
        a, sa = quant(p, op_p, 1)
        b, sb = quant(q, op_q, per)
        c = torch.empty(a.shape[0], b.shape[0], dtype=torch.bfloat16, device="cuda")
        dg.matmul_fp8(a, sa, b, sb, c, b_block_rows=per)
        want, d = fp8_ref(f64(a), f64(sa), f64(b), f64(sb), per)
        assert close(c, want, d, sa.shape[0], instruction=INSTRUCTION) <= 1
        # Each factor is off by at most 2^-4 of itself, or by half of e4m3's
        # smallest step (2^-10) of a scale of at most max / 448.
        full, top = exact(), float(np.abs(f64(p)).max() * np.abs(f64(q)).max())
        mags = fp8_ref(np.abs(f64(a)), f64(sa), np.abs(f64(b)), f64(sb), per)[0]
        assert np.all(np.abs(f64(c) - full) <= 0.15 * mags + a.shape[1] * top * 2.0 ** -17 + 2.0 ** -7 * np.abs(full))


# Many tiles: whole rounds of resident 256 x 256 tiles and a partly full one,
# with ragged edges in every dimension, whole tiles only, and one round.
MANY_TILES = [(5000, 4504, 272), (4352, 4096, 256), (2900, 3301, 400), (2048, 4096, 640)]


@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("size", MANY_TILES)
def test_product_of_many_tiles(size, b_rows):
    M, N, K = size
    note(f"fp8 {size} b_rows {b_rows}")
    up = -(-K // 16) * 16
    cpu, views = operands(M, N, K, b_rows, M + K, lda=up, ldb=up + 16)
    g = gen(M)
    c0, bias = torch.randn(M, N, generator=g).to(torch.bfloat16), torch.randn(N, generator=g).to(torch.bfloat16)
    ref = [f64(t) for t in cpu]
    for alpha, beta, act, with_bias in ((1.0, 0.0, dg.ACT_NONE, False), (0.5, -1.0, dg.ACT_RELU, True)):
        c = run_fp8(views, M, N, K, b_rows, alpha, beta, c0.cuda() if beta else None, bias if with_bias else None, act,
                    ldc=-(-N // 8) * 8)
        want, d = fp8_ref(*ref, b_rows, alpha, beta, f64(c0), f64(bias) if with_bias else None, act)
        assert close(c, want, d, -(-K // 128), instruction=INSTRUCTION) <= 1


# One case for each kernel and for the ragged forms of its pipeline.
CHECKED = [(16, 300, 1000, 128), (30, 8192, 400, 1), (200, 1000, 1040, 128), (500, 4096, 300, 1), (1000, 4100, 400, 128),
           (1500, 1500, 272, 1), (2100, 2050, 1000, 128), (4700, 4300, 272, 128), (4700, 4300, 272, 1)]


@pytest.mark.parametrize("check", ["poison", "sync"])
@pytest.mark.parametrize("case", CHECKED)
def test_lds_checking_builds_agree(case, check):
    """The builds that fill retired LDS stages with NaN and that complete every
    copy before the next read give the normal build's bits."""
    M, N, K, b_rows = case
    note(f"fp8 {check} {case}")
    lib = dg.load_check_build(check)
    up = -(-K // 16) * 16
    _, (a, sa, b, sb) = operands(M, N, K, b_rows, 9, lda=up, ldb=up)
    out = [torch.full((M, N + 4), float("nan"), dtype=torch.bfloat16, device="cuda")[:, :N] for _ in range(2)]
    for handle, c in zip((dg.load(), lib), out):
        st = handle.gemm_fp8(M, N, K, 1.0, a.data_ptr(), ld_of(a), sa.data_ptr(), ld_of(sa), b.data_ptr(), ld_of(b),
                             sb.data_ptr(), ld_of(sb), b_rows, 0.0, c.data_ptr(), c.stride(0), None, 0, None)
        torch.cuda.synchronize()
        assert st == dg.GEMM_OK
    assert torch.equal(out[0], out[1])


def test_conveniences_refuse():
    q = torch.zeros(64, 256, dtype=torch.uint8, device="cuda")
    s, s2 = torch.ones(2, 64, device="cuda"), torch.ones(2, 1, device="cuda")
    c = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(64, 256, dtype=torch.bfloat16, device="cuda")
    dg.matmul_fp8(q, s, q, s2, c)
    dg.quantize_fp8(x, q, s)
    for bad in (lambda: dg.matmul_fp8(q, s[:, :63], q, s2, c), lambda: dg.matmul_fp8(q, s, q[:, :200], s2, c),
                lambda: dg.matmul_fp8(q, s, q, s, c), lambda: dg.matmul_fp8(q, s, q, s2, c[:, :32]),
                lambda: dg.matmul_fp8(q.t(), s, q, s2, c), lambda: dg.matmul_fp8(q[:1].expand(64, 256), s, q, s2, c),
                lambda: dg.quantize_fp8(x, q, s[:1]), lambda: dg.quantize_fp8(x, q, s, dg.OP_T),
                lambda: dg.matmul_fp8(q, s, q, s2, c, bias=c[0, :3])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: dg.matmul_fp8(x, s, q, s2, c), lambda: dg.matmul_fp8(q, s.double(), q, s2, c),
                lambda: dg.matmul_fp8(q, s, q, s2, c.float()), lambda: dg.quantize_fp8(x.half(), q, s)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(dg.GemmError):
        dg.matmul_fp8(q, s, q, torch.ones(2, 32, device="cuda"), c, b_block_rows=2)
    with pytest.raises(dg.GemmError):
        dg.matmul_fp8(q, s, q, s2, c, act=9)
