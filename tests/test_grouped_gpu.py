"""GPU tests of the products grouped by expert and of their weight gradients
against plain 64-bit forms (ops_util)."""
import numpy as np
import pytest
import torch

import dense_gemm_04_amd as dg
from gpu_util import note
from ops_util import close, f64, gen, grouped_ref, put, rows_of, wgrad_ref

pytestmark = pytest.mark.gpu


def offsets_of(lengths, first=0):
    return np.concatenate([[first], first + np.cumsum(lengths)]).astype(np.int32)


def up(v, s):
    return -(-v // s) * s


def normal(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def run_grouped(A, B, tb, off, C0, aligned=True, alpha=1.0, beta=0.0, row_scale=None, bias=None, act=0, M=None):
    """One call on padded copies; every element outside the operands is NaN and
    must not reach C. Returns C (all M rows)."""
    M, K = A.shape
    E, N = B.shape[0], B.shape[1] if tb else B.shape[2]
    r, c = (N, K) if tb else (K, N)
    pad = (lambda v: up(v, 8) + 8) if aligned else (lambda v: v + 1)
    offset = 0 if aligned else 1
    _, a = rows_of(M, K, torch.bfloat16, pad(K), offset)
    put(a, A)
    ldb = pad(c)
    per = r * ldb + (8 if aligned else 3)
    bbuf = torch.full((E * per + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        bbuf[offset + e * per: offset + e * per + r * ldb].view(r, ldb)[:, :c].copy_(B[e])
    ldc = pad(N)
    cbuf, cv = rows_of(M, N, torch.bfloat16, ldc, offset)
    put(cv, C0)
    before = cbuf.clone()
    offs = torch.from_numpy(off).cuda()
    keep = [t.cuda() if t is not None else None for t in (row_scale, bias)]
    st = dg.gemm_bf16_grouped(dg.OP_T if tb else dg.OP_N, E, M, N, K, alpha, a.data_ptr(), pad(K),
                              bbuf.data_ptr() + 2 * offset, ldb, per, beta, cv.data_ptr(), ldc, offs.data_ptr(),
                              None if row_scale is None else keep[0].data_ptr(),
                              None if bias is None else keep[1].data_ptr(), 0 if bias is None else bias.stride(0), act)
    torch.cuda.synchronize()
    assert st == dg.GEMM_OK
    mask = torch.ones_like(cbuf, dtype=torch.bool)
    mask[offset:offset + M * ldc].view(M, ldc)[:, :N] = False
    assert torch.equal(cbuf[mask].view(torch.int16), before[mask].view(torch.int16))
    # Rows outside all groups keep their bits.
    out = np.ones(M, dtype=bool)
    out[int(off[0]):int(off[-1])] = False
    rows = torch.from_numpy(np.flatnonzero(out))
    assert torch.equal(cv.cpu()[rows].view(torch.int16), C0[rows].view(torch.int16))
    return cv


# lengths of the groups, first row, rows behind the last group, N, K
LAYOUTS = {
    "one row": ([1], 0, 0, 64, 64),
    "one row, odd": ([1], 0, 0, 1, 1),
    "decode": ([0, 2, 1, 0, 0, 5, 1, 3, 16, 0, 1, 0], 0, 3, 520, 512),
    "decode wide": ([3, 0, 1, 4], 2, 1, 2048, 2056),
    "seventeen": ([17, 15, 33, 1], 0, 0, 264, 200),
    "all empty": ([0, 0, 0], 4, 6, 96, 72),
    "tile edges": ([64, 128, 256, 0, 63, 65, 257, 1], 5, 7, 300, 328),
    "many groups": ([int(v) for v in np.random.default_rng(3).integers(0, 12, 150)], 0, 9, 136, 64),
    "large": ([700, 0, 1300, 37, 600], 0, 20, 776, 520),
    "large, one": ([2000], 0, 0, 1100, 1032),
    "ragged": ([33, 100, 7], 1, 1, 131, 77),
}


def case(name, tb, seed):
    lengths, first, spare, N, K = LAYOUTS[name]
    g = gen(seed)
    M = first + sum(lengths) + spare
    A, B = normal(g, M, K), normal(g, len(lengths), *((N, K) if tb else (K, N)))
    return A, B, offsets_of(lengths, first), normal(g, M, N)


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("name", list(LAYOUTS))
def test_grouped(name, aligned, tb):
    note(f"grouped {name} tb {tb} aligned {aligned}")
    A, B, off, C0 = case(name, tb, 100 + len(name))
    c = run_grouped(A, B, tb, off, C0, aligned)
    want, d = grouped_ref(f64(A), f64(B), tb, off, f64(C0))
    assert close(c, want, d, A.shape[1]) <= 1


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("name", ["decode", "seventeen", "tile edges", "large"])
@pytest.mark.parametrize("act,beta", [(dg.ACT_NONE, 1.0), (dg.ACT_RELU, 0.0), (dg.ACT_GELU_TANH, -0.5)])
def test_grouped_epilogue(act, beta, name, tb):
    A, B, off, C0 = case(name, tb, 7)
    g = gen(8)
    scale = torch.rand(A.shape[0], generator=g) * 2 - 0.5
    bias = normal(g, B.shape[0], C0.shape[1] + 3)[:, :C0.shape[1]]
    bias_rows = torch.empty(B.shape[0], C0.shape[1] + 3, dtype=torch.bfloat16)[:, :C0.shape[1]]
    bias_rows.copy_(bias)
    wide = torch.zeros(B.shape[0], C0.shape[1] + 3, dtype=torch.bfloat16)
    wide[:, :C0.shape[1]] = bias
    c = run_grouped(A, B, tb, off, C0, True, 0.5, beta, scale, wide, act)
    want, d = grouped_ref(f64(A), f64(B), tb, off, f64(C0), 0.5, beta, f64(scale), f64(bias), act)
    assert close(c, want, d, A.shape[1]) <= 1


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("name", ["decode", "tile edges", "large"])
def test_grouped_small_integers_are_exact(name, aligned):
    lengths, first, spare, N, K = LAYOUTS[name]
    g = gen(60)
    M = first + sum(lengths) + spare
    ints = lambda *s: torch.randint(-4, 5, s, generator=g).to(torch.bfloat16)
    A, B, C0, off = ints(M, K), ints(len(lengths), K, N), ints(M, N), offsets_of(lengths, first)
    c = run_grouped(A, B, False, off, C0, aligned, beta=2.0)
    want, _ = grouped_ref(f64(A), f64(B), False, off, f64(C0), beta=2.0)
    inside = slice(int(off[0]), int(off[-1]))
    assert torch.equal(c.cpu()[inside], torch.from_numpy(want[inside]).float().to(torch.bfloat16))


def test_grouped_product_free_calls():
    A, B, off, C0 = case("tile edges", False, 5)
    bias = normal(gen(6), B.shape[0], C0.shape[1])
    c = run_grouped(A, B, False, off, C0, True, alpha=0.0, beta=0.5, bias=bias, act=dg.ACT_RELU)
    want, d = grouped_ref(0 * f64(A), 0 * f64(B), False, off, f64(C0), 1.0, 0.5, None, f64(bias), dg.ACT_RELU)
    assert close(c, want, d, 2) <= 1
    # K == 0: C <- 0 in the groups' rows; beta == 1 then leaves C alone.
    _, c = rows_of(8, 40, torch.bfloat16, fill=3.0)
    o = torch.tensor([1, 4, 7], dtype=torch.int32, device="cuda")
    for beta, inside in ((1.0, 3.0), (0.0, 0.0)):
        st = dg.gemm_bf16_grouped(dg.OP_N, 2, 8, 40, 0, 1.0, None, 1, None, 40, 0, beta, c.data_ptr(), 40, o.data_ptr())
        torch.cuda.synchronize()
        assert st == dg.GEMM_OK
        assert bool((c[1:7] == inside).all()) and bool((c[0] == 3).all()) and bool((c[7] == 3).all())


def test_grouped_shared_matrix():
    A, B, off, C0 = case("tile edges", False, 12)
    one = B[:1].expand(B.shape[0], -1, -1)
    a, b, c = A.cuda(), B[:1].cuda().expand(B.shape[0], -1, -1), C0.cuda()
    dg.matmul_bf16_grouped(a, b, c, torch.from_numpy(off).cuda())
    want, d = grouped_ref(f64(A), f64(one.contiguous()), False, off, f64(C0))
    assert close(c, want, d, A.shape[1]) <= 1


@pytest.mark.parametrize("M", [300, 3000])
def test_offsets_that_break_the_rule_stay_inside(M):
    """Offsets below zero, past M and falling: the kernels cut every group to
    [0, M), so nothing outside C's rows is touched."""
    g = gen(2)
    off = np.array([-50, 40, 20, M + 1000, M + 7, 10, 2 ** 31 - 1], dtype=np.int32)
    A, B = normal(g, M, 64), normal(g, 6, 64, 72)
    a, b, offs = A.cuda(), B.cuda(), torch.from_numpy(off).cuda()
    buf = torch.full((M + 600, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    dg.matmul_bf16_grouped(a, b, buf[300:300 + M], offs)
    dw = torch.full((8, 64, 72), 5.0, device="cuda")
    dg.grouped_wgrad(a, buf[300:300 + M], dw[1:7], offs)
    torch.cuda.synchronize()
    assert bool((buf[:300] == 5).all()) and bool((buf[300 + M:] == 5).all())
    assert bool((dw[0] == 5).all()) and bool((dw[7] == 5).all())


# ---- weight gradients -----------------------------------------------------------

def run_wgrad(X, dY, off, dtype, aligned=True, alpha=1.0, beta=0.0, dW0=None):
    M, K = X.shape
    N, E = dY.shape[1], len(off) - 1
    pad = (lambda v: up(v, 8) + 8) if aligned else (lambda v: v + 1)
    offset = 0 if aligned else 1
    # Rows outside the groups are NaN: they must not be read into any sum.
    x, dy = X.clone(), dY.clone()
    out = np.ones(M, dtype=bool)
    out[int(off[0]):int(off[-1])] = False
    x[torch.from_numpy(out)] = float("nan")
    dy[torch.from_numpy(out)] = float("nan")
    _, xv = rows_of(M, K, torch.bfloat16, pad(K), offset)
    _, yv = rows_of(M, N, torch.bfloat16, pad(N), offset)
    put(xv, x), put(yv, dy)
    ldw = pad(N)
    per = K * ldw + (8 if aligned else 5)
    wbuf = torch.full((E * per + 64,), float("nan"), dtype=dtype, device="cuda")
    views = [wbuf[offset + e * per: offset + e * per + K * ldw].view(K, ldw)[:, :N] for e in range(E)]
    inside = torch.zeros_like(wbuf, dtype=torch.bool)
    for e in range(E):
        inside[offset + e * per: offset + e * per + K * ldw].view(K, ldw)[:, :N] = True
        if dW0 is not None:
            views[e].copy_(dW0[e])
    offs = torch.from_numpy(off).cuda()
    fn = dg.gemm_bf16_grouped_wgrad_f32 if dtype == torch.float32 else dg.gemm_bf16_grouped_wgrad
    st = fn(E, M, N, K, alpha, xv.data_ptr(), pad(K), yv.data_ptr(), pad(N), beta,
            wbuf.data_ptr() + offset * wbuf.element_size(), ldw, per, offs.data_ptr())
    torch.cuda.synchronize()
    assert st == dg.GEMM_OK
    assert bool(wbuf[~inside].isnan().all())
    return torch.stack(views)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("name", list(LAYOUTS))
def test_wgrad(name, aligned, dtype):
    note(f"wgrad {name} {dtype} aligned {aligned}")
    lengths, first, spare, N, K = LAYOUTS[name]
    g = gen(len(name))
    M = first + sum(lengths) + spare
    X, dY, off = normal(g, M, K), normal(g, M, N), offsets_of(lengths, first)
    dw = run_wgrad(X, dY, off, dtype, aligned)
    want, d = wgrad_ref(f64(X), f64(dY), off)
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    assert close(dw, want, d, max(lengths), step) <= 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", ["decode", "tile edges", "large", "all empty"])
def test_wgrad_accumulates(name, dtype):
    lengths, first, spare, N, K = LAYOUTS[name]
    g = gen(90)
    M = first + sum(lengths) + spare
    X, dY, off = normal(g, M, K), normal(g, M, N), offsets_of(lengths, first)
    dW0 = torch.randn(len(lengths), K, N, generator=g).to(dtype)
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    for alpha, beta in ((0.5, 1.0), (1.0, -0.25), (0.0, 0.5)):
        dw = run_wgrad(X, dY, off, dtype, True, alpha, beta, dW0)
        want, d = wgrad_ref(f64(X), f64(dY), off, alpha, beta, f64(dW0))
        assert close(dw, want, d, max(lengths) + 1, step) <= 1


def test_bias_gradient_is_a_column_of_ones():
    lengths, first, spare, N, _ = LAYOUTS["tile edges"]
    M, off = first + sum(lengths) + spare, offsets_of(lengths, first)
    dY = normal(gen(17), M, N)
    db = run_wgrad(torch.ones(M, 1, dtype=torch.bfloat16), dY, off, torch.float32)
    want, d = wgrad_ref(np.ones((M, 1)), f64(dY), off)
    assert close(db, want, d, max(lengths), 2.0 ** -24) <= 1


@pytest.mark.parametrize("lengths", [[3, 0, 20, 9], [300, 0, 170, 400]])
def test_layer_forward_and_gradients(lengths):
    """An expert layer's product and both gradients, as a training step calls
    them, against the formulas and against differences of the loss sum(G * Y),
    which is linear in X and in W: L(W + D) - L(W) = <dW, D> up to the rounding
    of dW (and of dX) to its own type."""
    E, N, K = len(lengths), 264, 136
    g = gen(50)
    M, off = sum(lengths), offsets_of(lengths)
    X, W, G = normal(g, M, K), normal(g, E, K, N), normal(g, M, N)
    x, w, dy, offs = X.cuda(), W.cuda(), G.cuda(), torch.from_numpy(off).cuda()
    y, dx = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    dw = torch.empty(E, K, N, device="cuda")
    dg.matmul_bf16_grouped(x, w, y, offs)
    dg.matmul_bf16_grouped(dy, w, dx, offs, opb=dg.OP_T)
    dg.grouped_wgrad(x, dy, dw, offs)
    want, d = grouped_ref(f64(X), f64(W), False, off, np.zeros((M, N)))
    assert close(y, want, d, K) <= 1
    want, d = grouped_ref(f64(G), f64(W), True, off, np.zeros((M, K)))
    assert close(dx, want, d, N) <= 1
    want, d = wgrad_ref(f64(X), f64(G), off)
    assert close(dw, want, d, max(lengths), 2.0 ** -24) <= 1
    loss = lambda a, b: float(np.sum(f64(G) * grouped_ref(a, b, False, off, np.zeros((M, N)))[0]))
    DW, DX = f64(normal(g, E, K, N)), f64(normal(g, M, K))
    base = loss(f64(X), f64(W))
    slack = np.sum(np.abs(f64(dw) * DW)) * 2.0 ** -14
    assert abs(loss(f64(X), f64(W) + DW) - base - np.sum(f64(dw) * DW)) <= slack
    slack = np.sum(np.abs(f64(dx) * DX)) * 2.0 ** -8 + 1e-3
    assert abs(loss(f64(X) + DX, f64(W)) - base - np.sum(f64(dx) * DX)) <= slack


@pytest.mark.parametrize("lengths", [[3, 0, 20, 9], [300, 0, 170, 400]])
def test_captured_calls_follow_the_offsets(lengths):
    """A captured step replayed after its offsets and inputs change gives the
    eager call's bits for the new ones; two streams at once give them too."""
    E, N, K = len(lengths), 520, 264
    g = gen(51)
    M, off = sum(lengths), offsets_of(lengths)
    x, w, dy = normal(g, M, K).cuda(), normal(g, E, K, N).cuda(), normal(g, M, N).cuda()
    offs = torch.from_numpy(off).cuda()
    y, dx, dw = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(x), torch.zeros(E, K, N, device="cuda")

    def step(y, dx, dw, stream=None):
        dg.matmul_bf16_grouped(x, w, y, offs, stream=stream)
        dg.matmul_bf16_grouped(dy, w, dx, offs, opb=dg.OP_T, stream=stream)
        dg.grouped_wgrad(x, dy, dw, offs, stream=stream)

    step(y, dx, dw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(y, dx, dw)
    for k in range(3):
        x.copy_(normal(g, M, K))
        offs.copy_(torch.from_numpy(offsets_of(np.roll(lengths, k))))
        want = [torch.full_like(t, 7.0) for t in (y, dx, dw)]
        both = [[torch.full_like(t, 7.0) for t in (y, dx, dw)] for _ in range(2)]
        step(*want)
        for t in (y, dx, dw):
            t.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for st, o in zip(streams, both):
            step(*o, stream=st)
        torch.cuda.synchronize()
        for t, u in zip((y, dx, dw), want):
            assert torch.equal(t, u)
        for o in both:
            assert all(torch.equal(t, u) for t, u in zip(o, want))


# Sizes that fill the GPU with 256 x 256 tiles: several rounds, ragged rows,
# columns and depth; the last with columns that fill no whole vector.
MANY_TILES = [([2500, 0, 1300, 37, 2163], 4096, 1032), ([4000, 2000], 4104, 1000), ([3000, 1999], 5003, 904)]


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("lengths,N,K", MANY_TILES)
def test_grouped_many_tiles(lengths, N, K, tb):
    note(f"grouped many tiles {lengths} {N} {K} tb {tb}")
    g = gen(N)
    M, E = sum(lengths) + 7, len(lengths)
    A, B = normal(g, M, K), normal(g, E, *((N, K) if tb else (K, N)))
    C0, off, bias = normal(g, M, N), offsets_of(lengths, 3), normal(g, E, N)
    scale = torch.rand(M, generator=g) + 0.5
    c = run_grouped(A, B, tb, off, C0, True)
    want, d = grouped_ref(f64(A), f64(B), tb, off, f64(C0))
    assert close(c, want, d, K) <= 1
    c = run_grouped(A, B, tb, off, C0, True, 1.0, 0.5, scale, bias, dg.ACT_RELU)
    s = f64(scale)[:, None]
    rows = slice(3, 3 + sum(lengths))
    group = np.repeat(np.arange(E), lengths)
    z = want[rows] * s[rows] + f64(bias)[group]
    full, mags = np.array(f64(C0)), np.zeros_like(d)
    full[rows] = np.maximum(z, 0) + 0.5 * f64(C0)[rows]
    mags[rows] = d[rows] * s[rows] + np.abs(f64(bias)[group]) + 0.5 * np.abs(f64(C0)[rows])
    assert close(c, full, mags, K) <= 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lengths,N,K", [([300, 0, 63, 1, 129, 107], 2304, 2304), ([700, 0, 1400], 2051, 2100)])
def test_wgrad_many_tiles(lengths, N, K, dtype):
    note(f"wgrad many tiles {lengths} {N} {K} {dtype}")
    g = gen(K)
    M, off = sum(lengths) + 5, offsets_of(lengths, 2)
    X, dY = normal(g, M, K), normal(g, M, N)
    want, d = wgrad_ref(f64(X), f64(dY), off)
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    dw = run_wgrad(X, dY, off, dtype)
    assert close(dw, want, d, max(lengths), step) <= 1
    dW0 = torch.randn(len(lengths), K, N, generator=g).to(dtype)
    dw = run_wgrad(X, dY, off, dtype, True, 1.0, 1.0, dW0)
    w0 = f64(dW0)
    assert close(dw, want + w0, d + np.abs(w0), max(lengths) + 1, step) <= 1


@pytest.mark.parametrize("many", [False, True])
def test_more_groups_than_lanes(many):
    """130 groups, with few rows each and with enough for the tiled kernels."""
    rng = np.random.default_rng(8)
    lengths = [int(v) for v in (rng.integers(0, 90, 130) if many else rng.integers(0, 4, 130))]
    g = gen(70)
    M, E, N, K = sum(lengths), 130, 200, 136
    A, B, off, C0 = normal(g, M, K), normal(g, E, K, N), offsets_of(lengths), normal(g, M, N)
    c = run_grouped(A, B, False, off, C0)
    want, d = grouped_ref(f64(A), f64(B), False, off, f64(C0))
    assert close(c, want, d, K) <= 1
    dY = normal(g, M, N)
    dw = run_wgrad(A, dY, off, torch.float32)
    want, d = wgrad_ref(f64(A), f64(dY), off)
    assert close(dw, want, d, max(lengths), 2.0 ** -24) <= 1


@pytest.mark.parametrize("lengths", [[0, 6000, 0, 0], [2000, 2000, 2000], [1, 1, 6000, 1], [700] * 9])
def test_skewed_and_equal_groups(lengths):
    """Orders of groups by length: one that holds all rows, equal ones (ties),
    and single rows beside a long one."""
    g = gen(71)
    M, E, N, K = sum(lengths), len(lengths), 264, 200
    A, dY, off = normal(g, M, K), normal(g, M, N), offsets_of(lengths)
    dw = run_wgrad(A, dY, off, torch.float32)
    want, d = wgrad_ref(f64(A), f64(dY), off)
    assert close(dw, want, d, max(lengths), 2.0 ** -24) <= 1
    B, C0 = normal(g, E, K, N), normal(g, M, N)
    c = run_grouped(A, B, False, off, C0)
    want, d = grouped_ref(f64(A), f64(B), False, off, f64(C0))
    assert close(c, want, d, K) <= 1


CHECKED = [([3, 0, 1, 4], 520, 1000), ([20, 33, 0, 11], 520, 328), ([700, 0, 300, 9], 776, 520), ([64, 130, 200, 0], 300, 264),
           ([2500, 0, 1300, 2163], 4096, 200)]


@pytest.mark.parametrize("check", ["poison", "sync"])
@pytest.mark.parametrize("lengths,N,K", CHECKED)
def test_lds_checking_builds_agree(lengths, N, K, check):
    note(f"grouped {check} {lengths} {N} {K}")
    g = gen(80)
    M, E = sum(lengths), len(lengths)
    x, dy = normal(g, M, K).cuda(), normal(g, M, N).cuda()
    offs = torch.from_numpy(offsets_of(lengths)).cuda()
    out = []
    for handle in (dg.load(), dg.load_check_build(check)):
        for tb in (False, True):
            w = normal(gen(81), E, *((N, K) if tb else (K, N))).cuda()
            y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
            assert handle.gemm_bf16_grouped(int(tb), E, M, N, K, 1.0, x.data_ptr(), K, w.data_ptr(), w.stride(1), w.stride(0),
                                            0.0, y.data_ptr(), N, offs.data_ptr(), None, None, 0, 0, None) == dg.GEMM_OK
            torch.cuda.synchronize()
            out.append(y)
        for dtype, fn in ((torch.float32, handle.gemm_bf16_grouped_wgrad_f32), (torch.bfloat16, handle.gemm_bf16_grouped_wgrad)):
            dw = torch.full((E, K, N), float("nan"), dtype=dtype, device="cuda")
            assert fn(E, M, N, K, 1.0, x.data_ptr(), K, dy.data_ptr(), N, 0.0, dw.data_ptr(), N, K * N, offs.data_ptr(),
                      None) == dg.GEMM_OK
            torch.cuda.synchronize()
            out.append(dw)
    for a, b in zip(out[:4], out[4:]):
        assert torch.equal(a, b)


def test_conveniences_refuse():
    x = torch.zeros(64, 32, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(4, 32, 48, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(64, 48, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(5, dtype=torch.int32, device="cuda")
    dg.matmul_bf16_grouped(x, w, y, o)
    dg.grouped_wgrad(x, y, w, o)
    for bad in (lambda: dg.matmul_bf16_grouped(x, w, y, o[:4]), lambda: dg.matmul_bf16_grouped(x, w, y, o, opb=dg.OP_T),
                lambda: dg.matmul_bf16_grouped(x[:, :31], w, y, o), lambda: dg.matmul_bf16_grouped(x, w, y[:63], o),
                lambda: dg.matmul_bf16_grouped(x, w.transpose(1, 2), y, o),
                lambda: dg.matmul_bf16_grouped(x, w, y, o, row_scale=torch.ones(63, device="cuda")),
                lambda: dg.matmul_bf16_grouped(x, w, y, o, bias=y[:3]), lambda: dg.grouped_wgrad(x, y[:63], w, o),
                lambda: dg.grouped_wgrad(x[:1].expand(64, 32), y, w, o), lambda: dg.grouped_wgrad(x, y, w[:, :31], o)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: dg.matmul_bf16_grouped(x, w, y, o.long()), lambda: dg.matmul_bf16_grouped(x.float(), w, y, o),
                lambda: dg.grouped_wgrad(x, y, w.half(), o)):
        with pytest.raises(TypeError):
            bad()
    # One gradient matrix for all groups: they would overwrite each other.
    with pytest.raises(dg.GemmError):
        dg.grouped_wgrad(x, y, w[:1].expand(4, -1, -1), o)
