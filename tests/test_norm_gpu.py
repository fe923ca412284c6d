"""Layer norm and its gradients against plain 64-bit forms (layer_util)."""
import itertools

import numpy as np
import pytest
import torch

import dense_gemm_04_amd as dg
from layer_util import BF16, F32, norm_allow, norm_grad_allow, norm_grad_ref, norm_ref, worst
from ops_util import f64, gen, put, rows_of

pytestmark = pytest.mark.gpu

# Rows x cols: every width class of the kernels and its edges, few and many rows.
SIZES = [(1, 1), (5, 2), (3, 7), (300, 8), (7, 9), (1000, 63), (33, 64), (64, 129), (257, 255), (1030, 256), (3, 511),
         (129, 513), (2, 1000), (4095, 1023), (700, 1024), (1, 2048), (530, 2050), (16, 4096), (1025, 4095), (40, 4104),
         (9, 8191), (260, 8192), (3, 12288), (17, 16384), (5, 16392), (2, 32768), (300, 20001), (3, 70001),
         (70, 1500), (33, 3000), (40, 5000), (37, 6100), (19, 10000), (12, 22000), (6, 26000), (9, 30001)]


def note(text):
    print(text, flush=True)


def inputs(rows, cols, dtype, seed):
    g = gen(seed)
    size = torch.exp(torch.randn(cols, generator=g) * 0.5)
    x = (torch.randn(rows, cols, generator=g) * size + 0.3 * torch.randn(cols, generator=g)).to(dtype)
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(dtype)
    b = (0.3 * torch.randn(cols, generator=g)).to(dtype)
    return x, w, b


def place(t, dtype, ld, offset):
    buf, view = rows_of(t.shape[0], t.shape[1], dtype, ld, offset)
    put(view, t)
    return buf, view


def untouched(buf, rows, cols, ld, offset):
    """The bytes around a rows x cols view still hold every bit set."""
    inside = torch.zeros(buf.numel(), dtype=torch.bool, device="cuda")
    inside[offset:offset + rows * ld].view(rows, ld)[:, :cols] = True
    raw = buf.view(torch.int16 if buf.element_size() == 2 else torch.int32)
    return bool((raw[~inside] == -1).all())


def layout(cols, dtype, aligned):
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return (-(-cols // per) * per + per, 0) if aligned else (cols + 1, 1)


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm(rows, cols, dtype, aligned):
    note(f"norm {rows} x {cols} {dtype} aligned {aligned}")
    x, w, b = inputs(rows, cols, dtype, rows + cols)
    ld, off = layout(cols, dtype, aligned)
    _, xv = place(x, dtype, ld, off)
    ybuf, yv = rows_of(rows, cols, dtype, ld + 1 - aligned, off)
    mean, rstd = torch.full((rows + 1,), 7.0, device="cuda"), torch.full((rows + 1,), 7.0, device="cuda")
    dg.layernorm(xv, yv, w.cuda(), b.cuda(), 1e-5, mean[:rows], rstd[:rows])
    torch.cuda.synchronize()
    y, m, r = norm_ref(f64(x), f64(w), f64(b), 1e-5)
    ay, am, ar = norm_allow(f64(x), f64(w), f64(b), 1e-5, dtype)
    assert worst(yv, y, ay) <= 1
    assert worst(mean[:rows], m, am) <= 1 and worst(rstd[:rows], r, ar) <= 1
    assert mean[rows] == 7 and rstd[rows] == 7
    assert untouched(ybuf, rows, cols, ld + 1 - aligned, off)
    dg.layernorm(xv, xv, w.cuda(), b.cuda(), 1e-5)                     # in place: the same bits
    assert torch.equal(xv, yv)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_without_weight_bias_or_statistics(dtype):
    for (rows, cols), ww, bb in itertools.product([(37, 200), (9, 3000)], (True, False), (True, False)):
        x, w, b = inputs(rows, cols, dtype, 5)
        y = torch.empty(rows, cols, dtype=dtype, device="cuda")
        xc = x.cuda()
        dg.layernorm(xc, y, w.cuda() if ww else None, b.cuda() if bb else None, 1e-3)
        args = (f64(x), f64(w) if ww else None, f64(b) if bb else None, 1e-3)
        assert worst(y, norm_ref(*args)[0], norm_allow(*args, dtype)[0]) <= 1
        # In place, the same bits.
        dg.layernorm(xc, xc, w.cuda() if ww else None, b.cuda() if bb else None, 1e-3)
        assert torch.equal(xc, y)


def test_norm_far_from_zero():
    """Rows whose mean is 4096 times their spread: the differences are taken first."""
    g = gen(9)
    for cols in (100, 1024, 5000, 20000):
        x = torch.randn(6, cols, generator=g) + 4096.0
        y = torch.empty(6, cols, device="cuda")
        dg.layernorm(x.cuda(), y, eps=1e-6)
        args = (f64(x), None, None, 1e-6)
        assert worst(y, norm_ref(*args)[0], norm_allow(*args, F32)[0]) <= 1


@pytest.mark.parametrize("cols", [8, 600, 4096, 20000])
def test_norm_of_rows_that_are_not_finite(cols):
    x = torch.randn(6, cols, generator=gen(2))
    x[1, cols // 2] = float("nan")
    x[2, 0] = float("inf")
    x[3, cols - 1] = -float("inf")
    x[4] = 3.0                                    # constant: y = bias
    for dtype in (BF16, F32):
        y = torch.empty(6, cols, dtype=dtype, device="cuda")
        b = torch.randn(cols, generator=gen(3)).to(dtype)
        dg.layernorm(x.to(dtype).cuda(), y, None, b.cuda())
        y = y.cpu()
        assert bool(y[1:4].isnan().all()) and not bool(y[[0, 5]].isnan().any())
        assert torch.equal(y[4], b)
        dg.layernorm(x.to(dtype).cuda(), yy := torch.empty(6, cols, dtype=dtype, device="cuda"), None, None, 0.0)
        assert bool(yy.cpu()[4].isnan().all())


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm_grad(rows, cols, dtype, aligned):
    for res in (False, True):
        note(f"norm gradient {rows} x {cols} {dtype} aligned {aligned} residual {res}")
        run_grad(rows, cols, dtype, aligned, res=res, beta=0.5 if (cols % 3 == 0) == res else 0.0)


def run_grad(rows, cols, dtype, aligned, res, beta, use_w=True, wants=(True, True), alias=None):
    x, w, _ = inputs(rows, cols, dtype, 3 * rows + cols)
    g = gen(cols)
    dy = (torch.randn(rows, cols, generator=g) * 0.5 + 0.1).to(dtype)
    r0 = torch.randn(rows, cols, generator=g).to(dtype)
    _, m, r = norm_ref(f64(x), None, None, 1e-5)
    mean, rstd = torch.from_numpy(m).float(), torch.from_numpy(r).float()
    ld, off = layout(cols, dtype, aligned)
    _, xv = place(x, dtype, ld, off)
    dybuf, dyv = place(dy, dtype, ld, off)
    rbuf, rv = place(r0, dtype, ld, off)
    out, dxv = (dybuf, dyv) if alias == "dY" else (rbuf, rv) if alias == "R" else rows_of(rows, cols, dtype, ld, off)
    start = torch.randn(2, cols, generator=g)
    dwb = torch.full((2, cols + 1), 7.0, device="cuda")
    dwb[:, :cols] = start.cuda() if beta else float("nan")
    ws = torch.full((dg.gemm_layernorm_grad_workspace_size(rows, cols),), 0xff, dtype=torch.uint8, device="cuda")
    dg.layernorm_grad(xv, dyv, dxv, mean.cuda(), rstd.cuda(), w.cuda() if use_w else None, rv if res else None,
                      dwb[0, :cols] if wants[0] else None, dwb[1, :cols] if wants[1] else None, beta,
                      ws if any(wants) else None)
    torch.cuda.synchronize()
    args = (f64(x), f64(w) if use_w else None, f64(mean), f64(rstd), f64(dy), f64(r0) if res else None)
    dx, dw, db = norm_grad_ref(*args)
    adx, adw, adb = norm_grad_allow(*args, dtype)
    assert worst(dxv, dx, adx) <= 1
    for i, (want, allow) in enumerate(((dw, adw), (db, adb))):
        if wants[i]:
            base = beta * f64(start[i]) if beta else 0.0
            assert worst(dwb[i, :cols], want + base, allow + 2.0 ** -23 * (np.abs(want) + np.abs(base))) <= 1
    assert bool((dwb[:, cols] == 7).all())
    if alias is None:
        assert untouched(out, rows, cols, ld, off)
    return dxv, dwb


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_grad_forms(dtype):
    for rows, cols in ((37, 200), (9, 3000), (600, 520), (11, 20000), (70, 100), (2100, 1031), (300, 5001), (5, 40000)):
        note(f"norm gradient forms {rows} x {cols} {dtype}")
        run_grad(rows, cols, dtype, True, True, 0.0, use_w=False)
        run_grad(rows, cols, dtype, True, False, 1.0, wants=(True, False))
        run_grad(rows, cols, dtype, True, True, -2.0, wants=(False, True))
        run_grad(rows, cols, dtype, False, False, 0.0, wants=(False, False))
        run_grad(rows, cols, dtype, True, True, 0.0, alias="dY")
        run_grad(rows, cols, dtype, False, True, 1.0, alias="R")


def test_norm_grad_of_no_rows():
    ws = torch.empty(dg.gemm_layernorm_grad_workspace_size(0, 70), dtype=torch.uint8, device="cuda")
    empty = torch.empty(0, 70, device="cuda")
    none = torch.empty(0, device="cuda")
    for beta, want in ((0.0, 0.0), (0.5, 1.5), (1.0, 3.0)):
        dw, db = torch.full((70,), 3.0, device="cuda"), torch.full((70,), 3.0, device="cuda")
        if beta == 0.0:
            dw[3] = float("nan")                  # not read
        dg.layernorm_grad(empty, empty, empty, none, none, None, None, dw, db, beta, ws)
        assert bool((dw == want).all()) and bool((db == want).all())


def test_norm_grad_same_bits_twice():
    for rows, cols, dtype in ((1030, 4096, BF16), (333, 1000, F32)):
        one = run_grad(rows, cols, dtype, True, True, 0.5)
        two = run_grad(rows, cols, dtype, True, True, 0.5)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_norm_grad_against_differences():
    """The forward call's own fp32 results along a direction against the gradient call's."""
    g = gen(77)
    rows, cols = 24, 320
    x, w, b, dy = (torch.randn(*s, generator=g) for s in ((rows, cols), (cols,), (cols,), (rows, cols)))
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    y = torch.empty(rows, cols, device="cuda")
    dg.layernorm(x.cuda(), y, w.cuda(), b.cuda(), 1e-3, mean, rstd)
    dx, dw, db = torch.empty_like(y), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(dg.gemm_layernorm_grad_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    dg.layernorm_grad(x.cuda(), dy.cuda(), dx, mean, rstd, w.cuda(), None, dw, db, 0.0, ws)
    step = 2.0 ** -8
    for i, grad in enumerate((dx, dw, db)):
        d = torch.randn(grad.shape, generator=g)
        ends = []
        for s in (step, -step):
            v = [t + s * d if i == n else t for n, t in enumerate((x, w, b))]
            dg.layernorm(v[0].cuda(), y, v[1].cuda(), v[2].cuda(), 1e-3)
            ends.append((f64(y) * f64(dy)).sum())
        # Each y is off by a few fp32 steps of about 1, so the quotient by about
        # sqrt(rows cols) 2^-22 / step; the third derivative adds step^2 of it.
        size = np.sqrt(rows * cols)
        assert abs((ends[0] - ends[1]) / (2 * step) - (f64(grad) * f64(d)).sum()) < size * (8 * 2.0 ** -22 / step + 8 * step ** 2)


def test_norm_past_32_bits():
    """Rows whose byte offsets pass 2^32, read and written through the same kernels."""
    ld, rows, cols = 1 << 20, 2300, 96                   # 4.8 GB in bf16
    buf = torch.empty(rows, ld, dtype=BF16, device="cuda")
    x, w, b = inputs(rows, cols, BF16, 1)
    v = buf[:, :cols]
    v.copy_(x)
    y = buf[:, 128:128 + cols]
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dg.layernorm(v, y, w.cuda(), b.cuda(), 1e-5, mean, rstd)
    args = (f64(x), f64(w), f64(b), 1e-5)
    assert worst(y, norm_ref(*args)[0], norm_allow(*args, BF16)[0]) <= 1
    dx = buf[:, 256:256 + cols]
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(dg.gemm_layernorm_grad_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    dg.layernorm_grad(v, y, dx, mean, rstd, w.cuda(), None, dw, db, 0.0, ws)
    args = (f64(x), f64(w), f64(mean), f64(rstd), f64(y), None)
    for got, want, allow in zip((dx, dw, db), norm_grad_ref(*args), norm_grad_allow(*args, BF16)):
        assert worst(got, want, allow) <= 1


def test_norm_of_more_rows_than_one_launch_takes():
    """2^27 short rows and a few, in place; the ends and rows between against a call on them alone."""
    rows, cols = (1 << 27) + 5, 8
    part = torch.randn(1 << 20, cols, generator=gen(6)).to(BF16).cuda()
    x = part.repeat(rows // part.shape[0] + 1, 1)[:rows]
    rstd = torch.zeros(rows, device="cuda")
    w = torch.randn(cols, generator=gen(7)).to(BF16).cuda()
    alone, r = torch.empty_like(part), torch.empty(part.shape[0], device="cuda")
    dg.layernorm(part, alone, w, None, 1e-5, None, r)
    dg.layernorm(x, x, w, None, 1e-5, None, rstd)
    torch.cuda.synchronize()
    args = (f64(part[:1000]), f64(w), None, 1e-5)
    for lo in (0, 5 << 20, 127 << 20, rows - 1005):
        at = lo % part.shape[0]
        some = part[at:at + 1000] if at + 1000 <= part.shape[0] else None
        if some is None:                                  # across the repeats' border
            some = torch.cat([part[at:], part[:1000 - (part.shape[0] - at)]])
        args = (f64(some), f64(w), None, 1e-5)
        assert worst(x[lo:lo + 1000], norm_ref(*args)[0], norm_allow(*args, BF16)[0]) <= 1
        assert worst(rstd[lo:lo + 1000], norm_ref(*args)[2], norm_allow(*args, BF16)[2]) <= 1
    assert bool((rstd > 0).all())
