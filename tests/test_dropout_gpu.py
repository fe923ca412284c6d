"""Dropout against the generator in 64-bit integers (layer_util)."""
import numpy as np
import pytest
import torch

import dense_gemm_04_amd as dg
from layer_util import BF16, F32, STEP, U, dropout_ref, philox, worst
from ops_util import f64, gen
from test_norm_gpu import layout, note, place, rows_of, untouched

pytestmark = pytest.mark.gpu

SEED, OFFSET = -0x123456789ABCDEF, 0x7000000012345


def rng(seed=SEED, offset=OFFSET):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def allow(x, res, want, p, dtype):
    return (STEP[dtype] + U) * np.abs(want) + 2 * U * (np.abs(x) / max(1 - p, 2.0 ** -16) + (0 if res is None else np.abs(res)))


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols,p", [(1, 1, 0.5), (3, 7, 0.1), (300, 8, 0.25), (5, 9, 0.9), (64, 129, 0.1), (1000, 63, 0.05),
                                         (257, 1023, 0.1), (2, 4096, 0.5), (130, 2050, 0.999), (1, 70001, 0.3), (4000, 16, 0.2)])
def test_dropout(rows, cols, p, dtype, aligned):
    note(f"dropout {rows} x {cols} p {p} {dtype} aligned {aligned}")
    g = gen(rows + cols)
    x, r = (torch.randn(rows, cols, generator=g).to(dtype) for _ in range(2))
    ld, off = layout(cols, dtype, aligned)
    _, xv = place(x, dtype, ld, off)
    _, rv = place(r, dtype, ld + 1 - aligned, off)
    for res in (None, rv):
        buf, yv = rows_of(rows, cols, dtype, ld, off)
        dg.dropout(xv, yv, p, rng(), res)
        torch.cuda.synchronize()
        rr = None if res is None else f64(r)
        want, keep = dropout_ref(f64(x), rr, p, SEED, OFFSET)
        assert worst(yv, want, allow(f64(x), rr, want, p, dtype)) <= 1
        assert untouched(buf, rows, cols, ld, off)
        if res is None:
            assert np.array_equal(f64(yv) != 0, keep & (f64(x) != 0))
    # In the residual's place, the same bits.
    again, av = place(r, dtype, ld, off)
    dg.dropout(xv, av, p, rng(), av)
    assert torch.equal(av, yv)
    # The mask is the same whatever the type and layout, and in place.
    dg.dropout(xv, xv, p, rng())
    assert np.array_equal(f64(xv) != 0, keep & (f64(x) != 0))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_dropout_ends(dtype):
    x = torch.randn(40, 200, generator=gen(1)).to(dtype).cuda()
    r = torch.randn(40, 200, generator=gen(2)).to(dtype).cuda()
    y = torch.empty_like(x)
    dg.dropout(x, y, 0.0, rng())
    assert torch.equal(y, x)
    dg.dropout(x, y, 1.0, rng())
    assert not bool(y.any())
    dg.dropout(x, y, 1.0, rng(), r)
    assert torch.equal(y, r)
    # What is dropped counts as zero, also where it is not finite; what is kept shows.
    bad = torch.full_like(x, float("nan"))
    bad[20:] = float("inf")
    dg.dropout(bad, y, 0.5, rng())
    _, keep = dropout_ref(np.ones((40, 200)), None, 0.5, SEED, OFFSET)
    keep = torch.from_numpy(keep)
    assert bool((y.cpu()[~keep] == 0).all())
    assert bool(y.cpu()[:20][keep[:20]].isnan().all()) and bool(y.cpu()[20:][keep[20:]].isinf().all())


def test_dropout_gradient_against_differences():
    """Y is linear in X for one mask, so differences are the gradient up to rounding."""
    g = gen(5)
    x, d, dy = (torch.randn(17, 100, generator=g).cuda() for _ in range(3))
    y1, y2, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dg.dropout(x + d, y1, 0.3, rng(7, 8))
    dg.dropout(x - d, y2, 0.3, rng(7, 8))
    dg.dropout(dy, dx, 0.3, rng(7, 8))
    left, right = ((f64(y1) - f64(y2)) / 2 * f64(dy)).sum(), (f64(dx) * f64(d)).sum()
    assert abs(left - right) < 8 * U * 2 * (np.abs(f64(x)) + np.abs(f64(d))).sum() * float(dy.abs().max())


def test_dropout_masks_differ_by_seed_offset_row_and_column():
    ones = torch.ones(64, 512, device="cuda")
    outs = []
    for state in ((1, 0), (2, 0), (1, 1), (1 + (1 << 32), 0), (1, 1 << 32)):
        y = torch.empty_like(ones)
        dg.dropout(ones, y, 0.5, rng(*state))
        outs.append(y.cpu() != 0)
    for i in range(len(outs)):
        for j in range(i):
            same = (outs[i] == outs[j]).float().mean()
            assert abs(float(same) - 0.5) < 5 * 0.5 / 181                  # 5 sigma of 32768 coins
    one = outs[0]
    assert abs(float((one[1:] == one[:-1]).float().mean()) - 0.5) < 5 * 0.5 / 179
    assert abs(float((one[:, 8:] == one[:, :-8]).float().mean()) - 0.5) < 5 * 0.5 / 179


def test_dropout_captured_follows_its_generator():
    x = torch.randn(100, 333, generator=gen(3)).cuda()
    y, state = torch.empty_like(x), rng(5, 0)
    dg.dropout(x, y, 0.2, state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.dropout(x, y, 0.2, state)
    for offset in (0, 1, 1 << 40, 3):
        state[1] = offset
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = dropout_ref(f64(x), None, 0.2, 5, offset)
        assert worst(y, want, allow(f64(x), None, want, 0.2, F32)) <= 1


def test_dropout_past_32_bits():
    ld, rows, cols = 1 << 20, 2300, 100
    buf = torch.empty(rows, ld, dtype=BF16, device="cuda")
    x = torch.randn(rows, cols, generator=gen(1)).to(BF16)
    buf[:, :cols].copy_(x)
    dg.dropout(buf[:, :cols], buf[:, 128:128 + cols], 0.1, rng())
    want, _ = dropout_ref(f64(x), None, 0.1, SEED, OFFSET)
    assert worst(buf[:, 128:128 + cols], want, allow(f64(x), None, want, 0.1, BF16)) <= 1


def test_dropout_of_more_vectors_than_32_bits_count():
    """2^32 vectors of 8 columns (69 GB), in place; rows from all over against the generator."""
    rows, cols = 1 << 20, 1 << 15
    x = torch.ones(rows, cols, dtype=BF16, device="cuda")
    dg.dropout(x, x, 0.5, rng(3, 4))
    torch.cuda.synchronize()
    ones = np.ones((1, cols // 8), dtype=np.uint64)
    for row in (0, 1, (1 << 17) - 1, (1 << 19) + 12345, rows - 2, rows - 1):
        w = philox((np.arange(cols // 8, dtype=np.uint64)[None, :], ones * np.uint64(row), ones * np.uint64(4), 0 * ones), (3, 0))
        u = np.stack([h for v in w for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))], 2).reshape(cols)
        assert np.array_equal(f64(x[row]), np.where(u >= 32768, 2.0, 0.0)), row
