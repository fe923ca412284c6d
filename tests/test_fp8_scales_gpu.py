"""GPU tests of the 8-bit product with scales at the ends of fp32's range, and
of exact sums on every kernel and at the depths in use.

The operands are whole numbers of magnitude up to 4, so a block's sum d is
exact. SA SB is formed in fp32 (here on the host as well), and every d * (SA SB)
and their sum are whole numbers of quanta that fp32 holds, or not finite: C is
their one rounding to bf16, whatever the order, on every kernel."""
import numpy as np
import pytest
import torch

import dense_gemm_04_amd as dg
from gpu_util import note
from ops_util import E4M3, f64, gen, put, rows_of
from test_fp8_gpu import run_fp8

pytestmark = pytest.mark.gpu

# M, N, K: few rows, lone 64 x 64 tiles that share K (the first three also
# unaligned, on the general kernel), then 64 x 64, 64 x 128 and 128 x 128 tiles
# alone and two to a CU, 192 x 256 and 256 x 256.
SIZES = [(9, 200, 500), (30, 4100, 260), (120, 260, 1040), (5500, 260, 272), (700, 2048, 400), (1500, 1500, 272),
         (1000, 4100, 260), (2880, 4090, 300), (4090, 4003, 400)]


def scales(kind, blocks, rows, g, left):
    """Powers of two, or for "subnormal" a mantissa beside one."""
    pow2 = lambda lo, hi: torch.exp2(torch.randint(lo, hi + 1, (blocks, rows), generator=g).float())
    if kind == "near":                       # products about 1
        return pow2(-2, 2)
    if kind == "apart":                      # far from 1, their products near it
        return pow2(98, 102) if left else pow2(-102, -98)
    if kind == "subnormal":                  # products 2^-141 .. 2^-139, up to three bits more
        return pow2(-101, -100) * (1 + torch.randint(0, 4, (blocks, rows), generator=g) / 4) if left else pow2(-40, -39)
    if kind == "vanishing":                  # 0 in fp32
        return pow2(-100, -98) if left else pow2(-60, -58)
    # Rows large in both operands meet in infinite products, others in 2^40 or 2^84.
    big = torch.rand(rows, generator=g) < 0.3
    big[0], big[1:2] = True, False
    return torch.where(big, 2.0 ** 64, 2.0 ** 20).expand(blocks, rows).contiguous()


def operands(M, N, K, b_rows, kind, aligned):
    g = gen(M + N + K)
    nk = -(-K // 128)
    ld = -(-K // 16) * 16 if aligned else K + 3
    out = []
    for rows, per in ((M, 1), (N, b_rows)):
        q = torch.randint(-4, 5, (rows, K), generator=g).float()
        if kind == "infinite":
            q[torch.rand(rows, generator=g) < 0.2] = 0       # rows of zeros: their blocks' sums are 0
        q = q.to(E4M3)
        s = scales(kind, nk, -(-rows // per), g, per == 1 and rows is M)
        out += [q, s]
    views = [put(rows_of(*t.shape, t.dtype if t.dtype == torch.float32 else torch.uint8,
                         ld if t.dtype == E4M3 else None, 0 if aligned else 1)[1],
                 t.view(torch.uint8) if t.dtype == E4M3 else t) for t in out]
    return out, views


def sample(M):
    """Rows to compare: all of a small product's, an odd step apart in a large one."""
    return torch.arange(0, M, M // 300 | 1)


def expected(ops, b_rows, alpha):
    a, sa, b, sb = ops
    a, sa = a.view(torch.uint8)[sample(a.shape[0])].view(E4M3), sa[:, sample(a.shape[0])]
    col = torch.arange(b.shape[0]) // b_rows
    total, most, quantum = np.zeros((a.shape[0], b.shape[0])), 0.0, np.inf
    with np.errstate(invalid="ignore", over="ignore"):
        for i, k in enumerate(range(0, a.shape[1], 128)):
            d = f64(a[:, k:k + 128]) @ f64(b[:, k:k + 128]).T
            factor = (sa[i].numpy()[:, None] * sb[i].numpy()[col.numpy()][None, :])      # fp32
            assert factor.dtype == np.float32
            terms = d * factor.astype(np.float64)
            total += terms
            finite = np.isfinite(factor) & (factor > 0)
            if finite.any():
                # Quanta of a quarter of the smallest factor of a row and column.
                most = most + np.abs(np.where(finite, terms, 0))
                quantum = np.minimum(quantum, np.where(finite, factor / 4.0, np.inf))
    assert np.all(most <= 2.0 ** 24 * quantum)           # so fp32 holds every partial sum
    return torch.from_numpy(total * alpha).float().to(torch.bfloat16)


def same(got, want):
    got = got.cpu()[sample(got.shape[0])]
    assert torch.equal(got.isnan(), want.isnan())
    keep = ~want.isnan()
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("kind", ["near", "apart", "subnormal", "vanishing", "infinite"])
@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("size,aligned", [(s, True) for s in SIZES] + [(s, False) for s in SIZES[:3]])
def test_scales_at_the_ends_of_the_range(size, aligned, b_rows, kind):
    M, N, K = size
    note(f"fp8 scales {size} {kind} b_rows {b_rows} aligned {aligned}")
    ops, views = operands(M, N, K, b_rows, kind, aligned)
    alpha = 2.0 ** 110 if kind == "subnormal" else 1.0
    c = run_fp8(views, M, N, K, b_rows, alpha, ldc=-(-N // 8) * 8)
    want = expected(ops, b_rows, alpha)
    if kind == "infinite":
        assert bool((want.isnan() | want.isinf()).any()) and bool(want.isfinite().any())
    if kind == "vanishing":
        assert not bool(want.any())
    same(c, want)


# The depths in use: each kernel and tile size over 32 to 64 blocks.
DEPTHS = (8192, 4100, 8176, 4000, 4000, 6000, 4096, 4112, 4000)


@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("size", [(M, N, K) for (M, N, _), K in zip(SIZES, DEPTHS)])
def test_deep_sums_of_small_integers_are_exact(size, b_rows):
    M, N, K = size
    note(f"fp8 deep {size} b_rows {b_rows}")
    ops, views = operands(M, N, K, b_rows, "near", True)
    c = run_fp8(views, M, N, K, b_rows, ldc=-(-N // 8) * 8)
    same(c, expected(ops, b_rows, 1.0))
