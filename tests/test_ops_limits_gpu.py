"""GPU tests of the 8-bit and grouped operators at their limits: operands whose
byte offsets pass 32 bits, values that are not finite beside a group, and sums
without terms."""
import pytest
import torch

import dense_gemm_04_amd as dg
from gpu_util import note
from ops_util import gen

pytestmark = pytest.mark.gpu


def spread(t, ld):
    """A copy of a matrix with rows ld elements apart (the rest is not set)."""
    buf = torch.empty((t.shape[0] - 1) * ld + t.shape[1] + 16, dtype=t.dtype, device="cuda")
    v = buf.as_strided(t.shape, (ld, 1))
    v.copy_(t)
    return v


def normal(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()


# The product's rows are 2^22 bytes apart (1 more: no alignment), 1300 of them
# 5 GB; the same values packed together have to give the same bits.
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("M", [20, 300, 1300])
def test_fp8_offsets_past_32_bits(M, odd):
    note(f"fp8 far M {M} odd {odd}")
    N, K, g = 1300, 200, gen(60)
    x, w = normal(g, M, K), normal(g, N, K)
    outs = []
    for far in (False, True):
        ld = (1 << 22) if far else 208
        xs, ws = (spread(x, ld // 2 + odd), spread(w, ld // 2 + odd)) if far else (x, w)
        ops = []
        for m, per in ((xs, 1), (ws, 128)):
            q = spread(torch.zeros(m.shape, dtype=torch.uint8, device="cuda"), ld + odd)
            s = torch.empty(2, -(-m.shape[0] // per), device="cuda")
            dg.quantize_fp8(m, q, s, dg.OP_N, per)
            ops += [q, s]
        c = spread(torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"), (ld // 2 if far else 1304) + odd)
        dg.matmul_fp8(*ops, c)
        torch.cuda.synchronize()
        outs.append([ops[0].clone(), ops[1], ops[2].clone(), ops[3], c.clone()])
        del xs, ws, ops, q, s, c, m
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("lengths", [[8, 0, 12], [300, 0, 1000]])
def test_grouped_offsets_past_32_bits(lengths, odd):
    note(f"grouped far {lengths} odd {odd}")
    M, N, K, E, g = sum(lengths), 264, 136, 3, gen(61)
    x, dy, w = normal(g, M, K), normal(g, M, N), normal(g, E, K, N)
    offs = torch.tensor([0, lengths[0], lengths[0] + lengths[1], M], dtype=torch.int32, device="cuda")
    outs = []
    for far in (False, True):
        ld = lambda n: ((1 << 21) if far else n) + odd
        per = (1 << 30) if far else K * N + 8
        xs, dys = spread(x, ld(K)), spread(dy, ld(N))
        wbuf = torch.empty(2 * per + K * (N + 1), dtype=torch.bfloat16, device="cuda")
        ws = wbuf.as_strided((E, K, N), (per, N, 1))
        ws.copy_(w)
        y = spread(torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"), ld(N))
        dx = spread(torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"), ld(K))
        dbuf = torch.empty(2 * per + K * (N + 1), device="cuda")
        dw = dbuf.as_strided((E, K, N), (per, N, 1))
        dg.matmul_bf16_grouped(xs, ws, y, offs)
        dg.matmul_bf16_grouped(dys, ws, dx, offs, opb=dg.OP_T)
        dg.grouped_wgrad(xs, dys, dw, offs)
        torch.cuda.synchronize()
        outs.append([y.clone(), dx.clone(), dw.clone()])
        del xs, dys, wbuf, ws, y, dx, dbuf, dw
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("lengths", [[5, 3, 0, 9], [130, 61, 0, 300]])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_in_their_group(lengths, value):
    """Group 1's rows and matrix hold them; every other group's results keep
    their bits."""
    E, N, K, g = len(lengths), 136, 264, gen(62)
    M, a, b = sum(lengths), lengths[0], lengths[0] + lengths[1]
    x, dy, w = normal(g, M, K), normal(g, M, N), normal(g, E, K, N)
    ends = [0, a, b, b + lengths[2], M]
    offs = torch.tensor(ends, dtype=torch.int32, device="cuda")

    def run():
        y, dx, dw = torch.zeros_like(dy), torch.zeros_like(x), torch.zeros(E, K, N, device="cuda")
        dg.matmul_bf16_grouped(x, w, y, offs)
        dg.matmul_bf16_grouped(dy, w, dx, offs, opb=dg.OP_T)
        dg.grouped_wgrad(x, dy, dw, offs)
        torch.cuda.synchronize()
        return y, dx, dw

    clean = run()
    x[a:b], dy[a:b], w[1] = value, value, value
    y, dx, dw = run()
    for got, want in ((y, clean[0]), (dx, clean[1])):
        assert torch.equal(got[:a], want[:a]) and torch.equal(got[b:], want[b:])
        assert not bool(got[a:b].isfinite().any())
    for e in (0, 2, 3):
        assert torch.equal(dw[e], clean[2][e])
    assert not bool(dw[1].isfinite().any())


@pytest.mark.parametrize("ld", [72, 73])
def test_sums_without_terms_are_zero_also_times_infinity(ld):
    inf = float("inf")
    offs = torch.tensor([0, 0, 4], dtype=torch.int32, device="cuda")
    ones = torch.ones(4, ld, dtype=torch.bfloat16, device="cuda")
    for fn, dtype in ((dg.gemm_bf16_grouped_wgrad, torch.bfloat16), (dg.gemm_bf16_grouped_wgrad_f32, torch.float32)):
        dw = torch.full((2, 16, ld), 3.0, dtype=dtype, device="cuda")
        assert fn(2, 4, 72, 16, inf, ones.data_ptr(), ld, ones.data_ptr(), ld, 2.0, dw.data_ptr(), ld, 16 * ld,
                  offs.data_ptr()) == dg.GEMM_OK
        torch.cuda.synchronize()
        assert bool((dw[0, :, :72] == 6).all()) and bool((dw[1, :, :72] == inf).all())
        assert fn(2, 0, 72, 16, inf, None, ld, None, ld, 2.0, dw.data_ptr(), ld, 16 * ld, offs.data_ptr()) == dg.GEMM_OK
        torch.cuda.synchronize()
        assert bool((dw[0, :, :72] == 12).all())
    c = torch.full((4, ld), 3.0, dtype=torch.bfloat16, device="cuda")
    assert dg.gemm_bf16_grouped(dg.OP_N, 2, 4, 72, 0, inf, None, 1, None, 72, 0, 2.0, c.data_ptr(), ld,
                                offs.data_ptr()) == dg.GEMM_OK
    torch.cuda.synchronize()
    assert bool((c[:, :72] == 6).all())
