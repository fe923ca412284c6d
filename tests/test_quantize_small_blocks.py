"""Quantisation of blocks whose largest value is tiny: the quotient 448 x / top
has to be rounded correctly there too, where a residual of its last correction
can be smaller than the smallest fp32 number.

The GPU tests hold the kernels to 64-bit quotients. The CPU test runs the
kernels' steps in exact arithmetic, each rounded to fp32 as the hardware rounds
it, over every bf16 value of a clamped block."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import dense_gemm_04_amd as dg
from ops_util import f64, gen, nearest_e4m3, quantize_ref, rows_of

CLAMP = 448 * 2.0 ** -126


def bf16(bits):
    return torch.as_tensor(np.asarray(bits, dtype=np.int64).astype(np.uint16).view(np.int16)).view(torch.bfloat16)


def clamped_values():
    """Every bf16 value of magnitude up to 448 * 2^-126, in rows of 128."""
    last = int(torch.tensor(CLAMP).to(torch.bfloat16).view(torch.int16))
    bits = np.arange(last + 1)
    bits = np.concatenate([bits, bits | 0x8000])
    return bf16(np.resize(bits, (-(-len(bits) // 128), 128)))


def small_tops():
    """Rows of one block each: its largest value, then every bf16 mantissa at one
    exponent below it. 1.75 makes every quotient a shift of x and most of them
    ties; 1, 1.125 and an odd mantissa others."""
    rows = []
    for e in range(9, 90):                               # 2^-118 .. 2^-38
        for m in (0x60, 0x00, 0x10, 0x2b):
            top = e << 7 | m
            for down in range(0, min(e, 18)):
                x = (e - down) << 7 | np.arange(128)
                rows.append(np.minimum(np.concatenate([[top], x[:127] | (np.arange(127) % 2) << 15]) & 0x7fff, top)
                            | np.concatenate([[0], (np.arange(127) % 2) << 15]))
    return bf16(np.stack(rows))


def to_f32(v):
    """A fraction rounded to the nearest fp32 number, ties to even (as a fraction)."""
    if v == 0:
        return v
    a, e = abs(v), 0
    while a >= 2:
        a, e = a / 2, e + 1
    while a < 1:
        a, e = a * 2, e - 1
    step = Fraction(2) ** (max(e, -126) - 23)
    n = abs(v) / step
    down = n.numerator // n.denominator
    rest = n - down
    n = down + (1 if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and down % 2) else 0)
    return (step * n) * (1 if v > 0 else -1)


def steps(x, top, shift):
    """The kernels' quotient: y and t scaled by 2^shift, every step in fp32."""
    y = to_f32(x * Fraction(7, 8) * Fraction(2) ** shift)
    t = to_f32(top * Fraction(2) ** (shift - 9))
    r = to_f32(1 / t)
    q0 = to_f32(y * r)
    return to_f32(to_f32(y - q0 * t) * r + q0)


def test_steps_round_every_value_of_a_clamped_block():
    values = [Fraction(float(v)) for v in clamped_values().float().flatten().unique()]
    top = Fraction(CLAMP)
    exact = np.array([float(v * 448 / top) for v in values])
    want = nearest_e4m3(exact)
    scaled = nearest_e4m3(np.array([float(steps(v, top, 64)) for v in values]))
    np.testing.assert_array_equal(scaled, want)
    # Unscaled, residuals vanish and some ties fall to the wrong side.
    plain = nearest_e4m3(np.array([float(steps(v, top, 0)) for v in values]))
    assert np.count_nonzero(plain != want) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("op", [dg.OP_N, dg.OP_T])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("values", [clamped_values, small_tops])
def test_bf16_is_rounded_correctly(values, block_rows, op):
    x = values()
    if block_rows == 128:
        # A block of 128 x 128 has one top: repeat a row's values 128 times less
        # its own top, with rows apart by blocks.
        x = x[:: max(1, x.shape[0] // 96)].repeat_interleave(128, 0)
    x = x if op == dg.OP_N else x.t().contiguous()
    r, k = x.shape if op == dg.OP_N else (x.shape[1], x.shape[0])
    q = rows_of(r, k, torch.uint8, -(-k // 16) * 16)[1]
    s = torch.empty(-(-k // 128), -(-r // block_rows), device="cuda")
    dg.quantize_fp8(x.cuda(), q, s, op, block_rows)
    torch.cuda.synchronize()
    v, scales = quantize_ref(f64(x if op == dg.OP_N else x.t()), block_rows)
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    np.testing.assert_array_equal(f64(q), nearest_e4m3(v))


@pytest.mark.gpu
@pytest.mark.parametrize("op", [dg.OP_N, dg.OP_T])
def test_fp32_is_within_two_roundings(op):
    """y = f x and the quotient are each rounded once: 2^-24 twice."""
    g = gen(12)
    size = torch.exp2(torch.randint(-126, -40, (400, 1), generator=g).float())
    x = torch.randn(400, 128, generator=g) * size
    x = x if op == dg.OP_N else x.t().contiguous()
    q = rows_of(400, 128, torch.uint8)[1]
    s = torch.empty(1, 400, device="cuda")
    dg.quantize_fp8(x.cuda(), q, s, op, 1)
    torch.cuda.synchronize()
    v, scales = quantize_ref(f64(x if op == dg.OP_N else x.t()), 1)
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    off = (2.0 ** -23 + 2.0 ** -48) * np.abs(v)
    lo, hi = nearest_e4m3(np.clip(v - off, -448, 448)), nearest_e4m3(np.clip(v + off, -448, 448))
    got = f64(q)
    assert np.all((got == lo) | (got == hi))
