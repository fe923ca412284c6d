"""The router and its rows against plain 64-bit forms (layer_util)."""
import numpy as np
import pytest
import torch

import dense_gemm_04_amd as dg
from layer_util import (BF16, F32, STEP, U, chain, prob_rel, route_grad_ref, route_ref, spread, softmax_ref, worst)
from ops_util import f64, gen
from test_norm_gpu import note, place, rows_of, untouched

pytestmark = pytest.mark.gpu

INT = torch.int32
# tokens, experts, k
ROUTES = [(0, 8, 2), (1, 1, 1), (1, 8, 8), (2, 3, 2), (16, 32, 2), (63, 16, 1), (64, 16, 2), (65, 17, 3), (127, 33, 4),
          (200, 64, 8), (257, 65, 6), (500, 128, 8), (255, 129, 2), (300, 256, 8), (90, 300, 5), (70, 513, 16),
          (40, 1024, 16), (1000, 24, 4), (1024, 60, 4), (1025, 8, 1), (4100, 64, 2), (3000, 256, 4)]


def logits(T, E, dtype, seed, odd=True):
    """Normal logits with ties; some rows of -infinity, some with few experts left."""
    g = gen(seed)
    x = torch.randn(T, E, generator=g) * 2
    if odd and T > 4:
        x[::3] = (x[::3] * 4).round() / 4                   # ties
        x[1::7] = -float("inf")
        x[2::11, 1:] = -float("inf")                         # one expert left
        x[3::13, ::2] = -float("inf")
        x[T - 1] = 1.25                                      # all equal
    return x.to(dtype)


def run_route(l, k, renormalize, ld=None, offset=0, with_loss=True, stream=None):
    T, E = l.shape
    _, v = place(l, l.dtype, ld or max(E, 1), offset)
    out = {"gates": torch.full((T, k), 9.0, device="cuda"), "choice": torch.full((T, k), 99, dtype=INT, device="cuda"),
           "slots": torch.full((T, k), 99, dtype=INT, device="cuda"),
           "offsets": torch.full((E + 1,), 99, dtype=INT, device="cuda"),
           "counts": torch.full((E + 1,), 99, dtype=INT, device="cuda"),
           "loss": torch.full((1,), 9.0, device="cuda") if with_loss else None}
    ws = torch.full((dg.gemm_moe_route_workspace_size(T, E, k) + 256,), 0xff, dtype=torch.uint8, device="cuda")
    dg.moe_route(v, out["gates"], out["choice"], out["slots"], out["offsets"], out["counts"], ws[:-256], out["loss"],
                 renormalize, stream)
    torch.cuda.synchronize()
    assert bool((ws[-256:] == 0xff).all())
    return out


def check_route(out, l, k, renormalize):
    x = f64(l)
    T, E = x.shape
    choice, gates, slots, offsets, counts, loss = route_ref(x, k, renormalize)
    for name, want in (("choice", choice), ("slots", slots), ("offsets", offsets), ("counts", counts)):
        np.testing.assert_array_equal(out[name].cpu().numpy(), want, err_msg=name)
    if T:
        rel = np.where(choice >= 0, np.take_along_axis(prob_rel(x), np.maximum(choice, 0), 1), 0.0)
        if renormalize:                     # the sum of the chosen carries theirs
            rel = rel + rel.max(1, keepdims=True) + 20 * U
        assert worst(out["gates"], gates, rel * np.abs(np.nan_to_num(gates)) + 1e-37) <= 1
    if out["loss"] is not None:
        rel = (T / 4 + E + 64 + 40) * U + (prob_rel(x).max() if T else 0)
        assert worst(out["loss"], np.array([loss]), rel * np.abs(np.nan_to_num(loss))) <= 1


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,k", ROUTES)
def test_route(T, E, k, dtype):
    note(f"route {T} x {E} k {k} {dtype}")
    for renormalize in (True, False):
        l = logits(T, E, dtype, T + E + k)
        check_route(run_route(l, k, renormalize), l, k, renormalize)
        check_route(run_route(l, k, renormalize, E + 3, 1, with_loss=False), l, k, renormalize)


def test_route_large():
    """More tokens than one round of workgroups takes at once."""
    for T, E, k in ((40000, 16, 2), (70000, 8, 1)):
        note(f"route {T} x {E} k {k}")
        l = logits(T, E, F32, 3)
        check_route(run_route(l, k, True), l, k, True)


def test_route_one_expert_takes_all():
    l = torch.zeros(700, 32)
    l[:, 5] = 9.0
    l[:, 6] = 8.0
    check_route(run_route(l, 2, True), l, 2, True)
    l = torch.full((300, 12), -float("inf"))                 # padding alone
    out = run_route(l, 2, True)
    check_route(out, l, 2, True)
    assert float(out["loss"]) == 0 and not bool(out["counts"].any()) and bool((out["slots"] == -1).all())


def test_route_rows_that_are_not_finite():
    for T in (40, 3000):
        l = logits(T, 20, F32, 8)
        l[4, 3] = float("nan")
        l[9, 0] = float("inf")
        l[13] = float("nan")
        for renormalize in (True, False):
            out = run_route(l, 3, renormalize)
            check_route(out, l, 3, renormalize)
            assert bool(out["loss"].isnan()) and bool(out["gates"][[4, 9, 13]].isnan().all())
            assert bool((out["choice"][[4, 9, 13]] == -1).all())


def test_route_wide_logits():
    """Differences that underflow exp, the largest finite values, and -0.0 beside 0.0 (equal)."""
    big = torch.finfo(F32).max
    l = torch.tensor([[0.0, -200.0, -300.0, -1e30], [big, -big, 0.0, big], [-big, -big, -float("inf"), -big],
                      [-0.0, 0.0, -1.0, -1.0]]).repeat(3, 1)
    for renormalize in (True, False):
        check_route(run_route(l, 3, renormalize), l, 3, renormalize)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,k", [r for r in ROUTES if r[0]])
def test_route_grad(T, E, k, dtype):
    note(f"route gradient {T} x {E} k {k} {dtype}")
    l = logits(T, E, dtype, T + E + k)
    g = gen(T)
    dgates = torch.randn(T, k, generator=g)
    for renormalize, dgate, dloss in ((True, True, 0.7), (False, True, -3.0), (True, False, 2.0), (False, True, None),
                                      (True, True, None)):
        choice, _, _, _, counts, _ = route_ref(f64(l), k, renormalize)
        poisoned = dgates.clone()
        poisoned[torch.from_numpy(choice) < 0] = float("nan")            # not read into any sum
        buf, out = rows_of(T, E, dtype, E + 1, 1)
        _, lv = place(l, dtype, E + 1, 1)
        dg.moe_route_grad(lv, torch.from_numpy(choice).to(INT).cuda(), torch.from_numpy(counts).to(INT).cuda(), out,
                          poisoned.cuda() if dgate else None,
                          None if dloss is None else torch.tensor([dloss], device="cuda"), renormalize)
        torch.cuda.synchronize()
        dl = None if dloss is None else float(np.float32(dloss))
        want, mag = route_grad_ref(f64(l), choice, counts, f64(dgates) if dgate else None, dl, renormalize)
        rel = 2 * prob_rel(f64(l)) + 2 * prob_rel(f64(l)).max(1, keepdims=True) + (chain(E) + k + 16) * U
        assert worst(out, want, rel * mag + (STEP[dtype] + U) * np.abs(want) + 1e-37) <= 1
        assert untouched(buf, T, E, E + 1, 1)


def test_route_grad_in_place_and_not_finite():
    l = logits(50, 20, F32, 8)
    choice, _, _, _, counts, _ = route_ref(f64(l), 2, True)
    c, n, d = torch.from_numpy(choice).to(INT).cuda(), torch.from_numpy(counts).to(INT).cuda(), torch.ones(50, 2).cuda()
    loss = torch.ones(1, device="cuda")
    a, b = l.cuda(), torch.empty(50, 20, device="cuda")
    dg.moe_route_grad(a, c, n, b, d, loss)
    dg.moe_route_grad(a, c, n, a, d, loss)
    assert torch.equal(a, b)
    l[4, 3] = float("nan")
    dg.moe_route_grad(l.cuda(), c, n, b, d, loss)
    assert bool(b[4].isnan().all()) and not bool(b[[0, 2, 3, 5, 6]].isnan().any())
    # Choices outside the experts are absent ones.
    c[0, 0], c[2, 1] = 20, -7
    dg.moe_route_grad(torch.zeros(50, 20, device="cuda"), c, n, b, d, None, False)
    assert bool(b.isfinite().all())


def test_route_grad_against_differences():
    g = gen(12)
    T, E, k = 48, 24, 3
    l, dgates = torch.randn(T, E, generator=g), torch.randn(T, k, generator=g)
    for renormalize in (True, False):
        out = run_route(l, k, renormalize)
        dl = torch.empty(T, E, device="cuda")
        dg.moe_route_grad(l.cuda(), out["choice"], out["counts"], dl, dgates.cuda(), torch.tensor([5.0], device="cuda"),
                          renormalize)
        d, step, ends = torch.randn(T, E, generator=g), 2.0 ** -9, []
        # Away from places where a choice changes within the step.
        top = l.sort(1, descending=True).values
        d[(top[:, :k] - top[:, 1:k + 1]).amin(1) < 16 * step] = 0
        for s in (step, -step):
            o = run_route(l + s * d, k, renormalize)
            assert torch.equal(o["choice"], out["choice"])
            ends.append((f64(o["gates"]) * f64(dgates)).sum() + 5 * f64(o["loss"])[0])
        size = np.sqrt(T * k) + 5
        assert abs((ends[0] - ends[1]) / (2 * step) - (f64(dl) * f64(d)).sum()) < size * (16 * U / step + 16 * step ** 2)


def test_route_past_32_bits():
    ld, T, E, k = 1 << 22, 300, 40, 3                        # 5 GB
    buf = torch.empty(T, ld, device="cuda")
    l = logits(T, E, F32, 1)
    v = buf[:, 64:64 + E]
    v.copy_(l)
    out = {n: torch.empty(T, k, dtype=d, device="cuda") for n, d in (("gates", F32), ("choice", INT), ("slots", INT))}
    out |= {n: torch.empty(E + 1, dtype=INT, device="cuda") for n in ("offsets", "counts")}
    out["loss"] = torch.empty(1, device="cuda")
    ws = torch.empty(dg.gemm_moe_route_workspace_size(T, E, k), dtype=torch.uint8, device="cuda")
    dg.moe_route(v, out["gates"], out["choice"], out["slots"], out["offsets"], out["counts"], ws, out["loss"])
    check_route(out, l, k, True)
    dl, d = buf[:, 256:256 + E], torch.randn(T, k, generator=gen(2))
    dg.moe_route_grad(v, out["choice"], out["counts"], dl, d.cuda())
    want, mag = route_grad_ref(f64(l), f64(out["choice"]).astype(int), f64(out["counts"]).astype(int), f64(d), None, True)
    rel = 4 * prob_rel(f64(l)).max(1, keepdims=True) + (chain(E) + k + 16) * U
    assert worst(dl, want, rel * mag + 2 * U * np.abs(want) + 1e-37) <= 1


def test_conveniences_refuse_what_the_calls_cannot_take():
    x, f = torch.zeros(4, 8, dtype=BF16, device="cuda"), torch.zeros(4, device="cuda")
    i, g = torch.zeros(4, 2, dtype=INT, device="cuda"), torch.zeros(4, 2, device="cuda")
    for call in (lambda: dg.layernorm(x, x[:3]), lambda: dg.layernorm(x, x.float()), lambda: dg.layernorm(x, x, weight=f),
                 lambda: dg.layernorm(x.t(), x.t()), lambda: dg.layernorm_grad(x, x, x, f, f[:3]),
                 lambda: dg.dropout(x, x, 0.1, f), lambda: dg.moe_gather(x, i.t(), x), lambda: dg.moe_gather(x, i[:3], x),
                 lambda: dg.moe_combine(x, i, x, gates=g[:, :1]), lambda: dg.moe_combine_grad(x, i, x, dgates=g),
                 lambda: dg.moe_combine(x[:1].expand(4, 8), i, x[:1].expand(4, 8))):
        with pytest.raises((TypeError, ValueError)):
            call()
    ws = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    for call in (lambda: dg.layernorm(x, x, eps=-1.0), lambda: dg.dropout(x, x, 1.5, torch.zeros(2, dtype=torch.int64, device="cuda")),
                 lambda: dg.layernorm_grad(x, x, x, f, f, dweight=torch.zeros(8, device="cuda")),
                 lambda: dg.layernorm_grad(x, x, x, f, f, dweight=torch.zeros(8, device="cuda"), workspace=ws[1:])):
        with pytest.raises(dg.GemmError) as bad:
            call()
        assert bad.value.status == dg.GEMM_ERR_INVALID_VALUE


# ---- rows ------------------------------------------------------------------------

def slots_of(T, k, seed, absent=0.1, spare=5):
    """Distinct slots in any order, a few absent, and rows that none names."""
    g = gen(seed)
    rows = T * k + spare
    s = torch.randperm(rows, generator=g)[:T * k].view(T, k).to(INT)
    s[torch.rand(T, k, generator=g) < absent] = -1
    return s, rows


ROWS = [(1, 1, 1), (1, 8, 4096), (3, 2, 7), (16, 4, 64), (5, 3, 9), (64, 2, 200), (33, 8, 513), (7, 16, 1000), (20, 6, 1024),
        (130, 1, 2050), (9, 5, 4099), (300, 2, 4096), (6, 7, 8192), (4, 2, 20001), (1100, 4, 256)]


@pytest.mark.parametrize("layout", ["lines", "aligned", "odd"])
@pytest.mark.parametrize("T,k,cols", ROWS)
def test_rows(T, k, cols, layout):
    note(f"rows {T} k {k} cols {cols} {layout}")
    g = gen(T + cols)
    slots, rows = slots_of(T, k, T)
    slots[0, 0] = rows if T > 1 else slots[0, 0]                   # past the rows: absent
    sc = slots.cuda()
    s = slots.long().numpy()
    there = (s >= 0) & (s < rows)
    # Whole cache lines (where the columns are), 16 bytes, and neither.
    ld, off = {"lines": (-(-cols // 64) * 64 + 64, 0), "aligned": (-(-cols // 8) * 8 + 8, 0), "odd": (cols + 1, 1)}[layout]
    bf = lambda *shape: torch.randn(*shape, generator=g).to(BF16)
    x, y, r, gates = bf(T, cols), bf(rows, cols), bf(T, cols), torch.rand(T, k, generator=g)
    named = np.zeros(rows, dtype=bool)
    named[s[there]] = True
    _, xv = place(x, BF16, ld, off)
    yy = y.clone()
    yy[torch.from_numpy(~named)] = float("nan")                    # rows that no slot names are not read
    _, yv = place(yy, BF16, ld, off)
    _, rv = place(r, BF16, ld, off)

    buf, out = rows_of(rows, cols, BF16, ld, off)
    dg.moe_gather(xv, sc, out)
    torch.cuda.synchronize()
    tok = np.repeat(np.arange(T), k).reshape(T, k)
    assert torch.equal(out.cpu()[s[there]], x[tok[there]])
    assert bool((out[torch.from_numpy(~named).cuda()].contiguous().view(torch.int16) == -1).all())
    assert untouched(buf, rows, cols, ld, off)

    y64 = np.where(there[:, :, None], f64(y)[np.where(there, s, 0)], 0.0)
    for gg, res in ((gates, r), (None, None), (gates, None), (None, r)):
        w = f64(gg) if gg is not None else np.ones((T, k))
        want = (y64 * w[:, :, None]).sum(1) + (0 if res is None else f64(res))
        mag = (np.abs(y64) * w[:, :, None]).sum(1) + (0 if res is None else np.abs(f64(res)))
        cbuf, c = rows_of(T, cols, BF16, ld, off)
        dg.moe_combine(yv, sc, c, None if gg is None else gg.cuda(), None if res is None else rv)
        torch.cuda.synchronize()
        assert worst(c, want, 2.0 ** -8 * np.abs(want) + (k + 2) * U * mag) <= 1
        assert untouched(cbuf, T, cols, ld, off)
        if res is not None:                                          # in place of the residual
            _, again = place(r, BF16, ld, off)
            dg.moe_combine(yv, sc, again, None if gg is None else gg.cuda(), again)
            assert torch.equal(again, c)

    dc64 = f64(x)
    for gg, want_gates in ((gates, True), (None, True), (gates, False)):
        w = f64(gg) if gg is not None else np.ones((T, k))
        dbuf, dy = rows_of(rows, cols, BF16, ld, off)
        dgates = torch.full((T, k), 9.0, device="cuda") if want_gates else None
        dg.moe_combine_grad(xv, sc, dy, yv if want_gates else None, None if gg is None else gg.cuda(), dgates)
        torch.cuda.synchronize()
        want = dc64[tok[there]] * w[there][:, None]
        assert worst(dy.cpu()[s[there]], want, (2.0 ** -8 + 2 * U) * np.abs(want)) <= 1
        assert bool((dy[torch.from_numpy(~named).cuda()].contiguous().view(torch.int16) == -1).all())
        assert untouched(dbuf, rows, cols, ld, off)
        if want_gates:
            terms = dc64[:, None, :] * y64
            assert worst(dgates, terms.sum(2), chain(cols) * U * np.abs(terms).sum(2)) <= 1
            # dY in Y's place.
            _, place_y = place(yy, BF16, ld, off)
            again = torch.empty_like(dgates)
            dg.moe_combine_grad(xv, sc, place_y, place_y, None if gg is None else gg.cuda(), again)
            assert torch.equal(again, dgates) and torch.equal(place_y.cpu()[s[there]], dy.cpu()[s[there]])


@pytest.mark.parametrize("T,k,cols", [(70000, 2, 24), (3, 2, 140000), (1100000, 1, 8)])
def test_rows_past_the_grid(T, k, cols):
    """More tokens or columns than a launch has workgroups for, each with its own value."""
    note(f"rows {T} k {k} cols {cols}")
    slots = torch.randperm(T * k, generator=gen(T)).view(T, k).to(INT).cuda()
    x = (torch.arange(T, device="cuda")[:, None] % 251 + torch.arange(cols, device="cuda")[None, :] % 5).to(BF16)
    y = torch.zeros(T * k, cols, dtype=BF16, device="cuda")
    dg.moe_gather(x, slots, y)
    assert torch.equal(y[slots.long().flatten()].view(T, k, cols), x[:, None, :].expand(-1, k, -1))
    c = torch.empty_like(x)
    dg.moe_combine(y, slots, c, torch.full((T, k), 1.0 / k, device="cuda"))
    assert torch.equal(c, x)
    dgates = torch.empty(T, k, device="cuda")
    dg.moe_combine_grad(x, slots, y, y, None, dgates)
    want = (x.double() ** 2).sum(1, keepdim=True).expand(-1, k)
    assert bool(((dgates.double() - want).abs() <= chain(cols) * U * want).all())


def test_rows_without_any_row():
    slots = torch.zeros(5, 2, dtype=INT, device="cuda")
    x = torch.randn(5, 40, generator=gen(1)).to(BF16).cuda()
    none, c = torch.empty(0, 40, dtype=BF16, device="cuda"), torch.empty_like(x)
    dg.moe_gather(x, slots, none)
    dg.moe_combine(none, slots, c, None, x)
    assert torch.equal(c, x)
    dgates = torch.full((5, 2), 9.0, device="cuda")
    dg.moe_combine_grad(x, slots, none, none, None, dgates)
    assert not bool(dgates.any())


def test_absent_rows_show_a_gate_that_is_not_a_number():
    slots = torch.tensor([[-1, -1], [0, -1]], dtype=INT, device="cuda")
    gates = torch.tensor([[float("nan"), float("nan")], [1.0, 0.0]], device="cuda")
    y, c = torch.ones(1, 70, dtype=BF16, device="cuda"), torch.empty(2, 70, dtype=BF16, device="cuda")
    dg.moe_combine(y, slots, c, gates)
    assert bool(c[0].isnan().all()) and bool((c[1] == 1).all())


def test_slots_outside_the_rows_touch_nothing():
    g = gen(4)
    slots = torch.tensor([[-2 ** 31, 2 ** 31 - 1], [50, -50], [3, 10 ** 6]], dtype=INT, device="cuda")
    x = torch.randn(3, 64, generator=g).to(BF16).cuda()
    buf = torch.full((150, 64), 5.0, dtype=BF16, device="cuda")
    dg.moe_gather(x, slots, buf[50:100])
    torch.cuda.synchronize()
    want = torch.full((150, 64), 5.0, dtype=BF16)
    want[53] = x[2].cpu()
    assert torch.equal(buf.cpu(), want)
    dgates = torch.full((3, 2), 9.0, device="cuda")
    dg.moe_combine_grad(x, slots, buf[50:100], buf[50:100], None, dgates)
    assert torch.equal(buf.cpu(), want)
    assert dgates.cpu().count_nonzero() == 1
    # The same slot twice leaves one of the two rows, whole.
    dg.moe_gather(x, torch.full((3, 1), 7, dtype=INT, device="cuda"), buf[50:100])
    assert any(torch.equal(buf[57], row) for row in x)


def test_rows_past_32_bits():
    ld, rows, cols, k = 1 << 20, 2300, 96, 2
    buf = torch.empty(rows, ld, dtype=BF16, device="cuda")
    g = gen(3)
    slots = torch.randperm(rows, generator=g)[:2200].view(1100, 2).to(INT)
    x, gates = torch.randn(1100, cols, generator=g).to(BF16), torch.rand(1100, 2, generator=g)
    sorted_rows = buf[:, 64:64 + cols]
    dg.moe_gather(x.cuda(), slots.cuda(), sorted_rows)
    assert torch.equal(sorted_rows.cpu()[slots.long()], x[:, None, :].expand(-1, 2, -1))
    c = buf[:1100, 256:256 + cols]
    dg.moe_combine(sorted_rows, slots.cuda(), c, gates.cuda())
    want = f64(x) * f64(gates).sum(1, keepdims=True)
    assert worst(c, want, 2.0 ** -8 * np.abs(want) + 4 * U * np.abs(want)) <= 1
    dgates = torch.empty(1100, 2, device="cuda")
    dg.moe_combine_grad(x.cuda(), slots.cuda(), sorted_rows, sorted_rows, gates.cuda(), dgates)
    terms = f64(x) ** 2
    assert worst(dgates, np.repeat(terms.sum(1)[:, None], 2, 1), chain(cols) * U * terms.sum(1)[:, None]) <= 1
