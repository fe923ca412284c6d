"""Refusals of the layer norm, dropout and routing entry points, and the tests'
own 64-bit forms: no HIP call is made, so they run without a GPU."""
import numpy as np
import pytest
import torch

import dense_gemm_04_amd as dg
from layer_util import dropout_bits, dropout_ref, norm_grad_ref, norm_ref, philox, route_grad_ref, route_ref

BAD = dg.GEMM_ERR_INVALID_VALUE
P = 0x10000            # suitably aligned addresses that validation never follows


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(dg.LIB_PATH):
        from dense_gemm_04_amd import build
        build.build()
    return dg.load()


def only_host(status):
    """A call that validation accepts, where no GPU can take it."""
    if not torch.cuda.is_available():
        assert status() == dg.GEMM_ERR_UNSUPPORTED_DEVICE


def norm(rows=300, cols=200, eps=1e-5, X=P, ldx=200, w=P, b=P, Y=P, ldy=200, mean=P, rstd=P, fn="bf16"):
    call = dg.gemm_layernorm_bf16 if fn == "bf16" else dg.gemm_layernorm_f32
    return call(rows, cols, eps, X, ldx, w, b, Y, ldy, mean, rstd)


@pytest.mark.parametrize("fn", ["bf16", "f32"])
def test_norm_refusals(fn):
    for bad in (dict(rows=-1), dict(cols=-1), dict(rows=1 << 31), dict(cols=1 << 31), dict(ldx=199), dict(ldy=199),
                dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")), dict(X=None), dict(Y=None),
                dict(X=P + 1), dict(Y=P + 1), dict(w=P + 1), dict(b=P + 1), dict(mean=P + 2), dict(rstd=P + 2),
                dict(ldx=1 << 58), dict(ldy=1 << 58)):
        assert norm(fn=fn, **bad) == BAD, bad
    assert norm(fn=fn, rows=0, X=None, Y=None) == norm(fn=fn, cols=0, X=None, Y=None) == dg.GEMM_OK
    only_host(lambda: norm(fn=fn))
    only_host(lambda: norm(fn=fn, w=None, b=None, mean=None, rstd=None, eps=0.0))
    assert norm(fn="f32", X=P + 2) == BAD


def norm_grad(rows=300, cols=200, X=P, ldx=200, w=P, mean=P, rstd=P, dY=P, lddy=200, R=P, ldr=200, dX=P, lddx=200,
              beta=0.0, dw=P, db=P, ws=P, wsb=None, fn="bf16"):
    call = dg.gemm_layernorm_grad_bf16 if fn == "bf16" else dg.gemm_layernorm_grad_f32
    wsb = dg.gemm_layernorm_grad_workspace_size(rows, cols) if wsb is None else wsb
    return call(rows, cols, X, ldx, w, mean, rstd, dY, lddy, R, ldr, dX, lddx, beta, dw, db, ws, wsb)


@pytest.mark.parametrize("fn", ["bf16", "f32"])
def test_norm_grad_refusals(fn):
    need = dg.gemm_layernorm_grad_workspace_size(300, 200)
    assert need > 0
    assert dg.gemm_layernorm_grad_workspace_size(-1, 4) == dg.gemm_layernorm_grad_workspace_size(4, 1 << 31) == 0
    for bad in (dict(rows=-1), dict(cols=-1), dict(rows=1 << 31), dict(ldx=199), dict(lddy=199), dict(ldr=199),
                dict(lddx=199), dict(X=None), dict(dY=None), dict(dX=None), dict(mean=None), dict(rstd=None),
                dict(X=P + 1), dict(dY=P + 1), dict(R=P + 1), dict(dX=P + 1), dict(w=P + 1), dict(mean=P + 2),
                dict(rstd=P + 1), dict(dw=P + 2), dict(db=P + 2), dict(ws=None, wsb=0), dict(ws=None), dict(ws=P + 128),
                dict(wsb=need - 1), dict(ldr=1 << 58), dict(lddx=1 << 58)):
        assert norm_grad(fn=fn, **bad) == BAD, bad
    nothing = dict(X=None, dY=None, dX=None, R=None, mean=None, rstd=None)
    assert norm_grad(fn=fn, cols=0, **nothing) == dg.GEMM_OK
    assert norm_grad(fn=fn, rows=0, beta=1.0, **nothing) == dg.GEMM_OK
    assert norm_grad(fn=fn, rows=0, dw=None, db=None, **nothing) == dg.GEMM_OK
    only_host(lambda: norm_grad(fn=fn))
    only_host(lambda: norm_grad(fn=fn, rows=0, **nothing))                    # dw, db <- 0
    only_host(lambda: norm_grad(fn=fn, dw=None, db=None, ws=None, wsb=0))     # needs no workspace
    only_host(lambda: norm_grad(fn=fn, R=None, ldr=0, w=None))


def drop(rows=300, cols=200, p=0.1, rng=P, X=P, ldx=200, R=P, ldr=200, Y=P, ldy=200, fn="bf16"):
    call = dg.gemm_dropout_bf16 if fn == "bf16" else dg.gemm_dropout_f32
    return call(rows, cols, p, rng, X, ldx, R, ldr, Y, ldy)


@pytest.mark.parametrize("fn", ["bf16", "f32"])
def test_dropout_refusals(fn):
    for bad in (dict(rows=-1), dict(cols=-1), dict(rows=1 << 31), dict(p=-0.01), dict(p=1.01), dict(p=float("nan")),
                dict(rng=None), dict(rng=P + 4), dict(X=None), dict(Y=None), dict(X=P + 1), dict(R=P + 1),
                dict(Y=P + 1), dict(ldx=199), dict(ldr=199), dict(ldy=199), dict(ldx=1 << 58)):
        assert drop(fn=fn, **bad) == BAD, bad
    assert drop(fn=fn, rows=0, X=None, Y=None, rng=None) == drop(fn=fn, cols=0, X=None, Y=None, rng=None) == dg.GEMM_OK
    only_host(lambda: drop(fn=fn))
    only_host(lambda: drop(fn=fn, R=None, ldr=0, p=1.0))


def route(T=300, E=64, k=4, norm=1, L=P, ldl=None, gates=P, choice=P, slots=P, offsets=P, counts=P, loss=P, ws=P,
          wsb=None, fn="f32"):
    call = dg.gemm_moe_route_bf16 if fn == "bf16" else dg.gemm_moe_route_f32
    wsb = dg.gemm_moe_route_workspace_size(T, E, k) if wsb is None else wsb
    return call(T, E, k, norm, L, max(E, 1) if ldl is None else ldl, gates, choice, slots, offsets, counts, loss, ws, wsb)


@pytest.mark.parametrize("fn", ["bf16", "f32"])
def test_route_refusals(fn):
    need = dg.gemm_moe_route_workspace_size(300, 64, 4)
    assert need > 0
    for sizes in ((-1, 64, 4), (300, 0, 4), (300, 64, 0), (300, 64, 17), (300, 3, 4), (300, 1025, 4), (1 << 30, 64, 2)):
        assert dg.gemm_moe_route_workspace_size(*sizes) == 0, sizes
        assert route(*sizes, wsb=1 << 40, fn=fn) == BAD, sizes
    for bad in (dict(ldl=63), dict(L=None), dict(gates=None), dict(choice=None), dict(slots=None), dict(offsets=None),
                dict(counts=None), dict(L=P + 1), dict(gates=P + 2), dict(choice=P + 2), dict(slots=P + 2),
                dict(offsets=P + 2), dict(counts=P + 2), dict(loss=P + 2), dict(ws=None), dict(ws=None, wsb=0),
                dict(ws=P + 64), dict(wsb=need - 1), dict(ldl=1 << 58)):
        assert route(fn=fn, **bad) == BAD, bad
    only_host(lambda: route(fn=fn))
    only_host(lambda: route(fn=fn, loss=None))
    only_host(lambda: route(fn=fn, T=0, L=None, gates=None, choice=None, slots=None))   # offsets and counts <- 0
    only_host(lambda: route(fn=fn, E=1024, k=16))


def route_grad(T=300, E=64, k=4, norm=1, L=P, ldl=64, choice=P, counts=P, dgates=P, dloss=P, dL=P, lddl=64, fn="f32"):
    call = dg.gemm_moe_route_grad_bf16 if fn == "bf16" else dg.gemm_moe_route_grad_f32
    return call(T, E, k, norm, L, ldl, choice, counts, dgates, dloss, dL, lddl)


@pytest.mark.parametrize("fn", ["bf16", "f32"])
def test_route_grad_refusals(fn):
    for bad in (dict(T=-1), dict(E=0), dict(E=1025, ldl=1025, lddl=1025), dict(k=0), dict(k=17), dict(E=3), dict(ldl=63),
                dict(lddl=63), dict(L=None), dict(choice=None), dict(counts=None), dict(dL=None), dict(L=P + 1),
                dict(dL=P + 1), dict(choice=P + 2), dict(counts=P + 2), dict(dgates=P + 2), dict(dloss=P + 2),
                dict(lddl=1 << 58)):
        assert route_grad(fn=fn, **bad) == BAD, bad
    assert route_grad(fn=fn, T=0, L=None, choice=None, counts=None, dL=None) == dg.GEMM_OK
    only_host(lambda: route_grad(fn=fn))
    only_host(lambda: route_grad(fn=fn, dgates=None, dloss=None))


def gather(T=300, k=2, cols=200, rows=600, X=P, ldx=200, slots=P, Y=P, ldy=200):
    return dg.gemm_moe_gather_bf16(T, k, cols, rows, X, ldx, slots, Y, ldy)


def combine(T=300, k=2, cols=200, rows=600, Y=P, ldy=200, slots=P, gates=P, R=P, ldr=200, C=P, ldc=200):
    return dg.gemm_moe_combine_bf16(T, k, cols, rows, Y, ldy, slots, gates, R, ldr, C, ldc)


def combine_grad(T=300, k=2, cols=200, rows=600, dC=P, lddc=200, Y=P, ldy=200, slots=P, gates=P, dY=P, lddy=200,
                 dgates=P):
    return dg.gemm_moe_combine_grad_bf16(T, k, cols, rows, dC, lddc, Y, ldy, slots, gates, dY, lddy, dgates)


def test_rows_refusals():
    sizes = (dict(T=-1), dict(k=0), dict(k=17), dict(cols=-1), dict(rows=-1), dict(T=1 << 30), dict(rows=1 << 31),
             dict(slots=None), dict(slots=P + 2))
    for bad in sizes + (dict(X=None), dict(Y=None), dict(X=P + 1), dict(Y=P + 1), dict(ldx=199), dict(ldy=199),
                        dict(ldy=1 << 58)):
        assert gather(**bad) == BAD, bad
    for bad in sizes + (dict(C=None), dict(Y=None), dict(C=P + 1), dict(Y=P + 1), dict(R=P + 1), dict(gates=P + 2),
                        dict(ldc=199), dict(ldy=199), dict(ldr=199)):
        assert combine(**bad) == BAD, bad
    for bad in sizes + (dict(dC=None), dict(Y=None), dict(dY=None), dict(dC=P + 1), dict(Y=P + 1), dict(dY=P + 1),
                        dict(gates=P + 2), dict(dgates=P + 2), dict(lddc=199), dict(ldy=199), dict(lddy=199)):
        assert combine_grad(**bad) == BAD, bad
    for empty in (dict(T=0), dict(cols=0), dict(rows=0)):
        assert gather(X=None, slots=None, Y=None, **empty) == dg.GEMM_OK
    for empty in (dict(T=0), dict(cols=0)):
        assert combine(Y=None, slots=None, C=None, R=None, **empty) == dg.GEMM_OK
    assert combine_grad(T=0, dC=None, Y=None, dY=None, slots=None) == dg.GEMM_OK
    assert combine_grad(rows=0, dgates=None, dC=None, Y=None, dY=None, slots=None) == dg.GEMM_OK
    only_host(gather)
    only_host(combine)
    only_host(combine_grad)
    only_host(lambda: combine(rows=0, Y=None))                       # C <- R
    only_host(lambda: combine_grad(rows=0, Y=None, dY=None))         # dgates <- 0
    only_host(lambda: combine_grad(dgates=None, Y=None, ldy=0))


def test_conveniences_refuse_host_tensors():
    x, f = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4)
    i, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    g, o = torch.zeros(4, 2), torch.zeros(9, dtype=torch.int32)
    for call in (lambda: dg.layernorm(x, x), lambda: dg.layernorm_grad(x, x, x, f, f),
                 lambda: dg.dropout(x, x, 0.1, torch.zeros(2, dtype=torch.int64)),
                 lambda: dg.moe_route(x, g, i, i, o, o, w), lambda: dg.moe_route_grad(x, i, o, x),
                 lambda: dg.moe_gather(x, i, x), lambda: dg.moe_combine(x, i, x),
                 lambda: dg.moe_combine_grad(x, i, x)):
        with pytest.raises(TypeError):
            call()


# ---- the tests' own forms ---------------------------------------------------------

def test_generator_against_its_published_vectors():
    for c, k, want in (((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
                       ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
                       ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
                        (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        assert tuple(int(v) for v in philox(c, k)) == want


def test_dropout_form():
    u = dropout_bits(64, 1000, 12345, 6)
    assert u.shape == (64, 1000) and u.min() >= 0 and u.max() < 65536
    assert abs(u.mean() - 32767.5) < 5 * 65536 / np.sqrt(12 * u.size)
    y, keep = dropout_ref(np.ones((64, 1000)), None, 0.25, 12345, 6)
    assert np.array_equal(y != 0, keep) and np.allclose(y[keep], 4 / 3)
    assert not dropout_ref(np.ones((2, 9)), None, 1.0, 1, 2)[0].any()


def test_norm_form_against_differences():
    g = np.random.default_rng(3)
    x, w, b, dy = g.normal(size=(5, 33)), g.normal(size=33), g.normal(size=33), g.normal(size=(5, 33))
    y, m, r = norm_ref(x, w, b, 1e-3)
    dx, dw, db = norm_grad_ref(x, w, m, r, dy, None)
    for move, grad in ((0, dx), (1, dw), (2, db)):
        d = g.normal(size=grad.shape)
        f = lambda s: (dy * norm_ref(*(v + s * d if i == move else v for i, v in enumerate((x, w, b))), 1e-3)[0]).sum()
        assert abs((f(1e-5) - f(-1e-5)) / 2e-5 - (grad * d).sum()) < 1e-7 * (1 + np.abs(grad * d).sum())


@pytest.mark.parametrize("renormalize", [False, True])
def test_route_form_against_differences(renormalize):
    g = np.random.default_rng(4)
    l, dgates = g.normal(size=(7, 12)), g.normal(size=(7, 3))
    l[2, 4] = -np.inf
    l[5] = -np.inf
    l[6, 2:] = -np.inf                                           # two experts for three choices
    choice, gates, slots, offsets, counts, loss = route_ref(l, 3, renormalize)
    assert choice[6, 2] == -1 and (choice[5] == -1).all() and counts[-1] == 6
    d = g.normal(size=l.shape)
    f = lambda s: ((lambda o: (o[1] * dgates).sum() + 0.7 * o[5])(route_ref(l + s * d, 3, renormalize)))
    grad, _ = route_grad_ref(l, choice, counts, dgates, 0.7, renormalize)
    assert abs((f(1e-5) - f(-1e-5)) / 2e-5 - (grad * d).sum()) < 1e-7 * (1 + np.abs(grad * d).sum())
