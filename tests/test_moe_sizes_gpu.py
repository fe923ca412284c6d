"""Routing at the sizes where its kernels change: 64 lanes to a token in two launches, more
than 8 choices on 16 lanes, and so many tokens that the workgroups' counts are added in
several rounds."""
import numpy as np
import pytest
import torch

import dense_gemm_04_amd as dg
from layer_util import BF16, F32, U, chain
from test_moe_gpu import INT, check_route, logits, note, run_route, test_route_grad as check_grad

pytestmark = pytest.mark.gpu

# tokens, experts, k
SIZES = [(300, 300, 5), (1000, 513, 16), (500, 1024, 16), (129, 1024, 1), (700, 700, 3), (200, 16, 16), (140, 40, 12),
         (300, 129, 9), (200, 256, 16), (2000, 32, 10), (128, 12, 11), (128, 400, 9)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_route(T, E, k, dtype):
    note(f"route {T} x {E} k {k} {dtype}")
    for renormalize in (True, False):
        l = logits(T, E, dtype, T + E + k)
        check_route(run_route(l, k, renormalize), l, k, renormalize)
        check_route(run_route(l, k, renormalize, E + 3, 1, with_loss=False), l, k, renormalize)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_route_gradient(T, E, k, dtype):
    check_grad(T, E, k, dtype)


@pytest.mark.parametrize("T,E,k,dtype", [(300000, 1024, 1, F32), (300000, 1024, 2, BF16), (2200000, 8, 1, F32),
                                         (2200000, 12, 3, BF16)])
def test_counts_added_in_several_rounds(T, E, k, dtype):
    """Nine tenths of the tokens choose one expert, so its 16-bit counts are as large as
    they get. The other logits are equal, and the chosen ones known."""
    note(f"route {T} x {E} k {k} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(T + E)
    first = torch.randint(0, E, (T, 1), generator=g, device="cuda")
    first[torch.rand(T, generator=g, device="cuda") < 0.9] = 5
    choice = (first + torch.arange(k, device="cuda")) % E
    l = torch.zeros(T, E, dtype=dtype, device="cuda")
    l.scatter_(1, choice, (4.0 - torch.arange(k, device="cuda")).to(dtype).expand(T, k))
    l[7::1000] = -float("inf")                           # padding
    some = torch.ones(T, dtype=torch.bool, device="cuda")
    some[7::1000] = False
    out = {n: torch.full((T, k), 9, dtype=d, device="cuda") for n, d in (("gates", F32), ("choice", INT), ("slots", INT))}
    out |= {n: torch.full((E + 1,), 9, dtype=INT, device="cuda") for n in ("offsets", "counts")}
    loss = torch.full((1,), 9.0, device="cuda")
    ws = torch.full((dg.gemm_moe_route_workspace_size(T, E, k),), 0xff, dtype=torch.uint8, device="cuda")
    dg.moe_route(l, out["gates"], out["choice"], out["slots"], out["offsets"], out["counts"], ws, loss)

    assert torch.equal(out["choice"], torch.where(some[:, None], choice, -1).to(INT))
    flat = choice[some].flatten()
    counts = torch.bincount(flat, minlength=E)
    assert torch.equal(out["counts"][:E].long(), counts) and int(out["counts"][E]) == int(some.sum())
    assert torch.equal(out["offsets"].long(), torch.cat([counts.new_zeros(1), counts.cumsum(0)]))
    order = flat.sort(stable=True).indices
    slots = torch.empty_like(order)
    slots[order] = torch.arange(order.numel(), device="cuda")
    assert torch.equal(out["slots"][some].flatten().long(), slots)
    assert bool((out["slots"][~some] == -1).all()) and not bool(out["gates"][~some].any())

    e = torch.exp(4.0 - torch.arange(k, dtype=torch.float64, device="cuda") - 4.0)
    want = e / e.sum()
    # exp's own steps and its argument's, the sum's and the division's, twice over.
    assert bool(((out["gates"][some].double() - want).abs() <= (2 * k + 32) * U * want).all())
    others = float(np.exp(-4.0))
    p = torch.full((E,), others * float(some.sum()), dtype=torch.float64, device="cuda")
    for j in range(k):
        p += torch.bincount(choice[some][:, j], minlength=E) * (e[j] - others)
    p /= float(e.sum()) + (E - k) * others
    balance = E * float((counts.double() / order.numel() * p).sum()) / float(some.sum())
    # A p goes through the additions of its thread (tokens of a workgroup by 8 at once), of lanes, waves
    # and workgroups, and through the sum over the experts; 48 U for the p itself and the quotients.
    assert abs(float(loss) - balance) <= (T / 256 / 8 + 256 + chain(E, 1) + 48) * U * balance
