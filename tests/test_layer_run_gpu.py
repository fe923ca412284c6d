"""An expert-routed layer as a program runs it, forward and backward:

    h = norm(x), router logits h Wr, the tokens' rows into the experts' order,
    the experts' products, their results back with the gates, dropout, residual

against the same in 64 bits (with the calls' choices and dropout mask), alone,
replayed from a graph, and twice at once on two streams.

Allowance: a result passes through at most 8 roundings to bf16 on its way (each
at most 2^-8 of what it rounds, and the maps between them at most double a
relative error here: weights of gain about 1, gates below 1, a norm of rows of
unit spread), so the 2-norm of its error stays below 8 * 2 * 2^-8 = 1/16 of its
own; the rounding errors are spread evenly over half a step and are
independent, which leaves a third of that and less.
"""
import numpy as np
import pytest
import torch

import dense_gemm_04_amd as dg
from layer_util import BF16, F32, dropout_ref
from ops_util import f64, gen

pytestmark = pytest.mark.gpu

INT = torch.int32
DROP, EPS = 0.2, 1e-5


class Layer:
    """Weights, inputs and every buffer of one pass."""

    def __init__(self, T, D, E, k, seed):
        g = gen(seed)
        bf = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(BF16).cuda()
        new = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device="cuda")
        self.sizes = T, D, E, k
        self.x, self.dout = bf(T, D), bf(T, D)
        self.w, self.b = (1 + 0.1 * bf(D).float()).to(BF16), bf(D, scale=0.1)
        self.wr, self.we = bf(D, E, scale=D ** -0.5 * 2), bf(E, D, D, scale=D ** -0.5)
        self.rng = torch.tensor([99, 0], dtype=torch.int64, device="cuda")
        self.dloss = torch.tensor([3.0], device="cuda")
        self.h, self.c, self.out, self.dc, self.dh, self.dx, self.dlr = (new(T, D) for _ in range(7))
        self.xs, self.ys, self.dys, self.dxs = (torch.zeros(T * k, D, dtype=BF16, device="cuda") for _ in range(4))
        self.logits, self.dlogits = new(T, E), new(T, E)
        self.mean, self.rstd = new(T, dtype=F32), new(T, dtype=F32)
        self.gates, self.dgates = new(T, k, dtype=F32), new(T, k, dtype=F32)
        self.choice, self.slots = new(T, k, dtype=INT), new(T, k, dtype=INT)
        self.offsets, self.counts, self.loss = new(E + 1, dtype=INT), new(E + 1, dtype=INT), new(1, dtype=F32)
        self.dwr, self.dwe = new(D, E), new(E, D, D, dtype=F32)
        self.dw, self.db = new(D, dtype=F32), new(D, dtype=F32)
        self.ws = new(max(dg.gemm_moe_route_workspace_size(T, E, k), dg.gemm_layernorm_grad_workspace_size(T, D)),
                      dtype=torch.uint8)

    def step(self):
        T, D, E, k = self.sizes
        dg.layernorm(self.x, self.h, self.w, self.b, EPS, self.mean, self.rstd)
        dg.matmul_bf16(self.h, self.wr, self.logits)
        dg.moe_route(self.logits, self.gates, self.choice, self.slots, self.offsets, self.counts, self.ws, self.loss)
        dg.moe_gather(self.h, self.slots, self.xs)
        dg.matmul_bf16_grouped(self.xs, self.we, self.ys, self.offsets)
        dg.moe_combine(self.ys, self.slots, self.c, self.gates)
        dg.dropout(self.c, self.out, DROP, self.rng, self.x)
        # Backward.
        dg.dropout(self.dout, self.dc, DROP, self.rng)
        dg.moe_combine_grad(self.dc, self.slots, self.dys, self.ys, self.gates, self.dgates)
        dg.grouped_wgrad(self.xs, self.dys, self.dwe, self.offsets)
        dg.matmul_bf16_grouped(self.dys, self.we, self.dxs, self.offsets, dg.OP_T)
        dg.moe_route_grad(self.logits, self.choice, self.counts, self.dlogits, self.dgates, self.dloss)
        stream = torch.cuda.current_stream().cuda_stream
        for st in (dg.gemm_bf16_op(dg.OP_T, dg.OP_N, D, E, T, 1.0, self.h.data_ptr(), D, self.dlogits.data_ptr(), E, 0.0,
                                   self.dwr.data_ptr(), E, stream=stream),
                   dg.gemm_bf16_op(dg.OP_N, dg.OP_T, T, D, E, 1.0, self.dlogits.data_ptr(), E, self.wr.data_ptr(), E, 0.0,
                                   self.dlr.data_ptr(), D, stream=stream)):
            assert st == dg.GEMM_OK
        dg.moe_combine(self.dxs, self.slots, self.dh, None, self.dlr)
        dg.layernorm_grad(self.x, self.dh, self.dx, self.mean, self.rstd, self.w, self.dout, self.dw, self.db, 0.0,
                          self.ws)

    RESULTS = ("out", "loss", "dx", "dw", "db", "dwr", "dwe", "choice", "slots", "offsets", "counts", "gates")

    def results(self):
        return {n: getattr(self, n).clone() for n in self.RESULTS}

    def in_64_bits(self):
        T, D, E, k = self.sizes
        leaf = lambda t: torch.from_numpy(f64(t)).requires_grad_()
        x, w, b, wr, we = (leaf(t) for t in (self.x, self.w, self.b, self.wr, self.we))
        h = (x - x.mean(1, keepdim=True)) / (x.var(1, correction=0, keepdim=True) + EPS).sqrt() * w + b
        p = torch.softmax(h @ wr, 1)
        choice = self.choice.cpu().long()
        gates = p.gather(1, choice)
        gates = gates / gates.sum(1, keepdim=True)
        c = torch.zeros(T, D, dtype=torch.float64)
        for e in range(E):
            t, j = torch.nonzero(choice == e, as_tuple=True)
            c = c.index_add(0, t, gates[t, j][:, None] * (h[t] @ we[e]))
        counts = torch.bincount(choice.flatten(), minlength=E).double()
        loss = E * (counts / counts.sum() * p.mean(0)).sum()
        _, keep = dropout_ref(np.ones((T, D)), None, DROP, *(int(v) for v in self.rng))
        drop = int(DROP * 65536 + 0.5)
        out = x + c * torch.from_numpy(keep) * (65536 / (65536 - drop))
        ((out * torch.from_numpy(f64(self.dout))).sum() + float(self.dloss) * loss).backward()
        return {"out": out, "loss": loss.view(1), "dx": x.grad, "dw": w.grad, "db": b.grad, "dwr": wr.grad, "dwe": we.grad}


@pytest.mark.parametrize("T,D,E,k", [(200, 256, 8, 2), (77, 200, 5, 3), (1, 128, 4, 1), (1500, 512, 16, 4)])
def test_layer_against_64_bits(T, D, E, k):
    print(f"layer {T} x {D}, {E} experts, {k} choices", flush=True)
    layer = Layer(T, D, E, k, T)
    layer.step()
    got = layer.results()
    for name, want in layer.in_64_bits().items():
        want = want.detach().numpy()
        off, size = np.linalg.norm(f64(got[name]) - want), np.linalg.norm(want)
        # With one choice the gates are 1 whatever the logits.
        assert off <= size / 16 + 1e-6, (name, off, size)


def same(a, b):
    return [n for n in a if not torch.equal(a[n], b[n])]


def test_layer_replayed_from_a_graph():
    layer = Layer(300, 256, 8, 2, 1)
    layer.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    for turn in range(4):
        layer.x.copy_(torch.randn(300, 256, generator=gen(50 + turn)))
        layer.rng[1] = turn
        layer.step()
        want = layer.results()
        for n in Layer.RESULTS:
            getattr(layer, n).zero_()
        layer.ws.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        assert not same(layer.results(), want)


def test_layers_on_two_streams_at_once():
    layers = [Layer(900, 256, 8, 2, 3), Layer(700, 512, 16, 4, 4)]
    wants = []
    for layer in layers:
        layer.step()
        wants.append(layer.results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for layer, stream in zip(layers, streams):
            with torch.cuda.stream(stream):
                layer.step()
    torch.cuda.synchronize()
    for layer, want in zip(layers, wants):
        assert not same(layer.results(), want)
