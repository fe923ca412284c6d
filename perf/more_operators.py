"""The operators around the products of an expert-routed layer, as cases to measure.

Four operators, each through the library's entry points where `own` is true
and in elementary torch operations otherwise:

  route    a router's k choices of experts for every token with their gates,
           each expert's count and place among the rows sorted by expert, and
           the balance loss; and the gradient of gates and loss in the logits;
  rows     rows brought into that order (gather), the experts' results added
           up with their gates (combine), and combine's gradient;
  norm     layer norm, and its gradients in the input, weight and bias;
  dropout  with a mask drawn anew from a counter wherever it is needed, and a
           residual added. Its gradient is the same call.

Matrices are contiguous, as torch allocates them: rows of odd lengths start
at any element.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # One decoding step's routing: latency.
        {"name": "route-decode", "do": "route", "tokens": 16, "experts": 32, "k": 2,
         "renormalize": True, "dtype": "f32", "padded": 0},
        # A training step's tokens over many experts; the end of the batch is
        # padding, whose logits are all -infinity.
        {"name": "route-train", "do": "route", "tokens": 16384, "experts": 128, "k": 8,
         "renormalize": True, "dtype": "f32", "padded": 333},
        # The router's gradient in a smaller layer, its logits from a bf16
        # product; an odd number of tokens.
        {"name": "route-grad", "do": "route-grad", "tokens": 8191, "experts": 64, "k": 4,
         "renormalize": False, "dtype": "bf16", "padded": 100},
        # A prompt's tokens brought into the experts' order.
        {"name": "gather-prompt", "do": "gather", "tokens": 8191, "k": 2, "experts": 16,
         "cols": 4096, "padded": 0},
        # The results of many small experts added up on the residual.
        {"name": "combine-train", "do": "combine", "tokens": 4096, "k": 8, "experts": 64,
         "cols": 2048, "padded": 50, "residual": True},
        # The gradients of the experts' results and of the gates.
        {"name": "combine-grad", "do": "combine-grad", "tokens": 8192, "k": 2, "experts": 16,
         "cols": 4096, "padded": 0},
        # The norm before a decoding step's projections: latency.
        {"name": "norm-decode", "do": "norm", "rows": 16, "cols": 8192, "dtype": "bf16"},
        # The norm of a full batch of tokens.
        {"name": "norm-train", "do": "norm", "rows": 8192, "cols": 4096, "dtype": "bf16"},
        # Its gradients, added to the residual path's.
        {"name": "norm-grad", "do": "norm-grad", "rows": 8192, "cols": 4096, "dtype": "bf16",
         "residual": True},
        # In fp32, with rows that start at any multiple of 4 bytes.
        {"name": "norm-grad-ragged", "do": "norm-grad", "rows": 4095, "cols": 1023, "dtype": "f32",
         "residual": False},
        # A block's output dropped and added to the residual.
        {"name": "dropout-train", "do": "dropout", "rows": 8192, "cols": 4096, "dtype": "bf16",
         "p": 0.1, "residual": True},
        # Its gradient in fp32, at an odd size.
        {"name": "dropout-grad-ragged", "do": "dropout", "rows": 4095, "cols": 1023, "dtype": "f32",
         "p": 0.25, "residual": False},
    ]


def _log(rng, lo, hi, step=1):
    """A whole number in [lo, hi], a multiple of `step`, spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    do = rng.choice(("route", "route-grad", "gather", "combine", "combine-grad", "norm",
                     "norm-grad", "dropout"))
    step = rng.choice((1, 8, 128))
    if do in ("norm", "norm-grad", "dropout"):
        case = {"do": do, "rows": _log(rng, 1, 16384), "cols": _log(rng, 128, 12288, step),
                "dtype": rng.choice(("bf16", "bf16", "f32"))}
        while case["rows"] * case["cols"] > 8192 * 4096 // (1 if case["dtype"] == "bf16" else 2):
            case["rows"] = case["rows"] * 2 // 3
        if do != "norm":
            case["residual"] = rng.random() < 0.5
        if do == "dropout":
            case["p"] = rng.choice((0.05, 0.1, 0.2, 0.5))
        return case
    tokens = _log(rng, 1, 16384)
    case = {"do": do, "tokens": tokens, "experts": _log(rng, 8, 256, rng.choice((1, 8))),
            "k": rng.randint(1, 8), "padded": rng.choice((0, 0, rng.randint(0, tokens // 4)))}
    if do in ("route", "route-grad"):
        case["renormalize"] = rng.random() < 0.5
        case["dtype"] = rng.choice(("f32", "f32", "bf16"))
        return case
    case["cols"] = _log(rng, 256, 8192, step)
    while case["tokens"] * (case["k"] + 1) * case["cols"] > 8192 * 3 * 4096:
        case["tokens"] = max(1, case["tokens"] * 2 // 3)
    case["padded"] = min(case["padded"], case["tokens"] // 4)
    if do == "combine":
        case["residual"] = rng.random() < 0.5
    return case


# ---- inputs -----------------------------------------------------------------

def _logits(gen, case):
    """Normal logits on top of the experts' own levels; padding's are -infinity."""
    T, E = case["tokens"], case["experts"]
    like = torch.randn(E, generator=gen, device="cuda") * 0.7
    x = torch.randn(T, E, generator=gen, device="cuda") * 1.5 + like
    x[T - case["padded"]:] = -math.inf
    return x.to(DTYPES[case.get("dtype", "f32")])


def _normal(gen, rows, cols, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(rows, cols, generator=gen, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    do = case["do"]
    if do in ("route", "route-grad"):
        T, E, k = case["tokens"], case["experts"], case["k"]
        s["logits"] = _logits(gen, case)
        if do == "route":
            s["gates"] = torch.empty(T, k, device="cuda")
            s["choice"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            s["slots"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
            s["counts"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
            s["loss"] = torch.empty(1, device="cuda")
            if own:
                import dense_gemm_04_amd as dg
                s["work"] = torch.empty(dg.gemm_moe_route_workspace_size(T, E, k),
                                        dtype=torch.uint8, device="cuda")
        else:
            out = _route(s["logits"], k, case["renormalize"])
            s["choice"], s["counts"] = out["choice"], out["counts"]
            s["dgates"] = torch.randn(T, k, generator=gen, device="cuda") * 1e-2
            s["dloss"] = torch.full((1,), 1e-2, device="cuda") * (1 + torch.rand(1, generator=gen, device="cuda"))
            s["dlogits"] = torch.empty_like(s["logits"])
    elif do in ("gather", "combine", "combine-grad"):
        T, k, cols = case["tokens"], case["k"], case["cols"]
        out = _route(_logits(gen, case), k, True)
        s["slots"], s["gates"] = out["slots"], out["gates"]
        # Padding's share of the sorted rows stays as it is: zero here.
        if do == "gather":
            s["x"] = _normal(gen, T, cols)
            s["y"] = torch.zeros(T * k, cols, dtype=torch.bfloat16, device="cuda")
            return s
        s["y"] = _normal(gen, T * k, cols)
        if do == "combine":
            s["r"] = _normal(gen, T, cols) if case["residual"] else None
            s["c"] = torch.empty(T, cols, dtype=torch.bfloat16, device="cuda")
        else:
            s["dc"] = _normal(gen, T, cols, scale=1e-2)
            s["dy"] = torch.zeros(T * k, cols, dtype=torch.bfloat16, device="cuda")
            s["dgates"] = torch.empty(T, k, device="cuda")
    elif do in ("norm", "norm-grad"):
        rows, cols, dtype = case["rows"], case["cols"], DTYPES[case["dtype"]]
        # A residual stream: channels of different sizes and levels, a few by far.
        size = torch.exp(torch.randn(cols, generator=gen, device="cuda") * 0.5)
        size[torch.rand(cols, generator=gen, device="cuda") < 0.005] *= 20.0
        level = torch.randn(cols, generator=gen, device="cuda") * 0.3
        s["x"] = (torch.randn(rows, cols, generator=gen, device="cuda") * size + level).to(dtype)
        s["w"] = (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(dtype)
        s["b"] = (0.1 * torch.randn(cols, generator=gen, device="cuda")).to(dtype)
        if do == "norm":
            s["y"] = torch.empty_like(s["x"])
            s["mean"] = torch.empty(rows, device="cuda")
            s["rstd"] = torch.empty(rows, device="cuda")
        else:
            out = _norm(s["x"], s["w"], s["b"])
            s["mean"], s["rstd"] = out["mean"], out["rstd"]
            s["dy"] = _normal(gen, rows, cols, dtype, 1e-2)
            s["r"] = _normal(gen, rows, cols, dtype, 1e-2) if case["residual"] else None
            s["dx"] = torch.empty_like(s["x"])
            s["dw"], s["db"] = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
            if own:
                import dense_gemm_04_amd as dg
                s["work"] = torch.empty(dg.gemm_layernorm_grad_workspace_size(rows, cols),
                                        dtype=torch.uint8, device="cuda")
    else:
        rows, cols, dtype = case["rows"], case["cols"], DTYPES[case["dtype"]]
        s["x"] = _normal(gen, rows, cols, dtype)
        s["r"] = _normal(gen, rows, cols, dtype) if case["residual"] else None
        s["y"] = torch.empty_like(s["x"])
        # The generator's seed, and how often it has been drawn from.
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=gen, device="cuda")
    return s


# ---- plain forms ------------------------------------------------------------

def _softmax(logits):
    """Rows of -infinity alone have no probabilities: zeros."""
    top = logits.amax(1, keepdim=True)
    e = torch.where(top == -math.inf, torch.zeros_like(logits), torch.exp(logits - top))
    return e / e.sum(1, keepdim=True).clamp_min(1e-30)


def _route(logits, k, renormalize):
    l = logits.float()
    T, E = l.shape
    top, choice = torch.sort(l, dim=1, descending=True, stable=True)
    none = top[:, :k] == -math.inf
    choice = torch.where(none, -1, choice[:, :k])
    p = _softmax(l)
    gates = torch.where(none, 0.0, p.gather(1, choice.clamp_min(0)))
    if renormalize:
        gates = gates / gates.sum(1, keepdim=True).clamp_min(1e-30)
    flat = choice.flatten()
    counts = (flat[:, None] == torch.arange(E, device=l.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    slots = torch.empty_like(flat)
    slots[order] = torch.arange(T * k, device=l.device)
    slots = torch.where(flat < 0, -1, slots).view(T, k)
    tokens = (choice[:, 0] >= 0).sum()
    loss = E * (counts * p.sum(0)).sum() / (counts.sum() * tokens).clamp_min(1)
    return {"gates": gates, "choice": choice.int(), "slots": slots.int(), "offsets": offsets.int(),
            "counts": torch.cat([counts, tokens[None]]).int(), "loss": loss.view(1)}


def _route_grad(s):
    p = _softmax(s["logits"].float())
    T, E = p.shape
    counts, tokens = s["counts"][:E].float(), s["counts"][E].float()
    there = s["choice"] >= 0
    choice = torch.where(there, s["choice"], 0).long()
    dg = torch.where(there, s["dgates"], 0.0)
    a = (s["dloss"] * E * counts / (counts.sum() * tokens).clamp_min(1)).expand(T, E).clone()
    if not s["renormalize"]:
        a.scatter_add_(1, choice, dg)
    dl = p * (a - (a * p).sum(1, keepdim=True))
    if s["renormalize"]:
        g = torch.where(there, p.gather(1, choice), 0.0)
        g = g / g.sum(1, keepdim=True).clamp_min(1e-30)
        dl.scatter_add_(1, choice, g * (dg - (g * dg).sum(1, keepdim=True)))
    return {"dlogits": dl.to(s["logits"].dtype)}


def _norm(x, w, b):
    x32 = x.float()
    mean = x32.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((x32 - mean) ** 2).mean(1, keepdim=True) + EPS)
    y = (x32 - mean) * rstd * w.float() + b.float()
    return {"y": y.to(x.dtype), "mean": mean[:, 0].contiguous(), "rstd": rstd[:, 0].contiguous()}


def _norm_grad(s):
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if s["r"] is not None:
        dx = dx + s["r"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def _philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10: four 32-bit words of each counter, held in 64-bit integers."""
    low = 0xFFFFFFFF
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def _dropout(s):
    x, low = s["x"], 0xFFFFFFFF
    rows, cols = x.shape
    seed, offset = s["rng"][0], s["rng"][1]
    eights = -(-cols // 8)
    c0 = torch.arange(eights, device=x.device).expand(rows, eights)
    c1 = torch.arange(rows, device=x.device)[:, None].expand(rows, eights)
    words = _philox(c0, c1, offset & low, (offset >> 32) & low, seed & low, (seed >> 32) & low)
    words = torch.stack(words, 2)
    u = torch.stack([words & 0xFFFF, words >> 16], 3).view(rows, eights * 8)[:, :cols]
    drop = math.floor(s["p"] * 65536 + 0.5)
    y = torch.where(u >= drop, x.float() * (65536 / (65536 - drop)), 0.0)
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(x.dtype)}


def _plain(s):
    do = s["do"]
    if do == "route":
        return _route(s["logits"], s["k"], s["renormalize"])
    if do == "route-grad":
        return _route_grad(s)
    if do == "norm":
        return _norm(s["x"], s["w"], s["b"])
    if do == "norm-grad":
        return _norm_grad(s)
    if do == "dropout":
        return _dropout(s)
    slots = s["slots"].long()
    there = slots >= 0
    if do == "gather":
        y = s["y"]
        y[slots[there]] = s["x"][:, None, :].expand(-1, s["k"], -1)[there]
        return {"y": y}
    rows = torch.where(there[:, :, None], s["y"][slots.clamp_min(0)].float(), 0.0)
    if do == "combine":
        c = (rows * s["gates"][:, :, None]).sum(1)
        if s["r"] is not None:
            c = c + s["r"].float()
        return {"c": c.to(torch.bfloat16)}
    dc = s["dc"].float()
    dy = s["dy"]
    dy[slots[there]] = (dc[:, None, :] * s["gates"][:, :, None])[there].to(torch.bfloat16)
    return {"dy": dy, "dgates": (rows * dc[:, None, :]).sum(2)}


# ---- the library's calls ----------------------------------------------------

def _ptr(t):
    return None if t is None else t.data_ptr()


def _own(s):
    import dense_gemm_04_amd as dg
    stream = torch.cuda.current_stream().cuda_stream
    do, bf16 = s["do"], s.get("dtype") == "bf16"
    if do == "route":
        l = s["logits"]
        call = dg.gemm_moe_route_bf16 if bf16 else dg.gemm_moe_route_f32
        status = call(s["tokens"], s["experts"], s["k"], int(s["renormalize"]), l.data_ptr(), l.stride(0),
                      s["gates"].data_ptr(), s["choice"].data_ptr(), s["slots"].data_ptr(),
                      s["offsets"].data_ptr(), s["counts"].data_ptr(), s["loss"].data_ptr(),
                      s["work"].data_ptr(), s["work"].numel(), stream)
        out = {n: s[n] for n in ("gates", "choice", "slots", "offsets", "counts", "loss")}
    elif do == "route-grad":
        l, dl = s["logits"], s["dlogits"]
        call = dg.gemm_moe_route_grad_bf16 if bf16 else dg.gemm_moe_route_grad_f32
        status = call(s["tokens"], s["experts"], s["k"], int(s["renormalize"]), l.data_ptr(), l.stride(0),
                      s["choice"].data_ptr(), s["counts"].data_ptr(), s["dgates"].data_ptr(),
                      s["dloss"].data_ptr(), dl.data_ptr(), dl.stride(0), stream)
        out = {"dlogits": dl}
    elif do == "gather":
        x, y = s["x"], s["y"]
        status = dg.gemm_moe_gather_bf16(s["tokens"], s["k"], s["cols"], y.shape[0], x.data_ptr(), x.stride(0),
                                         s["slots"].data_ptr(), y.data_ptr(), y.stride(0), stream)
        out = {"y": y}
    elif do == "combine":
        y, r, c = s["y"], s["r"], s["c"]
        status = dg.gemm_moe_combine_bf16(s["tokens"], s["k"], s["cols"], y.shape[0], y.data_ptr(), y.stride(0),
                                          s["slots"].data_ptr(), s["gates"].data_ptr(), _ptr(r),
                                          0 if r is None else r.stride(0), c.data_ptr(), c.stride(0), stream)
        out = {"c": c}
    elif do == "combine-grad":
        y, dc, dy = s["y"], s["dc"], s["dy"]
        status = dg.gemm_moe_combine_grad_bf16(s["tokens"], s["k"], s["cols"], y.shape[0], dc.data_ptr(),
                                               dc.stride(0), y.data_ptr(), y.stride(0), s["slots"].data_ptr(),
                                               s["gates"].data_ptr(), dy.data_ptr(), dy.stride(0),
                                               s["dgates"].data_ptr(), stream)
        out = {"dy": dy, "dgates": s["dgates"]}
    elif do == "norm":
        x, y = s["x"], s["y"]
        call = dg.gemm_layernorm_bf16 if bf16 else dg.gemm_layernorm_f32
        status = call(s["rows"], s["cols"], EPS, x.data_ptr(), x.stride(0), s["w"].data_ptr(), s["b"].data_ptr(),
                      y.data_ptr(), y.stride(0), s["mean"].data_ptr(), s["rstd"].data_ptr(), stream)
        out = {n: s[n] for n in ("y", "mean", "rstd")}
    elif do == "norm-grad":
        x, dy, r, dx = s["x"], s["dy"], s["r"], s["dx"]
        call = dg.gemm_layernorm_grad_bf16 if bf16 else dg.gemm_layernorm_grad_f32
        status = call(s["rows"], s["cols"], x.data_ptr(), x.stride(0), s["w"].data_ptr(), s["mean"].data_ptr(),
                      s["rstd"].data_ptr(), dy.data_ptr(), dy.stride(0), _ptr(r), 0 if r is None else r.stride(0),
                      dx.data_ptr(), dx.stride(0), 0.0, s["dw"].data_ptr(), s["db"].data_ptr(),
                      s["work"].data_ptr(), s["work"].numel(), stream)
        out = {n: s[n] for n in ("dx", "dw", "db")}
    else:
        x, r, y = s["x"], s["r"], s["y"]
        call = dg.gemm_dropout_bf16 if bf16 else dg.gemm_dropout_f32
        status = call(s["rows"], s["cols"], s["p"], s["rng"].data_ptr(), x.data_ptr(), x.stride(0), _ptr(r),
                      0 if r is None else r.stride(0), y.data_ptr(), y.stride(0), stream)
        out = {"y": y}
    if status != dg.GEMM_OK:
        raise dg.GemmError(status)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    do = case["do"]
    if do in ("route", "route-grad"):
        T, E, k = case["tokens"], case["experts"], case["k"]
        wide = 2 if case["dtype"] == "bf16" else 4
        if do == "route":
            return {"bytes": T * E * wide + 12 * T * k + 8 * (E + 1) + 4, "flops": T * E * (4 + k)}
        return {"bytes": 2 * T * E * wide + 8 * T * k + 4 * (E + 1) + 4, "flops": 8 * T * E}
    if do in ("gather", "combine", "combine-grad"):
        T, k, cols = case["tokens"], case["k"], case["cols"]
        sent = (T - case["padded"]) * k
        if do == "gather":
            return {"bytes": 2 * cols * (T - case["padded"] + sent) + 4 * T * k, "flops": 0}
        if do == "combine":
            return {"bytes": 2 * cols * (sent + T * (2 if case["residual"] else 1)) + 8 * T * k,
                    "flops": 2 * sent * cols}
        return {"bytes": 2 * cols * (2 * sent + T - case["padded"]) + 12 * T * k, "flops": 3 * sent * cols}
    rows, cols = case["rows"], case["cols"]
    wide = 2 if case["dtype"] == "bf16" else 4
    if do == "norm":
        return {"bytes": wide * (2 * rows * cols + 2 * cols) + 8 * rows, "flops": 8 * rows * cols}
    if do == "norm-grad":
        passes = 4 if case["residual"] else 3
        return {"bytes": wide * (passes * rows * cols + cols) + 8 * rows + 8 * cols, "flops": 15 * rows * cols}
    return {"bytes": wide * rows * cols * (3 if case["residual"] else 2) + 16, "flops": 2 * rows * cols}


# ---- the operators' definitions in 64 bits ------------------------------------

def _probabilities(logits):
    l = logits.double()
    out = torch.zeros_like(l)
    some = (l > -math.inf).any(1)
    l = l[some]
    out[some] = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    return out


def _exact_route(s, case):
    """The choices by k searches for the largest, the places by counting."""
    l, k = s["logits"].double(), case["k"]
    T, E = l.shape
    p = _probabilities(s["logits"])
    number = torch.arange(E, device=l.device)
    left, choice, gates = l.clone(), [], []
    for _ in range(k):
        top = left.amax(1, keepdim=True)
        at = torch.where(left == top, number, E).amin(1)
        gone = top[:, 0] == -math.inf
        choice.append(torch.where(gone, -1, at))
        gates.append(torch.where(gone, 0.0, p[torch.arange(T, device=l.device), at]))
        left[torch.arange(T, device=l.device), at] = -math.inf
    choice, gates = torch.stack(choice, 1), torch.stack(gates, 1)
    if case["renormalize"]:
        total = gates.sum(1, keepdim=True)
        gates = torch.where(total > 0, gates / torch.where(total > 0, total, 1.0), 0.0)
    hit = (choice[:, :, None] == number).any(1).long()              # tokens x experts
    before = hit.cumsum(0) - hit
    counts = hit.sum(0)
    offsets = torch.zeros(E + 1, dtype=torch.long, device=l.device)
    offsets[1:] = torch.cumsum(counts, 0)
    place = offsets[:E] + before
    slots = torch.where(choice < 0, -1, place.gather(1, choice.clamp(min=0)))
    tokens = hit.any(1).sum()
    share = counts.double() / max(int(counts.sum()), 1)
    loss = E * (share * p.sum(0)).sum() / max(int(tokens), 1)
    return {"gates": gates, "choice": choice, "slots": slots, "offsets": offsets,
            "counts": torch.cat([counts, tokens.view(1)]), "loss": loss.view(1)}


def _exact_route_grad(s, case):
    """Row by row through the softmax's Jacobian, the gates' as that of the chosen alone."""
    p = _probabilities(s["logits"])
    T, E = p.shape
    counts = s["counts"].double()
    share = counts[:E] / max(float(counts[:E].sum()), 1.0)
    d = float(s["dloss"]) * E * share.expand(T, E) / max(float(counts[E]), 1.0)
    dl = p * d - p * (p * d).sum(1, keepdim=True)
    for t_there, j in ((s["choice"][:, j] >= 0, j) for j in range(case["k"])):
        t = torch.nonzero(t_there)[:, 0]
        e = s["choice"][t, j].long()
        dg = s["dgates"][t, j].double()
        if case["renormalize"]:
            chosen = torch.zeros(t.numel(), E, dtype=torch.bool, device=p.device)
            for i in range(case["k"]):
                has = s["choice"][t, i] >= 0
                chosen[has.nonzero()[:, 0], s["choice"][t, i][has].long()] = True
            q = torch.where(chosen, p[t], 0.0)
            q = q / q.sum(1, keepdim=True)
        else:
            q = p[t]
        g = torch.where(chosen, q, 0.0) if case["renormalize"] else q
        own_g = g.gather(1, e[:, None])
        part = -g * own_g
        part.scatter_add_(1, e[:, None], own_g)
        dl[t] += part * dg[:, None]
    return {"dlogits": dl}


def _mul32(a, b):
    """(high, low) 32-bit words of a * b by 16-bit halves."""
    al, ah, bl, bh = a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16
    mid = ah * bl + ((al * bl) >> 16)
    mid2 = al * bh + (mid & 0xFFFF)
    return ah * bh + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | ((al * bl) & 0xFFFF)


def _exact_dropout(s, case):
    """The generator's words one column of eight at a time, by 16-bit halves."""
    x = s["x"].double()
    rows, cols = x.shape
    seed, offset = (int(v) for v in s["rng"])
    drop = int(case["p"] * 65536 + 0.5)
    keep = torch.empty(rows, -(-cols // 8), 8, dtype=torch.bool, device=x.device)
    step = max(1, (1 << 22) // max(rows, 1))
    row = torch.arange(rows, device=x.device)[:, None]
    for lo in range(0, keep.shape[1], step):
        col = torch.arange(lo, min(lo + step, keep.shape[1]), device=x.device)[None, :]
        word = [col + 0 * row, row + 0 * col, torch.full_like(row + col, offset % 2 ** 32),
                torch.full_like(row + col, offset // 2 ** 32 % 2 ** 32)]
        for r in range(10):
            key = ((seed + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32)
            h0, l0 = _mul32(word[0], 0xD2511F53)
            h1, l1 = _mul32(word[2], 0xCD9E8D57)
            word = [h1 ^ word[1] ^ key[0], l1, h0 ^ word[3] ^ key[1], l0]
        for i, w in enumerate(word):
            keep[:, lo:lo + step, 2 * i] = (w & 0xFFFF) >= drop
            keep[:, lo:lo + step, 2 * i + 1] = (w >> 16) >= drop
    y = torch.where(keep.view(rows, -1)[:, :cols], x / (1 - drop / 65536), 0.0)
    return {"y": y if s["r"] is None else y + s["r"].double()}


def exact(case, seed):
    s = prepare(case, seed)
    do = case["do"]
    if do == "route":
        return _exact_route(s, case)
    if do == "route-grad":
        return _exact_route_grad(s, case)
    if do == "dropout":
        return _exact_dropout(s, case)
    if do in ("norm", "norm-grad"):
        x, w = s["x"].double(), s["w"].double()
        if do == "norm":
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = (var + EPS) ** -0.5
            return {"y": torch.addcmul(s["b"].double(), (x - mean[:, None]) * rstd[:, None], w),
                    "mean": mean, "rstd": rstd}
        dy, rstd = s["dy"].double(), s["rstd"].double()
        xh = (x - s["mean"].double()[:, None]) * rstd[:, None]
        n = x.shape[1]
        along = (torch.matmul(dy, w) / n)[:, None]
        onto = ((dy * xh) @ w / n)[:, None]
        dx = rstd[:, None] * (dy * w - along - xh * onto)
        return {"dx": dx if s["r"] is None else dx + s["r"].double(),
                "dw": torch.einsum("rc,rc->c", dy, xh), "db": dy.sum(0)}
    T, k, cols = case["tokens"], case["k"], case["cols"]
    if do == "gather":
        y = torch.zeros(T * k, cols, dtype=torch.float64, device="cuda")
    elif do == "combine":
        y = torch.zeros(T, cols, dtype=torch.float64, device="cuda") if s["r"] is None else s["r"].double()
    else:
        y = torch.zeros(T * k, cols, dtype=torch.float64, device="cuda")
        dgates = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = (s["slots"][:, j] >= 0).nonzero()[:, 0]
        slot = s["slots"][t, j].long()
        if do == "gather":
            y[slot] = s["x"][t].double()
        elif do == "combine":
            y[t] += s["gates"][t, j].double()[:, None] * s["y"][slot].double()
        else:
            dc = s["dc"][t].double()
            y[slot] = s["gates"][t, j].double()[:, None] * dc
            dgates[t, j] = (dc * s["y"][slot].double()).sum(1)
    if do == "combine-grad":
        return {"dy": y, "dgates": dgates}
    return {"y" if do == "gather" else "c": y}
