"""The operators of a quantised or expert-routed linear layer, as cases to measure.

Four operators, each through the library's entry points where `own` is true
and in elementary torch operations otherwise:

  quantize  e4m3 values and fp32 scales of blocks of 128 (or 128 x 128)
            values along the dimension a product sums over, of a matrix or of
            its transpose;
  fp8       the product of two such matrices, C = sum over blocks b of
            SA(i,b) SB(j,b) sum over k in b of A(i,k) B(j,k);
  grouped   rows sorted by expert, each group of rows times its expert's
            matrix (stored K x N, or N x K for the input's gradient);
  wgrad     the gradient of the experts' matrices, X_e^T dY_e for each group.

Rows of every operand start at multiples of 16 bytes, as an allocator of
activations or weights lays them out; the sizes themselves may be odd.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
# Below this a block's largest value no longer makes its scale smaller, which
# stays a normal number.
MIN_TOP = E4M3_MAX * 2.0 ** -126
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # A decoding batch's activations before a product in 8 bits: latency.
        {"name": "quantize-decode", "do": "quantize", "rows": 16, "cols": 8192, "dtype": "bf16",
         "transpose": False, "block_rows": 1},
        # The gradient of a prompt-sized batch, transposed and quantised along
        # its tokens for the weight gradient; an odd number of tokens.
        {"name": "quantize-tokens-T", "do": "quantize", "rows": 8191, "cols": 4096,
         "dtype": "bf16", "transpose": True, "block_rows": 1},
        # fp32 master weights to 8 bits after an optimizer step.
        {"name": "quantize-weights", "do": "quantize", "rows": 12288, "cols": 4096,
         "dtype": "f32", "transpose": False, "block_rows": 128},
        # One decoding step's projection: 16 rows against a large weight.
        {"name": "fp8-decode", "do": "fp8", "M": 16, "N": 8192, "K": 8192, "block_rows": 128},
        # A short ragged prompt, with a last block of K that is not whole.
        {"name": "fp8-ragged", "do": "fp8", "M": 509, "N": 4096, "K": 4000, "block_rows": 128},
        # The projection of a full batch of tokens.
        {"name": "fp8-projection", "do": "fp8", "M": 8192, "N": 12288, "K": 4096,
         "block_rows": 128},
        # A weight's gradient in 8 bits: both operands quantised along the
        # tokens in blocks of 1 x 128.
        {"name": "fp8-wgrad", "do": "fp8", "M": 4096, "N": 4096, "K": 8192, "block_rows": 1},
        # One decoding step of 32 experts: a few rows each, some with none.
        {"name": "grouped-decode", "do": "grouped", "groups": 32, "rows": 64, "spare": 0,
         "N": 4096, "K": 2048, "transpose": False},
        # A prompt's tokens sorted by expert.
        {"name": "grouped-prefill", "do": "grouped", "groups": 16, "rows": 16384, "spare": 0,
         "N": 4096, "K": 4096, "transpose": False},
        # The gradient of the experts' input, weights read as they are stored;
        # a buffer larger than this step's rows.
        {"name": "grouped-dgrad", "do": "grouped", "groups": 8, "rows": 8001, "spare": 191,
         "N": 4096, "K": 2048, "transpose": True},
        # The experts' weight gradient of a training step, in fp32.
        {"name": "wgrad-train", "do": "wgrad", "groups": 16, "rows": 16384, "spare": 0,
         "N": 2048, "K": 4096, "out": "f32"},
        # A small model's, in bf16, with few rows for each expert.
        {"name": "wgrad-small", "do": "wgrad", "groups": 8, "rows": 999, "spare": 25,
         "N": 1024, "K": 1024, "out": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    """A whole number in [lo, hi], a multiple of `step`, spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    do = rng.choice(("quantize", "fp8", "grouped", "wgrad"))
    step = rng.choice((1, 8, 128))
    if do == "quantize":
        return {"do": do, "rows": _log(rng, 1, 8192), "cols": _log(rng, 128, 12288, step),
                "dtype": rng.choice(("bf16", "bf16", "f32")), "transpose": rng.random() < 0.4,
                "block_rows": rng.choice((1, 1, 128))}
    if do == "fp8":
        case = {"do": do, "M": _log(rng, 1, 8192), "N": _log(rng, 256, 12288, step),
                "K": _log(rng, 256, 8192, rng.choice((1, 16, 128))),
                "block_rows": rng.choice((1, 128, 128))}
        while case["M"] * case["N"] * case["K"] > 8192 * 12288 * 4096:
            case["M"] = case["M"] * 2 // 3
        return case
    case = {"do": do, "groups": _log(rng, 2, 64), "rows": _log(rng, 1, 16384),
            "spare": rng.choice((0, 0, rng.randint(1, 300))),
            "N": _log(rng, 256, 4096, step), "K": _log(rng, 256, 4096, rng.choice((8, 64, 128)))}
    if do == "grouped":
        case["transpose"] = rng.random() < 0.5
    else:
        case["out"] = rng.choice(("bf16", "f32"))
    most = (8 if case.get("out") == "f32" else 16) * 4096 * 4096
    while case["groups"] * case["N"] * case["K"] > most:
        case["groups"] = case["groups"] * 2 // 3
    return case


# ---- inputs -----------------------------------------------------------------

def _rows16(rows, cols, dtype):
    """An uninitialised rows x cols matrix whose rows start at multiples of 16 bytes."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.empty(rows, -(-cols // per) * per, dtype=dtype, device="cuda")[:, :cols]


def _normal(gen, rows, cols, dtype, scale=1.0):
    x = _rows16(rows, cols, dtype)
    x.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * scale)
    return x


def _activations(gen, rows, cols, dtype):
    """Normal values whose channels differ in size, a few of them by far."""
    size = torch.exp(torch.randn(cols, generator=gen, device="cuda") * 0.5)
    size[torch.rand(cols, generator=gen, device="cuda") < 0.005] *= 20.0
    x = _rows16(rows, cols, dtype)
    x.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * size)
    return x


def _lengths(seed, groups, rows):
    """How many rows each expert gets: a router with preferences of its own."""
    rng = np.random.default_rng(seed)
    like = np.exp(rng.normal(0.0, 0.7, groups))
    return rng.multinomial(rows, like / like.sum())


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["do"] == "quantize":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _activations(gen, rows, cols, DTYPES[case["dtype"]])
        r, c = (cols, rows) if case["transpose"] else (rows, cols)
        s["q"] = _rows16(r, c, torch.uint8)
        s["s"] = torch.empty(-(-c // 128), -(-r // case["block_rows"]), device="cuda")
    elif case["do"] == "fp8":
        M, N, K = case["M"], case["N"], case["K"]
        for name, rows, per, make in (("a", M, 1, _activations), ("b", N, case["block_rows"], _normal)):
            q, s["s" + name] = _quantize(make(gen, rows, K, torch.float32), per)
            s[name] = _rows16(rows, K, torch.uint8)
            s[name].copy_(q.view(torch.uint8))
        s["c"] = _rows16(M, N, torch.bfloat16)
    else:
        E, N, K, rows = case["groups"], case["N"], case["K"], case["rows"]
        lengths = _lengths(seed, E, rows)
        s["lengths"], s["longest"] = lengths, max(1, int(lengths.max()))
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
        s["x"] = _normal(gen, rows + case["spare"], K, torch.bfloat16)
        if case["do"] == "grouped":
            w = (N, K) if case["transpose"] else (K, N)
            s["w"] = _normal(gen, E * w[0], w[1], torch.bfloat16, 1.0 / math.sqrt(K)).unflatten(0, (E, w[0]))
            s["y"] = _rows16(rows + case["spare"], N, torch.bfloat16).zero_()
        else:
            s["dy"] = _normal(gen, rows + case["spare"], N, torch.bfloat16)
            s["dw"] = _rows16(E * K, N, DTYPES[case["out"]]).unflatten(0, (E, K))
    return s


# ---- plain forms ------------------------------------------------------------

def _quantize(x, block_rows):
    """(e4m3 values, scales [blocks of columns][blocks of rows]) of a matrix.

    A bf16 value divided by its block's scale often lies exactly between two
    e4m3 values; in 64 bits it stays there."""
    rows, cols = x.shape
    nb, nr = -(-cols // 128), -(-rows // block_rows)
    full = torch.zeros(nr * block_rows, nb * 128, device=x.device)
    full[:rows, :cols] = x
    blocks = full.view(nr, block_rows, nb, 128)
    top = blocks.abs().amax(dim=(1, 3)).clamp_min(MIN_TOP)
    q = (blocks.double() * E4M3_MAX / top.double()[:, None, :, None]).float().to(torch.float8_e4m3fn)
    return q.view(nr * block_rows, nb * 128)[:rows, :cols], (top / E4M3_MAX).t().contiguous()


def _dequantize(q, scale, block_rows):
    rows, cols = q.shape
    full = scale.t().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return q.view(torch.float8_e4m3fn).float() * full


def _by_group(x, s):
    """[groups, longest, columns] in fp32, zeros past each group's rows, and where each row went."""
    row = torch.arange(s["rows"], device=x.device)
    group = torch.searchsorted(s["offsets"][1:], row, right=True)
    place = row - s["offsets"][group]
    padded = torch.zeros(s["groups"], s["longest"], x.shape[1], device=x.device)
    padded[group, place] = x[:s["rows"]].float()
    return padded, group, place


def _plain(s):
    if s["do"] == "quantize":
        q, scale = _quantize(s["x"].float().t() if s["transpose"] else s["x"].float(), s["block_rows"])
        return {"q": q, "s": scale}
    if s["do"] == "fp8":
        a = _dequantize(s["a"], s["sa"], 1)
        b = _dequantize(s["b"], s["sb"], s["block_rows"])
        return {"c": torch.matmul(a, b.t()).to(torch.bfloat16)}
    x, group, place = _by_group(s["x"], s)
    if s["do"] == "grouped":
        w = s["w"].float()
        y = torch.bmm(x, w.transpose(1, 2) if s["transpose"] else w)
        out = torch.zeros(s["x"].shape[0], s["N"], dtype=torch.bfloat16, device=x.device)
        out[:s["rows"]] = y[group, place].to(torch.bfloat16)
        return {"y": out}
    dy, _, _ = _by_group(s["dy"], s)
    return {"dw": torch.bmm(x.transpose(1, 2), dy).to(DTYPES[s["out"]])}


# ---- the library's calls ----------------------------------------------------

def _own(s):
    import dense_gemm_04_amd as dg
    stream = torch.cuda.current_stream().cuda_stream
    if s["do"] == "quantize":
        x, q, scale = s["x"], s["q"], s["s"]
        call = dg.gemm_fp8_quantize_bf16 if s["dtype"] == "bf16" else dg.gemm_fp8_quantize_f32
        status = call(dg.OP_T if s["transpose"] else dg.OP_N, s["block_rows"], s["rows"], s["cols"],
                      x.data_ptr(), x.stride(0), q.data_ptr(), q.stride(0), scale.data_ptr(),
                      scale.stride(0), stream)
        out = {"q": q.view(torch.float8_e4m3fn), "s": scale}
    elif s["do"] == "fp8":
        a, b, c, sa, sb = s["a"], s["b"], s["c"], s["sa"], s["sb"]
        status = dg.gemm_fp8(s["M"], s["N"], s["K"], 1.0, a.data_ptr(), a.stride(0),
                             sa.data_ptr(), sa.stride(0), b.data_ptr(), b.stride(0),
                             sb.data_ptr(), sb.stride(0), s["block_rows"], 0.0, c.data_ptr(),
                             c.stride(0), None, dg.ACT_NONE, stream)
        out = {"c": c}
    elif s["do"] == "grouped":
        x, w, y = s["x"], s["w"], s["y"]
        status = dg.gemm_bf16_grouped(
            dg.OP_T if s["transpose"] else dg.OP_N, s["groups"], x.shape[0], s["N"], s["K"], 1.0,
            x.data_ptr(), x.stride(0), w.data_ptr(), w.stride(1), w.stride(0), 0.0, y.data_ptr(),
            y.stride(0), s["offsets"].data_ptr(), None, None, 0, dg.ACT_NONE, stream)
        out = {"y": y}
    else:
        x, dy, dw = s["x"], s["dy"], s["dw"]
        call = dg.gemm_bf16_grouped_wgrad if s["out"] == "bf16" else dg.gemm_bf16_grouped_wgrad_f32
        status = call(s["groups"], x.shape[0], s["N"], s["K"], 1.0, x.data_ptr(), x.stride(0),
                      dy.data_ptr(), dy.stride(0), 0.0, dw.data_ptr(), dw.stride(1), dw.stride(0),
                      s["offsets"].data_ptr(), stream)
        out = {"dw": dw}
    if status != dg.GEMM_OK:
        raise dg.GemmError(status)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    if case["do"] == "quantize":
        r, c = (case["cols"], case["rows"]) if case["transpose"] else (case["rows"], case["cols"])
        scales = -(-c // 128) * -(-r // case["block_rows"])
        wide = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": r * c * (wide + 1) + 4 * scales, "flops": 3 * r * c}
    N, K = case["N"], case["K"]
    if case["do"] == "fp8":
        M = case["M"]
        scales = -(-K // 128) * (M + -(-N // case["block_rows"]))
        return {"bytes": (M + N) * K + 2 * M * N + 4 * scales, "flops": 2 * M * N * K}
    E, rows = case["groups"], case["rows"]
    flops = 2 * rows * N * K
    if case["do"] == "grouped":
        # Of the experts' matrices, those of experts with rows; at most one a row.
        return {"bytes": 2 * (min(E, rows) * N * K + rows * (N + K)), "flops": flops}
    wide = 2 if case["out"] == "bf16" else 4
    return {"bytes": 2 * rows * (N + K) + wide * E * N * K, "flops": flops}


# ---- the operators' definitions in 64 bits ------------------------------------

def _e4m3_table():
    """Every finite value of the format, ascending: 4 exponent bits (bias 7), 3 of mantissa."""
    small = [m * 2.0 ** -9 for m in range(8)]
    rest = [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)]
    return torch.tensor(small + rest, dtype=torch.float64, device="cuda")


def _nearest_e4m3(v):
    """v rounded to the nearest value of the format, ties to the even one."""
    table = _e4m3_table()
    mag = v.abs().clamp(max=E4M3_MAX)
    above = torch.searchsorted(table, mag).clamp(max=table.numel() - 1)
    below = (above - 1).clamp(min=0)
    up, down = table[above] - mag, mag - table[below]
    take = torch.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
    return torch.copysign(table[take], v)


def exact(case, seed):
    s = prepare(case, seed)
    if case["do"] == "quantize":
        x = s["x"].double()
        x = x.t() if case["transpose"] else x
        r, c = x.shape
        per = case["block_rows"]
        q, scales = torch.empty(r, c, dtype=torch.float64, device="cuda"), []
        for k in range(0, c, 128):
            part = x[:, k:k + 128]
            top = part.abs().amax(1)
            top = torch.nn.functional.pad(top, (0, -r % per)).view(-1, per).amax(1)
            top = top.clamp(min=448 * 2.0 ** -126)
            q[:, k:k + 128] = _nearest_e4m3(part * 448 / top.repeat_interleave(per)[:r, None])
            scales.append(top / 448)
        return {"q": q, "s": torch.stack(scales)}
    if case["do"] == "fp8":
        total = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
        column = torch.arange(case["N"], device="cuda") // case["block_rows"]
        for b, k in enumerate(range(0, case["K"], 128)):
            left = s["a"][:, k:k + 128].view(torch.float8_e4m3fn).float().double() * s["sa"][b].double()[:, None]
            right = s["b"][:, k:k + 128].view(torch.float8_e4m3fn).float().double() * s["sb"][b].double()[column][:, None]
            total.addmm_(left, right.t())
        return {"c": total}
    ends = np.cumsum(s["lengths"])
    if case["do"] == "grouped":
        y = torch.zeros(s["x"].shape[0], case["N"], dtype=torch.float64, device="cuda")
        for e, end in enumerate(ends):
            lo, w = int(end - s["lengths"][e]), s["w"][e].double()
            y[lo:int(end)] = s["x"][lo:int(end)].double() @ (w.t() if case["transpose"] else w)
        return {"y": y}
    dw = torch.zeros(case["groups"], case["K"], case["N"], dtype=torch.float64, device="cuda")
    for e, end in enumerate(ends):
        lo = int(end - s["lengths"][e])
        dw[e] = s["x"][lo:int(end)].double().t() @ s["dy"][lo:int(end)].double()
    return {"dw": dw}
