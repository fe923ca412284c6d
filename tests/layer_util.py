"""Plain 64-bit forms of layer norm, dropout, the router and its rows, for
their tests, and the allowances of their results.

Allowances, derived once here. U = 2^-24 is fp32's half step, relative.
  * A result of n elements off by at most half a step of its type: 2^-8 of its
    value in bf16, 2^-24 in fp32.
  * A sum over a row: every kernel adds in at least 16 chains of equal
    lengths that meet in a tree, so a term goes through at most n / 16 + 16
    additions, each off by at most U of the running sum of magnitudes:
    chain(n) U of the sum of the terms' magnitudes. Sums down columns likewise
    with at least 4 chains.
  * exp is off by a few U (4 are allowed), and by U times its argument's
    magnitude from the argument's own rounding; a softmax's sum as the mean of
    those over the terms, and x exp(-x) <= 0.37 keeps that below 8 U for up to
    1024 terms.
"""
import math

import numpy as np
import torch

from ops_util import f64

U = 2.0 ** -24
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BF16, F32 = torch.bfloat16, torch.float32


def chain(n, chains=16):
    return n / chains + 16


def worst(got, want, allow):
    """Largest error over its allowance (1 or less passes); NaN and infinities have to agree."""
    got = f64(got) if torch.is_tensor(got) else np.asarray(got, dtype=np.float64)
    want = np.asarray(want, dtype=np.float64)
    assert got.shape == want.shape, (got.shape, want.shape)
    if not got.size:
        return 0.0
    special = ~np.isfinite(want)
    same = np.where(special, (got == want) | (np.isnan(got) & np.isnan(want)), np.isfinite(got))
    if not same.all():
        return math.inf
    err = np.abs(np.where(special, 0.0, got) - np.where(special, 0.0, want))
    allow = np.where(special, 1.0, np.broadcast_to(allow, want.shape))
    return float(np.max(np.where(err == 0, 0.0, err / np.maximum(allow, 1e-37))))


# ---- layer norm ---------------------------------------------------------------

def norm_ref(x, w, b, eps):
    """y, mean, rstd in 64 bits (w, b or None)."""
    m = x.mean(1)
    d = x - m[:, None]
    r = 1 / np.sqrt((d * d).mean(1) + eps)
    y = d * r[:, None]
    return (y if w is None else y * w) + (0.0 if b is None else b), m, r


def norm_allow(x, w, b, eps, dtype):
    """Allowances of y, mean and rstd. The mean is off by chain U mean|x| (dm); the
    variance by (chain + 4) U of itself and dm^2 (the differences sum to zero),
    so r by half of that and two steps; a difference by dm and a step."""
    y, m, r = norm_ref(x, w, b, eps)
    n = x.shape[1]
    dm = (chain(n) + 2) * U * np.abs(x).mean(1)
    rel = (chain(n) / 2 + 4) * U + 0.5 * dm * dm * r * r
    ww = 1.0 if w is None else np.abs(w)
    h = np.abs(x - m[:, None]) * r[:, None]
    ay = ww * (dm * r)[:, None] + ww * h * (rel[:, None] + 4 * U) + (0 if b is None else U * np.abs(b))
    return ay + (STEP[dtype] + U) * np.abs(y), dm + U * np.abs(m), r * rel


def norm_grad_ref(x, w, mean, rstd, dy, res):
    h = (x - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - h * (g * h).mean(1, keepdims=True))
    return dx + (0.0 if res is None else res), (dy * h).sum(0), dy.sum(0)


def norm_grad_allow(x, w, mean, rstd, dy, res, dtype):
    """h carries 2 steps, g one; their means chain(n) and what the terms carry; dx
    a few more for each of its terms. dw and db: sums down the rows."""
    n, rows = x.shape[1], x.shape[0]
    h = np.abs((x - mean[:, None]) * rstd[:, None])
    g = np.abs(dy if w is None else dy * w)
    mg, mgh = g.mean(1, keepdims=True), (g * h).mean(1, keepdims=True)
    dx, _, _ = norm_grad_ref(x, w, mean, rstd, dy, res)
    core = rstd[:, None] * (6 * U * (g + mg + h * mgh) + U * (chain(n) + 6) * (mg + h * mgh))
    adx = core + (0 if res is None else 2 * U * np.abs(res)) + (STEP[dtype] + 2 * U) * np.abs(dx)
    down = (chain(rows, 4) + 48) * U
    return adx, down * (np.abs(dy) * h).sum(0), down * np.abs(dy).sum(0)


# ---- dropout --------------------------------------------------------------------

def philox(counter, key):
    """Philox 4x32 of 10 rounds on arrays of 32-bit words (in 64-bit integers)."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [np.uint64(v) for v in key]
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ k[0], b & low, (a >> half) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return c


def dropout_bits(rows, cols, seed, offset):
    """u(i, j) of 16 bits each."""
    seed, offset = seed % (1 << 64), offset % (1 << 64)
    n8 = -(-cols // 8)
    ones = np.ones((rows, n8), dtype=np.uint64)
    w = philox((ones * np.arange(n8, dtype=np.uint64)[None, :], ones * np.arange(rows, dtype=np.uint64)[:, None],
                ones * np.uint64(offset & 0xFFFFFFFF), ones * np.uint64(offset >> 32)),
               (seed & 0xFFFFFFFF, seed >> 32))
    u = np.stack([h for v in w for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))], 2)
    return u.reshape(rows, n8 * 8)[:, :cols].astype(np.int64)


def dropout_ref(x, res, p, seed, offset):
    t = int(math.floor(np.float32(p) * 65536 + 0.5))
    keep = dropout_bits(*x.shape, seed, offset) >= t
    scale = 65536.0 / (65536 - t) if t < 65536 else 0.0
    return np.where(keep, np.where(keep, x, 0.0) * scale, 0.0) + (0.0 if res is None else res), keep


# ---- router ----------------------------------------------------------------------

def softmax_ref(l):
    """Rows of -infinity: zeros. Rows with a NaN or +infinity: NaN."""
    bad = (np.isnan(l) | (l == np.inf)).any(1)
    m = np.where(bad, 0.0, l.max(1, initial=-np.inf))
    m = np.where(np.isfinite(m), m, 0.0)
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.where(bad[:, None], 0.0, np.exp(np.where(bad[:, None], 0.0, l) - m[:, None]))
    s = e.sum(1)
    p = e / np.where(s > 0, s, 1.0)[:, None]
    p[bad] = np.nan
    return p, bad


def route_ref(l, k, renormalize):
    """Choices, gates, slots, offsets, counts and loss, token by token."""
    T, E = l.shape
    p, bad = softmax_ref(l)
    choice = np.full((T, k), -1, dtype=np.int64)
    gates = np.zeros((T, k))
    for t in range(T):
        if bad[t]:
            gates[t] = np.nan
            continue
        order = sorted((e for e in range(E) if l[t, e] > -np.inf), key=lambda e: (-l[t, e], e))[:k]
        choice[t, :len(order)] = order
        g = p[t, order]
        gates[t, :len(order)] = g / g.sum() if renormalize and len(order) else g
    counts = np.array([(choice == e).sum() for e in range(E)], dtype=np.int64)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    nxt, slots = offsets[:E].copy(), np.full((T, k), -1, dtype=np.int64)
    for t in range(T):
        for j in range(k):
            if choice[t, j] >= 0:
                slots[t, j] = nxt[choice[t, j]]
                nxt[choice[t, j]] += 1
    tokens = int((choice[:, 0] >= 0).sum()) if T else 0
    loss = E * (counts / max(counts.sum(), 1) * p.sum(0)).sum() / max(tokens, 1)
    return choice, gates, slots, offsets, np.concatenate([counts, [tokens]]), loss


def spread(l):
    """Each row's distances from its largest logit (0 where there is none)."""
    top = l.max(1, keepdims=True, initial=-np.inf)
    with np.errstate(invalid="ignore"):
        d = top - l
    return np.where(np.isfinite(d), d, 0.0)


def prob_rel(l):
    """Relative allowance of each p: the exponential's, the sum's and the division's."""
    return (spread(l) + chain(l.shape[1]) + 8 + 4 + 4) * U


def route_grad_ref(l, choice, counts, dgates, dloss, renormalize):
    """(gradient, magnitude its errors scale with)."""
    T, E = l.shape
    p, bad = softmax_ref(l)
    total, tokens = counts[:E].sum(), counts[E]
    a = np.zeros((T, E))
    if dloss is not None and total > 0:
        a += dloss * E * counts[:E] / (total * tokens)
    extra, mag = np.zeros((T, E)), np.zeros((T, E))
    if dgates is not None:
        for t in range(T):
            c = choice[t][choice[t] >= 0]
            d = dgates[t][choice[t] >= 0]
            if not len(c):
                continue
            if renormalize:
                q = p[t, c] / p[t, c].sum()
                extra[t, c] += q * (d - (q * d).sum())
                mag[t, c] += q * (np.abs(d) + (q * np.abs(d)).sum())
            else:
                a[t, c] += d
    out = p * (a - (a * p).sum(1, keepdims=True)) + extra
    return out, p * (np.abs(a) + (np.abs(a) * p).sum(1, keepdims=True)) + mag
