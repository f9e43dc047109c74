"""The serving operators in float64, from the definitions in
include/fp8bs_serve.h, with the error bounds that the kernels' roundings leave."""

import numpy as np

U16 = 2.0 ** -8       # relative error of rounding to BF16 (at most, to nearest)
U32 = 2.0 ** -24

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def fp4_quant(x):
    """x [n][512] float64 (BF16 numbers) -> (codes uint8 [n][256], exponent bytes
    uint8 [n][16]): nearest E2M1 number, halfway to the even code."""
    g = np.asarray(x, np.float64).reshape(len(x), 16, 32)
    amax = np.abs(g).max(-1)
    e = np.full(amax.shape, -126)
    while (small := amax > 6.0 * np.ldexp(1.0, e)).any():
        e[small] += 1
    e[amax == 0] = 0
    y = np.abs(g) / np.ldexp(1.0, e)[..., None]
    far = np.abs(y[..., None] - E2M1)                       # exact: differences of short numbers
    near = far == far.min(-1, keepdims=True)                # one, or the two neighbours of a middle
    even = np.arange(8) % 2 == 0
    code = np.where(near.sum(-1) == 1, near.argmax(-1), (near & even).argmax(-1)).astype(np.uint8)
    code |= (np.signbit(g).astype(np.uint8) << 3)
    code = code.reshape(len(x), 512)
    return code[:, ::2] | (code[:, 1::2] << 4), (e + 127).astype(np.uint8)


def fp4_values(codes, exps):
    """codes uint8 [..][256], exps uint8 [..][16] -> float64 [..][512]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 512)
    v = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    return v * np.repeat(np.ldexp(1.0, exps.astype(np.int64) - 127), 32, -1)


def slots(table, lens, cu, page, rows):
    """(page, slot in it, whether there is such a position) of each packed row,
    page -1 for rows of no request."""
    at = np.full((rows, 3), -1, np.int64)
    for b in range(len(lens)):
        for t in range(cu[b], cu[b + 1]):
            pos = int(lens[b]) - (int(cu[b + 1]) - t)
            ok = 0 <= pos < table.shape[1] * page
            at[t] = (table[b, pos // page] if ok else 0, pos % page if ok else 0, int(ok))
    return at


def silu(z):
    return z / (1.0 + np.exp(-z))


def moe_tokens(x, ids, weights, up, down):
    """x [T][K], ids and weights [T][topk], up [E][2F][K], down [E][K][F] (values).
    Returns (out, bound): FP32 products and sums, h and the output rounded to BF16."""
    T, K = x.shape
    E, F = len(up), up.shape[1] // 2
    out, bound = np.zeros((T, K)), np.full((T, K), 1e-30)
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < E:
                continue
            a, size = up[e] @ x[t], np.abs(up[e]) @ np.abs(x[t])
            g, u, eg, eu = a[:F], a[F:], K * U32 * size[:F], K * U32 * size[F:]
            h = silu(g) * u
            # |silu'| <= 1.1; the exponential and the quotient add a few steps of FP32
            dh = 1.1 * eg * (np.abs(u) + eu) + (np.abs(silu(g)) + 1.1 * eg) * eu + (U16 + 16 * U32) * np.abs(h)
            y, ysize = down[e] @ h, np.abs(down[e]) @ np.abs(h)
            w = float(weights[t, j])
            out[t] += w * y
            bound[t] += abs(w) * (np.abs(down[e]) @ dh + (F + 64) * U32 * ysize)
    return out, bound + U16 * np.abs(out)


def logprobs(x, targets, top):
    """x [T][V] float64: {name: value} with bounds {name: bound} of the computed numbers."""
    T, V = x.shape
    r = dict(logprob=np.zeros(T), entropy=np.zeros(T), norm=np.zeros((T, 2)), rank=np.zeros(T, np.int64),
             top_ids=np.zeros((T, top), np.int64), top_logprobs=np.zeros((T, top)))
    b = dict(logprob=np.zeros(T), entropy=np.zeros(T), norm=np.zeros((T, 2)), top_logprobs=np.zeros((T, top)))
    for t in range(T):
        row, y = x[t], int(targets[t])
        order = np.lexsort((np.arange(V), -(row + 0.0)))
        m = row.max()
        none = m == -np.inf
        d = np.where(row == -np.inf, -np.inf, row - (0 if none else m))
        e = np.exp(d)
        total = 1.0 if none else e.sum()
        n = np.log(total)
        with np.errstate(invalid="ignore"):
            mean = float(np.where(e > 0, e * d, 0.0).sum() / total)
        r["norm"][t], r["entropy"][t] = (m, n), n - mean
        # a term exp(d) errs by |d| 2^-23 (its exponent's rounding) and 2^-22, a sum of V terms in a tree by 64 steps
        rel = -mean * 2.0 ** -22 + 2.0 ** -18
        b["norm"][t] = 0.0, rel + 2 * U32 * n
        b["entropy"][t] = rel * (1 - mean)
        size = np.where(np.isfinite(d), np.abs(d), 0.0) + n
        if 0 <= y < V:
            r["logprob"][t], b["logprob"][t] = d[y] - n, rel + 4 * U32 * size[y]
            r["rank"][t] = np.flatnonzero(order == y)[0]
        else:
            r["rank"][t] = -1
        best = order[:top]
        r["top_ids"][t], r["top_logprobs"][t], b["top_logprobs"][t] = best, d[best] - n, rel + 4 * U32 * size[best]
    return r, b


def logprobs_bwd(x, targets, dl, dh, half_step):
    """Gradient of sum(dl * logprob + dh * entropy) and its bound; half_step: of
    the type it is rounded to."""
    T, V = x.shape
    out, bound = np.zeros((T, V)), np.full((T, V), 1e-30)
    for t in range(T):
        row, y = x[t], int(targets[t])
        m = row.max()
        if m == -np.inf:
            continue
        n = np.log(np.exp(row - m).sum())
        lp = (row - m) - n
        p = np.exp(lp)
        with np.errstate(invalid="ignore"):
            h = -np.where(p > 0, p * lp, 0.0).sum()
            token = 0 <= y < V
            g = float(dl[t]) if token else 0.0
            # p errs by its exponent's rounding and n's error, log p + entropy by both
            far = np.where(p > 0, np.abs(lp), 0.0)
            rel = 2.0 ** -17 * (1 + h) + (far + n) * 2.0 ** -22
            part = np.where(p > 0, p * (lp + h), 0.0)
            out[t] = -g * p - float(dh[t]) * part
            bound[t] += (abs(g) * p + abs(float(dh[t])) * p * (far + h + 1)) * rel
        if token:
            out[t, y] += g
            bound[t, y] += 4 * U32 * abs(g)
        bound[t] += half_step * np.abs(out[t])
    return out, bound
