"""Latent attention and draft verification in float64 (exact integers where the
definition has them), with the error bounds that BF16 rounding of the kernels'
operands leaves. Written from the definitions in include/fp8bs_attn.h."""

import numpy as np

U16 = 2.0 ** -8       # relative error of rounding to BF16, 8 significant bits (at most, to nearest)
U32 = 2.0 ** -24


def _visible(lq, lk, causal):
    i, j = np.arange(lq)[:, None], np.arange(lk)[None, :]
    return (j <= i + lk - lq) if causal else np.ones((lq, lk), bool)


def softmax_rows(S, visible):
    """(P, lse): rows with nothing visible give P = 0, lse = -inf."""
    S = np.where(visible, S, -np.inf)
    m = S.max(-1, initial=-np.inf, keepdims=True)
    e = np.exp(S - np.where(np.isfinite(m), m, 0.0))
    total = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, np.where(np.isfinite(m), m, 0.0) + np.log(total), -np.inf)[..., 0]
    return e / np.where(total > 0, total, 1.0), lse


def mla_head(q, k, v, scale, causal):
    """One head of one request: out, lse and the error bounds of both.

    A score is an FP32 sum of n products (error n * 2^-24 of their absolute
    sum), which moves its weight by that relative amount; the weight is then
    rounded to BF16, the output too."""
    vis = _visible(len(q), len(k), causal)
    P, lse = softmax_rows(q @ k.T * scale, vis)
    size = np.where(vis, np.abs(q) @ np.abs(k).T * scale, 0.0).max(-1, initial=0.0, keepdims=True)
    d = 2 * q.shape[1] * U32 * size + 2.0 ** -19
    out = P @ v
    bound = (U16 + 2 * d) * (P @ np.abs(v)) + U16 * np.abs(out) + 1e-30
    return out, lse, bound, d[:, 0] + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))


def mla_head_bwd(q, k, v, dout, scale, causal):
    """Gradients (dq, dk, dv) of one head and their bounds. D is formed from the
    BF16 output, P and dS are rounded to BF16 as operands."""
    vis = _visible(len(q), len(k), causal)
    P, _ = softmax_rows(q @ k.T * scale, vis)
    size = np.where(vis, np.abs(q) @ np.abs(k).T * scale, 0.0).max(-1, initial=0.0, keepdims=True)
    d = 4 * q.shape[1] * U32 * size + 2.0 ** -18
    out = P @ v
    dP = dout @ v.T
    D = (dout * out).sum(-1, keepdims=True)
    dS = P * (dP - D)
    err_out = (U16 + 2 * d) * (P @ np.abs(v)) + U16 * np.abs(out)
    err_D = (np.abs(dout) * err_out).sum(-1, keepdims=True)
    abs_dP = np.abs(dout) @ np.abs(v).T
    err_dS = P * (2 * d * (np.abs(dP) + np.abs(D)) + err_D + 256 * U32 * abs_dP) + U16 * np.abs(dS)
    slack = 2.0 ** -14                # FP32 sums over the tokens
    dq, dk, dv = dS @ k * scale, dS.T @ q * scale, P.T @ dout
    bq = scale * ((err_dS + slack * np.abs(dS)) @ np.abs(k)) + U16 * np.abs(dq) + 1e-30
    bk = scale * ((err_dS + slack * np.abs(dS)).T @ np.abs(q)) + U16 * np.abs(dk) + 1e-30
    bv = ((U16 + slack + 2 * d) * P).T @ np.abs(dout) + U16 * np.abs(dv) + 1e-30
    return (dq, dk, dv), (bq, bk, bv)


def mla_prefill(q, kv, k_rope, cu_q, cu_k, scale, causal, dout=None):
    """Packed requests, head by head: {name: (value, bound)} of out, lse and,
    with dout, dq, dkv, dk_rope."""
    Tq, H, _ = q.shape
    Tk = kv.shape[0]
    r = {"out": np.zeros((2, Tq, H, 128)), "lse": np.zeros((2, H, Tq))}
    r["lse"][0] = -np.inf
    if dout is not None:
        r.update(dq=np.zeros((2, Tq, H, 192)), dkv=np.zeros((2, Tk, H, 256)), dk_rope=np.zeros((2, Tk, 64)))
    for b in range(len(cu_q) - 1):
        i, j = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        for h in range(H):
            Q, V = q[i, h], kv[j, h, 128:]
            K = np.concatenate([kv[j, h, :128], k_rope[j]], -1)
            out, lse, bo, bl = mla_head(Q, K, V, scale, causal)
            r["out"][0, i, h], r["out"][1, i, h] = out, bo
            r["lse"][0, h, i], r["lse"][1, h, i] = lse, bl
            if dout is not None:
                g, e = mla_head_bwd(Q, K, V, dout[i, h], scale, causal)
                for n, (x, y) in enumerate(zip(g, e)):
                    if n == 0:
                        r["dq"][0, i, h], r["dq"][1, i, h] = x, y
                    elif n == 1:
                        r["dkv"][0, j, h, :128], r["dkv"][1, j, h, :128] = x[:, :128], y[:, :128]
                        r["dk_rope"][0, j] += x[:, 128:]
                        r["dk_rope"][1, j] += y[:, 128:]
                    else:
                        r["dkv"][0, j, h, 128:], r["dkv"][1, j, h, 128:] = x, y
    if dout is not None:
        r["dk_rope"][1] += U16 * np.abs(r["dk_rope"][0])
    return {k: (v[0], v[1]) for k, v in r.items()}


def mla_decode(q, keys, scale):
    """q [B][T][H][576] against keys[b] [n][576]; query t sees n - (T-1-t) of
    them (those before `fixed[b]` always, where keys[b] is a (fixed, keys)
    pair). Returns out, lse and their bounds."""
    B, T, H, _ = q.shape
    out, bound = np.zeros((B, T, H, 512)), np.zeros((B, T, H, 512))
    lse, lbound = np.full((B, T, H), -np.inf), np.zeros((B, T, H))
    for b in range(B):
        fixed, k = keys[b] if isinstance(keys[b], tuple) else (0, keys[b])
        for t in range(T):
            n = max(len(k) - (T - 1 - t), min(fixed, len(k)))
            if n <= 0:
                continue
            o, l, bo, bl = mla_head(q[b, t], k[:n], k[:n, :512], scale, False)
            out[b, t], lse[b, t], bound[b, t], lbound[b, t] = o, l, bo, bl
    return out, lse, bound, lbound


def verify_drafts(p, q, drafts, n_drafts, u, u_next):
    """Acceptance and next token, one request and one vocabulary entry at a
    time, float32 comparisons and exact integers."""
    B, K1, V = p.shape
    tokens, accepted = np.full((B, K1), -1, np.int32), np.zeros(B, np.int32)

    def weights(r):
        r = np.where(r > 0, np.minimum(r, np.float32(1)), np.float32(0)).astype(np.float64)
        return [int(x) for x in np.floor(r * 2.0 ** 38)]

    for b in range(B):
        n, a = int(min(max(n_drafts[b], 0), K1 - 1)), 0
        while a < n:
            x = int(drafts[b, a])
            if not 0 <= x < V:
                break
            qx = np.float32(1) if q is None else q[b, a, x]
            if not np.float32(u[b, a]) * qx < p[b, a, x]:
                break
            a += 1
        accepted[b] = a
        tokens[b, :a] = drafts[b, :a]
        w = weights(p[b, a])
        if a < n:
            if q is None:
                r = list(w)
                if 0 <= drafts[b, a] < V:
                    r[int(drafts[b, a])] = 0
            else:
                with np.errstate(invalid="ignore"):
                    r = weights(p[b, a] - q[b, a])
            if sum(r) > 0:
                w = r
        total = sum(w)
        if total > 0:
            goal = total * int(min(max(float(u_next[b]), 0.0), 1 - 2.0 ** -24) * 2 ** 24) >> 24
            run = 0
            for i, x in enumerate(w):
                run += x
                if run > goal:
                    tokens[b, a] = i
                    break
    return tokens, accepted
