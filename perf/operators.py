"""The attention and draft-verification operators: what is measured of them.

Five operators, in the two forms that `run` has:

  prefill   latent attention, expanded form: every head has its own keys and values (128 + 128 numbers a token,
            as the up-projection of the latent vector writes them) and shares one 64-wide rotary key
  train     the same with its gradients
  decode    latent attention, absorbed form: queries against the cached latent vectors themselves, one shared
            576-wide key a token whose first 512 numbers are also its value, in pages of a BF16 or FP8 cache
  shared    the absorbed form for a batch that shares a long prefix, computed once for all requests
  verify    acceptance of drafted tokens against the target's probabilities, and the token that follows them

With ``own`` false, `run` computes them from elementary torch operations in 32 bits; with ``own`` true it calls the
package. `exact` is written apart from both, in 64 bits.
"""

import math
import random

import torch

own = False

NOPE, ROPE, VDIM, LATENT = 128, 64, 128, 512     # numbers per head and token; the latent vector's width
QK = NOPE + ROPE
KEY = LATENT + ROPE
GROUP = 128                                      # FP8 cache: latent numbers that share one scale
SCALE = 1.0 / math.sqrt(QK)
WEIGHT_BITS = 38                                 # verify: sampling weights are whole multiples of 2^-38
MAX_SCORES = 1 << 28                             # scores that the plain form holds at a time


def _spread(low, high, n, seed):
    """n lengths of a ragged batch between low and high, fixed by seed."""
    r = random.Random(seed)
    return [r.randint(low, high) for _ in range(n)]


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # a scheduler's step over a handful of short prompts, one of them a single token: a small launch
        dict(name="prefill_short_ragged", op="prefill", batch=5, heads=8, new_low=1, new_high=300, past_low=0,
             past_high=0, len_seed=1, causal=True),
        # one chunk of a long prompt against all that was cached before it
        dict(name="prefill_chunk_on_context", op="prefill", batch=2, heads=32, new_low=500, new_high=600,
             past_low=7000, past_high=8000, len_seed=2, causal=True),
        # whole long prompts on all 128 heads: the largest matrix work
        dict(name="prefill_long", op="prefill", batch=2, heads=128, new_low=6000, new_high=8192, past_low=0,
             past_high=0, len_seed=3, causal=True),
        # a packed training batch of short documents with odd lengths
        dict(name="train_short_ragged", op="train", batch=6, heads=8, new_low=1, new_high=260, past_low=0,
             past_high=0, len_seed=4, causal=True),
        # a training sequence of 4096 tokens on 64 heads
        dict(name="train_4096", op="train", batch=1, heads=64, new_low=4096, new_high=4096, past_low=0, past_high=0,
             len_seed=5, causal=True),
        # one request, one token, a short context, 16 heads: pure latency
        dict(name="decode_one", op="decode", batch=1, heads=16, tokens=1, len_low=257, len_high=257, len_seed=6,
             page=64, cache="bf16"),
        # a full serving batch with ragged contexts, all 128 heads on one GPU
        dict(name="decode_batch_128_heads", op="decode", batch=128, heads=128, tokens=1, len_low=300, len_high=4500,
             len_seed=7, page=64, cache="bf16"),
        # long contexts in the FP8 cache, two tokens a request (one drafted), 16 heads: few rows, much to read
        dict(name="decode_long_fp8", op="decode", batch=8, heads=16, tokens=2, len_low=40000, len_high=70000,
             len_seed=8, page=64, cache="fp8"),
        # a few requests behind a short common instruction
        dict(name="shared_small", op="shared", batch=6, heads=16, tokens=1, prefix=1000, len_low=1, len_high=150,
             len_seed=9, page=16, cache="bf16"),
        # a large batch behind one long system prompt
        dict(name="shared_system_prompt", op="shared", batch=192, heads=32, tokens=1, prefix=16000, len_low=16,
             len_high=900, len_seed=10, page=64, cache="bf16"),
        # one request with one drafted token, a large vocabulary: pure latency
        dict(name="verify_one", op="verify", batch=1, drafts=1, vocab=129280, accept=0.3),
        # a serving batch with up to four drafted tokens a request
        dict(name="verify_batch", op="verify", batch=96, drafts=4, vocab=129280, accept=0.7),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["prefill", "train", "decode", "shared", "verify"])
    seed = rng.randrange(1 << 30)
    if op in ("prefill", "train"):
        limit = 4.0e12 if op == "prefill" else 1.2e12
        while True:
            high = _log_int(rng, 1, 8192 if op == "prefill" else 4096)
            low = max(1, int(high * rng.uniform(0.05, 1.0)))
            past = _log_int(rng, 1, 12000) if op == "prefill" and rng.random() < 0.4 else 0
            case = dict(op=op, batch=_log_int(rng, 1, 12), heads=rng.choice([1, 3, 8, 20, 32, 64, 128]), new_low=low,
                        new_high=high, past_low=past // 2, past_high=past, len_seed=seed,
                        causal=rng.random() < 0.8)
            if work(case)["flops"] <= limit and sum(k for _, k in _prefill_lengths(case)) * case["heads"] <= 3_000_000:
                return case
    if op in ("decode", "shared"):
        while True:
            shared = op == "shared"
            high = _log_int(rng, 1, 1500 if shared else 70000)
            case = dict(op=op, batch=_log_int(rng, 2 if shared else 1, 192), heads=rng.choice([1, 5, 16, 32, 64, 128]),
                        tokens=rng.choice([1, 1, 1, 2, 3, 4]), len_low=max(1, int(high * rng.uniform(0.02, 1.0))),
                        len_high=high, len_seed=seed, page=rng.choice([1, 16, 17, 64, 128]),
                        cache=rng.choice(["bf16", "fp8"]))
            if shared:
                case["prefix"] = _log_int(rng, 1, 16000)
            case["len_low"] = max(case["len_low"], case["tokens"])
            case["len_high"] = max(case["len_high"], case["len_low"])
            w = work(case)
            if w["flops"] <= 2.0e11 and case["batch"] * case["len_high"] <= 600_000:
                return case
    return dict(op=op, batch=_log_int(rng, 1, 96), drafts=rng.randint(1, 6), vocab=_log_int(rng, 5, 129280),
                accept=rng.choice([0.0, 0.3, 0.7, 1.0]))


def _prefill_lengths(case):
    new = _spread(case["new_low"], case["new_high"], case["batch"], case["len_seed"])
    past = _spread(case["past_low"], case["past_high"], case["batch"], case["len_seed"] + 1)
    return [(n, n + p) for n, p in zip(new, past)]


def _decode_lengths(case):
    return _spread(case["len_low"], case["len_high"], case["batch"], case["len_seed"])


def work(case):
    op = case["op"]
    if op in ("prefill", "train"):
        H, lens = case["heads"], _prefill_lengths(case)
        tq, tk = sum(q for q, _ in lens), sum(k for _, k in lens)
        pairs = sum(q * k - (q * (q - 1) // 2 if case["causal"] else 0) for q, k in lens)
        read = 2 * (tq * H * QK + tk * H * (NOPE + VDIM) + tk * ROPE)
        wrote = 2 * tq * H * VDIM + 4 * tq * H
        flops = 2 * pairs * H * (QK + VDIM)
        if op == "train":        # q, kv, k_rope and out once, dout read, three gradients written; S, dP, dV, dK, dQ
            return {"bytes": 2 * read + 2 * tq * H * VDIM * 2, "flops": flops + 2 * pairs * H * (3 * QK + 2 * VDIM)}
        return {"bytes": read + wrote, "flops": flops}
    if op in ("decode", "shared"):
        rows = case["tokens"] * case["heads"]
        lens = _decode_lengths(case)
        token = 2 * KEY if case["cache"] == "bf16" else LATENT + 4 * (LATENT // GROUP) + 2 * ROPE
        hidden = case["tokens"] * (case["tokens"] - 1) // 2 * case["heads"]
        prefix = case.get("prefix", 0)
        pairs = sum(rows * (n + prefix) - hidden for n in lens)
        io = len(lens) * rows * (2 * KEY + 2 * LATENT + 4)
        return {"bytes": (sum(lens) + prefix) * token + io, "flops": 2 * pairs * (KEY + LATENT)}
    # the row that the next token is drawn from, of both models where a draft was turned down
    return {"bytes": int(4 * case["batch"] * case["vocab"] * (2 - case["accept"] ** case["drafts"])),
            "flops": 3 * case["batch"] * case["vocab"]}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def _cache(case, g, pages):
    page = case["page"]
    rope = _normal(g, (pages, page, ROPE))
    latent = _normal(g, (pages, page, LATENT))
    if case["cache"] == "bf16":
        return torch.cat([latent, rope], dim=-1).contiguous()
    codes = torch.empty((pages, page, LATENT), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, page, LATENT // GROUP), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (page * LATENT))
    for a in range(0, pages, step):
        x = latent[a:a + step].float().reshape(-1, page, LATENT // GROUP, GROUP)
        s = x.abs().amax(-1) / 448.0
        s = torch.where(s == 0, torch.ones_like(s), s)
        scales[a:a + step] = s
        codes[a:a + step] = (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1, page, LATENT)
    return codes, scales, rope


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = {"op": op, "case": dict(case)}
    if op in ("prefill", "train"):
        H, lens = case["heads"], _prefill_lengths(case)
        tq, tk = sum(q for q, _ in lens), sum(k for _, k in lens)
        st.update(lens=lens, cu_q=_offsets([q for q, _ in lens]), cu_k=_offsets([k for _, k in lens]),
                  q=_normal(g, (tq, H, QK), 1.5), kv=_normal(g, (tk, H, NOPE + VDIM)), k_rope=_normal(g, (tk, ROPE)))
        if op == "train":
            st["dout"] = _normal(g, (tq, H, VDIM), 0.01)
    elif op in ("decode", "shared"):
        B, page, lens = case["batch"], case["page"], _decode_lengths(case)
        prefix = case.get("prefix", 0)
        most = max(-(-n // page) for n in lens)
        shared = -(-prefix // page)
        # pages in no order, as a pool hands them out after a while
        pool = torch.randperm(B * most + shared, generator=g, device="cuda").to(torch.int32)
        st.update(lens=lens, cache=_cache(case, g, B * most + shared), table=pool[:B * most].reshape(B, most).contiguous(),
                  seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                  q=_normal(g, (B, case["tokens"], case["heads"], KEY)))
        if op == "shared":
            st.update(prefix=prefix, prefix_table=pool[B * most:].contiguous(),
                      prefix_len=torch.tensor([prefix], dtype=torch.int32, device="cuda"))
    else:
        B, K, V = case["batch"], case["drafts"], case["vocab"]
        p = torch.softmax(2.0 * torch.randn((B, K + 1, V), generator=g, device="cuda"), -1)
        # the draft model's distribution is near the target's; `accept` of the drafts are ones that it accepts
        q = torch.softmax(torch.log(p[:, :K]) + 0.7 * torch.randn((B, K, V), generator=g, device="cuda"), -1)
        drafts = torch.argmax(torch.log(q) - torch.log(-torch.log(
            torch.rand((B, K, V), generator=g, device="cuda").clamp_min(1e-20))), -1).to(torch.int32)
        ratio = (p[:, :K].gather(2, drafts[..., None].long()) / q.gather(2, drafts[..., None].long()))[..., 0]
        u = torch.rand((B, K), generator=g, device="cuda")
        take = torch.rand((B, K), generator=g, device="cuda") < case["accept"]
        # below the ratio: accepted; above it: turned down where the ratio leaves room for that
        u = torch.where(take, u * ratio.clamp(max=1.0) * 0.99, ratio + (1.0 - ratio) * u).clamp(0.0, 1.0 - 2.0 ** -24)
        st.update(p=p, q=q, drafts=drafts, u=u, u_next=torch.rand(B, generator=g, device="cuda"),
                  n_drafts=torch.full((B,), K, dtype=torch.int32, device="cuda"))
    return st


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


def _run_own(st):
    import fp8_block_scaled_x1_amd as fb
    op = st["op"]
    if op in ("prefill", "train"):
        causal = st["case"]["causal"]
        out, lse = fb.fp8bs_mla_prefill(st["q"], st["kv"], st["k_rope"], st["cu_q"], st["cu_k"], SCALE, causal=causal)
        if op == "prefill":
            return out, lse
        return (out, *fb.fp8bs_mla_prefill_bwd(st["dout"], st["q"], st["kv"], st["k_rope"], out, lse, st["cu_q"],
                                               st["cu_k"], SCALE, causal=causal))
    if op == "decode":
        return fb.fp8bs_mla_decode(st["q"], st["cache"], st["table"], st["seq_lens"], SCALE)
    if op == "shared":
        return fb.fp8bs_mla_decode_shared(st["q"], st["cache"], st["prefix_table"], st["prefix_len"], st["table"],
                                          st["seq_lens"], SCALE)
    return fb.fp8bs_verify_drafts(st["p"], st["q"], st["drafts"], st["n_drafts"], st["u"], st["u_next"])


def _head_step(H, rows):
    return max(1, min(H, MAX_SCORES // max(1, rows)))


def _hide(S, causal):
    """Scores of the keys that a query must not see, to minus infinity; the last query sees every key."""
    if causal:
        lq, lk = S.shape[-2:]
        i = torch.arange(lq, device=S.device)[:, None]
        j = torch.arange(lk, device=S.device)[None, :]
        S.masked_fill_(j > i + (lk - lq), -math.inf)
    return S


def _plain_prefill(st):
    train, causal = st["op"] == "train", st["case"]["causal"]
    q, kv, kr = st["q"], st["kv"], st["k_rope"]
    H = q.shape[1]
    out = torch.empty((q.shape[0], H, VDIM), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((H, q.shape[0]), dtype=torch.float32, device=q.device)
    if train:
        dq, dkv = torch.empty_like(q), torch.empty_like(kv)
        dkr = torch.zeros(kr.shape, dtype=torch.float32, device=q.device)
    a = b = 0
    for lq, lk in st["lens"]:
        step = _head_step(H, lq * lk)
        for h in range(0, H, step):
            hs = slice(h, min(H, h + step))
            Q = q[a:a + lq, hs].float().transpose(0, 1)
            KV = kv[b:b + lk, hs].float().transpose(0, 1)
            Kr = kr[b:b + lk].float().expand(Q.shape[0], lk, ROPE)
            K, V = torch.cat([KV[..., :NOPE], Kr], -1), KV[..., NOPE:]
            S = _hide(torch.matmul(Q, K.transpose(1, 2)) * SCALE, causal)
            m = S.amax(-1, keepdim=True)
            P = torch.exp(S - m)
            total = P.sum(-1, keepdim=True)
            P = P / total
            O = torch.matmul(P, V)
            out[a:a + lq, hs] = O.transpose(0, 1).to(torch.bfloat16)
            lse[hs, a:a + lq] = (m + torch.log(total))[..., 0]
            if train:
                dO = st["dout"][a:a + lq, hs].float().transpose(0, 1)
                dV = torch.matmul(P.transpose(1, 2), dO)
                dP = torch.matmul(dO, V.transpose(1, 2))
                dS = P * (dP - (dO * O).sum(-1, keepdim=True)) * SCALE
                dK = torch.matmul(dS.transpose(1, 2), Q)
                dq[a:a + lq, hs] = torch.matmul(dS, K).transpose(0, 1).to(torch.bfloat16)
                dkv[b:b + lk, hs] = torch.cat([dK[..., :NOPE], dV], -1).transpose(0, 1).to(torch.bfloat16)
                dkr[b:b + lk] += dK[..., NOPE:].sum(0)
        a, b = a + lq, b + lk
    return (out, dq, dkv, dkr.to(torch.bfloat16)) if train else (out, lse)


def _gather(cache, table):
    """The cached keys of the pages in table [..., n], in 32 bits: [..., n * page, 576]."""
    idx = table.long()
    if isinstance(cache, tuple):
        codes, scales, rope = cache
        x = codes[idx].view(torch.float8_e4m3fn).float().unflatten(-1, (LATENT // GROUP, GROUP)) * scales[idx][..., None]
        x = torch.cat([x.flatten(-2), rope[idx].float()], -1)
    else:
        x = cache[idx].float()
    return x.flatten(-3, -2)


def _partial(Q, K, hidden):
    """Unnormalised attention of rows Q over keys K: row maxima, sums of weights and weighted values."""
    S = torch.matmul(Q, K.transpose(-1, -2)) * SCALE
    if hidden is not None:
        S.masked_fill_(hidden, -math.inf)
    m = S.amax(-1, keepdim=True)
    P = torch.exp(S - m)
    return m, P.sum(-1, keepdim=True), torch.matmul(P, K[..., :LATENT])


def _plain_decode(st):
    q = st["q"]
    B, T, H, _ = q.shape
    out = torch.empty((B, T, H, LATENT), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((B, T, H), dtype=torch.float32, device=q.device)
    if st["op"] == "shared":
        Kp = _gather(st["cache"], st["prefix_table"])[:st["prefix"]]
        rows, step = q.reshape(-1, KEY), max(1, MAX_SCORES // st["prefix"])
        parts = [_partial(rows[i:i + step].float(), Kp, None) for i in range(0, rows.shape[0], step)]
        mp, tp, op = (torch.cat(x).reshape(B, T * H, -1) for x in zip(*parts))
    width = st["table"].shape[1] * st["case"]["page"]
    step = max(1, min(MAX_SCORES // (T * H * width), (1 << 29) // (width * KEY)))
    late = torch.arange(T, device=q.device).repeat_interleave(H) - (T - 1)
    for b in range(0, B, step):
        K = _gather(st["cache"], st["table"][b:b + step])
        n = K.shape[0]
        Q = q[b:b + n].float().reshape(n, T * H, KEY)
        seen = st["seq_lens"][b:b + n, None] + late
        m, t, o = _partial(Q, K, torch.arange(width, device=q.device) >= seen[..., None])
        if st["op"] == "shared":
            top = torch.maximum(m, mp[b:b + n])
            x, y = torch.exp(m - top), torch.exp(mp[b:b + n] - top)
            m, t, o = top, t * x + tp[b:b + n] * y, o * x + op[b:b + n] * y
        out[b:b + n] = (o / t).reshape(n, T, H, LATENT).to(torch.bfloat16)
        lse[b:b + n] = (m + torch.log(t)).reshape(n, T, H)
    return out, lse


def _weights(r):
    """Sampling weights: whole multiples of 2^-38, so that their sums are exact in any order."""
    return torch.floor(r.clamp(0.0, 1.0) * 2.0 ** WEIGHT_BITS).to(torch.int64)


def _plain_verify(st):
    p, q, drafts = st["p"], st["q"], st["drafts"].long()
    B, K, V = q.shape
    px = p[:, :K].gather(2, drafts[..., None])[..., 0]
    qx = q.gather(2, drafts[..., None])[..., 0]
    slot = torch.arange(K + 1, device=p.device)
    ok = (st["u"] * qx < px) & (slot[:K] < st["n_drafts"][:, None])
    n = ok.to(torch.int64).cumprod(1).sum(1)
    row = torch.arange(B, device=p.device)
    target = p[row, n]
    draft = torch.where((n < st["n_drafts"])[:, None], q[row, n.clamp(max=K - 1)], torch.zeros_like(target))
    w = _weights(target - draft)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, _weights(target))
    total = w.sum(1)
    m = torch.floor(st["u_next"].clamp(0.0, 1.0 - 2.0 ** -24) * 2.0 ** 24).to(torch.int64)
    goal = (total >> 24) * m + (((total & 0xFFFFFF) * m) >> 24)
    nxt = (w.cumsum(1) <= goal[:, None]).sum(1)
    nxt = torch.where(total > 0, nxt, torch.full_like(nxt, -1))
    tokens = torch.cat([drafts, torch.full((B, 1), -1, device=p.device)], 1)
    tokens = torch.where(slot < n[:, None], tokens, torch.where(slot == n[:, None], nxt[:, None], -1))
    return tokens.to(torch.int32), n.to(torch.int32)


_PLAIN = {"prefill": _plain_prefill, "train": _plain_prefill, "decode": _plain_decode, "shared": _plain_decode,
          "verify": _plain_verify}


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "verify":
        return None                       # whole numbers: compared for equality
    if work(case)["flops"] > 8.0e12:      # over about 20 seconds in 64 bits
        return None
    st = prepare(case, seed)
    return _exact_prefill(st, case) if case["op"] in ("prefill", "train") else _exact_decode(st, case)


def _exact_prefill(st, case):
    """Head by head, each request's softmax(scale * q [k_nope k_rope]^T) v and its derivatives."""
    q, kv, kr = st["q"], st["kv"], st["k_rope"]
    H, dev = q.shape[1], q.device
    train = case["op"] == "train"
    kw = dict(dtype=torch.float64, device=dev)
    res = {"out": torch.empty((q.shape[0], H, VDIM), **kw)}
    if train:
        res.update(dq=torch.empty(q.shape, **kw), dkv=torch.empty(kv.shape, **kw), dkr=torch.zeros(kr.shape, **kw))
    else:
        res["lse"] = torch.empty((H, q.shape[0]), **kw)
    a = b = 0
    for lq, lk in st["lens"]:
        rope = kr[b:b + lk].double()
        visible = torch.ones((lq, lk), dtype=torch.bool, device=dev)
        if case["causal"]:
            visible = visible.tril(lk - lq)
        for h in range(H):
            qn, qr = q[a:a + lq, h].double().split([NOPE, ROPE], -1)
            kn, v = kv[b:b + lk, h].double().split([NOPE, VDIM], -1)
            logits = (qn @ kn.T + qr @ rope.T) * SCALE
            logits = torch.where(visible, logits, torch.full_like(logits, -math.inf))
            z = torch.logsumexp(logits, -1)
            prob = torch.exp(logits - z[:, None])
            o = prob @ v
            res["out"][a:a + lq, h] = o
            if not train:
                res["lse"][h, a:a + lq] = z
                continue
            go = st["dout"][a:a + lq, h].double()
            res["dkv"][b:b + lk, h, NOPE:] = prob.T @ go
            gs = go @ v.T
            gs = prob * (gs - (prob * gs).sum(-1, keepdim=True)) * SCALE
            res["dq"][a:a + lq, h] = torch.cat([gs @ kn, gs @ rope], -1)
            res["dkv"][b:b + lk, h, :NOPE] = gs.T @ qn
            res["dkr"][b:b + lk] += gs.T @ qr
        a, b = a + lq, b + lk
    return tuple(res.values())


def _exact_decode(st, case):
    """Request by request, the softmax over the prefix's and the request's own tokens together."""
    q, page = st["q"], case["page"]
    B, T, H, _ = q.shape

    def keys(pages, n):
        if case["cache"] == "fp8":
            codes, scales, rope = (c[pages.long()].reshape(-1, c.shape[-1])[:n] for c in st["cache"])
            latent = codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(GROUP, -1)
            return torch.cat([latent, rope.double()], -1)
        return st["cache"][pages.long()].reshape(-1, KEY)[:n].double()

    prefix = keys(st["prefix_table"], st["prefix"]) if case["op"] == "shared" else None
    out = torch.empty((B, T, H, LATENT), dtype=torch.float64, device=q.device)
    lse = torch.empty((B, T, H), dtype=torch.float64, device=q.device)
    for b, n in enumerate(st["lens"]):
        k = keys(st["table"][b, :-(-n // page)], n)
        if prefix is not None:
            k = torch.cat([prefix, k])
        for t in range(T):
            mine = k[:k.shape[0] - (T - 1 - t)]
            logits = (q[b, t].double() @ mine.T) * SCALE
            z = torch.logsumexp(logits, -1)
            out[b, t] = torch.exp(logits - z[:, None]) @ mine[:, :LATENT]
            lse[b, t] = z
    return out, lse
