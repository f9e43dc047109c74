"""The operators of a serving step around the latent attention: what is measured of them.

Four kinds, in the two forms that `run` has:

  cache     latent vectors quantised as they are written into a paged cache (BF16, FP8 with a scale per 128, FP4 with
            a power of two per 32), and read back as BF16, packed
  decode    latent attention, absorbed form, over the cache held in 4 bits; with a prefix, for a batch that shares one
  moe       a whole mixture-of-experts layer (gate and up, SiLU, down, weighted sum) for a few tokens, FP8 weights
  logprobs  log probabilities of given tokens, their ranks, the entropy and the most likely alternatives; with its
            gradient where it trains

With ``own`` false, `run` computes them from elementary torch operations in 32 bits; with ``own`` true it calls the
package. `exact` is written apart from both, in 64 bits.
"""

import math
import random

import torch

own = False

ROPE, LATENT = 64, 512                           # numbers of a cached token: rotary ones, latent ones
KEY = LATENT + ROPE
SCALE = 1.0 / math.sqrt(128 + ROPE)
GROUP8, GROUP4 = 128, 32                         # latent numbers that share one scale, FP8 and FP4 cache
BLOCK = 128                                      # weights: one scale per 128 x 128
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of a 4-bit code's lower three bits
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
        # a decoding step's own tokens (one, or up to two drafted ones with it) of a serving batch: a small launch
        dict(name="cache_decode_step", op="cache", batch=96, new_low=1, new_high=3, past_low=20, past_high=4000,
             len_seed=1, page=64, kind="fp8", back="new"),
        # a chunk of two prompts goes into the 4-bit cache; all that is cached comes back to be expanded
        dict(name="cache_prefill_chunk", op="cache", batch=2, new_low=500, new_high=600, past_low=7000, past_high=8000,
             len_seed=2, page=64, kind="fp4", back="all"),
        # whole long prompts into the FP8 cache, small pages
        dict(name="cache_prompts", op="cache", batch=9, new_low=1, new_high=8192, past_low=0, past_high=0, len_seed=3,
             page=16, kind="fp8", back="new"),
        # one request, one token, a short context, 16 heads: pure latency
        dict(name="decode_one", op="decode", batch=1, heads=16, tokens=1, len_low=257, len_high=257, len_seed=4,
             page=64, prefix=0),
        # a full serving batch with ragged contexts, all 128 heads on one GPU
        dict(name="decode_batch_128_heads", op="decode", batch=128, heads=128, tokens=1, len_low=300, len_high=4500,
             len_seed=5, page=64, prefix=0),
        # long contexts, what a 4-bit cache is for: two tokens a request (one drafted), 16 heads
        dict(name="decode_long", op="decode", batch=8, heads=16, tokens=2, len_low=40000, len_high=70000, len_seed=6,
             page=64, prefix=0),
        # a large batch behind one long system prompt
        dict(name="decode_system_prompt", op="decode", batch=192, heads=32, tokens=1, len_low=16, len_high=900,
             len_seed=7, page=64, prefix=16000),
        # one token through a layer of 32 experts: the weights of 8 of them, once
        dict(name="moe_one_token", op="moe", tokens=1, topk=8, experts=32, all_experts=32, width=7168, inner=2048,
             id_seed=8),
        # a small decoding batch that reaches nearly every expert of the layer
        dict(name="moe_batch", op="moe", tokens=32, topk=8, experts=32, all_experts=32, width=7168, inner=2048,
             id_seed=9),
        # small experts with an odd number of blocks, half of the experts on another GPU: latency and imbalance
        dict(name="moe_share_of_small_experts", op="moe", tokens=5, topk=6, experts=32, all_experts=64, width=2048,
             inner=1408, id_seed=10),
        # the sampled tokens of a serving batch with 20 alternatives each, most of the vocabulary banned by a grammar
        # in some rows
        dict(name="logprobs_top_20", op="logprobs", tokens=96, vocab=129280, pad=0, top=20, dtype="f32", banned=0.25,
             train=False),
        # policy-gradient training: log probability and entropy with their gradient, BF16 logits of a padded vocabulary
        dict(name="logprobs_train", op="logprobs", tokens=2048, vocab=129280, pad=96, top=0, dtype="bf16", banned=0.0,
             train=True),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["cache", "decode", "decode", "moe", "moe", "logprobs"])
    seed = rng.randrange(1 << 30)
    if op == "cache":
        while True:
            new, past = _log_int(rng, 1, 8192), _log_int(rng, 1, 12000) if rng.random() < 0.6 else 0
            case = dict(op=op, batch=_log_int(rng, 1, 192), new_low=max(1, int(new * rng.uniform(0.02, 1.0))),
                        new_high=new, past_low=past // 3, past_high=past, len_seed=seed,
                        page=rng.choice([1, 16, 17, 64, 128]), kind=rng.choice(["bf16", "fp8", "fp4"]),
                        back=rng.choice(["new", "all"]))
            if case["batch"] * new <= 60_000 and case["batch"] * (new + past) <= 80_000:
                return case
    if op == "decode":
        while True:
            high = _log_int(rng, 1, 70000)
            case = dict(op=op, batch=_log_int(rng, 1, 192), heads=rng.choice([1, 5, 16, 32, 64, 128]),
                        tokens=rng.choice([1, 1, 1, 2, 3, 4]), len_low=max(1, int(high * rng.uniform(0.02, 1.0))),
                        len_high=high, len_seed=seed, page=rng.choice([1, 16, 17, 64, 128]),
                        prefix=_log_int(rng, 1, 16000) if rng.random() < 0.35 else 0)
            case["len_low"] = max(case["len_low"], case["tokens"])
            case["len_high"] = max(case["len_high"], case["len_low"])
            if work(case)["flops"] <= 2.0e11 and case["batch"] * case["len_high"] <= 600_000:
                return case
    if op == "moe":
        while True:
            experts = rng.choice([4, 8, 16, 32, 40, 64, 128, 256])
            case = dict(op=op, tokens=_log_int(rng, 1, 64), topk=rng.randint(1, 9), experts=experts,
                        all_experts=experts * rng.choice([1, 1, 2, 4]), width=BLOCK * _log_int(rng, 4, 56),
                        inner=BLOCK * _log_int(rng, 1, 32), id_seed=seed)
            if case["topk"] <= experts and experts * case["width"] * case["inner"] * 3 <= 1_450_000_000 \
                    and case["tokens"] * case["topk"] * case["width"] * case["inner"] <= 32 * 8 * 7168 * 2048:
                return case
    while True:
        train = rng.random() < 0.5
        vocab = _log_int(rng, 30, 200_000)
        case = dict(op=op, tokens=_log_int(rng, 1, 4096), vocab=vocab, pad=rng.choice([0, 0, 1, 8, 96]),
                    top=0 if train else rng.choice([0, 1, 5, 20, 30]), dtype=rng.choice(["f32", "bf16"]),
                    banned=rng.choice([0.0, 0.0, 0.3]), train=train)
        if case["tokens"] * vocab * (2 if case["dtype"] == "bf16" else 4) <= 2048 * 129280 * 2:
            return case


def _cache_lengths(case):
    """(new, all) tokens of each request."""
    new = _spread(case["new_low"], case["new_high"], case["batch"], case["len_seed"])
    past = _spread(case["past_low"], case["past_high"], case["batch"], case["len_seed"] + 1)
    return [(n, n + p) for n, p in zip(new, past)]


def _decode_lengths(case):
    return _spread(case["len_low"], case["len_high"], case["batch"], case["len_seed"])


def _expert_ids(case):
    """Each token's experts, different ones; those from `experts` on are on other GPUs."""
    r = random.Random(case["id_seed"])
    return [r.sample(range(case["all_experts"]), case["topk"]) for _ in range(case["tokens"])]


def _token_bytes(kind):
    return {"bf16": 2 * KEY, "fp8": LATENT + 4 * (LATENT // GROUP8) + 2 * ROPE,
            "fp4": LATENT // 2 + LATENT // GROUP4 + 2 * ROPE}[kind]


def work(case):
    op = case["op"]
    if op == "cache":
        lens, token = _cache_lengths(case), _token_bytes(case["kind"])
        new = sum(n for n, _ in lens)
        back = new if case["back"] == "new" else sum(n for _, n in lens)
        return {"bytes": new * (2 * KEY + token) + back * (token + 2 * KEY), "flops": (2 * new + back) * LATENT}
    if op == "decode":
        rows, lens, prefix = case["tokens"] * case["heads"], _decode_lengths(case), case["prefix"]
        hidden = case["tokens"] * (case["tokens"] - 1) // 2 * case["heads"]
        pairs = sum(rows * (n + prefix) - hidden for n in lens)
        io = len(lens) * rows * (2 * KEY + 2 * LATENT + 4)
        return {"bytes": (sum(lens) + prefix) * _token_bytes("fp4") + io, "flops": 2 * pairs * (KEY + LATENT)}
    if op == "moe":
        weights = 3 * case["width"] * case["inner"]
        pairs = [e for row in _expert_ids(case) for e in row if e < case["experts"]]
        return {"bytes": len(set(pairs)) * (weights + weights // (BLOCK * BLOCK) * 4) + 4 * case["tokens"] * case["width"],
                "flops": 2 * weights * max(1, len(pairs))}
    numbers = case["tokens"] * case["vocab"]
    size = 4 if case["dtype"] == "f32" else 2
    return {"bytes": numbers * size * (2 if case["train"] else 1), "flops": numbers * (10 if case["train"] else 5)}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return _ints(off)


def _empty_cache(kind, pages, page):
    rope = torch.zeros((pages, page, ROPE), dtype=torch.bfloat16, device="cuda")
    if kind == "bf16":
        return torch.zeros((pages, page, KEY), dtype=torch.bfloat16, device="cuda")
    if kind == "fp8":
        return (torch.zeros((pages, page, LATENT), dtype=torch.uint8, device="cuda"),
                torch.ones((pages, page, LATENT // GROUP8), dtype=torch.float32, device="cuda"), rope)
    return (torch.zeros((pages, page, LATENT // 2), dtype=torch.uint8, device="cuda"),
            torch.full((pages, page, LATENT // GROUP4), 127, dtype=torch.uint8, device="cuda"), rope)


def _filled_cache(kind, g, pages, page):
    """What earlier steps left in the pages."""
    cache = _empty_cache(kind, pages, page)
    step = max(1, (1 << 26) // (page * LATENT))
    for a in range(0, pages, step):
        x = _normal(g, (min(step, pages - a), page, KEY))
        if kind == "bf16":
            cache[a:a + step] = x
            continue
        codes, scales = (_quantise8 if kind == "fp8" else _quantise4)(x[..., :LATENT])
        cache[0][a:a + step], cache[1][a:a + step], cache[2][a:a + step] = codes, scales, x[..., LATENT:]
    return cache


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = {"op": op, "case": dict(case)}
    if op == "cache":
        lens, page = _cache_lengths(case), case["page"]
        B, most = len(lens), max(-(-n // page) for _, n in lens)
        need = [-(-n // page) for _, n in lens]
        new = sum(n for n, _ in lens)
        # pages in no order, as a pool hands them out after a while; requests have as many as they need
        pool = torch.randperm(sum(need) + 3, generator=g, device="cuda").to(torch.int32)
        table, at = torch.full((B, most), -1, dtype=torch.int32, device="cuda"), 0
        for b, n in enumerate(need):
            table[b, :n] = pool[at:at + n]
            at += n
        st.update(table=table, lens=_ints([n for _, n in lens]), cu=_offsets([n for n, _ in lens]), new=new,
                  latent=_normal(g, (new, LATENT)), rope=_normal(g, (new, ROPE)),
                  cache=_filled_cache(case["kind"], g, pool.shape[0], page))
        if case["back"] == "all":
            st.update(cu_back=_offsets([n for _, n in lens]), back=sum(n for _, n in lens))
        else:
            st.update(cu_back=st["cu"], back=new)
    elif op == "decode":
        B, page, lens, prefix = case["batch"], case["page"], _decode_lengths(case), case["prefix"]
        most, shared = max(-(-n // page) for n in lens), -(-prefix // page)
        pool = torch.randperm(B * most + shared, generator=g, device="cuda").to(torch.int32)
        st.update(lengths=lens, cache=_filled_cache("fp4", g, B * most + shared, page),
                  table=pool[:B * most].reshape(B, most).contiguous(), lens=_ints(lens),
                  q=_normal(g, (B, case["tokens"], case["heads"], KEY)))
        if prefix:
            st.update(prefix_table=pool[B * most:].contiguous(), prefix_len=_ints([prefix]))
    elif op == "moe":
        E, K, F, T = case["experts"], case["width"], case["inner"], case["tokens"]

        def weights(rows, cols):
            q = torch.empty((E, rows, cols), dtype=torch.uint8, device="cuda")
            for e in range(E):      # blocks whose largest number is near 448, as a quantiser leaves them
                q[e] = (torch.randn((rows, cols), generator=g, device="cuda") * 105.0).clamp(-448.0, 448.0).to(
                    torch.float8_e4m3fn).view(torch.uint8)
            s = torch.rand((E, rows // BLOCK, cols // BLOCK), generator=g, device="cuda") * 1e-4 + 5e-5
            return q, s

        ids = _expert_ids(case)
        p = torch.rand((T, case["topk"]), generator=g, device="cuda") + 0.05
        st.update(x=_normal(g, (T, K)), ids=_ints(ids), weights=p / p.sum(1, keepdim=True), up=weights(2 * F, K),
                  down=weights(K, F))
    else:
        T, V = case["tokens"], case["vocab"]
        logits = torch.empty((T, V + case["pad"]), dtype=torch.float32 if case["dtype"] == "f32" else torch.bfloat16,
                             device="cuda")
        targets = torch.empty(T, dtype=torch.int32, device="cuda")
        step = max(1, (1 << 27) // (V + case["pad"]))
        for a in range(0, T, step):
            x = torch.randn((min(step, T - a), V + case["pad"]), generator=g, device="cuda") * 2.5
            if case["banned"]:      # in that share of the rows a grammar leaves one token of 50
                rows = torch.rand(x.shape[0], generator=g, device="cuda") < case["banned"]
                ban = rows[:, None] & (torch.rand(x.shape, generator=g, device="cuda") < 0.98)
                ban[:, 0] = False
                x.masked_fill_(ban, -math.inf)
            logits[a:a + step] = x
            # tokens as they are sampled
            noise = -torch.log(-torch.log(torch.rand((x.shape[0], V), generator=g, device="cuda").clamp(1e-9, 0.9999999)))
            targets[a:a + step] = (x[:, :V] + noise).argmax(1)
        st.update(logits=logits[:, :V], targets=targets)
        if case["train"]:
            st.update(d_logprob=torch.randn(T, generator=g, device="cuda") / T,
                      d_entropy=torch.full((T,), 0.01 / T, device="cuda"))
    return st


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


def _run_own(st):
    import fp8_block_scaled_x1_amd as fb
    op = st["op"]
    if op == "cache":
        fb.fp8bs_mla_cache_write(st["latent"], st["rope"], st["cache"], st["table"], st["lens"], st["cu"])
        return *fb.fp8bs_mla_cache_read(st["cache"], st["table"], st["lens"], st["cu_back"], st["back"]), \
            *_buffers(st["cache"])
    if op == "decode":
        if "prefix_len" in st:
            return fb.fp8bs_mla_decode_fp4_shared(st["q"], st["cache"], st["prefix_table"], st["prefix_len"],
                                                  st["table"], st["lens"], SCALE)
        return fb.fp8bs_mla_decode_fp4(st["q"], st["cache"], st["table"], st["lens"], SCALE)
    if op == "moe":
        return fb.fp8bs_moe_tokens(st["x"], st["ids"], st["weights"], *st["up"], *st["down"])
    logprob, entropy, lse, rank, ids, tops = fb.fp8bs_logprobs(st["logits"], st["targets"], st["case"]["top"])
    if not st["case"]["train"]:
        return logprob, entropy, rank, ids, tops
    return logprob, entropy, fb.fp8bs_logprobs_bwd(st["logits"], st["targets"], lse, entropy, st["d_logprob"],
                                                   st["d_entropy"])


def _buffers(cache):
    """The updated cache itself, codes of 8 bits as the numbers they are."""
    if not isinstance(cache, tuple):
        return (cache,)
    codes = cache[0].view(torch.float8_e4m3fn) if cache[0].shape[-1] == LATENT else cache[0]
    return codes, cache[1], cache[2]


def _quantise8(x):
    """E4M3 codes and scales of groups of 128, as FP32 quotients (formed in 64 bits: borders between two codes)."""
    x = x.double().unflatten(-1, (-1, GROUP8))
    s = (x.abs().amax(-1) / 448.0).float()
    s = torch.where(s == 0, torch.ones_like(s), s)
    y = (x / s.double()[..., None]).float()
    return y.to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2), s


def _quantise4(x):
    """E2M1 codes, two in a byte (the even column's in the lower half), and the exponents of groups of 32: the
    smallest power of two not below a sixth of the largest magnitude (1 for zeros), 127 added."""
    x = x.float().unflatten(-1, (-1, GROUP4))
    m, e = torch.frexp(x.abs().amax(-1))                     # m in [0.5, 1): m * 2^e <= 6 * 2^p
    p = torch.where(m <= 0.75, e - 3, e - 2).clamp(min=-126)
    p = torch.where(m == 0, torch.zeros_like(p), p)
    y = torch.ldexp(x, -p[..., None])
    a = y.abs()
    code = sum((a > b if i % 2 == 0 else a >= b).to(torch.uint8)      # halfway: to the even code
               for i, b in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
    code = (code + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2)
    return code[..., ::2] + 16 * code[..., 1::2], (p + 127).to(torch.uint8)


def _values(kind, latent_parts):
    """Latent numbers of codes and scales, in 32 bits."""
    codes, scales = latent_parts
    if kind == "fp8":
        x = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, GROUP8)) * scales[..., None]
        return x.flatten(-2)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    x = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    x = table[x.long()].unflatten(-1, (-1, GROUP4))
    return torch.ldexp(x, scales.int()[..., None] - 127).flatten(-2)


def _slots(st, cu, n):
    """Page and slot of each of the requests' newest tokens, packed as cu says."""
    i = torch.arange(n, device=cu.device)
    b = (i[:, None] >= cu[None, 1:]).sum(1)
    pos = st["lens"][b] - cu[b + 1] + i
    page = st["case"]["page"]
    return st["table"][b, pos // page].long(), pos % page


def _plain_cache(st):
    cache, kind = st["cache"], st["case"]["kind"]
    at = _slots(st, st["cu"], st["new"])
    if kind == "bf16":
        cache[at] = torch.cat([st["latent"], st["rope"]], -1)
    else:
        codes, scales = (_quantise8 if kind == "fp8" else _quantise4)(st["latent"])
        cache[0][at], cache[1][at], cache[2][at] = codes, scales, st["rope"]
    at = _slots(st, st["cu_back"], st["back"])
    if kind == "bf16":
        x = cache[at]
        return x[:, :LATENT].contiguous(), x[:, LATENT:].contiguous(), *_buffers(cache)
    latent = _values(kind, (cache[0][at], cache[1][at])).to(torch.bfloat16)
    return latent, cache[2][at], *_buffers(cache)


def _gather(cache, table):
    """The cached keys of the pages in table [..., n], in 32 bits: [..., n * page, 576]."""
    idx = table.long()
    return torch.cat([_values("fp4", (cache[0][idx], cache[1][idx])), cache[2][idx].float()], -1).flatten(-3, -2)


def _partial(Q, K, hidden):
    """Unnormalised attention of rows Q over keys K: row maxima, sums of weights and weighted values."""
    S = torch.matmul(Q, K.transpose(-1, -2)) * SCALE
    if hidden is not None:
        S.masked_fill_(hidden, -math.inf)
    m = S.amax(-1, keepdim=True)
    P = torch.exp(S - m)
    return m, P.sum(-1, keepdim=True), torch.matmul(P, K[..., :LATENT])


def _plain_decode(st):
    q, prefix = st["q"], st["case"]["prefix"]
    B, T, H, _ = q.shape
    out = torch.empty((B, T, H, LATENT), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((B, T, H), dtype=torch.float32, device=q.device)
    if prefix:
        Kp = _gather(st["cache"], st["prefix_table"])[:prefix]
        rows, step = q.reshape(-1, KEY), max(1, MAX_SCORES // prefix)
        parts = [_partial(rows[i:i + step].float(), Kp, None) for i in range(0, rows.shape[0], step)]
        mp, tp, op = (torch.cat(x).reshape(B, T * H, -1) for x in zip(*parts))
    width = st["table"].shape[1] * st["case"]["page"]
    step = max(1, min(MAX_SCORES // (T * H * width), (1 << 29) // (width * KEY)))
    late = torch.arange(T, device=q.device).repeat_interleave(H) - (T - 1)
    for b in range(0, B, step):
        K = _gather(st["cache"], st["table"][b:b + step])
        n = K.shape[0]
        Q = q[b:b + n].float().reshape(n, T * H, KEY)
        seen = st["lens"][b:b + n, None] + late
        m, t, o = _partial(Q, K, torch.arange(width, device=q.device) >= seen[..., None])
        if prefix:
            top = torch.maximum(m, mp[b:b + n])
            x, y = torch.exp(m - top), torch.exp(mp[b:b + n] - top)
            m, t, o = top, t * x + tp[b:b + n] * y, o * x + op[b:b + n] * y
        out[b:b + n] = (o / t).reshape(n, T, H, LATENT).to(torch.bfloat16)
        lse[b:b + n] = (m + torch.log(t)).reshape(n, T, H)
    return out, lse


def _weights32(q, s):
    """Experts' weights in 32 bits: codes times the scale of their block."""
    n, rows, cols = q.shape
    x = q.view(torch.float8_e4m3fn).float().view(n, rows // BLOCK, BLOCK, cols // BLOCK, BLOCK)
    return (x * s[:, :, None, :, None]).view(n, rows, cols)


def _plain_moe(st):
    ids, x = st["ids"].long(), st["x"].float()
    (qu, su), (qd, sd) = st["up"], st["down"]
    used = torch.unique(ids)
    used = used[(used >= 0) & (used < qu.shape[0])]
    # every expert that is used at all computes every token; weight 0 where the token did not choose it
    gate = ((ids[:, None, :] == used[None, :, None]) * st["weights"][:, None, :]).sum(2)          # [T][U]
    y = torch.matmul(x, _weights32(qu[used], su[used]).transpose(1, 2))                          # [U][T][2F]
    g, u = y.chunk(2, -1)
    h = g / (1.0 + torch.exp(-g)) * u
    z = torch.matmul(h, _weights32(qd[used], sd[used]).transpose(1, 2))                          # [U][T][K]
    return (z * gate.t()[:, :, None]).sum(0).to(torch.bfloat16)


def _plain_logprobs(st):
    x, targets, n = st["logits"].float(), st["targets"].long(), st["case"]["top"]
    T, V = x.shape
    m = x.amax(1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    lse = (m + torch.log(total))[:, 0]
    entropy = (torch.log(total) - torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1, keepdim=True) / total)[:, 0]
    xt = x.gather(1, targets[:, None])
    logprob = xt[:, 0] - lse
    if st["case"]["train"]:
        lp = x - lse[:, None]
        p = torch.exp(lp)
        grad = -p * st["d_logprob"][:, None]
        grad -= torch.where(p > 0, p * (lp + entropy[:, None]), torch.zeros_like(p)) * st["d_entropy"][:, None]
        grad.scatter_add_(1, targets[:, None], st["d_logprob"][:, None])
        return logprob, entropy, grad.to(st["logits"].dtype)
    at = torch.arange(V, device=x.device)
    rank = ((x > xt) | ((x == xt) & (at < targets[:, None]))).sum(1).to(torch.int32)
    # one whole number per entry that orders them: the value, then the lowest index
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF)) * (1 << 24) + (V - 1 - at)
    ids = V - 1 - torch.topk(key, n, 1).values % (1 << 24)
    return logprob, entropy, rank, ids.to(torch.int32), x.gather(1, ids) - lse[:, None]


_PLAIN = {"cache": _plain_cache, "decode": _plain_decode, "moe": _plain_moe, "logprobs": _plain_logprobs}


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "decode" and work(case)["flops"] > 8.0e11:
        return None
    st = prepare(case, seed)
    return {"cache": _exact_cache, "decode": _exact_decode, "moe": _exact_moe, "logprobs": _exact_logprobs}[case["op"]](st, case)


def _code_values(codes, scales):
    """Numbers of 4-bit codes and their groups' exponents."""
    def half(c):
        c = c.long()
        mag, exp = c & 1, (c >> 1) & 3
        v = torch.where(exp == 0, 0.5 * mag.double(), (1 + 0.5 * mag.double()) * 2.0 ** (exp - 1).double())
        return torch.where(c >= 8, -v, v)

    x = torch.empty(*codes.shape[:-1], LATENT, dtype=torch.float64, device=codes.device)
    x[..., 0::2], x[..., 1::2] = half(codes & 15), half(codes >> 4)
    return x * (2.0 ** (scales.double() - 127)).repeat_interleave(GROUP4, -1)


def _exact_cache(st, case):
    """What comes back: the cached numbers, those of the new tokens rounded to the nearest that their group's scale
    allows. (The buffers hold whole numbers, or what the inputs hold.)"""
    kind, page = case["kind"], case["page"]
    new = st["latent"].double()
    if kind == "fp8":
        grouped = new.reshape(-1, LATENT // GROUP8, GROUP8)
        s = (grouped.abs().amax(-1, keepdim=True) / 448).float().double()
        s = torch.where(s == 0, torch.ones_like(s), s)
        mag = (grouped / s).float().double().abs()       # the code is that of the FP32 quotient
        step = 2.0 ** (torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)
        new = (torch.round(mag / step) * step * grouped.sign() * s).reshape(new.shape)
    elif kind == "fp4":
        grouped = new.reshape(-1, LATENT // GROUP4, GROUP4)
        top = grouped.abs().amax(-1, keepdim=True)
        s = 2.0 ** torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 6.0)) / 6)).clamp(min=-126)
        mag = (grouped / s).abs()
        step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0))
        new = (torch.round(mag / step) * step * grouped.sign() * s).reshape(new.shape)
    back, ropes, at = [], [], 0
    for b, (n, total) in enumerate(_cache_lengths(case)):
        pages = st["table"][b, :-(-total // page)].long()
        if case["back"] == "all" and total > n:
            old = total - n
            parts = [c[pages].reshape(-1, c.shape[-1])[:old] for c in
                     (st["cache"] if kind != "bf16" else (st["cache"],))]
            if kind == "bf16":
                back.append(parts[0][:, :LATENT].double())
                ropes.append(parts[0][:, LATENT:])
            else:
                back.append(parts[0].view(torch.float8_e4m3fn).double() * parts[1].double().repeat_interleave(GROUP8, -1)
                            if kind == "fp8" else _code_values(parts[0], parts[1]))
                ropes.append(parts[2])
        back.append(new[at:at + n])
        ropes.append(st["rope"][at:at + n])
        at += n
    return torch.cat(back), torch.cat(ropes).double(), *(None for _ in _buffers(st["cache"]))


def _exact_decode(st, case):
    """Request by request, the softmax over the prefix's and the request's own tokens together."""
    q, page = st["q"], case["page"]
    B, T, H, _ = q.shape

    def keys(pages, n):
        codes, scales, rope = (c[pages.long()].reshape(-1, c.shape[-1])[:n] for c in st["cache"])
        return torch.cat([_code_values(codes, scales), rope.double()], -1)

    prefix = keys(st["prefix_table"], case["prefix"]) if case["prefix"] else None
    out = torch.empty((B, T, H, LATENT), dtype=torch.float64, device=q.device)
    lse = torch.empty((B, T, H), dtype=torch.float64, device=q.device)
    for b, n in enumerate(st["lengths"]):
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


def _exact_moe(st, case):
    """Expert by expert, the tokens that chose it."""
    x, F = st["x"].double(), case["inner"]
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)

    def matrix(parts, e):
        q, s = parts[0][e], parts[1][e].double()
        return q.view(torch.float8_e4m3fn).double() * s.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)

    chosen = {}
    for t, row in enumerate(_expert_ids(case)):
        for j, e in enumerate(row):
            if e < case["experts"]:
                chosen.setdefault(e, []).append((t, j))
    for e, pairs in chosen.items():
        t, j = (torch.tensor(v, device=x.device) for v in zip(*pairs))
        a = x[t] @ matrix(st["up"], e).T
        h = a[:, :F] * torch.sigmoid(a[:, :F]) * a[:, F:]
        out.index_add_(0, t, (h @ matrix(st["down"], e).T) * st["weights"][t, j].double()[:, None])
    return out


def _exact_logprobs(st, case):
    T = case["tokens"]
    kw = dict(dtype=torch.float64, device=st["logits"].device)
    logprob, entropy = torch.empty(T, **kw), torch.empty(T, **kw)
    tops = None if case["train"] else torch.empty((T, case["top"]), **kw)
    grad = torch.empty(st["logits"].shape, **kw) if case["train"] else None
    step = max(1, (1 << 26) // case["vocab"])
    for a in range(0, T, step):
        x = st["logits"][a:a + step].double()
        lp = x - torch.logsumexp(x, 1, keepdim=True)
        p = lp.exp()
        h = -torch.nan_to_num(p * lp, nan=0.0).sum(1)
        pick = st["targets"][a:a + step, None].long()
        logprob[a:a + step], entropy[a:a + step] = lp.gather(1, pick)[:, 0], h
        if case["train"]:
            dl, dh = st["d_logprob"][a:a + step, None].double(), st["d_entropy"][a:a + step, None].double()
            grad[a:a + step] = (torch.zeros_like(x).scatter_(1, pick, 1.0) - p) * dl \
                - torch.nan_to_num(p * (lp + h[:, None]), nan=0.0) * dh
        elif case["top"]:
            tops[a:a + step] = torch.topk(lp, case["top"], 1).values
    return (logprob, entropy, grad) if case["train"] else (logprob, entropy, None, None, tops)
