"""One layer of latent attention trained and served with the operators of
include/fp8bs_attn.h:

  train     packed ragged requests through the expanded form and its gradients
  generate  a shared system prompt and the requests' own prompts prefilled in
            the expanded form, their latent vectors put into a paged cache (BF16,
            or FP8 by the 1x128 quantizer), then steps of speculative decoding:
            a few drafted tokens scored at once by the absorbed form, which
            reads the shared prompt once for all requests, and verified

The weights are random and the model is one layer between an embedding and its
transpose: what is shown is how the operators fit together. Run on an MI355X:

  python examples/latent_attention.py [--cache bf16|fp8] [--steps 8] [--drafts 2]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_block_scaled_x1_amd as fb  # noqa: E402

NOPE, ROPE, VDIM, LATENT = 128, 64, 128, 512
SCALE = (NOPE + ROPE) ** -0.5


def offsets(lens, device):
    return torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device=device)


def rotate(x, pos):
    """Rotary positions on the last dimension (64), pos [tokens] for x [tokens][...][64]."""
    freq = 10000.0 ** (-torch.arange(0, ROPE, 2, device=x.device) / ROPE)
    a = (pos[:, None] * freq).reshape(len(pos), *[1] * (x.dim() - 2), ROPE // 2)
    u, v = x.float().chunk(2, -1)
    return torch.cat([u * a.cos() - v * a.sin(), u * a.sin() + v * a.cos()], -1).to(x.dtype)


class PrefillAttention(torch.autograd.Function):
    """fp8bs_mla_prefill with its gradient, causal."""

    @staticmethod
    def forward(ctx, q, kv, k_rope, cu_q, cu_k):
        out, lse = fb.fp8bs_mla_prefill(q, kv, k_rope, cu_q, cu_k, SCALE)
        ctx.save_for_backward(q, kv, k_rope, out, lse, cu_q, cu_k)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, kv, k_rope, out, lse, cu_q, cu_k = ctx.saved_tensors
        return *fb.fp8bs_mla_prefill_bwd(dout.contiguous(), q, kv, k_rope, out, lse, cu_q, cu_k, SCALE), None, None


class Layer:
    def __init__(self, device, heads=16, hidden=512, vocab=1024, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.vocab, self.device = heads, vocab, device

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g, device=device) * rows ** -0.5).requires_grad_()

        self.emb = weight(hidden, vocab)
        self.w_q = weight(hidden, heads * (NOPE + ROPE))
        self.w_c = weight(hidden, LATENT + ROPE)
        self.w_kv = weight(LATENT, heads * (NOPE + VDIM))        # keys then values of each head
        self.w_o = weight(heads * VDIM, hidden)
        self.weights = [self.emb, self.w_q, self.w_c, self.w_kv, self.w_o]

    def project(self, tokens, pos):
        """Embeddings, queries [T][H][192], latent vectors [T][512] and rotary keys [T][64]."""
        x = self.emb.t()[tokens] * self.emb.shape[0] ** 0.5
        xb = x.bfloat16()
        q = (xb @ self.w_q.bfloat16()).unflatten(-1, (self.heads, NOPE + ROPE))
        q = torch.cat([q[..., :NOPE], rotate(q[..., NOPE:], pos)], -1)
        c = xb @ self.w_c.bfloat16()
        return x, q, c[:, :LATENT].contiguous(), rotate(c[:, LATENT:], pos)

    def expand(self, latent):
        return (latent @ self.w_kv.bfloat16()).unflatten(-1, (self.heads, NOPE + VDIM))

    def logits(self, x, attended):
        """Next-token logits from embeddings and attention outputs [T][H][128]."""
        y = x + attended.flatten(1).bfloat16() @ self.w_o.bfloat16()
        return (y.bfloat16() @ self.emb.bfloat16()).float()

    def fold(self):
        """The up-projections as the absorbed form wants them: into the queries
        [H][128][512] and out of the latent outputs [H][512][128]."""
        w = self.w_kv.detach().bfloat16().unflatten(-1, (self.heads, NOPE + VDIM))
        return w[..., :NOPE].permute(1, 2, 0).contiguous(), w[..., NOPE:].permute(1, 0, 2).contiguous()


def train(layer, steps=20, lens=(70, 1, 129, 33, 200), seed=0, lr=3e-3):
    """Adam on random documents that repeat their first tokens; returns the losses."""
    g = torch.Generator(device=layer.device).manual_seed(seed)
    docs = [torch.randint(layer.vocab, (min(n, 16),), generator=g, device=layer.device).repeat(-(-(n + 1) // 16))[:n + 1]
            for n in lens]
    docs = [d if len(d) == n + 1 else torch.cat([d, d[:1]]) for d, n in zip(docs, lens)]
    tokens, targets = torch.cat([d[:-1] for d in docs]), torch.cat([d[1:] for d in docs])
    pos = torch.cat([torch.arange(n, device=layer.device) for n in lens])
    cu = offsets(lens, layer.device)
    opt, losses = torch.optim.Adam(layer.weights, lr=lr), []
    for _ in range(steps):
        x, q, latent, rope = layer.project(tokens, pos)
        out = PrefillAttention.apply(q, layer.expand(latent), rope, cu, cu)
        loss = torch.nn.functional.cross_entropy(layer.logits(x, out), targets)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


class Cache:
    """Latent vectors in pages: BF16, or FP8 codes with a scale per 128."""

    def __init__(self, pages, page, kind, device):
        self.page, self.kind = page, kind
        if kind == "fp8":
            self.data = (torch.zeros(pages, page, LATENT, dtype=torch.uint8, device=device),
                         torch.zeros(pages, page, LATENT // 128, device=device),
                         torch.zeros(pages, page, ROPE, dtype=torch.bfloat16, device=device))
        else:
            self.data = torch.zeros(pages, page, LATENT + ROPE, dtype=torch.bfloat16, device=device)

    def put(self, table, pos, latent, rope):
        """Tokens at positions pos [n] of the requests whose pages are table [n][width]."""
        pos = pos.long()
        page, slot = table.gather(1, (pos // self.page)[:, None])[:, 0].long(), pos % self.page
        if self.kind == "fp8":
            codes, scales = fb.fp8_quant_act_1x128(latent.contiguous())
            for to, what in zip(self.data, (codes, scales.t(), rope)):
                to[page, slot] = what
        else:
            self.data[page, slot] = torch.cat([latent, rope], -1)


@torch.no_grad()
def generate(layer, system=150, prompts=(40, 7, 100), steps=8, drafts=2, cache="bf16", page=16, seed=1):
    """Serves len(prompts) requests; returns a dict with each request's tokens
    (system prompt, own prompt, generated), the attention outputs of its
    generated tokens' positions, and the accepted drafts of every step."""
    device, H, V, B = layer.device, layer.heads, layer.vocab, len(prompts)
    g = torch.Generator(device=device).manual_seed(seed)

    def ints(*shape):
        return torch.randint(V, shape, generator=g, device=device)

    shared, own = ints(system), [ints(n) for n in prompts]
    width = -(-(max(prompts) + steps * (drafts + 1)) // page)
    n_shared = -(-system // page)
    pool = torch.randperm(n_shared + B * width, generator=g, device=device).int()
    shared_pages, table = pool[:n_shared], pool[n_shared:].view(B, width).contiguous()
    store = Cache(len(pool), page, cache, device)

    # the system prompt, once; only its latent vectors are kept
    pos = torch.arange(system, device=device)
    _, _, c0, r0 = layer.project(shared, pos)
    store.put(shared_pages.expand(system, -1), pos, c0, r0)

    # the requests' own prompts but for their last token, packed, behind the system prompt's keys
    lens = [n - 1 for n in prompts]
    pos = torch.cat([torch.arange(n, device=device) for n in lens])
    owner = torch.cat([torch.full((n,), b, device=device) for b, n in enumerate(lens)])
    _, q, c, r = layer.project(torch.cat([t[:-1] for t in own]), pos + system)
    store.put(table[owner], pos, c, r)
    keys, ropes = layer.expand(torch.cat([torch.cat([c0, x]) for x in c.split(lens)])), \
        torch.cat([torch.cat([r0, x]) for x in r.split(lens)])
    fb.fp8bs_mla_prefill(q, keys, ropes, offsets(lens, device), offsets([system + n for n in lens], device), SCALE)
    # (a model of several layers would go on from this output; here the next layer is the head, and only the last
    # token's, which the first decoding step computes, is wanted)

    w_in, w_out = layer.fold()
    T = drafts + 1
    system_len = torch.tensor([system], dtype=torch.int32, device=device)
    length = torch.tensor(lens, dtype=torch.int32, device=device)
    last = torch.stack([t[-1] for t in own])
    done = [list(torch.cat([shared, t]).tolist()) for t in own]
    outs, accepts = [[] for _ in own], []
    for _ in range(steps):
        # drafts from the model without its attention, one after the other
        toks, qs = [last], []
        for _ in range(drafts):
            x = layer.emb.t()[toks[-1]] * layer.emb.shape[0] ** 0.5
            p = (layer.logits(x, torch.zeros(B, H, VDIM, device=device)) / 4).softmax(-1)
            qs.append(p)
            toks.append(torch.multinomial(p, 1, generator=g)[:, 0])
        x_tok = torch.stack(toks, 1)                                             # [B][T]
        at = length[:, None] + torch.arange(T, device=device)                    # positions among the request's own
        x, q, c, r = layer.project(x_tok.flatten(), (at + system).flatten())
        store.put(table.repeat_interleave(T, 0), at.flatten(), c, r)

        # all T tokens of every request at once, the queries with the keys' up-projection folded in
        heads_first = q[..., :NOPE].transpose(0, 1).contiguous()
        folded = torch.bmm(heads_first, w_in).transpose(0, 1)
        qa = torch.cat([folded, q[..., NOPE:]], -1).view(B, T, H, LATENT + ROPE)
        o, _ = fb.fp8bs_mla_decode_shared(qa, store.data, shared_pages, system_len, table, length + T, SCALE)
        o = torch.bmm(o.view(B * T, H, LATENT).transpose(0, 1).contiguous(), w_out).transpose(0, 1)

        p = (layer.logits(x, o) / 4).softmax(-1).view(B, T, V)
        tokens, accepted = fb.fp8bs_verify_drafts(
            p, torch.stack(qs, 1) if drafts else None, x_tok[:, 1:].int().contiguous(),
            torch.full((B,), drafts, dtype=torch.int32, device=device),
            torch.rand(B, drafts, generator=g, device=device), torch.rand(B, generator=g, device=device))
        for b, a in enumerate(accepted.tolist()):
            done[b] += tokens[b, :a + 1].tolist()
            outs[b].append(o.unflatten(0, (B, T))[b, :a + 1])
        accepts.append(accepted)
        length = length + accepted + 1          # the last token and the accepted drafts stay in the cache
        last = tokens.gather(1, accepted[:, None].long())[:, 0].long()
    return dict(tokens=done, outputs=[torch.cat(x) for x in outs], accepted=torch.stack(accepts))


@torch.no_grad()
def attention_of(layer, tokens):
    """Attention outputs [n][H][128] of one whole sequence, expanded form."""
    tokens = torch.tensor(tokens, device=layer.device)
    _, q, c, r = layer.project(tokens, torch.arange(len(tokens), device=layer.device))
    cu = offsets([len(tokens)], layer.device)
    return fb.fp8bs_mla_prefill(q, layer.expand(c), r, cu, cu, SCALE)[0]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--cache", choices=["bf16", "fp8"], default="bf16")
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=2)
    args = ap.parse_args()
    layer = Layer(torch.device("cuda"))
    res = generate(layer, steps=args.steps, drafts=args.drafts, cache=args.cache)
    for b, (toks, o) in enumerate(zip(res["tokens"], res["outputs"])):
        want = attention_of(layer, toks[:-1])[-len(o):].float()
        off = ((o.float() - want).norm() / want.norm()).item()
        print(f"request {b}: {len(o)} tokens in {args.steps} steps, {res['accepted'][:, b].sum().item()} drafts accepted, "
              f"attention within {off:.4f} of the expanded form")
    losses = train(layer)
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f} in {len(losses)} steps")


if __name__ == "__main__":
    main()
