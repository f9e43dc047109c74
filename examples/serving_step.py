"""A block of latent attention and a mixture of experts served and tuned with
the operators of include/fp8bs_serve.h:

  generate  prompts prefilled in the expanded form, the second half of each over
            the first half read back from the cache, as chunks are; then one
            token a step: its latent vector written into its page (BF16, FP8 or
            FP4), the absorbed form over that cache, the experts' layer for few
            tokens, and the log probability, entropy and best alternatives of
            the token that was chosen
  tune      a policy gradient step on sampled tokens: their log probabilities
            and entropies with gradients into logits and weights

The weights are random: what is shown is how the operators fit together. Run on
an MI355X:

  python examples/serving_step.py [--cache bf16|fp8|fp4] [--steps 8] [--top 5]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_block_scaled_x1_amd as fb  # noqa: E402
from latent_attention import LATENT, NOPE, ROPE, SCALE, Layer, offsets  # noqa: E402


class LogProbs(torch.autograd.Function):
    """fp8bs_logprobs with its gradient: (log probability, entropy) of each row's token."""

    @staticmethod
    def forward(ctx, logits, targets):
        logprob, entropy, norm, *_ = fb.fp8bs_logprobs(logits, targets)
        ctx.save_for_backward(logits, targets, norm, entropy)
        return logprob, entropy

    @staticmethod
    def backward(ctx, d_logprob, d_entropy):
        logits, targets, norm, entropy = ctx.saved_tensors
        return fb.fp8bs_logprobs_bwd(logits, targets, norm, entropy, d_logprob.contiguous(), d_entropy.contiguous()), None


def blockwise(w):
    """[E][rows][cols] as E4M3 codes (uint8) with a scale per 128 x 128 block."""
    E, rows, cols = w.shape
    blocks = w.float().view(E, rows // 128, 128, cols // 128, 128)
    scale = (blocks.abs().amax((2, 4)) / 448).clamp_min(1e-12)
    codes = (blocks / scale[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(E, rows, cols).view(torch.uint8), scale


class Block(Layer):
    """The layer of latent_attention.py with experts behind its attention."""

    def __init__(self, device, experts=8, topk=2, inner=256, seed=0, **kw):
        super().__init__(device, seed=seed, **kw)
        hidden = self.emb.shape[0]
        g = torch.Generator(device=device).manual_seed(seed + 1)
        self.topk, self.gate = topk, torch.randn(hidden, experts, generator=g, device=device) * hidden ** -0.5
        self.up = blockwise(torch.randn(experts, 2 * inner, hidden, generator=g, device=device) * hidden ** -0.5)
        self.down = blockwise(torch.randn(experts, hidden, inner, generator=g, device=device) * inner ** -0.5)

    def experts(self, y):
        """y [T][hidden] BF16 with what its experts make of it added."""
        p, ids = (y.float() @ self.gate).softmax(-1).topk(self.topk)
        return y + fb.fp8bs_moe_tokens(y, ids.int(), (p / p.sum(-1, keepdim=True)).contiguous(), *self.up, *self.down)

    def head(self, x, attended):
        """Next-token logits: the attention's output projection, the experts, the embedding's transpose."""
        y = (x + attended.flatten(1).bfloat16() @ self.w_o.bfloat16()).bfloat16()
        return self.experts(y) @ self.emb.bfloat16()


def new_cache(kind, pages, page, device):
    """An empty cache of a kind that fp8bs_mla_cache_write fills."""
    def zeros(n, dtype):
        return torch.zeros(pages, page, n, dtype=dtype, device=device)

    if kind == "bf16":
        return zeros(LATENT + ROPE, torch.bfloat16)
    if kind == "fp8":
        return zeros(LATENT, torch.uint8), zeros(LATENT // 128, torch.float32), zeros(ROPE, torch.bfloat16)
    return zeros(LATENT // 2, torch.uint8), zeros(LATENT // 32, torch.uint8), zeros(ROPE, torch.bfloat16)


class Server:
    """Requests with their pages. A decoding step keeps its state in tensors
    that stay where they are (tokens, lens), so it can be captured into a graph."""

    def __init__(self, block, prompts, room, cache="fp4", page=16, top=5, seed=1):
        device, B = block.device, len(prompts)
        g = torch.Generator(device=device).manual_seed(seed)
        self.block, self.top, self.kind = block, top, cache
        self.fold = block.fold()
        width = -(-(max(prompts) + room) // page)
        self.table = torch.randperm(B * width, generator=g, device=device).int().view(B, width).contiguous()
        self.cache = new_cache(cache, B * width, page, device)
        self.prompts = [torch.randint(block.vocab, (n,), generator=g, device=device) for n in prompts]
        self.one_each = torch.arange(B + 1, dtype=torch.int32, device=device)
        # all but a prompt's last token, in two chunks
        self.lens = torch.zeros(B, dtype=torch.int32, device=device)
        have = [0] * B
        for want in ([(n - 1) // 2 for n in prompts], [n - 1 for n in prompts]):
            self.prefill(have, want)
            have = want
        self.tokens = torch.stack([p[-1] for p in self.prompts])

    @torch.no_grad()
    def prefill(self, have, want):
        """Positions have[b] .. want[b]-1 of each prompt, over the whole of what the cache then holds."""
        block, device = self.block, self.block.device
        new = [w - h for h, w in zip(have, want)]
        pos = torch.cat([torch.arange(h, w, device=device) for h, w in zip(have, want)])
        _, q, c, r = block.project(torch.cat([p[h:w] for p, h, w in zip(self.prompts, have, want)]), pos)
        self.lens = torch.tensor(want, dtype=torch.int32, device=device)
        cu_q, cu_k = offsets(new, device), offsets(want, device)
        fb.fp8bs_mla_cache_write(c, r, self.cache, self.table, self.lens, cu_q)
        c, r = fb.fp8bs_mla_cache_read(self.cache, self.table, self.lens, cu_k, sum(want))
        if sum(new):
            # (a model of several blocks would go on from this output; the last token's is computed by the first step)
            fb.fp8bs_mla_prefill(q, block.expand(c), r, cu_q, cu_k, SCALE)

    @torch.no_grad()
    def step(self, chosen):
        """The last tokens' positions are added, tokens are chosen by `chosen`
        (logits [B][vocab] -> [B]) and kept in self.tokens. Returns the attention
        outputs [B][H][128], the logits and what fp8bs_logprobs says of the tokens."""
        block, B, H = self.block, len(self.prompts), self.block.heads
        x, q, c, r = block.project(self.tokens, self.lens)
        self.lens += 1
        fb.fp8bs_mla_cache_write(c, r, self.cache, self.table, self.lens, self.one_each)
        w_in, w_out = self.fold
        heads_first = q[..., :NOPE].transpose(0, 1).contiguous()
        qa = torch.cat([torch.bmm(heads_first, w_in).transpose(0, 1), q[..., NOPE:]], -1).view(B, 1, H, LATENT + ROPE)
        decode = fb.fp8bs_mla_decode_fp4 if self.kind == "fp4" else fb.fp8bs_mla_decode
        o, _ = decode(qa, self.cache, self.table, self.lens, SCALE)
        o = torch.bmm(o.view(B, H, LATENT).transpose(0, 1).contiguous(), w_out).transpose(0, 1)
        logits = block.head(x, o)
        self.tokens.copy_(chosen(logits))
        return o, logits, fb.fp8bs_logprobs(logits, self.tokens.int(), self.top)


def tune(block, tokens, targets, advantages, entropy_bonus=0.01):
    """Gradients of -mean(advantage * log p(target) + entropy_bonus * entropy)
    with respect to the embedding and the attention's output projection, for
    tokens [T] taken each by itself, targets and advantages [T]."""
    x = block.emb.t()[tokens] * block.emb.shape[0] ** 0.5
    logits = block.logits(x, torch.ones(len(tokens), block.heads, 128, device=block.device))
    logprob, entropy = LogProbs.apply(logits, targets.int())
    loss = -(advantages * logprob + entropy_bonus * entropy).mean()
    return loss.detach(), torch.autograd.grad(loss, [block.emb, block.w_o])


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--cache", choices=["bf16", "fp8", "fp4"], default="fp4")
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--top", type=int, default=5)
    args = ap.parse_args()
    block = Block(torch.device("cuda"))
    server = Server(block, (40, 7, 100), args.steps, args.cache, top=args.top)
    for _ in range(args.steps):
        _, _, (logprob, entropy, _, rank, top_ids, top_logprobs) = server.step(lambda logits: logits.argmax(-1))
    for b, n in enumerate(server.lens.tolist()):
        best = ", ".join(f"{i} {p:.3f}" for i, p in zip(top_ids[b].tolist(), top_logprobs[b].tolist()))
        print(f"request {b}: {n} tokens in the cache, the last one's log probability {logprob[b]:.3f} (place {rank[b]}), "
              f"entropy {entropy[b]:.3f}; best: {best}")
    g = torch.Generator(device=block.device).manual_seed(3)
    t = torch.randint(block.vocab, (2, 64), generator=g, device=block.device)
    loss, grads = tune(block, t[0], t[1], torch.randn(64, generator=g, device=block.device))
    print(f"tuning step: loss {loss:.4f}, gradient norms {', '.join(f'{x.norm():.4f}' for x in grads)}")


if __name__ == "__main__":
    main()
