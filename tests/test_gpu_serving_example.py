"""The operators of a serving step run together, as the example does, and the
gradients of its tuning step."""

import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

from oracle import serve as os_

import fp8_block_scaled_x1_amd as fb
import serving_step as ex

pytestmark = pytest.mark.gpu

PROMPTS = (40, 7, 100, 1)


def _argmax(logits):
    return logits.argmax(-1)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp4"])
def test_attention_of_the_steps_is_that_of_the_cache(dev, cache):
    """The attention of every step against the expanded form in 64 bits over the
    numbers that the cache gives back."""
    block = ex.Block(dev)
    server = ex.Server(block, PROMPTS, 3, cache)
    for _ in range(3):
        _, q, *_ = block.project(server.tokens, server.lens)
        o, *_ = server.step(_argmax)
        lens = server.lens.tolist()
        c, r = fb.fp8bs_mla_cache_read(server.cache, server.table, server.lens, ex.offsets(lens, dev), sum(lens))
        w = block.w_kv.detach().bfloat16().double().cpu()
        at = 0
        for b, n in enumerate(lens):
            kv = (c[at:at + n].double().cpu() @ w).unflatten(-1, (block.heads, 256))
            k = torch.cat([kv[..., :128], r[at:at + n].double().cpu()[:, None].expand(-1, block.heads, -1)], -1)
            s = torch.einsum("hd,nhd->hn", q[b].detach().double().cpu(), k) * ex.SCALE
            want = torch.einsum("hn,nhd->hd", s.softmax(-1), kv[..., 128:])
            # folded queries, weights, latent outputs and outputs are rounded to BF16: 2^-8 / sqrt(12) * 1.5 of the
            # norm each, twice that for the weights' part that comes by the scores
            assert (o[b].double().cpu() - want).norm() <= 5 * 0.0017 * want.norm()
            at += n


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp4"])
def test_log_probabilities_of_the_steps(dev, cache):
    server = ex.Server(ex.Block(dev), PROMPTS, 4, cache, top=7)
    for i in range(4):
        _, logits, got = server.step(_argmax if i % 2 else lambda x: x.argmin(-1))
        want, bound = os_.logprobs(logits.double().cpu().numpy(), server.tokens.cpu().numpy(), 7)
        for n, t in zip(("logprob", "entropy", "norm", "rank", "top_ids", "top_logprobs"), got):
            t = t.cpu().numpy()
            if n in ("rank", "top_ids"):
                assert np.array_equal(t, want[n])
            else:
                assert (np.abs(t.astype(np.float64) - want[n]) <= bound[n]).all(), n
    assert server.lens.tolist() == [n - 1 + 4 for n in PROMPTS]


@pytest.mark.parametrize("cache", ["fp8", "fp4"])
def test_captured_steps_of_two_servers(dev, cache):
    """Two servers' steps, each captured once and replayed in turn, with an eager
    server's steps between: the same numbers, step by step, as eager servers give."""
    block = ex.Block(dev)

    def servers():
        return [ex.Server(block, PROMPTS, 8, cache), ex.Server(block, (3, 60), 8, cache, page=17, seed=5)]

    eager, captured, between = servers(), servers(), ex.Server(block, (9,), 40, cache)
    graphs, results = [], []
    for s in captured:
        keep = s.tokens.clone(), s.lens.clone()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            s.step(_argmax)                      # (libraries set themselves up)
        torch.cuda.current_stream().wait_stream(stream)
        torch.cuda.synchronize()
        s.tokens.copy_(keep[0])
        s.lens.copy_(keep[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = s.step(_argmax)
        s.tokens.copy_(keep[0])
        s.lens.copy_(keep[1])
        graphs.append(graph)
        results.append(out)
    for _ in range(5):
        want = [s.step(_argmax) for s in eager]
        for g in graphs:
            g.replay()
            between.step(_argmax)
        torch.cuda.synchronize()
        for w, r, a, b in zip(want, results, eager, captured):
            assert torch.equal(a.tokens, b.tokens) and torch.equal(a.lens, b.lens)
            assert torch.equal(w[0], r[0]) and torch.equal(w[1], r[1])
            for x, y in zip(w[2], r[2]):
                assert torch.equal(x, y)


def test_steps_on_streams_beside_each_other(dev):
    block = ex.Block(dev)
    args = [(PROMPTS, 6, "fp4"), ((3, 60), 6, "fp8"), ((200,), 6, "bf16")]
    want = []
    for a in args:
        s = ex.Server(block, *a)
        want.append([s.step(_argmax) for _ in range(6)])
    servers, streams = [ex.Server(block, *a) for a in args], [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    got = [[] for _ in args]
    for _ in range(6):
        for s, stream, to in zip(servers, streams, got):
            with torch.cuda.stream(stream):
                to.append(s.step(_argmax))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for x, y in zip(w, g):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1]) and all(torch.equal(p, q) for p, q in zip(x[2], y[2]))


def test_tuning_gradients(dev):
    """Against the formula's gradient of the logits in 64 bits, carried to the weights by torch."""
    block = ex.Block(dev)
    g = torch.Generator(device=dev).manual_seed(4)
    t = torch.randint(block.vocab, (2, 37), generator=g, device=dev)
    adv = torch.randn(37, generator=g, device=dev)
    loss, grads = ex.tune(block, t[0], t[1], adv)
    x = block.emb.t()[t[0]] * block.emb.shape[0] ** 0.5
    logits = block.logits(x, torch.ones(37, block.heads, 128, device=dev))
    lp = logits.detach().double().requires_grad_()
    p = lp.log_softmax(-1)
    plain = -(adv.double() * p.gather(1, t[1][:, None])[:, 0] - 0.01 * (p.exp() * p).sum(-1)).mean()
    plain.backward()
    assert abs(loss.item() - plain.item()) <= 2 ** -18 * p.abs().max().item() * adv.abs().max().item()
    want = torch.autograd.grad(logits, [block.emb, block.w_o], lp.grad.float())
    for a, b in zip(grads, want):
        # FP32 gradients of the logits, some 2^-22 of their largest apart, rounded to BF16 on the way through the
        # products: where a rounding falls the other way it differs by 2^-8, which is rare
        assert (a - b).norm() <= 2 ** -8 * b.norm()


def test_only_one_of_the_outputs_is_used(dev):
    logits = torch.randn(5, 300, generator=torch.Generator().manual_seed(0)).to(dev).requires_grad_()
    targets = torch.tensor([0, 299, 5, -1, 17], dtype=torch.int32, device=dev)
    for pick in (0, 1):
        got, = torch.autograd.grad(ex.LogProbs.apply(logits, targets)[pick].sum(), logits)
        x = logits.detach().double().requires_grad_()
        p = x.log_softmax(-1)
        inside = (targets >= 0).double()
        value = (p.gather(1, targets.clamp_min(0).long()[:, None])[:, 0] * inside).sum() if pick == 0 else -(p.exp() * p).sum()
        want, = torch.autograd.grad(value, x)
        assert (got.double() - want).abs().max() <= 2 ** -18


def test_outputs_may_be_changed_in_place(dev):
    """Masking ignored tokens in place, as a training loss does: the outputs share nothing, with what is kept for the
    gradient neither."""
    x = torch.randn(6, 300, generator=torch.Generator().manual_seed(3)).to(dev).requires_grad_()
    y = torch.tensor([0, 299, 5, -1, 17, 100], dtype=torch.int32, device=dev)
    ignored = torch.tensor([0, 1, 0, 0, 1, 0], dtype=torch.bool, device=dev)
    logprob, entropy = ex.LogProbs.apply(x, y)
    want, = torch.autograd.grad((logprob * ~ignored).sum() + entropy.sum(), x)
    logprob, entropy = ex.LogProbs.apply(x, y)
    logprob.masked_fill_(ignored, 0.0)
    got, = torch.autograd.grad(logprob.sum() + entropy.sum(), x)
    assert torch.equal(got, want)
    assert len({t.untyped_storage().data_ptr() for t in fb.fp8bs_logprobs(x.detach(), y, 2)}) == 6
