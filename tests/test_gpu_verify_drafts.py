"""Draft verification on the GPU against the oracle: whole numbers, so equal."""

import numpy as np
import pytest
import torch

from oracle import attention as oa

import fp8_block_scaled_x1_amd as fb

pytestmark = pytest.mark.gpu


def _case(B, K, V, seed, dtype=torch.float32, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    p = torch.softmax(sharp * torch.randn((B, K + 1, V), generator=g), -1).to(dtype)
    q = torch.softmax(sharp * torch.randn((B, K, V), generator=g) * 0.3 + torch.log(p[:, :K].float() + 1e-9), -1).to(dtype)
    drafts = torch.randint(0, V, (B, K), generator=g, dtype=torch.int32)
    n = torch.randint(0, K + 1, (B,), generator=g, dtype=torch.int32)
    u = torch.rand((B, K), generator=g) ** 2
    return p, q, drafts, n, u, torch.rand(B, generator=g)


def _compare(dev, p, q, drafts, n, u, un):
    got = fb.fp8bs_verify_drafts(*(None if x is None else x.to(dev) for x in (p, q, drafts, n, u, un)))
    f = lambda x: None if x is None else x.float().numpy()
    want = oa.verify_drafts(f(p), f(q), drafts.numpy(), n.numpy(), u.numpy(), un.numpy())
    for a, b, what in zip(got, want, ("tokens", "accepted")):
        assert np.array_equal(a.cpu().numpy(), b), f"{what}: {a.cpu().numpy()} against {b}"
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,K,V", [(1, 1, 1), (3, 2, 5), (7, 4, 63), (4, 3, 64), (5, 1, 4095), (2, 6, 4096), (3, 2, 4097),
                                   (4, 0, 1000), (2, 63, 300), (2, 2, 70001)])
def test_against_oracle(dev, B, K, V, dtype):
    p, q, *rest = _case(B, K, V, B * 1000 + V, dtype)
    _compare(dev, p, q, *rest)
    _compare(dev, p, None, *rest)


def test_all_accepted_and_none(dev):
    p, q, drafts, n, u, un = _case(6, 4, 500, 1)
    n[:] = 4
    tokens, accepted = _compare(dev, p, p[:, :4].clone(), drafts, n, u * 0 + 0.999, un)
    assert accepted.tolist() == [4] * 6 and torch.equal(tokens[:, :4].cpu(), drafts)
    tokens, accepted = _compare(dev, p, q, drafts, n, u * 0 + float("inf"), un)
    assert accepted.tolist() == [0] * 6 and torch.all(tokens[:, 1:] == -1)


def test_edges(dev):
    # ends of u_next, no weight anywhere, nothing left of p - q, drafts and counts out of range, NaN entries
    p, q, drafts, n, u, un = _case(8, 2, 1000, 2)
    un[0], un[1], un[2] = 0.0, 1.0 - 2.0 ** -24, 1.5
    p[3] = 0.0
    q[4] = 1.0
    drafts[5], n[5] = 1000, 2
    drafts[6], n[6] = -1, 99
    n[7] = -3
    p[7, 0, ::2] = float("nan")
    _compare(dev, p, q, drafts, n, u, un)


def test_first_and_last_entry_and_ties(dev):
    # equal weights: the running sums are whole multiples, so the limits are hit exactly
    V = 8192
    p = torch.full((V + 1, 1, V), 1.0 / V)
    un = torch.arange(V + 1).float() / V
    un[-1] = 1.0 - 2.0 ** -24
    z = torch.zeros((V + 1, 0))
    tokens, _ = fb.fp8bs_verify_drafts(*(x.to(dev) for x in (p, torch.zeros((V + 1, 0, V)), z.int(),
                                                             torch.zeros(V + 1).int(), z, un)))
    assert tokens[:-1, 0].tolist() == list(range(V)) and tokens[-1, 0] == V - 1


def test_same_in_a_graph(dev):
    args = [x.to(dev) for x in _case(5, 3, 10007, 4)]
    ref = [x.clone() for x in fb.fp8bs_verify_drafts(*args)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = fb.fp8bs_verify_drafts(*args)
    for _ in range(3):
        for x in res:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, ref):
            assert torch.equal(a, b)
