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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [8191, 8192, 8193, 8196, 16384, 129280])
def test_sizes_around_whole_chunks(dev, V, dtype):
    # a row's sums are taken 8192 entries at a time; four entries a load where V is a multiple of four
    p, q, drafts, n, u, un = _case(6, 2, V, V, dtype, sharp=0.5)
    n[:] = torch.tensor([2, 2, 2, 1, 0, 2])
    for b in (0, 3):         # likely drafts (accepted at a small u), the others are turned down
        drafts[b] = p[b, :2].float().argmax(-1)
        u[b] = 0.0
    un[:] = torch.tensor([0.0, 0.999999, 0.5, 0.93, 0.07, 0.3])
    _compare(dev, p, q, drafts, n, u, un)
    _compare(dev, p, None, drafts, n, u, un)


@pytest.mark.parametrize("dtype,skip", [(torch.float32, 1), (torch.bfloat16, 2)])
def test_rows_that_are_not_aligned_for_wide_loads(dev, dtype, skip):
    # four bytes behind an aligned address, rows of whole groups of four entries
    p, q, *rest = _case(4, 2, 9000, 9, dtype)

    def shifted(x):
        buf = torch.zeros(x.numel() + skip, dtype=dtype, device=dev)
        view = buf[skip:].view(x.shape)
        view.copy_(x)
        assert view.data_ptr() % 16 == 4
        return view

    want = fb.fp8bs_verify_drafts(*(x.to(dev) for x in (p, q, *rest)))
    _compare(dev, p, q, *rest)
    for a, b in ((shifted(p), q.to(dev)), (p.to(dev), shifted(q)), (shifted(p), shifted(q))):
        got = fb.fp8bs_verify_drafts(a, b, *(x.to(dev) for x in rest))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_more_than_64_chunks(dev, dtype):
    # 128 chunks of equal weights: token floor(u * V); at the chunks' limits, and the random number before each
    V = 1 << 20
    at = torch.tensor([0, 1, 63, 64, 65, 100, 127])
    un = torch.cat([at / 128, (at[1:] / 128) - 2.0 ** -24, torch.tensor([1 - 2.0 ** -24, 0.51, 0.4999])]).float()
    B = len(un)
    p = torch.full((B, 1, V), 2.0 ** -20, dtype=dtype)
    z = torch.zeros((B, 0))
    args = p, None, z.int(), torch.zeros(B).int(), z, un
    got = fb.fp8bs_verify_drafts(*(None if x is None else x.to(dev) for x in args))
    assert got[0][:, 0].tolist() == torch.floor(un.double() * V).int().tolist() and got[1].tolist() == [0] * B


def test_more_than_64_chunks_of_random_weights(dev):
    V = 600001
    p, q, drafts, n, u, un = _case(3, 1, V, 12, sharp=0.5)
    un[:] = torch.tensor([1e-6, 0.9, 0.9999])
    _compare(dev, p[:, :1].contiguous(), q[:, :0].contiguous(), drafts[:, :0].contiguous(), n * 0, u[:, :0].contiguous(), un)
    u[:] = float("inf")
    _compare(dev, p, q, drafts, n * 0 + 1, u, un)
