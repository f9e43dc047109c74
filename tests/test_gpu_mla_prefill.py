"""Expanded latent attention on the GPU, forward and gradients, against the
float64 oracle: every element inside the bound that follows from rounding the
probabilities (and dS) and the outputs to BF16."""

import numpy as np
import pytest
import torch

from oracle import attention as oa

import fp8_block_scaled_x1_amd as fb

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5
NAN = float("nan")


def _f64(t):
    return t.detach().double().cpu().numpy()


def _off(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _inputs(dev, lens, H, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    cq, ck = _off([a for a, _ in lens]), _off([b for _, b in lens])
    q = (torch.randn((cq[-1], H, 192), generator=g) * std).to(torch.bfloat16).to(dev)
    kv = torch.randn((ck[-1], H, 256), generator=g).to(torch.bfloat16).to(dev)
    kr = torch.randn((ck[-1], 64), generator=g).to(torch.bfloat16).to(dev)
    dout = torch.randn((cq[-1], H, 128), generator=g).to(torch.bfloat16).to(dev)
    return q, kv, kr, dout, cq, ck


def _inside(got, ref, what):
    want, bound = ref
    got = _f64(got)
    assert got.shape == want.shape, what
    same_inf = np.isneginf(want) & np.isneginf(got)
    with np.errstate(invalid="ignore"):
        bad = ~(same_inf | (np.abs(got - want) <= bound))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first at {tuple(np.argwhere(bad)[0])}: " \
                          f"{got[bad][0]} against {want[bad][0]} +- {bound[bad][0]}"


def _check(dev, lens, H, causal, seed=0, scale=SCALE, std=1.5):
    q, kv, kr, dout, cq, ck = _inputs(dev, lens, H, seed, std)
    tq, tk = torch.from_numpy(cq).to(dev), torch.from_numpy(ck).to(dev)
    out, lse = fb.fp8bs_mla_prefill(q, kv, kr, tq, tk, scale, causal=causal)
    grads = fb.fp8bs_mla_prefill_bwd(dout, q, kv, kr, out, lse, tq, tk, scale, causal=causal)
    torch.cuda.synchronize()
    ref = oa.mla_prefill(_f64(q), _f64(kv), _f64(kr), cq, ck, scale, causal, _f64(dout))
    _inside(out, ref["out"], f"out {lens} {causal}")
    _inside(lse, ref["lse"], f"lse {lens} {causal}")
    for name, x in zip(("dq", "dkv", "dk_rope"), grads):
        _inside(x, ref[name], f"{name} {lens} {causal}")


LENS = [
    [(1, 1)],
    [(1, 200)],
    [(64, 64), (65, 65), (63, 63)],
    [(128, 128), (129, 129)],
    [(33, 97), (1, 64), (127, 191)],                # chunks behind cached tokens, ends inside tiles
    [(260, 260)],
    [(5, 0), (0, 7), (3, 3), (0, 0)],               # no keys, no queries, neither
    [(70, 20), (200, 130), (2, 1)],                 # causal rows that see nothing
    [(40, 300), (150, 513)],
]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_against_oracle(dev, lens, causal):
    _check(dev, lens, 3, causal, seed=len(lens))


@pytest.mark.parametrize("lens", [
    [(3, 5000)],
    [(1, 1300), (130, 2049), (33, 700)],            # parts ending on and off the causal edge, one block without parts
    [(257, 1500), (1, 1), (0, 4000), (64, 1023)],
    [(1500, 1200)],                                 # causal: the first 300 queries see nothing
], ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_keys_in_parts(dev, lens, causal):
    sizes = len(lens), sum(a for a, _ in lens), sum(b for _, b in lens)
    assert fb.attn_lib().fp8bs_mla_prefill_workspace_bytes(*sizes, 2) > 0
    _check(dev, lens, 2, causal, seed=3)


@pytest.mark.parametrize("H", [1, 2, 5, 8, 16, 24])
def test_head_counts(dev, H):
    _check(dev, [(77, 77), (1, 130)], H, True, seed=H)


@pytest.mark.parametrize("std,scale", [(0.01, SCALE), (12.0, SCALE), (1.0, 1e-4), (1.0, 1.0)])
def test_flat_and_peaked_scores(dev, std, scale):
    _check(dev, [(90, 90), (40, 100)], 2, True, seed=7, scale=scale, std=std)


def test_many_short_requests(dev):
    rng = np.random.default_rng(2)
    _check(dev, [(int(n), int(n + e)) for n, e in zip(rng.integers(0, 9, 150), rng.integers(0, 4, 150))], 2, True)


def test_tokens_with_gaps(dev):
    # q, kv and k_rope as slices of wider rows, as a fused projection leaves them
    q, kv, kr, dout, cq, ck = _inputs(dev, [(50, 50), (90, 120)], 4, 3)
    tq, tk = torch.from_numpy(cq).to(dev), torch.from_numpy(ck).to(dev)
    ref = fb.fp8bs_mla_prefill(q, kv, kr, tq, tk, SCALE)
    wide = torch.full((len(q), 4 * 192 + 64), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, 64:] = q.reshape(len(q), -1)
    wkv = torch.full((len(kv), 4 * 256 + 8), float("nan"), dtype=torch.bfloat16, device=dev)
    wkv[:, :-8] = kv.reshape(len(kv), -1)
    lat = torch.full((len(kr), 576), float("nan"), dtype=torch.bfloat16, device=dev)
    lat[:, 512:] = kr
    views = wide[:, 64:].unflatten(1, (4, 192)), wkv[:, :-8].unflatten(1, (4, 256)), lat[:, 512:]
    got = fb.fp8bs_mla_prefill(*views, tq, tk, SCALE)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    for a, b in zip(fb.fp8bs_mla_prefill_bwd(dout, *views, *got, tq, tk, SCALE),
                    fb.fp8bs_mla_prefill_bwd(dout, q, kv, kr, *ref, tq, tk, SCALE)):
        assert torch.equal(a, b)
    with pytest.raises(fb.Fp8bsError):          # 193 numbers apart: not 16-byte aligned
        fb.fp8bs_mla_prefill(torch.zeros(8, 193, dtype=torch.bfloat16, device=dev)[:, :192].unflatten(1, (1, 192)),
                             kv[:8, :1].contiguous(), kr[:8], tq[:2] * 0, tk[:2] * 0, SCALE)
    with pytest.raises(ValueError, match="contiguous"):
        fb.fp8bs_mla_prefill(q.transpose(0, 1).contiguous().transpose(0, 1), kv, kr, tq, tk, SCALE)


def test_requests_do_not_see_each_other(dev):
    # a request's results do not depend on its neighbours in the batch, nor on their values
    q, kv, kr, dout, cq, ck = _inputs(dev, [(60, 60), (61, 100), (200, 200)], 2, 4)
    tq, tk = torch.from_numpy(cq).to(dev), torch.from_numpy(ck).to(dev)
    out, lse = fb.fp8bs_mla_prefill(q, kv, kr, tq, tk, SCALE)
    i, j = slice(cq[1], cq[2]), slice(ck[1], ck[2])
    one = [torch.tensor([0, n], dtype=torch.int32, device=dev) for n in (61, 100)]
    o1, l1 = fb.fp8bs_mla_prefill(q[i].contiguous(), kv[j].contiguous(), kr[j].contiguous(), *one, SCALE)
    assert torch.equal(out[i], o1) and torch.equal(lse[:, i], l1)
    q[:cq[1]] = float("nan")
    kv[ck[2]:], kr[ck[2]:] = float("inf"), float("nan")
    o2, l2 = fb.fp8bs_mla_prefill(q, kv, kr, tq, tk, SCALE)
    assert torch.equal(o2[i], o1) and torch.equal(l2[:, i], l1)
    g1 = fb.fp8bs_mla_prefill_bwd(dout[i].contiguous(), q[i].contiguous(), kv[j].contiguous(), kr[j].contiguous(), o1, l1,
                                  *one, SCALE)
    g2 = fb.fp8bs_mla_prefill_bwd(dout, q, kv, kr, o2, l2, tq, tk, SCALE)
    assert torch.equal(g2[0][i], g1[0]) and torch.equal(g2[1][j], g1[1]) and torch.equal(g2[2][j], g1[2])


@pytest.mark.parametrize("causal", [True, False])
def test_gradients_of_few_keys_keep_their_precision(dev, causal):
    # A rounding to BF16 is 2^-7 / sqrt(12) of its power of two, 0.00166 of the values' norm. dQ and dK hold two of
    # them, of dS and of the result: 0.00235, one and a half single ones with room for the sample. The rounding of the
    # output must not come in through D = dO . O, where few keys make it as large as theirs.
    lens = [(n, n) for n in (2, 5, 17, 33, 48, 64)]
    q, kv, kr, dout, cq, ck = _inputs(dev, lens, 8, 11)
    tq, tk = torch.from_numpy(cq).to(dev), torch.from_numpy(ck).to(dev)
    out, lse = fb.fp8bs_mla_prefill(q, kv, kr, tq, tk, SCALE, causal=causal)
    grads = fb.fp8bs_mla_prefill_bwd(dout, q, kv, kr, out, lse, tq, tk, SCALE, causal=causal)
    ref = oa.mla_prefill(_f64(q), _f64(kv), _f64(kr), cq, ck, SCALE, causal, _f64(dout))
    for name, x in zip(("dq", "dkv", "dk_rope"), grads):
        want = ref[name][0]
        assert np.linalg.norm(_f64(x) - want) <= 0.0025 * np.linalg.norm(want), name


def test_long_rows_against_float32(dev):
    # long enough to rescale often, with ends off every tile: the sampled rows of one head
    lens = [(1500, 2777)]
    q, kv, kr, dout, cq, ck = _inputs(dev, lens, 8, 6)
    tq, tk = torch.from_numpy(cq).to(dev), torch.from_numpy(ck).to(dev)
    out, lse = fb.fp8bs_mla_prefill(q, kv, kr, tq, tk, SCALE)
    for h in (0, 7):
        K = np.concatenate([_f64(kv[:, h, :128]), _f64(kr)], -1)
        for row in (0, 1, 127, 128, 700, 1499):
            n = row + 1 + 2777 - 1500
            o, l, bo, bl = oa.mla_head(_f64(q[row:row + 1, h]), K[:n], _f64(kv[:n, h, 128:]), SCALE, False)
            _inside(out[row:row + 1, h], (o, bo), f"row {row} head {h}")
            _inside(lse[h, row:row + 1], (l, bl), f"lse {row} head {h}")


@pytest.mark.parametrize("lens", [[(130, 130), (70, 200)], [(70, 3000)]], ids=str)      # (whole, in parts)
def test_same_bits_every_time_and_in_a_graph(dev, lens):
    q, kv, kr, dout, cq, ck = _inputs(dev, lens, 8, 9)
    tq, tk = torch.from_numpy(cq).to(dev), torch.from_numpy(ck).to(dev)

    def step():
        out, lse = fb.fp8bs_mla_prefill(q, kv, kr, tq, tk, SCALE)
        return (out, lse, *fb.fp8bs_mla_prefill_bwd(dout, q, kv, kr, out, lse, tq, tk, SCALE))

    ref = [x.clone() for x in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a, b in zip(step(), ref):
            assert torch.equal(a, b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for _ in range(3):
        for x in res:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, ref):
            assert torch.equal(a, b)


def _sampled(dev, lens, H, heads, causal, seed):
    """out, lse, dq, dkv of some heads of a problem large enough for blocks of 256 queries, and
    dk_rope where these are all the heads."""
    q, kv, kr, dout, cq, ck = _inputs(dev, lens, H, seed)
    tq, tk = torch.from_numpy(cq).to(dev), torch.from_numpy(ck).to(dev)
    out, lse = fb.fp8bs_mla_prefill(q, kv, kr, tq, tk, SCALE, causal=causal)
    dq, dkv, dk_rope = fb.fp8bs_mla_prefill_bwd(dout, q, kv, kr, out, lse, tq, tk, SCALE, causal=causal)
    torch.cuda.synchronize()
    at = torch.tensor(heads)
    pick = lambda t: _f64(t[:, at.to(t.device)])
    ref = oa.mla_prefill(pick(q), pick(kv), _f64(kr), cq, ck, SCALE, causal, pick(dout))
    what = f"{lens} H {H} causal {causal}"
    for name, x in (("out", out), ("dq", dq), ("dkv", dkv)):
        _inside(x[:, at.to(dev)], ref[name], f"{name} {what}")
    _inside(lse[at.to(dev)], ref["lse"], f"lse {what}")
    if len(heads) == H:
        _inside(dk_rope, ref["dk_rope"], f"dk_rope {what}")
    return (q, kv, kr, dout, tq, tk), (out, lse, dq, dkv, dk_rope)


# causal ends inside blocks and tiles, chunks, waves without queries, no keys, rows that see nothing
MIXED = [(257, 257), (1, 70), (300, 513), (5, 0), (70, 20), (255, 256)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H", [128, 200])
def test_blocks_of_256_queries(dev, H, causal):
    # (groups of four heads per XCD: 128 has four whole ones, 200 six and one of a single head)
    _sampled(dev, MIXED, H, [0, 7, 31, 63, 100, H - 9, H - 1], causal, seed=H)


@pytest.mark.parametrize("H", [40, 48])
def test_blocks_of_256_queries_every_head(dev, H):
    # five and six heads per XCD: the last group has one and two; the rotary gradient sums them all
    lens = [(33, 33), (1, 90), (64, 64), (20, 85), (3, 2)] * 6
    _sampled(dev, lens, H, list(range(H)), True, seed=H)


@pytest.mark.parametrize("H", [56, 64, 65, 72, 128, 256, 344])
def test_both_sides_of_the_block_size_rule(dev, H):
    _sampled(dev, [(300, 300), (212, 700)], H, [0, 3, H // 2, H - 1], True, seed=H)


@pytest.mark.parametrize("H", [192, 193])
def test_one_and_a_half_blocks_per_compute_unit(dev, H):
    # (two blocks of 256 queries, by the average, on 256 compute units: blocks of 128 up to here, of 256 from here on)
    _sampled(dev, [(300, 300), (212, 700)], H, [0, 3, 100, H - 1], True, seed=H)


def test_blocks_of_256_queries_with_gaps_and_in_a_graph(dev):
    H = 128
    (q, kv, kr, dout, tq, tk), ref = _sampled(dev, MIXED, H, [5], True, seed=1)
    ref = [x.clone() for x in ref]
    wide = torch.full((len(q), H * 192 + 8), NAN, dtype=torch.bfloat16, device=dev)
    wide[:, 8:] = q.reshape(len(q), -1)
    wkv = torch.full((len(kv), H * 256 + 64), NAN, dtype=torch.bfloat16, device=dev)
    wkv[:, :-64] = kv.reshape(len(kv), -1)
    lat = torch.full((len(kr), 576), NAN, dtype=torch.bfloat16, device=dev)
    lat[:, 512:] = kr
    views = wide[:, 8:].unflatten(1, (H, 192)), wkv[:, :-64].unflatten(1, (H, 256)), lat[:, 512:]

    def step():
        out, lse = fb.fp8bs_mla_prefill(*views, tq, tk, SCALE)
        return (out, lse, *fb.fp8bs_mla_prefill_bwd(dout, *views, out, lse, tq, tk, SCALE))

    for a, b in zip(step(), ref):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for _ in range(3):
        for x in res:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, ref):
            assert torch.equal(a, b)
