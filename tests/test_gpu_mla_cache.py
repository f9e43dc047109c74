"""Writing to and reading from the paged cache on the GPU against the oracle:
codes, scales and untouched slots equal, bit for bit; what is read back is the
value rounded once."""

import numpy as np
import pytest
import torch

import oracle
from oracle import serve as os_

import fp8_block_scaled_x1_amd as fb

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "fp8", "fp4"]


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


def _bytes_of(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def _empty(dev, kind, pages, page, seed=0):
    """A cache full of arbitrary bytes."""
    g = torch.Generator().manual_seed(seed)

    def fill(*shape):
        return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).to(dev)

    rope = fill(pages, page, 128).view(torch.bfloat16)
    if kind == "bf16":
        return fill(pages, page, 1152).view(torch.bfloat16)
    if kind == "fp8":
        return fill(pages, page, 512), fill(pages, page, 16).view(torch.float32), rope
    return fill(pages, page, 256), fill(pages, page, 16), rope


def _parts(cache):
    return list(cache) if isinstance(cache, tuple) else [cache]


def _want_parts(kind, latent, rope):
    """The bytes of each token's slot, part by part."""
    x = latent.float().numpy()
    if kind == "bf16":
        return [_bytes_of(torch.cat([latent, rope], -1))]
    if kind == "fp8":
        q, s = oracle.quant_act_1x128(x)
        return [q, np.ascontiguousarray(s.T).view(np.uint8), _bytes_of(rope)]
    q, e = os_.fp4_quant(x.astype(np.float64))
    return [q, e, _bytes_of(rope)]


def _values(kind, parts):
    """BF16 numbers of slots' bytes (n rows), as the read gives them."""
    if kind == "bf16":
        x = torch.from_numpy(parts[0].copy()).view(torch.bfloat16)
        return x[:, :512], x[:, 512:]
    rope = torch.from_numpy(parts[2].copy()).view(torch.bfloat16)
    if kind == "fp8":
        code = torch.from_numpy(parts[0].copy()).view(torch.float8_e4m3fn).float()
        s = torch.from_numpy(parts[1].copy()).view(torch.float32).repeat_interleave(128, -1)
        return (code * s).to(torch.bfloat16), rope
    return _bf16(os_.fp4_values(parts[0], parts[1])), rope


def _tables(lens, page, seed, width=None):
    rng = np.random.default_rng(seed)
    need = [max(0, -(-n // page)) for n in lens]
    pages = sum(need) + 3
    order = rng.permutation(pages)
    width = max(need + [1]) + 1 if width is None else width
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :min(n, width)] = order[at:at + min(n, width)]
        at += n
    return table, pages


def _cu(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def _run(dev, kind, page, new, lens, seed=0, extra=0, latent=None, gap=0):
    table, pages = _tables(lens, page, seed)
    cu, T = _cu(new), sum(new) + extra
    g = torch.Generator().manual_seed(seed + 1)
    if latent is None:
        latent = (torch.randn((T, 512), generator=g) * torch.exp2(torch.randint(-20, 20, (T, 1), generator=g).float())).bfloat16()
    rope = torch.randn((T, 64), generator=g).bfloat16()
    cache = _empty(dev, kind, pages, page, seed)
    before = [_bytes_of(p) for p in _parts(cache)]
    wide = torch.zeros((T, 512 + 64 + gap), dtype=torch.bfloat16)
    wide[:, :512], wide[:, 512:576] = latent, rope
    wide = wide.to(dev)
    up = [torch.from_numpy(np.asarray(a, np.int32)).to(dev) for a in (table, lens, cu)]
    fb.fp8bs_mla_cache_write(wide[:, :512], wide[:, 512:576], cache, *up)
    want = [p.copy() for p in before]
    rows = _want_parts(kind, latent, rope)
    at = os_.slots(table, lens, cu, page, T)
    for t, (pg, slot, ok) in enumerate(at):
        if ok == 1 and 0 <= pg < pages:
            for w, r in zip(want, rows):
                w[pg, slot] = r[t]
    for n, (got, w) in enumerate(zip(_parts(cache), want)):
        got = _bytes_of(got)
        bad = np.argwhere(got != w)
        assert not len(bad), f"part {n}: {len(bad)} bytes differ, first {tuple(bad[0])}: {got[tuple(bad[0])]} against {w[tuple(bad[0])]}"
    # and back; rows of no request stay as they were
    out = tuple(torch.full((T, n), 7.0, dtype=torch.bfloat16, device=dev) for n in (512, 64))
    got = fb.fp8bs_mla_cache_read(cache, *up, T, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    for t, (pg, slot, ok) in enumerate(at):
        for x, v in zip(got, _values(kind, [w[min(max(pg, 0), pages - 1), slot][None] for w in want])):
            row = x[t].cpu()
            if ok < 0:
                assert torch.all(row == 7.0)
            elif ok == 0:
                assert torch.all(row == 0.0)
            else:
                assert torch.equal(row.view(torch.int16), v[0].view(torch.int16)) or torch.equal(row, v[0]), t
    return cache, up


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [1, 7, 16, 64, 100])
@pytest.mark.parametrize("new,lens", [([1], [1]), ([1, 1, 1], [5, 64, 65]), ([3, 0, 70, 1], [3, 9, 200, 129]),
                                      ([130], [130]), ([0, 0, 2], [0, 0, 2])], ids=str)
def test_write_and_read(dev, kind, page, new, lens):
    _run(dev, kind, page, new, lens, seed=page, extra=2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B", [64, 65, 129, 4097])
def test_many_requests(dev, kind, B):
    rng = np.random.default_rng(B)
    new = [int(x) for x in rng.integers(0, 3, B)]
    _run(dev, kind, 4, new, [n + int(p) for n, p in zip(new, rng.integers(0, 9, B))], seed=B)


@pytest.mark.parametrize("kind", KINDS)
def test_positions_without_a_slot(dev, kind):
    # more new tokens than the request is long, negative lengths, and lengths past the table
    _run(dev, kind, 16, [5, 2, 3], [3, -4, 1000], seed=2)


@pytest.mark.parametrize("kind", KINDS)
def test_entries_outside_the_pool_are_not_written(dev, kind):
    cache = _empty(dev, kind, 3, 4)
    before = [_bytes_of(p) for p in _parts(cache)]
    x = torch.randn((4, 512), device=dev).bfloat16()
    up = [torch.tensor(a, dtype=torch.int32, device=dev) for a in ([[3], [-1], [1 << 30], [-(1 << 31)]], [2] * 4, [0, 1, 2, 3, 4])]
    fb.fp8bs_mla_cache_write(x, x[:, :64], cache, *up)
    for p, b in zip(_parts(cache), before):
        assert np.array_equal(_bytes_of(p), b)


def test_fp4_every_group_maximum(dev):
    # every positive finite BF16 number as a group's largest, among multiples of its sixteenth: all codes and ties
    bits = np.arange(1, 0x7F80, dtype=np.uint16)
    top = torch.from_numpy(bits.astype(np.int16)).view(torch.bfloat16)
    g = torch.Generator().manual_seed(0)
    frac = torch.randint(-16, 17, (len(bits), 32), generator=g).float() / 16
    x = (top.float()[:, None] * frac).bfloat16()
    x[:, 5] = top
    x[:, 6] = -0.0
    x = torch.cat([x, torch.zeros(-len(x) % 16, 32).bfloat16()]).reshape(-1, 512)
    _run(dev, "fp4", 64, [len(x)], [len(x)], latent=x)


def test_fp4_every_number(dev):
    # every finite BF16 number against maxima of 4, 6 and 7 (and smaller)
    bits = np.concatenate([np.arange(0, 0x40E1), np.arange(0x8000, 0xC0E1)]).astype(np.uint16)
    v = torch.from_numpy(bits.astype(np.int16)).view(torch.bfloat16)
    for top in (4.0, 6.0, 7.0):
        w = v[v.float().abs() <= top]
        w = torch.cat([w, torch.zeros(-len(w) % 31).bfloat16()]).reshape(-1, 31)
        x = torch.cat([w, torch.full((len(w), 1), top).bfloat16()], 1)
        x = torch.cat([x, torch.zeros(-len(x) % 16, 32).bfloat16()]).reshape(-1, 512)
        _run(dev, "fp4", 64, [len(x)], [len(x)], latent=x)


@pytest.mark.parametrize("kind", KINDS)
def test_zeros_and_strides(dev, kind):
    x = torch.zeros((5, 512)).bfloat16()
    x[1, 3], x[2] = -1.0, -0.0
    _run(dev, kind, 2, [5], [5], latent=x, gap=64)


@pytest.mark.parametrize("kind", KINDS)
def test_same_in_a_graph_and_on_a_stream(dev, kind):
    new, lens = [2, 1, 40], [2, 17, 60]
    table, pages = _tables(lens, 16, 3)
    up = [torch.from_numpy(np.asarray(a, np.int32)).to(dev) for a in (table, lens, _cu(new))]
    x = torch.randn((43, 512), device=dev).bfloat16()
    r = torch.randn((43, 64), device=dev).bfloat16()
    cache, eager = _empty(dev, kind, pages, 16), _empty(dev, kind, pages, 16)

    def step(c):
        fb.fp8bs_mla_cache_write(x, r, c, *up)
        return fb.fp8bs_mla_cache_read(c, *up, 43)

    step(cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(cache)
    for i in range(3):
        x.copy_(torch.randn((43, 512), device=dev))
        up[1].copy_(torch.tensor([n - i for n in lens], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, step(eager)):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step(eager)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(res, again):
        assert torch.equal(a, b)


def test_written_cache_is_the_one_that_decoding_reads(dev):
    # the FP8 and BF16 kinds against the layouts that the absorbed form documents
    lens, page = [70, 3], 16
    table, pages = _tables(lens, page, 1)
    up = [torch.from_numpy(np.asarray(a, np.int32)).to(dev) for a in (table, lens, _cu(lens))]
    x = torch.randn((73, 512), device=dev).bfloat16()
    r = torch.randn((73, 64), device=dev).bfloat16()
    q = torch.randn((2, 1, 4, 576), device=dev).bfloat16()
    for kind in KINDS:
        cache = _empty(dev, kind, pages, page)
        fb.fp8bs_mla_cache_write(x, r, cache, *up)
        latent, rope = fb.fp8bs_mla_cache_read(cache, *up, 73)
        plain = _empty(dev, "bf16", pages, page)
        fb.fp8bs_mla_cache_write(latent, rope, plain, *up)
        want = fb.fp8bs_mla_decode(q, plain, up[0], up[1], 0.07)
        got = (fb.fp8bs_mla_decode_fp4 if kind == "fp4" else fb.fp8bs_mla_decode)(q, cache, up[0], up[1], 0.07)
        # FP8: the numbers read back are rounded once more to BF16 (2^-9 of each, on scores of a few units)
        assert torch.allclose(got[1], want[1], atol=2e-2 if kind == "fp8" else 1e-5, rtol=0)
        limit = 0.02 if kind == "fp8" else 0.008       # each side's weights and output to BF16
        assert (got[0].float() - want[0].float()).norm() <= limit * want[0].float().norm()
