"""Absorbed latent attention over the 4-bit cache on the GPU, alone and behind a
shared prefix, against the float64 oracle, with the bounds that follow from
rounding the weights and the output to BF16."""

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import serve as os_

import fp8_block_scaled_x1_amd as fb

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def _f64(t):
    return t.detach().double().cpu().numpy()


class Paged:
    """Requests' tokens in scattered pages; unused slots hold infinite scales and NaN."""

    def __init__(self, dev, page, lens, seed, prefix=0, spare=3, exps=(125, 129)):
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        npre = -(-prefix // page)
        pages = sum(need) + npre + spare
        order = rng.permutation(pages)
        table = np.full((len(lens), max(need + [1]) + 1), -7, np.int32)       # never read behind a request's last token
        codes = rng.integers(0, 256, (pages, page, 256)).astype(np.uint8)
        scales = rng.integers(exps[0], exps[1] + 1, (pages, page, 16)).astype(np.uint8)
        rope = torch.from_numpy(rng.standard_normal((pages, page, 64))).to(torch.bfloat16)
        live = np.zeros((pages, page), bool)
        at = 0

        def take(n, count):
            nonlocal at
            mine = order[at:at + count]
            at += count
            pos = np.arange(n)
            live[mine[pos // page], pos % page] = True
            return mine, (mine[pos // page], pos % page)

        pre_pages, pre = take(prefix, npre)
        self.slots = []
        for b, n in enumerate(lens):
            mine, s = take(n, need[b])
            table[b, :need[b]] = mine
            self.slots.append(s)
        vals = np.concatenate([os_.fp4_values(codes, scales), _f64(rope)], -1)
        codes[~live], scales[~live], rope[torch.from_numpy(~live)] = 0x77, 0xFF, float("nan")
        self.cache = (torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev), rope.to(dev))
        self.prefix_keys = vals[pre]
        self.keys = [vals[s] for s in self.slots]
        self.table = torch.from_numpy(table).to(dev)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.prefix_table = torch.from_numpy(pre_pages.astype(np.int32)).to(dev)
        self.prefix_len = torch.tensor([prefix], dtype=torch.int32, device=dev)


def _inside(got, want, bound, what):
    got = _f64(got)
    with np.errstate(invalid="ignore"):
        bad = ~((np.isneginf(want) & np.isneginf(got)) | (np.abs(got - want) <= bound))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first at {tuple(np.argwhere(bad)[0])}: " \
                          f"{got[bad][0]} against {want[bad][0]} +- {bound[bad][0]}"


def _q(dev, B, T, H, seed, std=1.0):
    g = torch.Generator().manual_seed(seed + 100)
    return (torch.randn((B, T, H, 576), generator=g) * std).to(torch.bfloat16).to(dev)


def _check(dev, page, lens, T, H, seed=0, qstd=0.5):
    c = Paged(dev, page, lens, seed)
    q = _q(dev, len(lens), T, H, seed, qstd)
    out, lse = fb.fp8bs_mla_decode_fp4(q, c.cache, c.table, c.lens, SCALE)
    torch.cuda.synchronize()
    o, l, bo, bl = oa.mla_decode(_f64(q), c.keys, SCALE)
    what = f"page {page} lens {lens} T {T} H {H}"
    _inside(out, o, bo, "out " + what)
    _inside(lse, l, bl, "lse " + what)
    return c, q, out, lse


def _groups(B, T, H, width, page):
    """Workgroup ranges that the tiles of 64 tokens are shared by, from the workspace."""
    return fb.serve_lib().fp8bs_mla_decode_fp4_workspace_bytes(B, T, H, width, page, 0) // (2 * T * H * 514 * 4)


def _tiles(lens):
    return sum(-(-n // 64) for n in lens)


@pytest.mark.parametrize("lens", [[1], [2], [31], [32], [33], [127], [128], [129], [257], [1000]], ids=str)
def test_one_request(dev, lens):
    _check(dev, 64, lens, 1, 16, seed=lens[0])


def test_every_column_has_its_own_place(dev):
    # one token: the output is its latent numbers, exactly, in order
    c = Paged(dev, 16, [1, 1, 1], 3)
    q = _q(dev, 3, 1, 5, 3)
    out, _ = fb.fp8bs_mla_decode_fp4(q, c.cache, c.table, c.lens, SCALE)
    for b in range(3):
        assert np.array_equal(_f64(out)[b], np.broadcast_to(c.keys[b][:, :512], (1, 5, 512)))


@pytest.mark.parametrize("H,T", [(1, 1), (16, 1), (16, 2), (5, 3), (32, 1), (40, 1), (64, 1), (128, 1), (33, 4)])
def test_rows(dev, H, T):
    _check(dev, 64, [4, 70, 129, 300], T, H, seed=H)


@pytest.mark.parametrize("page", [1, 7, 16, 64, 100, 128])
def test_pages(dev, page):
    _check(dev, page, [1, 63, 64, 65, 257], 1, 16, seed=page)


@pytest.mark.parametrize("lens", [[0], [0, 0, 5], [3, 0, 700, 0], [2000], [64] * 70, list(range(0, 130))], ids=str)
def test_lengths(dev, lens):
    _check(dev, 16, lens, 1, 16, seed=len(lens))


@pytest.mark.parametrize("T", [2, 4, 7])
def test_drafted_tokens_hide_later_ones(dev, T):
    # lengths below T: the first queries see nothing at all
    _check(dev, 16, [0, 1, 2, 3, 5, 32, 33, 34, 64, 66, 128, 130], T, 4, seed=T)
    _check(dev, 16, [1, T, 65], T, 20, seed=T)


@pytest.mark.parametrize("qstd", [0.01, 10.0])
def test_flat_and_peaked(dev, qstd):
    _check(dev, 64, [300, 1000], 1, 16, seed=3, qstd=qstd)


def test_scales_far_apart(dev):
    c = Paged(dev, 16, [40, 200], 6, exps=(100, 128))
    q = _q(dev, 2, 1, 16, 6, 0.5)
    out, lse = fb.fp8bs_mla_decode_fp4(q, c.cache, c.table, c.lens, SCALE)
    o, l, bo, bl = oa.mla_decode(_f64(q), c.keys, SCALE)
    _inside(out, o, bo, "out")
    _inside(lse, l, bl, "lse")


SHORT = [100 + 37 * i % 600 for i in range(600)]
MANY_TILES = [(4, 128, [3000, 65, 700, 0, 129]), (3, 40, [2000, 1, 64, 900, 1500, 1100, 2500, 3000] * 3),
              (1, 16, [19000, 6400, 3, 0, 22000]), (1, 20, SHORT)]


@pytest.mark.parametrize("T,H,lens", MANY_TILES, ids=["512 rows", "120 rows", "long", "600 requests"])
def test_several_tiles_per_workgroup(dev, T, H, lens):
    c, *_ = _check(dev, 64, lens, T, H, seed=T + H)
    assert _tiles(lens) > 1.2 * _groups(len(lens), T, H, c.table.shape[1], 64)


@pytest.mark.parametrize("page", [1, 48])
def test_several_tiles_per_workgroup_of_other_pages(dev, page):
    lens = [2000, 64, 0, 333, 1]
    c, *_ = _check(dev, page, lens, 8, 128, seed=page)
    assert _tiles(lens) > 1.2 * _groups(len(lens), 8, 128, c.table.shape[1], page)


def test_reference_raised_over_sums(dev):
    # scores that grow along the request: each tile of a range raises the reference over what has been added up
    lens, T, H = [3000, 2300], 8, 128
    c = Paged(dev, 64, lens, 4)
    q = _q(dev, 2, T, H, 4, 2.0)
    q[..., 512] = 30.0
    keys = [k.copy() for k in c.keys]
    for b, n in enumerate(lens):
        ramp = (torch.arange(n) * 16 // n).float().to(torch.bfloat16)
        pages, pos = c.slots[b]
        c.cache[2][torch.from_numpy(pages).to(dev), torch.from_numpy(pos).to(dev), 0] = ramp.to(dev)
        keys[b][:, 512] = ramp.double().numpy()
    out, lse = fb.fp8bs_mla_decode_fp4(q, c.cache, c.table, c.lens, SCALE)
    assert _tiles(lens) > 1.2 * _groups(2, T, H, c.table.shape[1], 64)
    o, l, bo, bl = oa.mla_decode(_f64(q), keys, SCALE)
    _inside(out, o, bo, "out")
    _inside(lse, l, bl, "lse")


@pytest.mark.parametrize("prefix,lens,T,H,page", [
    (1, [1], 1, 1, 16), (100, [1, 70, 5], 1, 16, 16), (64, [64, 1], 2, 8, 64), (1000, [3, 0, 200, 65], 1, 16, 7),
    (500, [4] * 40, 1, 32, 128), (0, [5, 9], 1, 16, 16), (2000, [130, 2], 3, 20, 64),
    (1300, [1 + 13 * i % 250 for i in range(40)], 1, 128, 64), (4000, [2 + 29 * i % 260 for i in range(60)], 2, 16, 64),
])
def test_shared_prefix(dev, prefix, lens, T, H, page):
    c = Paged(dev, page, lens, 5, prefix=prefix)
    q = _q(dev, len(lens), T, H, 5, 0.5)
    out, lse = fb.fp8bs_mla_decode_fp4_shared(q, c.cache, c.prefix_table, c.prefix_len, c.table, c.lens, SCALE)
    torch.cuda.synchronize()
    keys = [(prefix, np.concatenate([c.prefix_keys, k])) for k in c.keys]
    o, l, bo, bl = oa.mla_decode(_f64(q), keys, SCALE)
    _inside(out, o, bo, f"shared {prefix} {lens}")
    _inside(lse, l, bl, f"shared lse {prefix} {lens}")


def test_prefix_and_own_tokens_empty(dev):
    c = Paged(dev, 16, [0, 3], 5, prefix=0)
    q = _q(dev, 2, 1, 4, 1)
    table = torch.zeros(2, dtype=torch.int32, device=dev)
    out, lse = fb.fp8bs_mla_decode_fp4_shared(q, c.cache, table, c.prefix_len, c.table, c.lens, SCALE)
    assert torch.all(out[0] == 0) and torch.all(torch.isneginf(lse[0])) and torch.all(torch.isfinite(lse[1]))
    # and no table at all
    out, lse = fb.fp8bs_mla_decode_fp4(q, c.cache, c.table[:, :0].contiguous(), c.lens, SCALE)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


def test_lengths_and_entries_are_clamped(dev):
    c, q, out, lse = _check(dev, 16, [40, 16], 1, 16, seed=1)
    lens = torch.tensor([40, -5], dtype=torch.int32, device=dev)
    o2, l2 = fb.fp8bs_mla_decode_fp4(q, c.cache, c.table, lens, SCALE)
    assert torch.equal(o2[0], out[0]) and torch.all(o2[1] == 0) and torch.all(torch.isneginf(l2[1]))
    wide = c.table[:, :1].contiguous()
    o3, _ = fb.fp8bs_mla_decode_fp4(q, c.cache, wide, torch.tensor([1 << 30, 16], dtype=torch.int32, device=dev), SCALE)
    o4, _ = fb.fp8bs_mla_decode_fp4(q, c.cache, wide, torch.tensor([16, 16], dtype=torch.int32, device=dev), SCALE)
    assert torch.equal(o3, o4)
    clean = (c.cache[0], c.cache[1].clamp(max=130), torch.nan_to_num(c.cache[2]))
    high, last = wide.clone(), wide.clone()
    high[1], last[1] = 1 << 30, c.cache[0].shape[0] - 1                # past the last page: the last page
    n = torch.tensor([16, 16], dtype=torch.int32, device=dev)
    assert torch.equal(fb.fp8bs_mla_decode_fp4(q, clean, high, n, SCALE)[0], fb.fp8bs_mla_decode_fp4(q, clean, last, n, SCALE)[0])


def test_nan_stays_with_the_rows_that_see_it(dev):
    c = Paged(dev, 16, [300, 200], 9)
    q = _q(dev, 2, 2, 16, 9, 0.5)
    pages, pos = c.slots[0]
    c.cache[2][int(pages[299]), int(pos[299]), 3] = float("nan")        # seen by the last query token of request 0 only
    q[1, 0, 4, 17] = float("nan")                                       # held by one row of request 1
    out, lse = fb.fp8bs_mla_decode_fp4(q, c.cache, c.table, c.lens, SCALE)
    bad = torch.zeros((2, 2, 16), dtype=torch.bool, device=dev)
    bad[0, 1] = bad[1, 0, 4] = True
    assert torch.equal(torch.isnan(lse), bad) and torch.equal(torch.isnan(out).all(-1), bad)
    assert torch.isfinite(out[~bad]).all()


def test_same_bits_on_a_stream_and_in_a_graph(dev):
    c = Paged(dev, 16, [900, 3, 64, 130], 2, prefix=200)
    q = _q(dev, 4, 1, 16, 2)

    def step():
        return (*fb.fp8bs_mla_decode_fp4(q, c.cache, c.table, c.lens, SCALE),
                *fb.fp8bs_mla_decode_fp4_shared(q, c.cache, c.prefix_table, c.prefix_len, c.table, c.lens, SCALE))

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
    for lens in ([900, 3, 64, 130], [17, 3, 0, 130], [900, 3, 64, 130]):     # lengths change between replays
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, step()):
            assert torch.equal(a, b)
    for a, b in zip(res, ref):
        assert torch.equal(a, b)


def test_binding_refusals(dev):
    c = Paged(dev, 16, [5, 9], 1)
    q = _q(dev, 2, 1, 4, 1)
    codes, scales, rope = c.cache
    bad = [
        (ValueError, (q, c.cache, c.table[:1], c.lens)), (ValueError, (q, c.cache, c.table, c.lens[:1])),
        (TypeError, (q.float(), c.cache, c.table, c.lens)), (TypeError, (q, c.cache, c.table.long(), c.lens)),
        (ValueError, (q, (codes[..., :128], scales, rope), c.table, c.lens)), (TypeError, (q, (codes, scales.float(), rope), c.table, c.lens)),
        (ValueError, (q, (codes, scales[:1], rope), c.table, c.lens)), (ValueError, (q, (codes, scales), c.table, c.lens)),
        (ValueError, (q, codes, c.table, c.lens)), (ValueError, (q, c.cache, c.table.cpu(), c.lens)),
        (ValueError, (torch.cat([q, q], 1)[:, ::2], c.cache, c.table, c.lens)), (ValueError, (q, c.cache, c.table[:, ::2], c.lens)),
    ]
    for error, args in bad:
        with pytest.raises(error):
            fb.fp8bs_mla_decode_fp4(*args, SCALE)
    with pytest.raises(fb.Fp8bsError):
        fb.fp8bs_mla_decode_fp4(q, c.cache, c.table, c.lens, -1.0)
    with pytest.raises(ValueError):
        fb.fp8bs_mla_decode_fp4_shared(q, c.cache, c.table, c.prefix_len, c.table, c.lens, SCALE)
