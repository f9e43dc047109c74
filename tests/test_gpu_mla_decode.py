"""Absorbed latent attention over a paged cache on the GPU, alone and behind a
shared prefix, against the float64 oracle, with the bounds that follow from
rounding the weights and the output to BF16."""

import numpy as np
import pytest
import torch

from oracle import attention as oa

import fp8_block_scaled_x1_amd as fb

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def _f64(t):
    return t.detach().double().cpu().numpy()


class Paged:
    """Requests' tokens in scattered pages of a cache whose unused slots hold NaN."""

    def __init__(self, dev, kind, page, lens, seed, prefix=0, spare=3, std=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        npre = -(-prefix // page)
        pages = sum(need) + npre + spare
        order = rng.permutation(pages)
        width = max(need + [1]) + 1
        table = np.full((len(lens), width), -7, np.int32)       # never read behind a request's last token
        x = (torch.randn((pages, page, 576), generator=g) * std).to(torch.bfloat16).to(dev)
        live = np.zeros((pages, page), bool)
        at = 0
        self.slots = []

        def take(n, count):
            nonlocal at
            mine = order[at:at + count]
            at += count
            pos = np.arange(n)
            live[mine[pos // page], pos % page] = True
            return mine, (mine[pos // page], pos % page)

        self.prefix_pages, pre = take(prefix, npre)
        for b, n in enumerate(lens):
            mine, s = take(n, need[b])
            table[b, :need[b]] = mine
            self.slots.append(s)
        hole = torch.from_numpy(~live).to(dev)
        if kind == "bf16":
            vals = _f64(x)
            x[hole] = float("nan")
            self.cache = x
        else:
            codes, scales = fb.fp8_quant_act_1x128(x[..., :512].reshape(-1, 512).contiguous())
            codes = codes.reshape(pages, page, 512)
            scales = scales.t().reshape(pages, page, 4).contiguous()
            lat = codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, -1)
            vals = np.concatenate([lat.cpu().numpy(), _f64(x[..., 512:])], -1)
            rope = x[..., 512:].contiguous()
            codes[hole], scales[hole], rope[hole] = 0x7F, float("inf"), float("nan")
            self.cache = (codes, scales, rope)
        self.prefix_keys = vals[pre]
        self.keys = [vals[s] for s in self.slots]
        self.table = torch.from_numpy(table).to(dev)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.prefix_table = torch.from_numpy(self.prefix_pages.astype(np.int32)).to(dev)
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


def _check(dev, kind, page, lens, T, H, seed=0, qstd=1.0):
    c = Paged(dev, kind, page, lens, seed)
    q = _q(dev, len(lens), T, H, seed, qstd)
    out, lse = fb.fp8bs_mla_decode(q, c.cache, c.table, c.lens, SCALE)
    torch.cuda.synchronize()
    o, l, bo, bl = oa.mla_decode(_f64(q), c.keys, SCALE)
    what = f"{kind} page {page} lens {lens} T {T} H {H}"
    _inside(out, o, bo, "out " + what)
    _inside(lse, l, bl, "lse " + what)
    return c, q, out, lse


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("H,T", [(1, 1), (16, 1), (16, 2), (5, 3), (32, 1), (40, 1), (64, 1), (128, 1), (33, 4)])
def test_rows(dev, kind, H, T):
    _check(dev, kind, 64, [4, 70, 129, 300], T, H, seed=H)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("page", [1, 7, 16, 64, 100, 128])
def test_pages(dev, kind, page):
    _check(dev, kind, page, [1, 63, 64, 65, 257], 1, 16, seed=page)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("lens", [[0], [1], [0, 0, 5], [3, 0, 700, 0], [2000], [64] * 70, list(range(0, 130))], ids=str)
def test_lengths(dev, kind, lens):
    _check(dev, kind, 16, lens, 1, 16, seed=len(lens))


@pytest.mark.parametrize("T", [2, 4, 7])
def test_drafted_tokens_hide_later_ones(dev, T):
    # lengths below T: the first queries see nothing at all
    _check(dev, "bf16", 16, [0, 1, 2, 3, 5, 64, 66, 130], T, 4, seed=T)
    _check(dev, "fp8", 16, [1, T, 65], T, 20, seed=T)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("qstd", [0.01, 20.0])
def test_flat_and_peaked(dev, kind, qstd):
    _check(dev, kind, 64, [300, 1000], 1, 16, seed=3, qstd=qstd)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_long_contexts_are_cut_and_joined(dev, kind):
    # one long request among short ones: cut over many workgroups
    _check(dev, kind, 64, [9000, 3, 64, 0, 1501], 1, 16, seed=8)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("prefix,lens,T,H,page", [
    (1, [1], 1, 1, 16), (100, [1, 70, 5], 1, 16, 16), (64, [64, 1], 2, 8, 64), (1000, [3, 0, 200, 65], 1, 16, 7),
    (500, [4] * 40, 1, 32, 128), (0, [5, 9], 1, 16, 16), (2000, [130, 2], 3, 20, 64),
])
def test_shared_prefix(dev, kind, prefix, lens, T, H, page):
    c = Paged(dev, kind, page, lens, 5, prefix=prefix)
    q = _q(dev, len(lens), T, H, 5)
    out, lse = fb.fp8bs_mla_decode_shared(q, c.cache, c.prefix_table, c.prefix_len, c.table, c.lens, SCALE)
    torch.cuda.synchronize()
    keys = [(prefix, np.concatenate([c.prefix_keys, k])) for k in c.keys]
    o, l, bo, bl = oa.mla_decode(_f64(q), keys, SCALE)
    _inside(out, o, bo, f"shared {prefix} {lens}")
    _inside(lse, l, bl, f"shared lse {prefix} {lens}")


def test_prefix_and_own_tokens_empty(dev):
    c = Paged(dev, "bf16", 16, [0, 3], 5, prefix=0)
    q = _q(dev, 2, 1, 4, 1)
    table = torch.zeros(2, dtype=torch.int32, device=dev)
    out, lse = fb.fp8bs_mla_decode_shared(q, c.cache, table, c.prefix_len, c.table, c.lens, SCALE)
    assert torch.all(out[0] == 0) and torch.all(torch.isneginf(lse[0])) and torch.all(torch.isfinite(lse[1]))
    # and no table at all
    out, lse = fb.fp8bs_mla_decode(q, c.cache, c.table[:, :0].contiguous(), c.lens, SCALE)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


def test_lengths_and_entries_are_clamped(dev):
    c, q, out, lse = _check(dev, "bf16", 16, [40, 16], 1, 16, seed=1)
    lens = torch.tensor([40, -5], dtype=torch.int32, device=dev)
    o2, l2 = fb.fp8bs_mla_decode(q, c.cache, c.table, lens, SCALE)
    assert torch.equal(o2[0], out[0]) and torch.all(o2[1] == 0) and torch.all(torch.isneginf(l2[1]))
    wide = c.table[:, :1].contiguous()
    o3, _ = fb.fp8bs_mla_decode(q, c.cache, wide, torch.tensor([1 << 30, 16], dtype=torch.int32, device=dev), SCALE)
    o4, _ = fb.fp8bs_mla_decode(q, c.cache, wide, torch.tensor([16, 16], dtype=torch.int32, device=dev), SCALE)
    assert torch.equal(o3, o4)
    high = wide.clone()
    high[1] = 1 << 30                                # past the last page: the last page
    last = wide.clone()
    last[1] = c.cache.shape[0] - 1
    n = torch.tensor([16, 16], dtype=torch.int32, device=dev)
    clean = torch.nan_to_num(c.cache)
    assert torch.equal(fb.fp8bs_mla_decode(q, clean, high, n, SCALE)[0], fb.fp8bs_mla_decode(q, clean, last, n, SCALE)[0])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_same_bits_on_a_stream_and_in_a_graph(dev, kind):
    c = Paged(dev, kind, 16, [900, 3, 64, 130], 2, prefix=200)
    q = _q(dev, 4, 1, 16, 2)

    def step():
        return (*fb.fp8bs_mla_decode(q, c.cache, c.table, c.lens, SCALE),
                *fb.fp8bs_mla_decode_shared(q, c.cache, c.prefix_table, c.prefix_len, c.table, c.lens, SCALE))

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
    c = Paged(dev, "bf16", 16, [5, 9], 1)
    q = _q(dev, 2, 1, 4, 1)
    bad = [
        (ValueError, (q, c.cache, c.table[:1], c.lens)), (ValueError, (q, c.cache, c.table, c.lens[:1])),
        (TypeError, (q.float(), c.cache, c.table, c.lens)), (TypeError, (q, c.cache, c.table.long(), c.lens)),
        (ValueError, (q, c.cache[..., :512], c.table, c.lens)), (ValueError, (q, c.cache.transpose(0, 1), c.table, c.lens)),
        (ValueError, (q, (c.cache, c.cache), c.table, c.lens)), (ValueError, (q, c.cache, c.table.cpu(), c.lens)),
        (ValueError, (torch.cat([q, q], 1)[:, ::2], c.cache, c.table, c.lens)), (ValueError, (q, c.cache, c.table[:, ::2], c.lens)),
    ]
    for error, args in bad:
        with pytest.raises(error):
            fb.fp8bs_mla_decode(*args, SCALE)
    with pytest.raises(fb.Fp8bsError):
        fb.fp8bs_mla_decode(q, c.cache, c.table, c.lens, -1.0)
    with pytest.raises(ValueError):
        fb.fp8bs_mla_decode_shared(q, c.cache, c.table, c.prefix_len, c.table, c.lens, SCALE)


def _groups(B, T, H, width, page):
    """Workgroup ranges that the tiles of 64 tokens are shared by, from the workspace: two partials
    (512 + 2 numbers, FP32) of a request's rows each."""
    return fb.attn_lib().fp8bs_mla_decode_workspace_bytes(B, T, H, width, page, 0) // (2 * T * H * 514 * 4)


def _tiles(lens):
    return sum(-(-n // 64) for n in lens)


SHORT = [100 + 37 * i % 600 for i in range(300)]
MANY_TILES = [
    (4, 128, [3000, 65, 700, 0, 129]),       # a request cut over ranges, ranges that hold several requests' ends
    (3, 40, [2000, 1, 64, 900, 1500, 1100, 2500, 3000]),
    (1, 16, [9000, 6400, 3, 0, 12000]),      # few rows, more tiles than workgroups
    (1, 20, SHORT),                          # whole requests one after the other inside a range
]


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H,lens", MANY_TILES, ids=["512 rows", "120 rows", "long", "300 requests"])
def test_several_tiles_per_workgroup(dev, kind, T, H, lens):
    c, *_ = _check(dev, kind, 64, lens, T, H, seed=T + H)
    assert _tiles(lens) > 1.2 * _groups(len(lens), T, H, c.table.shape[1], 64)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("page", [1, 48])
def test_several_tiles_per_workgroup_of_other_pages(dev, kind, page):
    lens = [1000, 64, 0, 333, 1]
    c, *_ = _check(dev, kind, page, lens, 8, 128, seed=page)
    assert _tiles(lens) > 1.2 * _groups(len(lens), 8, 128, c.table.shape[1], page)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_reference_raised_over_sums(dev, kind):
    # scores that grow along the request: each tile of a range raises the reference over what has been added up
    lens, T, H = [2000, 1300], 8, 128
    c = Paged(dev, kind, 64, lens, 4)
    q = _q(dev, 2, T, H, 4, 6.0)
    own = [torch.from_numpy(c.table[b, :-(-n // 64)].cpu().numpy()).long() for b, n in enumerate(lens)]
    rope = c.cache[..., 512:] if kind == "bf16" else c.cache[2]
    keys = [k.copy() for k in c.keys]
    q[..., 512] = 30.0
    for b, n in enumerate(lens):
        # (whole numbers below 16: BF16 values)
        ramp = (torch.arange(n) * 16 // n).float().to(torch.bfloat16)
        pos = torch.arange(n)
        rope[own[b][pos // 64].to(dev), (pos % 64).to(dev), 0] = ramp.to(dev)
        keys[b][:, 512] = ramp.double().numpy()
    out, lse = fb.fp8bs_mla_decode(q, c.cache, c.table, c.lens, SCALE)
    torch.cuda.synchronize()
    assert _tiles(lens) > 1.2 * _groups(2, T, H, c.table.shape[1], 64)
    o, l, bo, bl = oa.mla_decode(_f64(q), keys, SCALE)
    _inside(out, o, bo, "out")
    _inside(lse, l, bl, "lse")


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("B,T,H,prefix", [(20, 1, 128, 1000), (11, 3, 70, 900), (60, 2, 16, 3000), (150, 1, 16, 700)])
def test_shared_prefix_of_several_tiles_per_workgroup(dev, kind, B, T, H, prefix):
    # more tiles than workgroups in the prefix (one request per 64 rows there), and both joins of rows with a prefix
    assert -(-B * T * H // 64) * -(-prefix // 64) > 1.2 * 256
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(T, 260, B)]
    c = Paged(dev, kind, 64, lens, 6, prefix=prefix)
    q = _q(dev, B, T, H, 6)
    out, lse = fb.fp8bs_mla_decode_shared(q, c.cache, c.prefix_table, c.prefix_len, c.table, c.lens, SCALE)
    torch.cuda.synchronize()
    keys = [(prefix, np.concatenate([c.prefix_keys, k])) for k in c.keys]
    o, l, bo, bl = oa.mla_decode(_f64(q), keys, SCALE)
    _inside(out, o, bo, f"shared {prefix} {lens}")
    _inside(lse, l, bl, f"shared lse {prefix} {lens}")
