"""A mixture-of-experts layer for a few tokens on the GPU against the float64
oracle, with the bounds that follow from FP32 sums and two roundings to BF16."""

import numpy as np
import pytest
import torch

from oracle import serve as os_

import fp8_block_scaled_x1_amd as fb

pytestmark = pytest.mark.gpu


def _weights(E, rows, cols, g, scale):
    q = (torch.randn((E, rows, cols), generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = (torch.rand((E, rows // 128, cols // 128), generator=g) + 0.5) * scale
    return q, s


def _values(q, s):
    return q.double().numpy() * s.double().repeat_interleave(128, -1).repeat_interleave(128, -2).numpy()


class Layer:
    def __init__(self, dev, E, K, F, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.up, self.down = _weights(E, 2 * F, K, g, 0.01 / K ** 0.5), _weights(E, K, F, g, 0.01 / F ** 0.5)
        self.args = [t.to(dev) for t in (self.up[0].view(torch.uint8), self.up[1], self.down[0].view(torch.uint8), self.down[1])]
        self.values = _values(*self.up), _values(*self.down)
        self.E, self.K, self.F = E, K, F


def _x(T, K, seed, std=1.0):
    return (torch.randn((T, K), generator=torch.Generator().manual_seed(seed + 7)) * std).to(torch.bfloat16)


def _check(dev, layer, x, ids, w):
    ids, w = np.asarray(ids, np.int32), np.asarray(w, np.float32)
    out = fb.fp8bs_moe_tokens(x.to(dev), torch.from_numpy(ids).to(dev), torch.from_numpy(w).to(dev), *layer.args)
    want, bound = os_.moe_tokens(x.double().numpy(), ids, w, *layer.values)
    got = out.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, first at {tuple(np.argwhere(bad)[0])}: " \
                          f"{got[bad][0]} against {want[bad][0]} +- {bound[bad][0]}"
    return out


def _ids(T, topk, E, seed):
    rng = np.random.default_rng(seed)
    return np.stack([rng.permutation(E)[:topk] for _ in range(T)]), rng.random((T, topk)) + 0.05


@pytest.fixture(scope="module")
def small(dev):
    return Layer(dev, 8, 256, 128)


@pytest.mark.parametrize("T", [1, 2, 3, 15, 16, 17, 31, 33, 48, 63, 64])
@pytest.mark.parametrize("topk", [1, 3, 8])
def test_tokens(dev, small, T, topk):
    _check(dev, small, _x(T, 256, T), *_ids(T, topk, 8, T * 10 + topk))


@pytest.mark.parametrize("E,K,F", [(1, 128, 128), (3, 128, 640), (2, 1152, 128), (40, 384, 256), (5, 640, 384), (100, 128, 128)])
def test_shapes(dev, E, K, F):
    layer = Layer(dev, E, K, F, seed=E)
    for T in (1, 20):
        _check(dev, layer, _x(T, K, T), *_ids(T, min(E, 6), E, T))


def test_all_tokens_choose_one_expert(dev, small):
    _check(dev, small, _x(64, 256, 1), np.full((64, 1), 5), np.ones((64, 1)))


@pytest.mark.parametrize("tokens", [9, 31, 32, 33, 50, 64])
def test_tokens_of_one_expert_beside_others(dev, small, tokens):
    """Expert 2 is chosen by so many of 64 tokens, in the order of a shuffle; some name it several times."""
    rng = np.random.default_rng(tokens)
    ids = rng.integers(3, 8, (64, 5))
    chose = rng.permutation(64)[:tokens]
    ids[chose, 1] = 2
    ids[chose[::2], 3:] = 2
    _check(dev, small, _x(64, 256, tokens), ids, rng.random((64, 5)))


@pytest.mark.parametrize("T", [1, 5, 16, 17, 32, 33, 64])
def test_waves_with_columns_of_their_own(dev, T):
    """Many columns and few inner numbers: 6 experts of 128 x 1024, some or all of them for every token."""
    layer = Layer(dev, 6, 128, 1024, seed=T)
    for topk in (3, 6):
        _check(dev, layer, _x(T, 128, T), *_ids(T, topk, 6, T + topk))
    _check(dev, layer, _x(T, 128, T + 1), *_ids(T, 6, 12, T))


@pytest.mark.parametrize("T", [16, 17, 32, 33, 64])
@pytest.mark.parametrize("E,K,F", [(8, 128, 2048), (8, 768, 2048), (4, 4096, 128)])
def test_strips_around_the_rules_limits(dev, T, E, K, F):
    """Many strips of short and of longer columns (1024 at least), and few of rows a multiple of 4096 bytes apart;
    ids of experts elsewhere among the tokens'."""
    layer = Layer(dev, E, K, F, seed=T)
    _check(dev, layer, _x(T, K, T), *_ids(T, 4, E, T))
    _check(dev, layer, _x(T, K, T + 1), *_ids(T, 4, 3 * E, T))


@pytest.mark.parametrize("E", [70, 1024])
def test_most_tokens_and_slots(dev, E):
    layer = Layer(dev, E, 128, 128, seed=E)
    _check(dev, layer, _x(64, 128, 3), *_ids(64, 64, E, 3))


@pytest.mark.parametrize("T", [17, 64])
def test_one_share_of_the_second_kernel(dev, T):
    layer = Layer(dev, 2, 6144, 128, seed=5)
    _check(dev, layer, _x(T, 6144, T), *_ids(T, 2, 2, T))


@pytest.mark.parametrize("T", [5, 33])
@pytest.mark.parametrize("K", [128, 1408, 2816, 4096, 4352])
def test_shares_of_the_second_kernel(dev, K, T):
    layer = Layer(dev, 3, K, 128, seed=K)
    _check(dev, layer, _x(T, K, T), *_ids(T, 2, 3, T))


def test_experts_elsewhere_and_named_twice(dev, small):
    rng = np.random.default_rng(3)
    ids = rng.integers(-2, 12, (30, 6))
    ids[0] = -1                              # nothing of this token here
    ids[1] = 3                               # one expert in every slot
    ids[2] = [1 << 30, -(1 << 31), 8, -1, 7, 7]
    out = _check(dev, small, _x(30, 256, 3), ids, rng.random((30, 6)))
    assert torch.all(out[0] == 0)


def test_nobody_here(dev, small):
    out = _check(dev, small, _x(5, 256, 3), np.full((5, 2), 8), np.ones((5, 2)))
    assert torch.all(out == 0)


def test_large_and_negative_gates(dev, small):
    # silu far out on both sides, weights of either sign and zero
    ids, w = _ids(9, 4, 8, 5)
    w = w * np.where(np.arange(4) % 2, -3.0, 1.0)
    w[:, 2] = 0.0
    _check(dev, small, _x(9, 256, 5, std=300.0), ids, w)


def test_one_tokens_overflow_stays_its_own(dev, small):
    # an infinite activation of one token; the others share experts and tiles with it
    x = _x(6, 256, 6)
    ids, w = _ids(6, 8, 8, 6)
    clean = _check(dev, small, x, ids, w)
    x[2, 5] = float("inf")
    out = fb.fp8bs_moe_tokens(x.to(dev), *(torch.from_numpy(a).to(dev) for a in (ids.astype(np.int32), w.astype(np.float32))),
                              *small.args)
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(out[keep], clean[keep]) and not torch.isfinite(out[2]).any()


def test_more_experts_than_a_bitmap_word_and_many_slots(dev):
    layer = Layer(dev, 300, 128, 128, seed=9)
    rng = np.random.default_rng(9)
    ids = rng.integers(0, 300, (64, 40))
    _check(dev, layer, _x(64, 128, 9), ids, rng.random((64, 40)) * 0.1)


def test_layer_of_the_decode_workload(dev):
    # 7168 wide, 2048 inner, two experts of it
    layer = Layer(dev, 2, 7168, 2048, seed=4)
    _check(dev, layer, _x(3, 7168, 4), [[0, 1], [1, 0], [0, 5]], np.full((3, 2), 0.5))


def test_agrees_with_the_grouped_path(dev, small):
    # dispatch, grouped GEMMs and combine quantize the activations twice (E4M3, 2^-4 of each number at most, 0.027 of
    # the norm of a group), the layer does not
    T, topk = 20, 4
    x = _x(T, 256, 11).to(dev)
    ids, w = _ids(T, topk, 8, 11)
    ids, w = torch.from_numpy(ids.astype(np.int32)).to(dev), torch.from_numpy(w.astype(np.float32)).to(dev)
    q, s, off, pos, _ = fb.fp8_moe_dispatch(x, ids, 8)
    a = fb.fp8_grouped_gemm_blockscaled(q, s, small.args[0], small.args[1], off).float()
    h = (torch.nn.functional.silu(a[:, :128]) * a[:, 128:]).bfloat16()
    hq, hs = fb.fp8_quant_act_1x128(h)
    y = fb.fp8_grouped_gemm_blockscaled(hq, hs, small.args[2], small.args[3], off)
    want = fb.fp8_moe_combine(y, pos, w).float()
    got = fb.fp8bs_moe_tokens(x, ids, w, *small.args).float()
    assert (got - want).norm() <= 0.12 * want.norm()


def test_same_bits_in_a_graph_and_on_a_stream(dev, small):
    T, topk = 12, 3
    x, (ids, w) = _x(T, 256, 12).to(dev), _ids(T, topk, 8, 12)
    ids, w = torch.from_numpy(ids.astype(np.int32)).to(dev), torch.from_numpy(w.astype(np.float32)).to(dev)

    def step():
        return fb.fp8bs_moe_tokens(x, ids, w, *small.args)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for i in range(3):
        ids.copy_(torch.from_numpy(_ids(T, topk, 8, 20 + i)[0].astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res, step())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(res, again)


def test_no_tokens(dev, small):
    out = fb.fp8bs_moe_tokens(_x(0, 256, 0).to(dev), torch.zeros((0, 2), dtype=torch.int32, device=dev),
                              torch.zeros((0, 2), device=dev), *small.args)
    assert out.shape == (0, 256)


def test_binding_refusals(dev, small):
    x, ids, w = _x(2, 256, 0).to(dev), torch.zeros((2, 2), dtype=torch.int32, device=dev), torch.ones((2, 2), device=dev)
    a, b, c, d = small.args
    bad = [(TypeError, (x.float(), ids, w, a, b, c, d)), (TypeError, (x, ids.long(), w, a, b, c, d)),
           (ValueError, (x, ids, w[:1], a, b, c, d)), (ValueError, (x, ids, w, a[:1], b, c, d)),
           (ValueError, (x, ids, w, a, b[:, :1], c, d)), (ValueError, (x, ids, w, a, b, c[:, :128], d)),
           (ValueError, (x, ids, w, a, b, c, d.transpose(1, 2))), (ValueError, (x[:, :128].contiguous(), ids, w, a, b, c, d)),
           (ValueError, (x, ids[0], w, a, b, c, d)), (ValueError, (x, ids, w, a, b, c.cpu(), d))]
    for error, args in bad:
        with pytest.raises(error):
            fb.fp8bs_moe_tokens(*args)
    with pytest.raises(fb.Fp8bsError):
        fb.fp8bs_moe_tokens(_x(65, 256, 0).to(dev), ids[:1].expand(65, 2).contiguous(), w[:1].expand(65, 2).contiguous(), a, b, c, d)
