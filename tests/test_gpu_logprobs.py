"""Log probabilities, entropy, ranks and alternatives on the GPU against the
float64 oracle: whole numbers equal, the others within the bounds of FP32; the
gradient against the formula and against differences."""

import numpy as np
import pytest
import torch

from oracle import serve as os_

import fp8_block_scaled_x1_amd as fb

pytestmark = pytest.mark.gpu
NAMES = ("logprob", "entropy", "norm", "rank", "top_ids", "top_logprobs")
DTYPES = [torch.float32, torch.bfloat16]


def _logits(T, V, seed, dtype, std=3.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, V + pad), generator=g) * std).to(dtype)[:, :V]


def _inside(got, want, bound, what):
    got = got.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        bad = ~((np.isneginf(want) & np.isneginf(got)) | (np.abs(got - want) <= bound))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first at {tuple(np.argwhere(bad)[0])}: " \
                          f"{got[bad][0]} against {want[bad][0]} +- {bound[bad][0]}"


def _on(dev, x):
    """The same view of a copy on the GPU, rows as far apart."""
    base = torch.empty((x.shape[0], x.stride(0) if x.shape[0] > 1 else x.shape[1]), dtype=x.dtype, device=dev)
    y = base[:, :x.shape[1]]
    y.copy_(x)
    return y


def _check(dev, x, targets, top):
    targets = torch.as_tensor(targets, dtype=torch.int32)
    xd = _on(dev, x)
    got = dict(zip(NAMES, fb.fp8bs_logprobs(xd, targets.to(dev), top)))
    want, bound = os_.logprobs(x.double().numpy(), targets.numpy(), top)
    for n in ("rank", "top_ids"):
        assert np.array_equal(got[n].cpu().numpy(), want[n]), f"{n}: {got[n].cpu().numpy()} against {want[n]}"
    for n in bound:
        _inside(got[n], want[n], bound[n], n)
    g = torch.Generator().manual_seed(5)
    dl, dh = torch.randn(len(x), generator=g), torch.randn(len(x), generator=g)
    grad = fb.fp8bs_logprobs_bwd(xd, targets.to(dev), got["norm"], got["entropy"], dl.to(dev), dh.to(dev))
    w, b = os_.logprobs_bwd(x.double().numpy(), targets.numpy(), dl.numpy(), dh.numpy(), torch.finfo(x.dtype).eps / 2)
    assert grad.dtype == x.dtype and grad.is_contiguous()
    _inside(grad, w, b, "gradient")
    return got


def _targets(T, V, seed):
    return np.random.default_rng(seed).integers(0, V, T)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 2, 3, 7, 64, 255, 256, 1000, 8191, 8192, 8193, 16385, 40000])
def test_vocabularies(dev, V, dtype):
    _check(dev, _logits(5, V, V, dtype), _targets(5, V, V), min(V, 20))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("top", [0, 1, 2, 33, 63, 64])
@pytest.mark.parametrize("V", [64, 9000])
def test_alternatives(dev, top, V, dtype):
    _check(dev, _logits(4, V, top, dtype), _targets(4, V, top), top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad", [1, 3, 8, 96])
def test_rows_apart(dev, pad, dtype):
    _check(dev, _logits(6, 8200 + pad, pad, dtype, pad=pad), _targets(6, 8200, pad), 5)


@pytest.mark.parametrize("dtype", DTYPES)
def test_ties_go_to_the_lowest_index(dev, dtype):
    x = torch.zeros((4, 17000), dtype=dtype)
    x[1, ::7] = 1.0
    x[2] = torch.arange(17000) % 3
    x[3, 16000:16010] = -0.0                 # equal to 0
    x[3, 100] = -1.0
    _check(dev, x, [16999, 14, 5, 16005], 64)


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_entries(dev, dtype):
    x = _logits(6, 20000, 4, dtype)
    inf = float("inf")
    x[0, 1:] = -inf                          # one entry left
    x[1, :] = -inf                           # none
    x[2, :19990] = -inf                      # fewer than alternatives asked for, all in the last chunk
    x[3, ::2] = torch.finfo(dtype).min       # the type's lowest value
    x[4, :] = torch.finfo(dtype).min
    x[5, 8192:] = -inf
    _check(dev, x, [0, 3, 5, 2, 7, 9000], 20)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("top", [0, 30])
@pytest.mark.parametrize("V", [5, 13, 77, 8195, 8199, 8205, 12943])
def test_masked_tokens_in_the_last_chunk(dev, V, top, dtype):
    """Most entries masked, the tokens' own among them, where the row's end cuts an access."""
    x = _logits(5, V, V, dtype)
    x[torch.rand(x.shape, generator=torch.Generator().manual_seed(V)) < 0.98] = -float("inf")
    targets = [V - 1, V - 2, V - 3, V - 4, V // 2]
    x[range(4), targets[:4]] = -float("inf")
    _check(dev, x, targets, min(V, top))


@pytest.mark.parametrize("dtype", DTYPES)
def test_far_apart_and_large(dev, dtype):
    x = _logits(4, 9000, 6, dtype, std=100.0)
    x[1] += 10000.0
    x[2] -= 10000.0
    x[3] = 0.0
    _check(dev, x, [1, 2, 3, 4], 10)


def test_targets_that_are_no_token(dev):
    got = _check(dev, _logits(4, 500, 7, torch.float32), [-1, 500, -100, 499], 3)
    assert got["rank"].tolist()[:3] == [-1, -1, -1] and got["logprob"][:3].tolist() == [0, 0, 0]


@pytest.mark.parametrize("V", [300, 20000])
def test_nan_and_infinity_stay_in_their_rows(dev, V):
    x = _logits(5, V, 8, torch.float32)
    y = _targets(5, V, 8)
    clean = _check(dev, x, y, 7)
    x[1, V - 5] = float("nan")
    x[3, 17] = float("inf")
    args = x.to(dev), torch.as_tensor(y, dtype=torch.int32, device=dev)
    got = dict(zip(NAMES, fb.fp8bs_logprobs(*args, 7)))
    for n in NAMES:
        assert torch.equal(got[n][[0, 2, 4]], clean[n][[0, 2, 4]]), n
    for n in ("logprob", "entropy"):
        assert torch.isnan(got[n][[1, 3]]).all(), n
    assert torch.isnan(got["norm"][[1, 3], 1]).all()
    assert ((got["top_ids"] >= 0) & (got["top_ids"] < V)).all() and ((got["rank"] >= 0) & (got["rank"] < V)).all()
    one = torch.ones(5, device=dev)
    grad = fb.fp8bs_logprobs_bwd(*args, got["norm"], got["entropy"], one, one)
    assert torch.isnan(grad[[1, 3]]).any(1).all() and torch.isfinite(grad[[0, 2, 4]]).all()


def test_adversarial_order(dev):
    # one thread's entries above all others, then everything ascending and descending
    x = _logits(3, 8192, 9, torch.float32)
    x[0, 40:44] += 100.0
    x[1] = torch.arange(8192).float()
    x[2] = -torch.arange(8192).float()
    _check(dev, x, [41, 8191, 8191], 64)


def test_one_row_and_many(dev):
    _check(dev, _logits(1, 129280, 10, torch.float32), [77], 20)
    _check(dev, _logits(700, 50, 10, torch.bfloat16), _targets(700, 50, 10), 5)


def test_largest_vocabulary(dev):
    _check(dev, _logits(1, 1 << 20, 11, torch.bfloat16), [1 << 19], 64)


def test_gradient_is_that_of_differences(dev):
    # in 64 bits by central differences of the definition
    T, V, eps = 3, 11, 1e-4
    x, y = _logits(T, V, 12, torch.float32), _targets(T, V, 12)
    dl, dh = np.array([0.7, -1.3, 0.2]), np.array([0.5, 0.1, -2.0])

    def value(z):
        r, _ = os_.logprobs(z, y, 0)
        return r["logprob"] * dl + r["entropy"] * dh

    want = np.zeros((T, V))
    for i in range(V):
        z = x.double().numpy()
        up, down = z.copy(), z.copy()
        up[:, i] += eps
        down[:, i] -= eps
        want[:, i] = (value(up) - value(down)) / (2 * eps)
    args = x.to(dev), torch.as_tensor(y, dtype=torch.int32, device=dev)
    _, entropy, norm, *_ = fb.fp8bs_logprobs(*args)
    grad = fb.fp8bs_logprobs_bwd(*args, norm, entropy, *(torch.from_numpy(a).float().to(dev) for a in (dl, dh)))
    # third derivatives of a few units times eps^2 / 6, and FP32
    assert np.abs(grad.double().cpu().numpy() - want).max() <= 1e-6 + 2e-5


@pytest.mark.parametrize("top", [0, 8])
def test_same_bits_in_a_graph_and_on_a_stream(dev, top):
    x, y = _logits(9, 30000, 13, torch.float32).to(dev), torch.as_tensor(_targets(9, 30000, 13), dtype=torch.int32, device=dev)
    d = torch.randn(2, 9, device=dev)

    def step():
        r = fb.fp8bs_logprobs(x, y, top)
        return (*r, fb.fp8bs_logprobs_bwd(x, y, r[2], r[1], d[0], d[1]))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for i in range(3):
        x.copy_(torch.randn(9, 30000, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, step()):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(res, again):
        assert torch.equal(a, b)


def test_no_rows_and_refusals(dev):
    y = torch.zeros(3, dtype=torch.int32, device=dev)
    r = fb.fp8bs_logprobs(torch.zeros((0, 5), device=dev), y[:0], 2)
    assert r[0].shape == (0,) and r[4].shape == (0, 2)
    x = torch.zeros((3, 10), device=dev)
    for error, args in [(TypeError, (x.half(), y)), (TypeError, (x, y.long())), (ValueError, (x, y[:2])), (ValueError, (x.t(), y)),
                        (ValueError, (x[0], y)), (ValueError, (x[:1].expand(3, 10), y)), (ValueError, (x.cpu(), y))]:
        with pytest.raises(error):
            fb.fp8bs_logprobs(*args)
    for top in (-1, 11, 65):
        with pytest.raises(fb.Fp8bsError):
            fb.fp8bs_logprobs(x, y, top)
    with pytest.raises(ValueError):
        fb.fp8bs_logprobs_bwd(x, y, x[:, :2].contiguous(), x[0, :3].clone(), x[0, :2].clone(), x[0, :3].clone())


def _masked_rows(V, dtype, masks, seed):
    """Rows masked with finite values, for each of them: three entries left, one of 50 left, a chunk of 8192 masked."""
    x = _logits(3 * len(masks), V, seed, dtype)
    keep = torch.zeros((3, V), dtype=torch.bool)
    keep[0, [5, V // 2, V - 1]] = True
    keep[1, 7::50] = True
    keep[2, 8192:] = True
    for i, value in enumerate(masks):
        x[3 * i:3 * i + 3][~keep] = value
    targets = [5, 7, V - 2] * len(masks)
    targets[2::6] = [100] * len(targets[2::6])         # (a masked token)
    return x, targets


def _check_masked(dev, V, top, dtype, masks):
    x, targets = _masked_rows(V, dtype, masks, V)
    got = _check(dev, x, targets, top)
    # the gradient of the log probability alone, as a policy gradient takes it
    xd, y = x.to(dev), torch.as_tensor(targets, dtype=torch.int32, device=dev)
    one, none = torch.ones(len(x), device=dev), torch.zeros(len(x), device=dev)
    grad = fb.fp8bs_logprobs_bwd(xd, y, got["norm"], got["entropy"], one, none)
    w, b = os_.logprobs_bwd(x.double().numpy(), targets, np.ones(len(x)), np.zeros(len(x)), torch.finfo(dtype).eps / 2)
    _inside(grad, w, b, "gradient of the log probability")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("top", [0, 20])
@pytest.mark.parametrize("V", [20000, 129280])
def test_masks_near_the_lowest_value(dev, V, top, dtype):
    """Parts of a row whose sum of exponentials times their distance to the row's maximum overflows."""
    _check_masked(dev, V, top, dtype, [torch.finfo(dtype).min, -1e38, -1e36])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("top", [0, 20])
@pytest.mark.parametrize("V", [20000, 129280])
def test_masks_of_large_finite_values(dev, V, top, dtype):
    """Maxima of a part whose product with log2 e has a rounding error beyond the range of an exponential."""
    _check_masked(dev, V, top, dtype, [-1e30, -1e20, -1e10, -1e9, -3e6, -1e6])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("top", [0, 5])
def test_large_maxima(dev, top, dtype):
    """The same at the rows' own maxima, of either sign, next to what is their rounding away."""
    x = _logits(10, 9000, 3, dtype)
    for i, m in enumerate([2.0 ** 18, 2.0 ** 20, 1e7, 1e9, 1e30]):
        x[2 * i:2 * i + 2] *= m * 2.0 ** -22           # differences from a fraction of one to far more
        x[2 * i] += m
        x[2 * i + 1] -= m
    _check(dev, x, [1, 8999, 2, 8998, 3, 8997, 4, 8996, 5, 8995], top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,pad", [(2048, 16385, 3), (700, 40000, 0), (700, 40000, 5), (1100, 24576, 8), (400, 60001, 1)])
def test_many_rows_of_several_chunks(dev, T, V, pad, dtype):
    """Without alternatives, a workgroup goes over several chunks: all three of a row's (2048 rows), two and one of
    three (1100) or of five (700), two of eight (400). Usual rows, and rows that only some chunks decide."""
    x = _logits(T, V, V, dtype, pad=pad)
    targets = _targets(T, V, V)
    low, inf, at = torch.finfo(dtype).min, float("inf"), 8192
    x[0] = torch.arange(V) // 7 / V * 30               # every chunk raises the maximum
    x[1] = -x[0]
    x[2, :at] = x[3, at:2 * at] = x[4, 2 * at:] = -inf
    x[5, :at] = x[6, at:2 * at] = x[7, 2 * at:] = low
    x[8], x[9], x[10] = -inf, low, 0.0
    x[11, :V - 1] = x[12, 1:] = -inf
    x[13, :V - 1] = x[14, 1:] = low
    x[15] = torch.arange(V) % 3                        # ties, here and over chunks' ends
    x[16, :2 * at] -= 10000.0
    x[17, at:] += 10000.0
    x[18] *= 100.0
    x[19, ::2] = low
    targets[:20] = [V - 1, V - 1, at, at - 1, 0, at - 1, 2 * at, V - 1, 2 * at, 5, at, V - 1, 0, V - 1, V - 1, 2 * at, V - 1, at, 3, 2]
    targets[20:24] = [-1, V, at - 1, 2 * at - 1]
    rows = list(range(28)) + [T // 2, T - 2, T - 1]
    xd = _on(dev, x)
    y = torch.as_tensor(targets, dtype=torch.int32, device=dev)
    got = dict(zip(NAMES, fb.fp8bs_logprobs(xd, y)))
    some = x[rows].double().numpy()
    want, bound = os_.logprobs(some, targets[rows], 0)
    assert np.array_equal(got["rank"][rows].cpu().numpy(), want["rank"])
    for n in ("logprob", "entropy", "norm"):
        _inside(got[n][rows], want[n], bound[n], n)
    g = torch.Generator().manual_seed(5)
    dl, dh = torch.randn(T, generator=g), torch.randn(T, generator=g)
    grad = fb.fp8bs_logprobs_bwd(xd, y, got["norm"], got["entropy"], dl.to(dev), dh.to(dev))
    w, b = os_.logprobs_bwd(some, targets[rows], dl[rows].numpy(), dh[rows].numpy(), torch.finfo(dtype).eps / 2)
    _inside(grad[rows], w, b, "gradient")
    # the other rows: the same numbers as when they are asked for by themselves, a chunk per workgroup
    for first in range(28, T - 9, T // 3):
        few = slice(first, first + 9)
        alone = dict(zip(NAMES, fb.fp8bs_logprobs(xd[few], y[few])))
        assert torch.equal(alone["rank"], got["rank"][few])
        # (each within FP32's bound of the same number: a few units times 2^-17)
        for n in ("logprob", "entropy", "norm"):
            assert torch.allclose(alone[n], got[n][few], rtol=2.0 ** -17, atol=2.0 ** -16), n
