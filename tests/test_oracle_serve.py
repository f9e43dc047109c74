"""The serving operators' oracle against values worked out by hand, and against
direct forms of the definitions."""

import numpy as np

from oracle import serve as os_


def test_e2m1_halfway_goes_to_the_even_code():
    x = np.zeros((1, 512))
    x[0, :9] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0]
    q, e = os_.fp4_quant(x)
    v = os_.fp4_values(q, e)[0]
    assert e[0, 0] == 127 and v[:9].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -4.0]
    assert q[0, 0] == 0x07 and q[0, 1] == 0x22          # column 0 in the lower half


def test_fp4_scale_is_the_smallest_that_holds_the_maximum():
    x = np.zeros((5, 512))
    x[:, 0] = [6.0, 6.03125, 12.0, 2.0 ** -133, 2.0 ** 127 * 1.9921875]
    _, e = os_.fp4_quant(x)
    assert e[:, 0].tolist() == [127, 128, 128, 1, 253]
    assert np.all(e[:, 1:] == 127)                       # groups of zeros


def test_fp4_numbers_of_the_format_are_kept():
    rng = np.random.default_rng(0)
    x = rng.choice(os_.E2M1, (8, 16, 32)) * rng.choice([-1.0, 1.0], (8, 16, 32))
    x[..., 0] = 6.0
    x = (x * np.ldexp(1.0, rng.integers(-100, 100, (8, 16, 1)))).reshape(8, 512)
    assert np.array_equal(os_.fp4_values(*os_.fp4_quant(x)), x)


def test_slots():
    at = os_.slots(np.array([[4, 9], [7, 2]]), [3, 1], [0, 2, 5], 2, 6)
    assert at.tolist() == [[4, 1, 1], [9, 0, 1], [0, 0, 0], [0, 0, 0], [7, 0, 1], [-1, -1, -1]]


def test_moe_by_hand():
    up = np.zeros((2, 2, 1))
    up[:, 0], up[:, 1] = 1.0, [[2.0], [3.0]]             # gate 1, up 2 and 3
    down = np.array([[[5.0]], [[7.0]]])
    out, bound = os_.moe_tokens(np.array([[1.0], [-2.0]]), [[0, 1], [1, 2]], np.array([[0.5, 0.25], [1.0, 9.0]]), up, down)
    s = 1 / (1 + np.exp(-1.0))
    assert np.isclose(out[0, 0], 0.5 * 5 * 2 * s + 0.25 * 7 * 3 * s)
    assert np.isclose(out[1, 0], 7 * (-2 / (1 + np.exp(2.0))) * -6)
    assert np.all(bound > 0) and np.all(bound < 0.05 * np.abs(out))


def test_logprobs_by_hand():
    x = np.log(np.array([[1.0, 2.0, 5.0], [1.0, 1.0, 2.0]]))
    r, _ = os_.logprobs(x, [1, -1], 2)
    assert np.allclose(r["logprob"], [np.log(0.25), 0.0]) and r["rank"].tolist() == [1, -1]
    assert np.allclose(r["entropy"][1], 1.5 * np.log(2.0)) and np.allclose(r["norm"].sum(1), np.log([8.0, 4.0]))
    assert r["top_ids"].tolist() == [[2, 1], [2, 0]] and np.allclose(np.exp(r["top_logprobs"]), [[0.625, 0.25], [0.5, 0.25]])


def test_rows_of_nothing():
    x = np.full((1, 4), -np.inf)
    r, _ = os_.logprobs(x, [2], 2)
    assert r["logprob"][0] == -np.inf and r["entropy"][0] == 0 and r["rank"][0] == 2 and r["top_ids"].tolist() == [[0, 1]]
    g, _ = os_.logprobs_bwd(x, [2], [1.0], [1.0], 0.0)
    assert np.all(g == 0)


def test_gradient_is_that_of_differences():
    rng = np.random.default_rng(1)
    x, y, dl, dh = rng.standard_normal((2, 6)) * 2, [3, -1], [0.3, 0.8], [-1.1, 0.4]
    x[0, 1] = -np.inf
    g, _ = os_.logprobs_bwd(x, y, dl, dh, 0.0)

    def value(z):
        r, _ = os_.logprobs(z, y, 0)
        return r["logprob"] * dl + r["entropy"] * dh

    for i in range(6):
        up, down = x.copy(), x.copy()
        up[:, i] += 1e-6
        down[:, i] -= 1e-6
        assert np.allclose((value(up) - value(down)) / 2e-6, g[:, i], atol=1e-8)
