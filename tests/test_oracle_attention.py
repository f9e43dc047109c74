"""Pins of the attention oracle: against closed forms and differences, and of
the draft verification against its distribution."""

import numpy as np

from oracle import attention as oa


def _rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


def test_uniform_scores_average_the_values():
    q, k, v = np.zeros((4, 192)), _rand(7, 192), _rand(7, 128, seed=1)
    out, lse, _, _ = oa.mla_head(q, k, v, 0.1, True)
    for i in range(4):
        np.testing.assert_allclose(out[i], v[:i + 4].mean(0), rtol=1e-13)
        np.testing.assert_allclose(lse[i], np.log(i + 4), rtol=1e-13)


def test_rows_that_see_nothing():
    out, lse, _, _ = oa.mla_head(_rand(5, 192), _rand(3, 192), _rand(3, 128), 0.1, True)
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.all(np.isfinite(lse[2:]))
    assert oa.softmax_rows(np.zeros((2, 0)), np.zeros((2, 0), bool))[0].shape == (2, 0)


def test_gradients_against_differences():
    rng = np.random.default_rng(3)
    for lq, lk, causal in ((5, 5, True), (3, 6, True), (6, 4, True), (4, 3, False)):
        q, k, v = rng.standard_normal((lq, 192)), rng.standard_normal((lk, 192)), rng.standard_normal((lk, 128))
        dout = rng.standard_normal((lq, 128))
        (dq, dk, dv), _ = oa.mla_head_bwd(q, k, v, dout, 0.2, causal)

        def value():
            return float((oa.mla_head(q, k, v, 0.2, causal)[0] * dout).sum())

        for x, g in ((q, dq), (k, dk), (v, dv)):
            for _ in range(12):
                at = tuple(rng.integers(0, s) for s in x.shape)
                keep, h = x[at], 1e-5
                x[at] = keep + h
                up = value()
                x[at] = keep - h
                down = value()
                x[at] = keep
                # second-order differences: h^2 of the third derivative, and 1e-16/h of the sum
                assert abs((up - down) / (2 * h) - g[at]) < 1e-7 * (1 + abs(g[at])), (lq, lk, at)


def test_verify_follows_the_target_distribution():
    # the emitted first token has the target's distribution whatever the draft model is
    rng = np.random.default_rng(5)
    V, N = 6, 40000
    p = rng.dirichlet(np.ones(V)).astype(np.float32)
    q = rng.dirichlet(np.ones(V)).astype(np.float32)
    drafts = rng.choice(V, N, p=q.astype(np.float64) / q.astype(np.float64).sum()).astype(np.int32)
    P = np.broadcast_to(p, (N, 2, V))
    Q = np.broadcast_to(q, (N, 1, V))
    tokens, _ = oa.verify_drafts(P, Q, drafts[:, None], np.ones(N, np.int32), rng.random((N, 1)).astype(np.float32),
                                 rng.random(N).astype(np.float32))
    share = np.bincount(tokens[:, 0], minlength=V) / N
    assert np.all(np.abs(share - p) < 5 * np.sqrt(p * (1 - p) / N) + 1e-6)


def test_verify_hand_cases():
    f = np.float32
    p = np.array([[[0.5, 0.5, 0.0], [0.0, 0.25, 0.75]]], f)
    q = np.array([[[1.0, 0.0, 0.0]]], f)
    d, n = np.array([[0]], np.int32), np.array([1], np.int32)
    # accepted (0.4 * 1 < 0.5), then 0.3 falls in the third entry
    t, a = oa.verify_drafts(p, q, d, n, np.array([[0.4]], f), np.array([0.3], f))
    assert t.tolist() == [[0, 2]] and a.tolist() == [1]
    # at the limit it is turned down; what is left of p is entry 1
    t, a = oa.verify_drafts(p, q, d, n, np.array([[0.5]], f), np.array([0.9], f))
    assert t.tolist() == [[1, -1]] and a.tolist() == [0]
    # no drafts: plain sampling; no weight at all: -1
    t, a = oa.verify_drafts(p[:, :1], q[:, :0], d[:, :0], n * 0, np.zeros((1, 0), f), np.array([0.49], f))
    assert t.tolist() == [[0]] and a.tolist() == [0]
    t, _ = oa.verify_drafts(p[:, :1] * 0, q[:, :0], d[:, :0], n * 0, np.zeros((1, 0), f), np.array([0.49], f))
    assert t.tolist() == [[-1]]
    # a certain draft model (no q): the draft itself is left out after a rejection
    t, _ = oa.verify_drafts(p, None, d, n, np.array([[0.7]], f), np.array([0.1], f))
    assert t.tolist() == [[1, -1]]
