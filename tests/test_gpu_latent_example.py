"""The example of training and serving one layer of latent attention: what the
paged, absorbed, speculative path computed is what the expanded form computes
for the whole sequences."""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import latent_attention as ex

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("drafts", [0, 3])
def test_generation_is_the_expanded_form(dev, cache, drafts):
    layer = ex.Layer(dev)
    res = ex.generate(layer, steps=5, drafts=drafts, cache=cache)
    for toks, o in zip(res["tokens"], res["outputs"]):
        want = ex.attention_of(layer, toks[:-1])[-len(o):].float()
        # up to eight roundings to BF16 (2^-8 / sqrt(12) * 1.5 of the norm each, at most) on either side, added up;
        # the E4M3 codes add one of 2^-4 / sqrt(12) * 1.5 of the latent vectors to keys and to values
        limit = 16 * 0.0017 + (2 * 0.027 if cache == "fp8" else 0)
        assert (o.float() - want).norm() <= limit * want.norm()
    made = [len(t) - 150 - n for t, n in zip(res["tokens"], (40, 7, 100))]
    assert made == [int(a) + 5 for a in res["accepted"].sum(0)]
    assert all(0 <= t < layer.vocab for toks in res["tokens"] for t in toks)


def test_training_step_learns(dev):
    losses = ex.train(ex.Layer(dev), steps=25)
    assert all(x == x for x in losses) and losses[-1] < 0.7 * losses[0]
