"""The log-probability and embedding oracles against closed forms and finite differences (CPU)."""
import math

import numpy as np
import pytest

from oracle import embed as oembed
from oracle import logprobs as olp


def test_uniform_and_one_hot_distributions():
    o = olp.slot(np.zeros(8), token=3, k=3)
    assert abs(o["logprob"] + math.log(8)) < 1e-15 and abs(o["entropy"] - math.log(8)) < 1e-15
    assert list(o["top_ids"]) == [0, 1, 2]
    x = np.full(5, -np.inf)
    x[2] = 4.0
    o = olp.slot(x, token=2, k=5)
    assert o["logprob"] == 0 and o["entropy"] == 0 and o["m"] == 4 and o["logS"] == 0
    assert list(o["top_ids"]) == [2, 0, 1, 3, 4] and np.isneginf(o["top_logprobs"][1:]).all()


def test_two_columns_by_hand():
    # odds 3 to 1
    o = olp.slot([math.log(3.0), 0.0], token=1, k=2)
    assert abs(o["logprob"] - math.log(0.25)) < 1e-15
    assert abs(o["entropy"] - (-0.75 * math.log(0.75) - 0.25 * math.log(0.25))) < 1e-15


@pytest.mark.parametrize("x", [[-np.inf, -np.inf], [np.inf, 0.0], [np.nan, 1.0]])
def test_slots_without_a_distribution(x):
    o = olp.slot(x, token=0)
    assert np.isnan(o["logprob"]) and np.isnan(o["entropy"])


@pytest.mark.parametrize("gl,gh", [(1.0, 0.0), (0.0, 1.0), (-0.7, 0.3)])
def test_gradient_against_differences(gl, gh):
    rng = np.random.default_rng(3)
    x = rng.normal(size=17) * 2
    tok = 5

    def f(y):
        o = olp.slot(y, token=tok)
        return gl * o["logprob"] + gh * o["entropy"]
    g = olp.grad(x, tok, gl, gh)
    h = 1e-5
    num = np.array([(f(x + h * np.eye(17)[i]) - f(x - h * np.eye(17)[i])) / (2 * h) for i in range(17)])
    # central differences: h^2 f'''/6 plus rounding eps/h
    assert np.abs(g - num).max() < 1e-9 and abs(g.sum()) < 1e-14


def test_embedding_by_hand():
    table = np.arange(12.0).reshape(4, 3)
    out = oembed.lookup(table, [2, 0, 9, -1, 3], valid=[1, 1, 1, 1, 0], scale=2.0)
    assert np.array_equal(out, [[12, 14, 16], [0, 2, 4], [0, 0, 0], [0, 0, 0], [0, 0, 0]])
    g = np.arange(15.0).reshape(5, 3)
    total, size, count = oembed.gradient(g, [1, 1, 7, 0, 1], 4, valid=[1, 1, 1, 0, 1], scale=-1.0)
    assert np.array_equal(total[1], -(g[0] + g[1] + g[4])) and np.array_equal(size[1], g[0] + g[1] + g[4])
    assert list(count) == [0, 3, 0, 0] and not total[[0, 2, 3]].any()
