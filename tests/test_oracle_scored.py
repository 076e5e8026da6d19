"""The oracle of routing by scores and of low-rank adapters, against closed
forms, brute force and the plain routing rule."""

import itertools

import numpy as np
import pytest

from oracle import route as oroute
from oracle import scored


def test_softmax_without_bias_and_groups_is_the_plain_rule():
    rng = np.random.default_rng(0)
    logits = rng.normal(0, 2, (9, 37)).astype(np.float32)
    logits[3, 5], logits[4] = np.nan, np.round(logits[4])
    ids, w = scored.route(logits, 5, sigmoid=False)
    want = oroute.route_topk(logits, 5)
    assert np.array_equal(ids, want[0])
    assert np.abs(w - want[1]).max() <= 2.0 ** -24


@pytest.mark.parametrize("sigmoid", [True, False])
def test_groups_and_choice_by_brute_force(sigmoid):
    """The chosen groups and experts are the ones of the largest sums among all subsets."""
    rng = np.random.default_rng(1)
    logits, bias = rng.normal(0, 1, (6, 12)).astype(np.float32), rng.normal(0, 0.2, 12).astype(np.float32)
    ids, w = scored.route(logits, 3, bias, sigmoid, groups=4, keep=2, best=2, scale=2.5)
    c = scored.scores(logits, sigmoid) + bias.astype(np.float64)
    for t in range(6):
        value = lambda g: np.sort(c[t, 3 * g:3 * g + 3])[-2:].sum()  # noqa: E731
        pair = max(itertools.combinations(range(4), 2), key=lambda p: value(p[0]) + value(p[1]))
        inside = [e for e in range(12) if e // 3 in pair]
        three = max(itertools.combinations(inside, 3), key=lambda p: sum(c[t, list(p)]))
        assert set(ids[t]) == set(three)
        assert list(c[t, ids[t]]) == sorted(c[t, ids[t]], reverse=True)
        s = scored.scores(logits, sigmoid)[t, ids[t]]
        assert np.allclose(w[t], 2.5 * s / s.sum(), rtol=1e-14)


def test_weights_hold_where_scores_underflow():
    l = np.array([[-1000.0, -1001.0, -3.4e38, -1002.0]], np.float32)
    ids, w = scored.route(l, 3)
    e = np.exp([0.0, -1.0, -2.0])
    assert ids.tolist() == [[0, 1, 3]] and np.allclose(w[0], e / e.sum(), rtol=1e-14)
    ids, w = scored.route(np.full((1, 4), -3.4e38, np.float32), 2)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.5, 0.5]]


def test_unavailable_experts():
    n, i = np.nan, np.inf
    l = np.array([[n, -i, 1.0, 2.0], [n, -i, n, -i], [0.0, i, i, 1.0]], np.float32)
    ids, w = scored.route(l, 3, sigmoid=False)
    assert ids.tolist() == [[3, 2, -1], [-1, -1, -1], [1, 2, 3]]
    assert w[0, 2] == 0 and not w[1].any() and w[2].tolist() == [0.5, 0.5, 0.0]
    ids, _ = scored.route(np.zeros((1, 4), np.float32), 4, [0.0, n, i, -i])
    assert ids.tolist() == [[2, 0, -1, -1]]


def test_ties_go_to_the_lower_index():
    ids, _ = scored.route(np.array([[0.0, -0.0, 0.0, 0.0]], np.float32), 2)
    assert ids.tolist() == [[0, 1]]
    ids, _ = scored.route(np.zeros((1, 8), np.float32), 2, np.zeros(8, np.float32), groups=4, keep=2)
    assert ids.tolist() == [[0, 1]]


def test_lora_against_the_merged_matrix():
    rng = np.random.default_rng(2)
    x, y = rng.normal(size=(7, 10)), rng.normal(size=(7, 6))
    a, b, scale = rng.normal(size=(3, 4, 10)), rng.normal(size=(3, 6, 4)), rng.random(3)
    slots = [0, 2, -1, 1, 3, 2, 0]
    out = scored.lora(x, slots, a, b, y, scale)
    for m, s in enumerate(slots):
        want = y[m] + (x[m] @ (scale[s] * b[s] @ a[s]).T if 0 <= s < 3 else 0.0)
        assert np.allclose(out[m], want, rtol=1e-12, atol=1e-12)
