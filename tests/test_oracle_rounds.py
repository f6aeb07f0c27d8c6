"""The 64-bit oracle of the operators around a round, on cases that can be worked by hand,
and the host arithmetic of the rotation's frequencies (CPU only)."""
import math

import numpy as np
import pytest

from oracle import mixing, rounds


def test_pages_by_hand():
    # page of 4; sequence 0 grows by two pages, 1 gives one back, 2 needs nothing
    out = rounds.assign([5, 6, 7, 0], 3, [[1, -1, -1], [2, 3, -1], [4, -1, -1]], [1, 2, 1], 4, [4, 2, 0], [5, 2, 3], 5)
    # the page given back lies on top of 7, and is taken first
    assert out["table"] == [[1, 3, 7], [2, -1, -1], [4, -1, -1]]
    assert out["held"] == [3, 1, 1] and out["n_free"] == 2 and out["free"][:2] == [5, 6]
    assert out["granted"] == [5, 2, 3]
    assert out["positions"][0] == [4, 5, 6, 7, 8] and out["positions"][1] == [2, 3, -1, -1, -1]
    assert out["slots"][0] == [12, 13, 14, 15, 28] and out["slots"][2] == [16, 17, 18, -1, -1]


def test_a_shortage_ends_the_taking():
    out = rounds.assign([5, 6], 2, [[-1] * 3, [-1] * 3, [4, -1, -1]], [0, 0, 1], 4, [0, 0, 0], [4, 8, 6], 8)
    assert out["held"] == [1, 0, 1] and out["n_free"] == 1
    assert out["granted"] == [4, 0, 4]  # the last has the rows of the page that it holds


def test_giving_back_restores_the_list():
    free, table, held = [9, 8, 7, 6, 5, 4], [[0, -1, -1], [1, 2, -1]], [1, 2]
    up = rounds.assign(free, 6, table, held, 2, [2, 3], [4, 3], 4)
    down = rounds.assign(up["free"], up["n_free"], up["table"], up["held"], 2, [2, 3], [0, 0], 4)
    assert down["free"] == free and down["n_free"] == 6 and down["table"] == table and down["held"] == held


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_a_quarter_turn(layout):
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    y = rounds.norm_rope(x, None, 0.0, np.array([1]), [math.pi / 2] * 2, 1.0, layout)[0, 0]
    want = [-3, -4, 1, 2] if layout == "half" else [-2, 1, -4, 3]
    assert np.allclose(y, want + [5, 6, 7, 8])


def test_norm():
    x = np.array([[[3.0, 4.0]]])
    assert np.allclose(rounds.norm_rope(x, np.array([1.0, 2.0]), 0.0, np.array([0]), [], 1.0, "half"),
                       [[[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]]])


def test_a_prefix_is_the_first_positions():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 6, 2, 4, 8))
    q = rng.standard_normal((2, 2, 4, 8))
    # pages 0, 1 hold the prefix of 8 positions of both; the same as tables that begin with them
    got = rounds.prefix_attention(q, k, v, [0, 1], 8, [[2, 3], [4, 5]], [3, 0], [2, 1], None, 0.3)
    want = mixing.attention(q, k, v, [[0, 1, 2, 3], [0, 1, 4, 5]], [11, 8], [2, 1], None, 0.3)
    assert np.allclose(got["out"], want["out"]) and np.allclose(got["lse"], want["lse"])


def test_drafted_tokens_by_hand():
    logits = np.log(np.array([[0.5, 0.25, 0.25], [0.2, 0.2, 0.6]]))
    # kept (0.4 < 0.5), then a draw from the second row: running 0.2, 0.4, 1
    assert rounds.verify(logits, 1.0, [0], 1, None, np.array([0.4, 0.3]))[:2] == (1, 1)
    # not kept: from the others, halves
    assert rounds.verify(logits, 1.0, [0], 1, None, np.array([0.6, 0.49]))[:2] == (0, 1)
    assert rounds.verify(logits, 1.0, [0], 1, None, np.array([0.6, 0.51]))[:2] == (0, 2)
    # a drafter that says 0 with 1 and more than the target: kept with 0.5
    q = np.array([[1.0, 0.0, 0.0]])
    assert rounds.verify(logits, 1.0, [0], 1, q, np.array([0.49, 0.9]))[:2] == (1, 2)
    assert rounds.verify(logits, 1.0, [0], 1, q, np.array([0.5, 0.9]))[:2] == (0, 2)
    # greedy, a token outside, no token left
    assert rounds.verify(logits, 0.0, [0], 1, None, np.array([0.99, 0.0]))[:2] == (1, 2)
    assert rounds.verify(logits, 1.0, [7], 1, None, np.array([0.0, 0.0]))[:2] == (0, 0)
    assert rounds.verify(np.full((1, 3), -np.inf), 1.0, [], 0, None, np.array([0.5]))[:2] == (0, -1)
