"""Pins for the 64-bit token-mixing oracle (CPU only): closed forms and cases
worked by hand."""
import numpy as np

from oracle import mixing


def _pages(rows, table, page, heads=1):
    """Pages holding rows [L, heads, dim] through ``table``."""
    out = np.full((max(table) + 1, heads, page, rows.shape[-1]), np.nan)
    for p in range(rows.shape[0]):
        out[table[p // page], :, p % page] = rows[p]
    return out


def test_one_position_gives_its_value():
    k, v = np.array([[[2.0, 0.0]]]), np.array([[[5.0, -3.0]]])
    r = mixing.attention(np.ones((1, 1, 1, 2)), _pages(k, [1], 4), _pages(v, [1], 4), [[1]], [0], [1], None, 0.5)
    assert r["out"][0, 0, 0].tolist() == [5.0, -3.0] and r["lse"][0, 0, 0] == 1.0


def test_equal_scores_give_the_mean():
    rng = np.random.default_rng(0)
    v = rng.normal(size=(11, 1, 3))
    k = np.zeros((11, 1, 3))
    t = [2, 0, 5]
    r = mixing.attention(rng.normal(size=(1, 1, 2, 3)), _pages(k, t, 4), _pages(v, t, 4), [t], [10], [1], None, 1.0)
    np.testing.assert_allclose(r["out"][0, 0], np.tile(v[:, 0].mean(0), (2, 1)))
    np.testing.assert_allclose(r["lse"][0, 0], np.log(11.0))


def test_a_mask_word_selects_positions_and_an_empty_one_gives_nothing():
    v = np.arange(8.0).reshape(4, 1, 2)
    k = np.zeros((4, 1, 2))
    mask = [[0b1010, 0b0001, 0, 0b10000]]
    r = mixing.attention(np.ones((1, 4, 1, 2)), _pages(k, [0], 4), _pages(v, [0], 4), [[0]], [0], [4], mask, 1.0)
    np.testing.assert_allclose(r["out"][0, 0, 0], (v[1, 0] + v[3, 0]) / 2)
    np.testing.assert_allclose(r["out"][0, 1, 0], v[0, 0])
    assert not r["out"][0, 2].any() and r["lse"][0, 2, 0] == -np.inf
    assert not r["out"][0, 3].any() and r["lse"][0, 3, 0] == -np.inf  # a bit past the window


def test_causal_rows_grow_by_one_position():
    rng = np.random.default_rng(1)
    k, v = rng.normal(size=(5, 1, 4)), rng.normal(size=(5, 1, 4))
    q = rng.normal(size=(1, 3, 1, 4))
    pk, pv = _pages(k, [0, 1], 3), _pages(v, [0, 1], 3)
    r = mixing.attention(q, pk, pv, [[0, 1]], [2], [3], None, 0.7)
    for i in range(3):
        s = k[:3 + i, 0] @ q[0, i, 0] * 0.7
        w = np.exp(s) / np.exp(s).sum()
        np.testing.assert_allclose(r["out"][0, i, 0], w @ v[:3 + i, 0])


def test_append_writes_its_rows_and_no_others():
    pages = np.zeros((4, 2, 3, 1))
    rows = np.arange(1.0, 9.0).reshape(1, 4, 2, 1)
    out = mixing.append(pages, rows, [[3, 1]], [2], [3])
    assert out[3, :, 2, 0].tolist() == [1.0, 2.0] and out[1, :, 0, 0].tolist() == [3.0, 4.0]
    assert out[1, :, 1, 0].tolist() == [5.0, 6.0] and out.sum() == 21.0


def test_without_decay_the_state_is_a_sum_of_outer_products():
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(1, 6, 1, 3)), rng.normal(size=(1, 6, 1, 3)), rng.normal(size=(1, 6, 2, 4))
    r = mixing.linear(q, k, v, np.zeros((1, 6, 2)), 0.5, [6], np.zeros((1, 2, 3, 4)))
    for h in range(2):
        np.testing.assert_allclose(r["state"][0, h], k[0, :, 0].T @ v[0, :, h])
        full = np.tril(q[0, :, 0] @ k[0, :, 0].T) @ v[0, :, h]
        np.testing.assert_allclose(r["o"][0, :, h], 0.5 * full)


def test_decay_is_geometric_and_a_dropped_state_is_gone():
    k, v = np.ones((1, 3, 1, 1)), np.ones((1, 3, 1, 1))
    g = np.full((1, 3, 1), np.log(0.5))
    r = mixing.linear(k, k, v, g, 1.0, [3], np.full((1, 1, 1, 1), 8.0))
    np.testing.assert_allclose(r["o"][0, :, 0, 0], [5.0, 3.5, 2.75])
    g[0, 1] = -np.inf
    r = mixing.linear(k, k, v, g, 1.0, [3], np.full((1, 1, 1, 1), np.inf))
    assert r["o"][0, 1:, 0, 0].tolist() == [1.0, 1.5] and r["state"][0, 0, 0, 0] == 1.5
    r = mixing.linear(k, k, v, g, 1.0, [1], np.full((1, 1, 1, 1), 8.0))
    assert r["o"][0, :, 0, 0].tolist() == [5.0, 0.0, 0.0] and r["state"][0, 0, 0, 0] == 5.0
