"""Pins of oracle/trees.py against closed forms, the batch oracle and planted mistakes."""

import numpy as np
import pytest

from oracle import accept as oacc
from oracle import batch as obat
from oracle import trees as otree

D = 128


def normal(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def test_prompt_rows_are_the_batch_oracles():
    q, k, v = normal(1, 9, 2, 3, D), normal(2, 9, 2, D), normal(3, 9, 2, D)
    starts = [1, 4, 4, 8]
    out, spread = otree.attention_prompt(q, k, v, starts)
    assert not out[0].any() and not out[8].any() and not spread[0].any()
    for a, b in ((1, 4), (4, 8)):
        kk, vv = k[a:b].transpose(1, 0, 2), v[a:b].transpose(1, 0, 2)
        ref, rs = obat.attention_batch(q[a:b][None], kk[:, :0], vv[:, :0], kk[None], vv[None], [0])
        np.testing.assert_allclose(out[a:b], ref[0], rtol=1e-12)
        np.testing.assert_allclose(spread[a:b], rs[0], rtol=1e-12)


def test_first_row_of_a_prompt_is_its_value():
    q, k, v = normal(1, 5, 1, 2, D), normal(2, 5, 1, D), normal(3, 5, 1, D)
    out, _ = otree.attention_prompt(q, k, v, [0, 2, 5])
    for r in (0, 2):
        np.testing.assert_allclose(out[r], np.broadcast_to(v[r, :, None], out[r].shape), rtol=1e-14)


def test_paths():
    parents = [-1, 0, 0, 1, 3, 2, -1]
    assert [otree.tree_path(parents, i) for i in range(7)] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4], [0, 2, 5], []]


def test_a_chain_is_the_batch_oracle():
    q, sk, sv = normal(1, 2, 4, 2, 3, D), normal(2, 2, 5, D), normal(3, 2, 5, D)
    k, v = normal(4, 2, 2, 20, D), normal(5, 2, 2, 20, D)
    chain = [[-1, 0, 1, 2]] * 2
    got, ref = (f[0] for f in (otree.attention_tree(q, sk, sv, k, v, [7, -1], chain),
                               obat.attention_batch(q, sk, sv, k, v, [7, -1])))
    np.testing.assert_allclose(got, ref, rtol=1e-12)


def test_a_node_sees_its_path_alone():
    q, k, v = normal(1, 1, 4, 1, 1, D), normal(2, 1, 1, 12, D), normal(3, 1, 1, 12, D)
    none = np.zeros((1, 0, D))
    out, _ = otree.attention_tree(q, none, none, k, v, [6], [[-1, 0, 0, 2]])
    k2, v2 = k.copy(), v.copy()
    k2[0, 0, 7], v2[0, 0, 7] = 9.0, -9.0      # node 1, on no path but its own
    moved, _ = otree.attention_tree(q, none, none, k2, v2, [6], [[-1, 0, 0, 2]])
    same = [np.array_equal(out[0, i], moved[0, i]) for i in range(4)]
    assert same == [True, False, True, True]
    # node 3's path 0, 2, 3 laid out one after the other, as serial decoding has it
    at = list(range(7)) + [8, 9]
    serial, _ = obat.attention_batch(q[:, 3:], none, none, k[:, :, at], v[:, :, at], [8])
    np.testing.assert_allclose(out[0, 3], serial[0, 0], rtol=1e-12)


def test_acceptance_along_a_chain_is_the_chains():
    rng = np.random.default_rng(0)
    for _ in range(200):
        n = int(rng.integers(1, 7))
        tokens, sampled = rng.integers(0, 2, n), rng.integers(0, 2, n)
        a, bonus = oacc.accept(tokens[1:], sampled)
        got = otree.accept_tree([-1] + list(range(n - 1)), tokens, sampled)
        assert got == (a, bonus, list(range(a + 1)), list(sampled[: a + 1]))


def test_acceptance_takes_the_first_child_that_fits():
    parents, tokens = [-1, 0, 0, 0, 1, 3, -1], [0, 5, 6, 6, 6, 8, 7]
    assert otree.accept_tree(parents, tokens, [6, 0, 9, 0, 0, 0, 0]) == (1, 9, [0, 2], [6, 9])
    assert otree.accept_tree(parents, tokens, [5, 6, 0, 0, 3, 0, 0]) == (2, 3, [0, 1, 4], [5, 6, 3])
    assert otree.accept_tree(parents, tokens, [7, 0, 0, 0, 0, 0, 0]) == (0, 7, [0], [7])     # an unused row's token


@pytest.mark.parametrize("wrong", ["future", "sibling", "scale"])
def test_planted_mistakes_are_caught(wrong):
    q, k, v = normal(1, 6, 1, 1, D), normal(2, 6, 1, D), normal(3, 6, 1, D)
    out, _ = otree.attention_prompt(q, k, v, [0, 6])
    if wrong == "future":
        bad = otree._attend(q[2, 0], k[:4, 0], v[:4, 0])[0]
    elif wrong == "sibling":
        bad = otree._attend(q[2, 0], k[[0, 2], 0], v[[0, 2], 0])[0]
    else:
        bad = otree._attend(q[2, 0] * np.sqrt(D), k[:3, 0], v[:3, 0])[0]
    assert np.abs(bad - out[2, 0]).max() > 1e-2
