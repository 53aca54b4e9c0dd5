"""Pins of the oracle of the score rules, the rotation on several axes and the
lists of a step, by worked values and invariants."""
import numpy as np
import pytest

import oracle
from oracle import rules as ref
from oracle.draft import tree_attention
from tests._rules import RulesBatch


def test_seen_ranges_by_hand():
    assert ref.seen(5, 8) == (0, 6)
    assert ref.seen(5, 8, window=1) == (5, 6)
    assert ref.seen(5, 8, window=4) == (2, 6)
    assert ref.seen(5, 8, window=6) == (0, 6)
    assert ref.seen(5, 8, see_from=3) == (3, 6)
    assert ref.seen(5, 8, window=2, see_from=3) == (4, 6)
    assert ref.seen(5, 8, see_to=7) == (0, 7)
    assert ref.seen(5, 8, see_to=70) == (0, 8)
    assert ref.seen(5, 8, see_to=2) == (0, 6)
    assert ref.seen(5, 8, see_from=6) == (6, 6)          # nothing


def test_two_keys_by_hand():
    """One query, two keys: scores 2 and 0, capped at 1: tanh 2 and 0; V 1 and 3."""
    k = np.array([[[2.0, 0.0]], [[0.0, 0.0]]])
    v = np.array([[[1.0, 1.0]], [[3.0, 3.0]]])
    q = np.array([[[1.0, 0.0]]])
    rtt = np.array([[0, 1]])
    o, lse, a = ref.attention(q, k, v, rtt, [0], [1], [1], 1.0, cap=1.0, slopes=[0.5])
    x = np.array([np.tanh(2.0) - 0.5, 0.0])              # the first key is one position back
    w = np.exp(x) / np.exp(x).sum()
    assert np.allclose(o[0, 0], w[0] + 3 * w[1], rtol=1e-14)
    assert np.allclose(lse[0, 0], np.log(np.exp(x).sum()), rtol=1e-14)
    assert np.allclose(a, o)


def test_without_rules_it_is_the_attention_of_chains():
    b = RulesBatch(1, 4, 2, 8, [5, 0, 9], [3, 4, 1])
    see = [np.tril(np.ones((t, t), bool)) for t in b.new_len]
    want = tree_attention(b.q, b.k.astype(np.float64), b.v.astype(np.float64), b.rtt, b.req_idx, b.prefix_len, b.indptr, see,
                          b.scale)
    got = b.oracle(b.q, b.k.astype(np.float64), b.v.astype(np.float64))
    for x, y in zip(got, want):
        assert np.allclose(x, y, rtol=1e-12, atol=1e-12)


def test_documents_do_not_see_one_another():
    """A packed request gives what its documents give alone."""
    b = RulesBatch(2, 2, 1, 8, [0], [69], mask="docs")
    k, v = b.k.astype(np.float64), b.v.astype(np.float64)
    o, lse, _ = b.oracle(b.q, k, v)
    for s in range(0, 69, 23):
        rtt = b.rtt[b.req_idx[0]:b.req_idx[0] + 1, s:s + 23]
        alone, l, _ = ref.attention(b.q[s:s + 23], k, v, rtt, [0], [0], [23], b.scale)
        assert np.allclose(o[s:s + 23], alone, rtol=1e-12) and np.allclose(lse[s:s + 23], l, rtol=1e-12)


def test_a_large_cap_is_none():
    b = RulesBatch(3, 2, 1, 8, [7], [5])
    k, v = b.k.astype(np.float64), b.v.astype(np.float64)
    plain = b.oracle(b.q, k, v)
    b.cap = 1e6
    assert np.allclose(b.oracle(b.q, k, v)[0], plain[0], atol=1e-9)


@pytest.mark.parametrize("d", [64, 128])
def test_equal_axes_are_one_axis(d):
    rng = np.random.default_rng(4)
    x, pos = rng.standard_normal((6, 3, d)), rng.integers(-50, 100000, 6)
    axis = rng.integers(0, 3, d // 2)
    got = ref.rope_axes(x, np.stack([pos] * 3), axis, 10000.0)
    assert np.allclose(got, oracle.rope_f64(x, pos, 10000.0), atol=1e-9)


def test_axes_turn_their_own_pairs():
    """A position on axis 1 leaves the pairs of axis 0 alone."""
    x = np.ones((1, 1, 4))
    got = ref.rope_axes(x, np.array([[0], [3]]), [0, 1], 100.0)[0, 0]
    a = 3 * 100.0 ** -0.5
    assert np.allclose(got, [1, np.cos(a) - np.sin(a), 1, np.cos(a) + np.sin(a)])


def test_maps_by_hand():
    rtt = np.array([[10, 11, 12, 13], [20, 21, 22, 23]])
    got = ref.step_maps([1, 0], [1, 0], [2, 3], rtt, 100, 99)
    assert got[0] == [0, 2, 5] and got[1] == [3, 3]
    assert got[2] == [1, 2, 0, 1, 2] and got[3] == [21, 22, 10, 11, 12] and not got[5] and not got[6]
    pages = np.array([[7, 3], [5, 1]])
    got = ref.step_maps([1, 0], [1, 0], [2, 3], rtt, 100, 99, pages, 2)
    assert got[3] == [11, 2, 14, 15, 6] and got[4].tolist() == [[14, 15, 6, 13], [20, 11, 2, 23]]
