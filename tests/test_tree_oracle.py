"""Pins for the oracles of speculative decoding (CPU only)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle.attn import decode_attention
from oracle.tree import Pages, ancestors, tree_attention, verify_drafts


def test_ancestors_of_a_chain_and_a_fork():
    np.testing.assert_array_equal(ancestors([-1, 0, 1]), np.tril(np.ones((3, 3), bool)))
    sees = ancestors([-1, 0, 0, 2, -2])
    assert sees[3].tolist() == [True, False, True, True, False] and not sees[4].any()


@pytest.mark.parametrize("parent", [[-1], [-1, 0, 1, 2], [-1, 0, 0, 1, -1]])
def test_tree_attention_is_single_token_attention_over_what_a_node_sees(parent):
    r = np.random.default_rng(0)
    n, L = len(parent), 9
    q, kn, vn = r.normal(size=(n, 4, 16)), r.normal(size=(n, 2, 16)), r.normal(size=(n, 2, 16))
    ko, vo = r.normal(size=(L, 2, 16)), r.normal(size=(L, 2, 16))
    o = tree_attention(q, ko, vo, kn, vn, parent)[0]
    sees = ancestors(parent)
    for i in range(n):
        ref = decode_attention(q[i], np.concatenate([ko, kn[sees[i]]]), np.concatenate([vo, vn[sees[i]]]))
        np.testing.assert_allclose(o[i], ref, rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("parent,drafted", [([-1, 0], True), ([-1, 0, 0, 0], True), ([-1, 0, 0], False)])
def test_verification_leaves_the_targets_distribution(parent, drafted):
    """The first token after the root follows p exactly: summed over drawn drafts, by frequency.
    60,000 walks: a frequency of 1/2 at most is off by 6 standard deviations 6 * sqrt(1/4 / 60000) = 0.0122."""
    r = np.random.default_rng(1)
    V, walks = 5, 60000
    p = r.dirichlet(np.ones(V), len(parent))
    q = r.dirichlet(np.ones(V), len(parent))
    seen = np.zeros(V)
    kids = [j for j in range(1, len(parent))]
    draws = r.choice(V, (walks, len(parent)), p=q[0])
    ua, us = r.random((walks, len(parent))), r.random(walks)
    for w in range(walks):
        tok = draws[w] if drafted else np.array([0, 3, 1, 2])[:len(parent)]
        path, nxt = verify_drafts(p, q if drafted else None, tok, parent, ua[w], us[w])
        seen[tok[path[1]] if len(path) > 1 else nxt] += 1
    assert kids and np.abs(seen / walks - p[0]).max() < 0.0122


def test_verification_of_a_perfect_draft_takes_it():
    p = np.array([[0.25, 0.75], [0.5, 0.5], [1.0, 0.0]])
    path, nxt = verify_drafts(p, p, [0, 1, 0], [-1, 0, 1], [0.9, 0.999, 0.999], 0.3)
    assert path == [0, 1, 2] and nxt == 0


def test_verification_draws_from_the_residual():
    # child token 0 refused (u q = 0.9 * 0.8 >= 0.5); R = max(p - q, 0) = [0, 0.3, 0]
    path, nxt = verify_drafts([[0.5, 0.5, 0.0], [1, 0, 0]], [[0.8, 0.2, 0.0], [1, 0, 0]], [0, 0], [-1, 0], [0, 0.9], 0.0)
    assert path == [0] and nxt == 1


def test_pages_share_copy_and_free():
    k = np.arange(6 * 4 * 2, dtype=float).reshape(1, 6, 4, 1, 2)
    c = Pages(k, k + 100, np.zeros(6, int), np.full((3, 3), -1), np.zeros(3, int))
    rows = np.arange(12, dtype=float).reshape(1, 6, 1, 2)
    c.append([(0, rows, rows)])
    assert c.table[0].tolist() == [0, 1, -1] and c.refs.tolist() == [1, 1, 0, 0, 0, 0]
    c.fork([(0, 1)])
    assert c.table[1].tolist() == [0, 2, -1] and c.refs.tolist() == [2, 1, 1, 0, 0, 0]
    np.testing.assert_array_equal(c.rows(1)[0], rows[0])
    c.trim(1, 3)  # inside the shared page: appending moves its rows first
    c.append([(1, rows[:, :1] + 50, rows[:, :1])])
    assert c.table[1].tolist() == [2, -1, -1] and c.refs.tolist() == [1, 1, 1, 0, 0, 0]
    np.testing.assert_array_equal(c.rows(0)[0], rows[0])
    np.testing.assert_array_equal(c.rows(1)[0], np.concatenate([rows[0, :3], rows[0, :1] + 50]))
    c.trim(0, 0)
    assert c.refs.tolist() == [0, 0, 1, 0, 0, 0]
