"""Pins of the oracle's operators around the indexer: worked examples, closed forms and distributions."""

import math

import numpy as np

from oracle import step


def test_slots_by_hand():
    # page 4; request 0: 5 cached + 3 new -> 2 pages, owns 2; request 1: 0 + 5 -> 2 pages, owns none; request 2: 4 + 1, owns 3
    table = np.array([[7, 3, -1], [-1, -1, -1], [0, 1, 2]])
    o = step.build_slots([5, 0, 4], [3, 5, 1], [2, 0, 3], table, [9, 8, 6, 5], 1, 10, 4, 11)
    assert o["block_table"].tolist() == [[7, 3, -1], [8, 6, -1], [0, 1, 2]]
    assert o["cu_tokens"].tolist() == [0, 3, 8, 9]
    assert o["seq_lens"].tolist() == [8, 5, 5] and o["pages_out"].tolist() == [2, 2, 3] and o["cursor_out"] == 3
    assert o["slots"].tolist() == [13, 14, 15, 32, 33, 34, 35, 24, 4, -1, -1]
    assert o["positions"].tolist() == [5, 6, 7, 0, 1, 2, 3, 4, 4, 0, 0]
    assert o["status"] == 0


def test_slots_shortage_and_trees():
    table = np.full((2, 3), -1)
    o = step.build_slots([0, 0], [5, 5], [0, 0], table, [4, 2, 1], 0, 5, 4, 10, parents=[-1, 0, 0, 1, 3, -1, 0, 1, 1, 5])
    assert o["block_table"].tolist() == [[4, 2, -1], [1, -1, -1]]
    assert o["slots"].tolist()[5:] == [4, 5, 6, 7, -1] and o["pages_out"].tolist() == [2, 1] and o["cursor_out"] == 3
    assert o["status"] == 16 | 32  # too few blocks; parent 5 of node 4 is no earlier node
    assert o["tree_mask"].tolist() == [1, 3, 5, 11, 27, 1, 3, 7, 11, 16]
    assert o["positions"].tolist() == [0, 1, 1, 2, 3, 0, 1, 2, 2, 0]


def test_rotation_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 12))
    f, m = step.rope_frequencies(8, 10000.0, 0)
    for inter in (False, True):
        y = step.rotate(x, [0, 5, 100_000], f, 1.0, inter)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 8:], x[..., 8:])
        np.testing.assert_allclose((y**2).sum(-1), (x**2).sum(-1), rtol=1e-12)
        back = step.rotate(y, [0, -5, -100_000], f, 1.0, inter)
        np.testing.assert_allclose(back, x, atol=1e-12)
        # products of rotated rows depend on the distance alone
        a, b = step.rotate(x[:1], [7], f, 1.0, inter), step.rotate(x[1:2], [3], f, 1.0, inter)
        c, d = step.rotate(x[:1], [1007], f, 1.0, inter), step.rotate(x[1:2], [1003], f, 1.0, inter)
        np.testing.assert_allclose((a * b).sum(-1), (c * d).sum(-1), atol=1e-10)


def test_frequency_scaling_ends():
    plain, _ = step.rope_frequencies(128, 10000.0, 0)
    ramp, m = step.rope_frequencies(128, 10000.0, 2, 4.0, 4096.0)
    assert ramp[0] == plain[0] and math.isclose(ramp[-1], plain[-1] / 4, rel_tol=1e-12)
    assert np.all(ramp <= plain) and math.isclose(m, 0.1 * math.log(4.0) + 1)


def test_attention_of_a_chain_is_the_causal_softmax():
    rng = np.random.default_rng(1)
    n, ctx, d, page = 5, 6, 8, 4
    k = rng.standard_normal((4, page, 1, d))
    v = rng.standard_normal((4, page, 1, d))
    q = rng.standard_normal((n, 2, d))
    table = np.array([[2, 0, 3]])
    out, lse, *_ = step.tree_attention(q, k, v, table, [ctx + n], [0, n], 0.3)
    kk, vv = k[table[0]].reshape(-1, d), v[table[0]].reshape(-1, d)
    for i in range(n):
        x = 0.3 * kk[: ctx + i + 1] @ q[i].T
        p = np.exp(x) / np.exp(x).sum(0)
        np.testing.assert_allclose(out[i], p.T @ vv[: ctx + i + 1], atol=1e-12)
        np.testing.assert_allclose(lse[i], np.log(np.exp(x).sum(0)), atol=1e-12)
    # the same as a tree whose masks are the chain's, and over lists of all pages
    mask = [(1 << (i + 1)) - 1 for i in range(n)]
    again, *_ = step.tree_attention(q, k, v, table, [ctx + n], [0, n], 0.3, mask, np.tile([[[2, 0, 1, 1, -1]]], (n, 1, 1)))
    np.testing.assert_allclose(again, out, atol=1e-12)
    none, l0, *_ = step.tree_attention(q, k, v, table, [n], [0, n], 0.3, [0] * n)
    assert not none.any() and np.all(np.isneginf(l0))


def test_verification_by_hand():
    p = np.array([[0.5, 0.3, 0.2, 0.0], [0.0, 0.0, 1.0, 0.0], [0.25, 0.25, 0.25, 0.25]])
    q = np.array([[0.1, 0.9, 0.0, 0.0], [0.5, 0.5, 0.0, 0.0], [1.0, 0.0, 0.0, 0.0]])
    # draft token 1: 0.3 / 0.9; u below it stands, then token 0 is refused by p = 0, residual is p itself: token 2
    a, t, n = step.verify(p, q, [0, 1, 0], None, [0, 3], [0, 0.33, 0.0], [0.9], 3)
    assert (a.tolist(), t.tolist(), n.tolist()) == ([1], [[1, 2, -1]], [[1, -1, -1]])
    # refused: residual (0.4, 0, 0.2): token 0 below 2/3, token 2 above
    for u, want in ((0.66, 0), (0.67, 2)):
        a, t, n = step.verify(p, q, [0, 1, 0], None, [0, 3], [0, 0.34, 0.0], [u], 3)
        assert (a.tolist(), t.tolist(), n.tolist()) == ([0], [[want, -1, -1]], [[-1, -1, -1]])
    # without draft rows: siblings 0 then 1 of node 0; 0 refused leaves half the mass
    a, t, n = step.verify(p, None, [9, 0, 1], [-1, 0, 0], [0, 3], [0, 0.5, 0.59], [0.3], 2)
    assert (a.tolist(), t.tolist()) == ([1], [[1, 1]])  # 0.59 * 0.5 < 0.3; node 2's row is uniform
    a, t, n = step.verify(p, None, [9, 0, 1], [-1, 0, 0], [0, 3], [0, 0.5, 0.61], [0.3], 2)
    assert (a.tolist(), t.tolist()) == ([0], [[2, -1]])


def test_closed_form_of_the_residual():
    # after k refusals the normalised residual is max(p - c_k q, 0) / W_k with c_{k+1} = c_k + W_k
    rng = np.random.default_rng(2)
    p, q = rng.dirichlet(np.ones(50)), rng.dirichlet(np.ones(50))
    rest, c, w = p.copy(), 0.0, 1.0
    for _ in range(5):
        rest = np.maximum(rest - q, 0)
        rest /= rest.sum()
        c += w
        w = np.maximum(p - c * q, 0).sum()
        np.testing.assert_allclose(np.maximum(p - c * q, 0) / w, rest, atol=1e-12)


def test_verification_keeps_the_target_distribution():
    # drafts from q, two siblings a node: the first token out follows p whatever q is
    rng = np.random.default_rng(3)
    v, runs = 4, 40_000
    p, q = np.array([0.1, 0.2, 0.3, 0.4]), np.array([0.4, 0.4, 0.1, 0.1])
    target, draft = np.tile(p, (3, 1)), np.tile(q, (3, 1))
    got = np.zeros(v)
    toks, us = rng.choice(v, size=(runs, 3), p=q), rng.random((runs, 4))
    for i in range(runs):
        _, t, _ = step.verify(target, draft, toks[i], [-1, 0, 0], [0, 3], us[i, :3], us[i, 3:], 3)
        got[t[0, 0]] += 1
    # 5 standard deviations of a count
    assert np.all(np.abs(got - runs * p) < 5 * np.sqrt(runs * p * (1 - p)))
