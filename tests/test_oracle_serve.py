"""The oracle of the calls between a decoding step's own, against brute force and closed forms."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import formats, serve


def test_norm_rotate():
    r = np.random.default_rng(0)
    x, w, f = r.normal(size=(3, 2, 6)), r.normal(size=6), np.array([0.7, 0.01])
    got = serve.norm_rotate(x, w, 1e-3, 1.0, np.array([0, 5, 7]), f, 1.0, False)
    for t, pos in enumerate((0, 5, 7)):
        for h in range(2):
            n = (1.0 + w) * x[t, h] / np.sqrt((x[t, h] ** 2).sum() / 6 + 1e-3)
            z = [(n[i] + 1j * n[i + 2]) * np.exp(1j * pos * f[i]) for i in range(2)]
            np.testing.assert_allclose(got[t, h], [z[0].real, z[1].real, z[0].imag, z[1].imag, n[4], n[5]], rtol=1e-13)
    assert np.array_equal(serve.norm_rotate(x, None, 0.0, 0.0, np.zeros(3), f, 1.0, True), x)


def test_nearest_code():
    x = np.random.default_rng(1).normal(size=3000) * 100
    assert np.array_equal(serve.nearest_code(x, serve.E4M3), [formats.e4m3_encode_rational(v) for v in x])
    # halves go to the even code, in both formats
    for values in (serve.E4M3, serve.E2M1):
        for c in range(len(values) - 1):
            assert serve.nearest_code((values[c] + values[c + 1]) / 2, values) == c + c % 2
    assert serve.nearest_code(-5.1, serve.E2M1) == 15 and serve.nearest_code(1e9, serve.E2M1) == 7


def test_index_rows():
    r = np.random.default_rng(2)
    q = r.normal(size=(2, 1, 128))
    codes, s = serve.index_queries(q, None, 0.0, 0.0, np.zeros(2), np.zeros(0), 1.0, False, 0.5, np.array([[2.0], [4.0]]))
    np.testing.assert_allclose(s[:, 0], np.abs(q[:, 0]).max(-1) / 448 * 0.5 * [2.0, 4.0], rtol=1e-14)
    for t in range(2):
        top = np.abs(q[t, 0]).max()
        assert [int(c) for c in codes[t, 0]] == [formats.e4m3_encode_rational(Fraction(float(v)) * 448 / Fraction(float(top))) for v in q[t, 0]]
    k = r.normal(size=(2, 128))
    k[1, 16:32] = 0.0
    code, scale = serve.index_keys(k, None, 0.0, 0.0, np.zeros(2), np.zeros(0), 1.0, False)
    assert scale[1, 1] == 0 and not code[1, 8:16].any()
    for t in range(2):
        for b in range(8):
            sv = formats.e4m3_value(int(scale[t, b]))
            assert int(scale[t, b]) == formats.e4m3_encode_rational(np.abs(k[t, 16 * b : 16 * b + 16]).max() / 6)
            for i in range(16):
                c = int(code[t, 8 * b + i // 2]) >> (4 * (i % 2)) & 15
                value = serve.E2M1[c & 7] * (-1 if c & 8 else 1) * sv
                assert abs(value - k[t, 16 * b + i]) <= min(abs(v * s * sv - k[t, 16 * b + i]) for v in serve.E2M1 for s in (1, -1)) + 1e-12


def test_logit_probs():
    logits = np.array([[2.0, -1.0, 0.5, 3.0], [1.0, 1.0, 0.0, 1.0]])
    counts = np.array([[2, 0, 0, 0]], dtype=np.int32)
    counts[0, 1] = -(2**31)  # in the prompt
    kw = dict(repetition=np.array([2.0]), presence=np.array([0.25]), frequency=np.array([0.5]), counts=counts, temperature=np.array([0.5]))
    p, lse = serve.logit_probs(logits[:1], [0, 1], **kw)
    x = np.array([2.0 / 2 - (0.5 * 2 + 0.25), -1.0 * 2, 0.5, 3.0]) / 0.5
    np.testing.assert_allclose(p[0], np.exp(x) / np.exp(x).sum(), rtol=1e-14)
    assert abs(lse[0] - np.log(np.exp(x).sum())) < 1e-13
    # a chain: node 1's row counts its own token too; a mask of the grammar; a bias
    p, _ = serve.logit_probs(logits, [0, 2], tokens=np.array([3, 2]), biases=[[(1, 1.5)]], allowed=np.array([[15], [7]], dtype=np.int32), **kw)
    x = np.array([1.0 / 2 - 1.25, 1.0 / 2 + 1.5, 0.0 * 2 - (0.5 + 0.25), -np.inf]) / 0.5
    np.testing.assert_allclose(p[1], np.exp(x) / np.exp(x).sum(), rtol=1e-14)
    # the lowest of equal ones; nothing allowed
    p, lse = serve.logit_probs(logits, [0, 2], temperature=np.array([0.0]), allowed=np.array([[0], [14]], dtype=np.int32))
    assert not p[0].any() and lse[0] == -np.inf and list(p[1]) == [0, 1, 0, 0] and lse[1] == 1.0


def test_settle():
    cache = np.arange(2 * 3 * 4 * 2.0).reshape(2, 3, 4, 2)
    slots = np.array([5, 6, 7, 8, 9])  # places in blocks 1 and 2
    new, ctx, counts = serve.settle([cache], slots, [0, 5], np.array([[1, 1, 2, -1]]), np.array([[2, 4, -1, -1]]), [2], np.array([10]),
                                    np.zeros((1, 3), dtype=np.int32))
    rows, old = new[0].reshape(2, 12, 2), cache.reshape(2, 12, 2)
    assert np.array_equal(rows[:, 6], old[:, 7]) and np.array_equal(rows[:, 7], old[:, 9])
    assert np.array_equal(np.delete(rows, [6, 7], 1), np.delete(old, [6, 7], 1))
    assert ctx[0] == 13 and list(counts[0]) == [0, 2, 1]


def test_a_place_without_a_fork_names_no_parent():
    ctx, owned, table = np.array([6, 0, 0]), np.array([2, 0, 0]), np.array([[3, 1], [-1, -1], [-1, -1]])
    _, ctx, owned, table, refs, cursor, status = serve.fork([], [0, 1], [1, -1], ctx, owned, table, np.zeros(5, dtype=np.int32), np.array([0, 2, 4]), 0, 4, 5)
    assert status == 0 and list(ctx) == [6, 6, 0] and list(owned) == [2, 2, 0] and list(table[1]) == [3, 0] and list(refs) == [0, 0, 0, 1, 0] and cursor == 1


@pytest.mark.parametrize("seed", range(4))
def test_forks_and_releases_balance(seed):
    """Random forks, then everything released: every block comes back once."""
    r = np.random.default_rng(seed)
    page, blocks, reqs, width = 4, 60, 8, 6
    perm = r.permutation(blocks)
    ctx, owned = np.zeros(reqs, dtype=np.int64), np.zeros(reqs, dtype=np.int64)
    table = np.full((reqs, width), -1)
    cursor = 0
    for p in range(3):
        ctx[p] = r.integers(0, width * page + 1)
        owned[p] = -(-ctx[p] // page)
        table[p, : owned[p]] = perm[cursor : cursor + owned[p]]
        cursor += owned[p]
    cache = r.normal(size=(1, blocks, page, 1))
    refs = np.zeros(blocks, dtype=np.int32)
    (cache2,), ctx, owned, table, refs, cursor, status = serve.fork([cache], [0, 1, 2, 0, 2], [3, 4, 5, 6, 7], ctx, owned, table, refs, perm, cursor, page, blocks)
    assert status == 0
    for c, p in ((3, 0), (4, 1), (5, 2), (6, 0), (7, 2)):
        for i in range(ctx[p]):
            assert cache2[0, table[c, i // page], i % page] == cache[0, table[p, i // page], i % page]
    refs, free, cursor, kept, status = serve.release(np.zeros(reqs), owned, table, refs, perm.copy(), cursor, page)
    assert status == 0 and cursor == 0 and not refs.any() and not kept.any()
    assert sorted(free) == list(range(blocks))
