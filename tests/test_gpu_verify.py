"""idx_verify_drafts against its definition: tokens and nodes equal in every entry."""

import numpy as np
import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu


def make(seed, counts, vocab, tree, with_draft, spread=3.0, near=0.8, pad=0):
    rng = np.random.default_rng(seed)
    tokens = int(sum(counts))
    logits = rng.standard_normal((tokens, vocab)) * spread
    soft = lambda x: (np.exp(x - x.max(1, keepdims=True)) / np.exp(x - x.max(1, keepdims=True)).sum(1, keepdims=True)).astype(np.float32)
    target = soft(logits)
    draft = soft(logits + near * rng.standard_normal((tokens, vocab))) if with_draft else None
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    parents = np.full(tokens, -1, dtype=np.int32)
    toks = np.zeros(tokens, dtype=np.int32)
    for r, n in enumerate(counts):
        for i in range(1, n):
            parents[cu[r] + i] = max(0, i - 1 - int(rng.random() * min(i, 4))) if tree else i - 1
            src = (draft if with_draft else target)[cu[r] + parents[cu[r] + i]].astype(np.float64)
            toks[cu[r] + i] = rng.choice(vocab, p=src / src.sum())
    c = dict(target=target, draft=draft, tokens=toks, parents=parents if tree else None, cu=cu,
             accept=rng.random(tokens, dtype=np.float32), sample=rng.random(len(counts), dtype=np.float32), pad=pad)
    return c


def run(lib, c, max_out):
    d = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()

    def rows(x):  # rows with `pad` columns behind them
        if x is None:
            return None
        w = torch.full((x.shape[0], x.shape[1] + c["pad"]), float("nan"), device="cuda")
        w[:, : x.shape[1]] = d(x)
        return w[:, : x.shape[1]]

    reqs = len(c["cu"]) - 1
    e = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")
    acc, out_t, out_n = e(reqs), e(reqs, max_out), e(reqs, max_out)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.idx_verify_drafts(rows(c["target"]), rows(c["draft"]), d(c["tokens"]), d(c["cu"]), d(c["accept"]), d(c["sample"]), out_t, out_n,
                          acc, parents=d(c["parents"]), status=status)
    torch.cuda.synchronize()
    return acc.cpu().numpy(), out_t.cpu().numpy(), out_n.cpu().numpy(), int(status.item())


def check(lib, c, max_out, status=0):
    got = run(lib, c, max_out)
    want = step.verify(c["target"], c["draft"], c["tokens"], c["parents"], c["cu"], c["accept"], c["sample"], max_out)
    for g, w in zip(got, want):
        assert np.array_equal(g, w), np.argwhere(g != w)[:5]
    assert got[3] == status
    return got


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("vocab", [1, 2, 31, 1000, 4097, 50_001])
def test_matches_definition(lib, vocab, tree, with_draft):
    check(lib, make(vocab + tree, [5, 1, 8, 3, 0, 2, 8, 8], vocab, tree, with_draft), 8)


@pytest.mark.parametrize("with_draft", [True, False])
def test_far_drafts_refuse_many_siblings(lib, with_draft):
    for seed in range(6):
        check(lib, make(seed, [30] * 12, 700, True, with_draft, near=3.0), 30)


def test_short_outputs_stop_the_walk(lib):
    for max_out in (1, 2, 3):
        check(lib, make(1, [9] * 20, 300, True, True, near=0.1), max_out)
        check(lib, make(2, [9] * 20, 300, False, False, spread=12.0), max_out)


def test_many_requests(lib):
    check(lib, make(3, [3] * 700, 501, False, True), 3)


def test_row_strides(lib):
    for pad in (1, 3, 8):
        c = make(4, [6] * 9, 1003, True, True)
        c["pad"] = pad
        check(lib, c, 6)


def test_one_hot_rows_are_greedy(lib):
    c = make(5, [6] * 10, 400, False, False)
    best = c["target"].argmax(1)
    c["target"] = np.eye(400, dtype=np.float32)[best]
    cu = c["cu"]
    for r in range(10):  # the first r tokens follow the target
        for i in range(1, 6):
            c["tokens"][cu[r] + i] = best[cu[r] + i - 1] if i <= r else (best[cu[r] + i - 1] + 1) % 400
    acc, out_t, _, _ = check(lib, c, 6)
    assert acc.tolist() == [min(r, 5) for r in range(10)]


def test_same_rows_accept_everything(lib):
    c = make(6, [7] * 20, 900, False, True)
    c["draft"] = c["target"].copy()
    acc, *_ = check(lib, c, 7)
    assert (acc == 6).all()


def test_residuals_without_mass(lib):
    """Rows that are no distributions: a draft above the target everywhere, and rows of zeros."""
    c = make(7, [4] * 8, 257, True, True)
    c["draft"] = c["target"] * 2
    c["accept"][:] = 0.75
    check(lib, c, 4)
    c["target"][:] = 0
    _, out_t, _, _ = check(lib, c, 4)
    assert (out_t[:, 0] == 256).all()


def test_bad_entries_and_tokens(lib):
    c = make(8, [8] * 12, 300, True, True)
    c["target"][:, ::7] = np.nan
    c["target"][:, 3::11] = -1
    c["tokens"][::5] = 300
    c["tokens"][2::9] = -1
    c["parents"][4::13] = 7
    c["parents"][5::17] = -3
    check(lib, c, 8)


def test_random_numbers_at_the_ends(lib):
    c = make(9, [5] * 16, 333, True, True)
    c["accept"][::2], c["accept"][1::2] = 0.0, np.float32(1 - 2**-24)
    c["sample"][::2], c["sample"][1::2] = 0.0, np.float32(1 - 2**-24)
    check(lib, c, 5)
    c["target"][:, 0] = c["target"][:, -1] = 0.0  # the draw skips entries without probability
    check(lib, c, 5)


def test_siblings_with_the_same_token(lib):
    c = make(10, [6] * 10, 50, True, False)
    c["parents"] = np.tile(np.array([-1, 0, 0, 0, 0, 0], dtype=np.int32), 10)
    c["tokens"][:] = np.tile(np.array([0, 7, 7, 9, 7, 9], dtype=np.int32), 10)
    c["accept"][:] = 0.99
    check(lib, c, 6)


def test_more_nodes_than_are_tried(lib):
    c = make(11, [1500, 4], 40, False, False, spread=30.0)
    c["accept"][:] = 0.0
    acc, _, _, st = run(lib, c, 1600)
    assert acc[0] <= 1023 and st == lib.ST_BAD_TREE


def test_large_vocabulary(lib):
    check(lib, make(12, [4, 2], 262_147, True, True), 4)


def test_graph_and_repeats(lib):
    c = make(13, [6] * 30, 2000, True, True)
    first = check(lib, c, 6)
    for _ in range(4):
        again = run(lib, c, 6)
        assert all(np.array_equal(x, y) for x, y in zip(first[:3], again[:3]))
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    t, q, tok, cu, par, au, su = (d(c[k]) for k in ("target", "draft", "tokens", "cu", "parents", "accept", "sample"))
    e = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")
    acc, out_t, out_n = e(30), e(30, 6), e(30, 6)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        lib.idx_verify_drafts(t, q, tok, cu, au, su, out_t, out_n, acc, parents=par)
    c2 = make(14, [6] * 30, 2000, True, True)
    for dst, key in ((t, "target"), (q, "draft"), (tok, "tokens"), (par, "parents"), (au, "accept"), (su, "sample")):
        dst.copy_(d(c2[key]))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    want = step.verify(c2["target"], c2["draft"], c2["tokens"], c2["parents"], c2["cu"], c2["accept"], c2["sample"], 6)
    assert np.array_equal(acc.cpu().numpy(), want[0]) and np.array_equal(out_t.cpu().numpy(), want[1])
