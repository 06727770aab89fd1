"""The example that serves, forks and releases requests: every stage of its steps against the oracle.

Rows in the caches, codes, counts, lengths, tables and the free list are equal
in every entry; normed rows and probabilities within the tolerances that the
tests of their calls derive.
"""

import importlib.util
import os

import numpy as np
import pytest
import torch

from test_gpu_norm_rope import bound

from oracle import serve, step

pytestmark = pytest.mark.gpu


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_steps.py")
    spec = importlib.util.spec_from_file_location("serve_steps", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def np_(t):
    return t.cpu().numpy()


def wide(t):
    return t.double().cpu().numpy()


def as_bytes(c):
    return c.contiguous().view(torch.uint8).cpu().numpy()


def check_step(ex, s):
    s.draw()
    n, t = s.active, s.active * ex.DRAFTS
    ctx = np_(s.ctx[:n])
    s.attend()
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    slots, pos, freq = s.slots[:t], np_(s.positions[:t]), np_(s.freq)
    rows = s.cache.flatten(1, 2)
    eps = float(np.float32(s.eps))
    for x, w, got in ((s.q[:t], s.q_weight, s.q_turned[:t]), (s.k[:t], s.k_weight, rows[0][slots])):
        normed = serve.norm_rotate(wide(x), wide(w), eps, 0.0, pos, freq[:0], 1.0, False)
        want = step.rotate(normed, pos, freq, 1.0, False)
        assert (np.abs(wide(got) - want) <= bound(normed, want, len(freq), False, 1.0, x.dtype)).all()
    assert torch.equal(rows[1][slots], s.v[:t])
    codes, scales = serve.index_queries(wide(s.index_rows[:t, : ex.LISTS]), wide(s.iq_weight), eps, 0.0, pos, freq, 1.0, False, 128**-0.5, None)
    assert np.array_equal(np_(s.index_q[:n]).reshape(codes.shape) & 0x7F, codes & 0x7F)
    assert np.all(np.abs(wide(s.index_scale[:n]).reshape(scales.shape) - scales) <= 32 * 2.0**-24 * scales)
    code, scale = serve.index_keys(wide(s.index_rows[:t, ex.LISTS]), wide(s.ik_weight), eps, 0.0, pos, freq, 1.0, False)
    flat = s.index_k.view(s.blocks, -1)
    b, o = slots // ex.PAGE, slots % ex.PAGE
    got = flat[b[:, None], o[:, None] * 64 + torch.arange(64, device="cuda")]
    assert np.array_equal(np_(got) & 0x77, code & 0x77)
    assert np.array_equal(np_(flat[b[:, None], 64 * ex.PAGE + o[:, None] * 8 + torch.arange(8, device="cuda")]), scale)
    assert torch.isfinite(s.out[:t]).all()

    counts = np_(s.counts[:n]).copy()
    s.judge()
    torch.cuda.synchronize()
    want, _ = serve.logit_probs(wide(s.logits[:t]), np_(s.cu_).tolist(), np_(s.temperature), np_(s.repetition), np_(s.presence), np_(s.frequency), counts,
                                np_(s.drafted[:t]), np_(s.mask[:t]), None, np_(s.allowed[:t]))
    p = np_(s.target[:t])
    # 4 d + 128 + 12 X / T units of 2^-24 (X, the magnitudes on an entry's way, at most 20; T 0.8)
    d = np.where(want > 0, np.log(want.max(1, keepdims=True)) - np.log(np.where(want > 0, want, 1.0)), 0.0)
    assert np.all(np.abs(p - want) <= want * 2.0**-24 * (4 * d + 128 + 12 * 20 / 0.8) + 2.0**-126)
    acc, toks, nodes = step.verify(p, np_(s.draft[:t]), np_(s.drafted[:t]), np_(s.parents[:t]), np_(s.cu_), np_(s.accept_u[:t]), np_(s.sample_u[:n]),
                                   ex.DRAFTS)
    assert np.array_equal(np_(s.accepted[:n]), acc) and np.array_equal(np_(s.out_tokens[:n]), toks) and np.array_equal(np_(s.out_nodes[:n]), nodes)

    before = [as_bytes(c) for c in s.caches]
    s.settle()
    torch.cuda.synchronize()
    caches, ctx_out, counted = serve.settle(before, np_(slots), np_(s.cu_), toks, nodes, acc, ctx, counts)
    for c, w in zip(s.caches, caches):
        assert np.array_equal(as_bytes(c), w)
    assert np.array_equal(np_(s.ctx[:n]), ctx_out) and np.array_equal(np_(s.counts[:n]), counted)
    assert int(s.status.item()) == 0


def test_steps_forks_and_releases(lib):
    ex = load()
    s = ex.Server(9, 700, q_heads=8, kv_heads=4, vocab=2003)
    s.admit(5, 500)
    for _ in range(2):
        check_step(ex, s)
    before = [as_bytes(c) for c in s.caches], np_(s.ctx), np_(s.owned), np_(s.table), np_(s.refs), int(s.cursor.item())
    s.fork([0, 3, 0])
    want = serve.fork(before[0], [0, 3, 0], [5, 6, 7], *before[1:5], np_(s.free), before[5], ex.PAGE, s.blocks)
    for c, w in zip(s.caches, want[0]):
        assert np.array_equal(as_bytes(c), w)
    for got, w in zip((s.ctx, s.owned, s.table, s.refs), want[1:5]):
        assert np.array_equal(np_(got), w)
    assert int(s.cursor.item()) == want[5] and s.active == 8
    for _ in range(2):
        check_step(ex, s)
    keep = np_(s.ctx[:8]).tolist()
    keep[2], keep[6], keep[7] = 130, 0, 0  # one cut back, two ended
    want = serve.release(np.array(keep + [0]), np_(s.owned), np_(s.table), np_(s.refs), np_(s.free), int(s.cursor.item()), ex.PAGE)
    s.release(keep)
    for got, w in zip((s.refs, s.free, s.owned), (want[0], want[1], want[3])):
        assert np.array_equal(np_(got), w)
    assert int(s.cursor.item()) == want[2] and s.active == 6
    check_step(ex, s)
    s.release([0] * s.active)
    torch.cuda.synchronize()
    assert int(s.cursor.item()) == 0 and not s.refs.any() and int(s.status.item()) == 0
    assert torch.equal(s.free.sort().values, torch.arange(s.blocks, dtype=torch.int32, device="cuda"))


def test_a_captured_step_is_the_same(lib):
    ex = load()
    servers = [ex.Server(4, 600, q_heads=8, kv_heads=4, vocab=1000, seed=3) for _ in range(2)]
    for s in servers:
        s.admit(4, 300)
        s.draw()
        s.step()
    s, other = servers
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    for _ in range(3):
        for x in servers:
            x.draw()
        graph.replay()
        other.step()
    torch.cuda.synchronize()
    for name in ("ctx", "table", "counts", "cache", "index_k", "target", "out_tokens", "accepted", "cursor", "pages", "out"):
        assert torch.equal(getattr(s, name), getattr(other, name)), name


def test_the_program_runs(lib, capsys, monkeypatch):
    ex = load()
    monkeypatch.setattr("sys.argv", ["serve_steps.py", "--reqs", "6", "--forks", "2", "--context", "1000", "--steps", "3"])
    ex.main()
    assert "free again" in capsys.readouterr().out
