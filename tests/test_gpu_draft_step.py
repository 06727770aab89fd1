"""The example's decoding steps, every stage against the oracle.

Slots, pages (of the GPU's own scores), verified tokens and moved cache rows
are equal in every entry; turned rows and attention within the tolerances that
the tests of idx_rope_append and idx_tree_attention derive.
"""

import importlib.util
import os

import numpy as np
import pytest
import torch

from test_gpu_rope import bound
from test_gpu_tree_attention import compare

from oracle import step
from oracle.indexer import decode_step

pytestmark = pytest.mark.gpu


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_step.py")
    spec = importlib.util.spec_from_file_location("draft_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def np_(t):
    return t.cpu().numpy()


def state(d):
    return {k: getattr(d, k).clone() for k in ("ctx", "new", "owned", "table", "cursor", "cache")}


def check_step(ex, d, before):
    """Runs a step on d (drawn already) and checks every stage; `before` is its state at the begin."""
    d.attend()
    torch.cuda.synchronize()
    slots = step.build_slots(np_(before["ctx"]), np_(before["new"]), np_(before["owned"]), np_(before["table"]), np_(d.free),
                             int(before["cursor"].item()), d.blocks, ex.PAGE, len(d.positions), np_(d.parents))
    assert slots["status"] == 0 and int(d.status.item()) == 0
    for name, got in (("block_table", d.table), ("cu_tokens", d.cu), ("seq_lens", d.seq), ("pages_out", d.pages_out),
                      ("positions", d.positions), ("slots", d.slots)):
        assert np.array_equal(np_(got), slots[name]), name
    assert np.array_equal(np_(d.mask).view(np.uint64), slots["tree_mask"])
    assert int(d.cursor_out.item()) == slots["cursor_out"]

    freq, half = np_(d.freq), len(d.freq)
    m32 = float(np.float32(d.mscale))
    rows = d.cache.flatten(1, 2)
    for x, got in ((d.q, d.q_turned), (d.k, rows[0][d.slots])):
        x = x.double().cpu().numpy()
        want = step.rotate(x, slots["positions"], freq, m32, False)
        assert (np.abs(got.double().cpu().numpy() - want) <= bound(x, want, half, False, m32, d.q.dtype)).all()
    assert torch.equal(rows[1][d.slots], d.v)

    width = d.scores.shape[-1]
    want, _, _ = decode_step(np_(d.index_q), np_(d.index_scale), np_(d.index_k), slots["block_table"].astype(np.int32),
                             slots["seq_lens"], ex.DRAFTS, width, width, scores=np_(d.scores))
    assert np.array_equal(np_(d.pages), want)

    c = dict(dt=d.q.dtype)
    cache = d.cache.double().cpu().numpy()
    ref = step.tree_attention(d.q_turned.double().cpu().numpy(), cache[0], cache[1], slots["block_table"], slots["seq_lens"],
                              slots["cu_tokens"], d.scale, slots["tree_mask"], np_(d.pages).reshape(len(d.positions), ex.LISTS, ex.PICKED))
    compare(c, d.out, None, ref)

    held = d.cache.clone()
    d.settle()
    torch.cuda.synchronize()
    acc, toks, nodes = step.verify(np_(d.target), np_(d.draft), np_(d.drafted), np_(d.parents), slots["cu_tokens"], np_(d.accept_u),
                                   np_(d.sample_u), ex.DRAFTS)
    assert np.array_equal(np_(d.accepted), acc) and np.array_equal(np_(d.out_tokens), toks) and np.array_equal(np_(d.out_nodes), nodes)
    old = held.flatten(1, 2)
    want = old.clone()
    for r in range(d.reqs):
        for i in range(int(acc[r])):
            want[:, slots["slots"][r * ex.DRAFTS + 1 + i]] = old[:, slots["slots"][r * ex.DRAFTS + int(nodes[r, i])]]
    assert torch.equal(d.cache.flatten(1, 2), want)
    assert np.array_equal(np_(d.ctx), np_(before["ctx"]) + 1 + acc)
    return int(acc.sum())


@pytest.mark.parametrize("reqs,context,heads,dtype", [(3, 2500, (64, 4), torch.bfloat16), (2, 0, (8, 8), torch.float16),
                                                      (5, 1021, (8, 4), torch.bfloat16)])
def test_steps(lib, reqs, context, heads, dtype):
    ex = load()
    d = ex.Decoder(reqs, context, context + 64, q_heads=heads[0], kv_heads=heads[1], vocab=1000, dtype=dtype, seed=reqs)
    for _ in range(3):
        d.draw()
        check_step(ex, d, state(d))


def test_captured(lib):
    """A replayed step gives what the calls give one by one."""
    ex = load()
    made = [ex.Decoder(4, 1500, 1600, q_heads=16, kv_heads=4, vocab=1000, seed=7) for _ in range(2)]
    for d in made:
        for _ in range(2):
            d.draw()
            d.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made[1].step()
    for _ in range(3):
        for d in made:
            d.draw()
        made[0].step()
        graph.replay()
        torch.cuda.synchronize()
        for name in ("out", "pages", "out_tokens", "out_nodes", "accepted", "ctx", "table", "cursor"):
            assert torch.equal(getattr(made[0], name), getattr(made[1], name)), name
        assert torch.equal(made[0].cache, made[1].cache)
    assert int(made[0].status.item()) == 0 and int(made[1].status.item()) == 0
