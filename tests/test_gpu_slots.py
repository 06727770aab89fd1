"""idx_build_slots against its definition: whole numbers, equal in every entry."""

import numpy as np
import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu


def case(seed, reqs, new_hi, ctx_hi, page, tree, extra_owned=1, short=0, cap=None, width_cut=0):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_hi + 1, reqs)
    new = rng.integers(0, new_hi + 1, reqs)
    need = -(-(ctx + new) // page)
    owned = np.minimum(need + 1, -(-ctx // page) + rng.integers(0, extra_owned + 1, reqs))
    width = max(1, int(max(need.max(initial=0), owned.max(initial=0))) - width_cut)
    owned = np.minimum(owned, width)
    blocks = int(np.maximum(need, owned).sum()) + 5
    ids = rng.permutation(blocks).astype(np.int32)
    table = np.full((reqs, width), -1, dtype=np.int32)
    at = 0
    for r in range(reqs):
        table[r, : owned[r]] = ids[at : at + owned[r]]
        at += owned[r]
    free = ids[at : len(ids) - short] if short < len(ids) - at else ids[:0]
    total = int(new.sum())
    cap = total + 3 if cap is None else cap
    parents = None
    if tree:
        parents = np.full(cap, -1, dtype=np.int32)
        t = 0
        for m in new:
            for i in range(m):
                if t + i < cap:
                    parents[t + i] = rng.integers(-1, i) if i else -1
            t += m
    return dict(ctx=ctx.astype(np.int32), new=new.astype(np.int32), owned=owned.astype(np.int32), table=table, free=free,
                blocks=blocks, page=page, cap=cap, parents=parents, cursor=1 if len(free) > 2 else 0)


def run(lib, c):
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    reqs, cap = len(c["ctx"]), c["cap"]
    e = lambda n, t=torch.int32: torch.full((n,), -77, dtype=t, device="cuda")
    o = dict(block_table=d(c["table"]), cu_tokens=e(reqs + 1), seq_lens=e(reqs), pages_out=e(reqs), cursor_out=e(1), positions=e(cap),
             slots=e(cap, torch.int64), tree_mask=e(cap, torch.int64) if c["parents"] is not None else None)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.idx_build_slots(d(c["ctx"]), d(c["new"]), d(c["owned"]), o["block_table"], d(c["free"].astype(np.int32)),
                        d(np.array([c["cursor"]], dtype=np.int32)), c["blocks"], c["page"], o["cu_tokens"], o["seq_lens"],
                        o["pages_out"], o["cursor_out"], o["positions"], o["slots"],
                        parents=None if c["parents"] is None else d(c["parents"]), tree_mask=o["tree_mask"], status=status)
    return o, int(status.item())


def check(lib, c):
    o, status = run(lib, c)
    ref = step.build_slots(c["ctx"], c["new"], c["owned"], c["table"], c["free"], c["cursor"], c["blocks"], c["page"], c["cap"], c["parents"])
    for k, v in o.items():
        if v is None:
            continue
        got = v.cpu().numpy()
        got = got.astype(np.uint64) if k == "tree_mask" else got
        assert np.array_equal(got, np.asarray(ref[k]).reshape(got.shape)), k
    assert status == ref["status"]


@pytest.mark.parametrize("reqs,new_hi,ctx_hi,page,tree", [
    (1, 1, 0, 128, False), (1, 64, 1000, 128, True), (3, 5, 10, 1, True), (64, 8, 172032, 128, True), (37, 300, 500, 16, False),
    (1023, 3, 300, 32, True), (1024, 1, 100, 16, False), (1025, 2, 100, 64, True), (2600, 40, 1000, 256, False), (7, 20000, 9, 24, False),
])
def test_matches_definition(lib, reqs, new_hi, ctx_hi, page, tree):
    check(lib, case(reqs + page, reqs, new_hi, ctx_hi, page, tree))


def test_empty_batches(lib):
    check(lib, case(1, 5, 0, 100, 16, False))  # no tokens at all
    c = case(2, 4, 3, 50, 16, True)
    c.update(ctx=c["ctx"][:0], new=c["new"][:0], owned=c["owned"][:0], table=c["table"][:0])
    check(lib, c)  # no requests: only padding


def test_shortage_of_blocks(lib):
    for short in (1, 7, 10_000):
        check(lib, case(3, 50, 60, 200, 16, False, short=short))


def test_clamped_by_table_and_by_tokens(lib):
    check(lib, case(4, 20, 60, 200, 16, False, width_cut=3))
    check(lib, case(5, 20, 30, 200, 16, True, cap=100))


def test_negative_lengths_and_wide_trees(lib):
    c = case(6, 6, 10, 50, 16, False)
    c["ctx"][2], c["new"][3], c["owned"][4] = -5, -1, -3
    c["cap"] = 200
    check(lib, c)
    check(lib, case(7, 3, 90, 50, 16, True))  # more than 64 nodes
    c = case(8, 3, 20, 50, 16, True)
    c["parents"][::3] = 5  # not always an earlier node
    check(lib, c)


def test_blocks_outside_the_pool(lib):
    c = case(9, 12, 40, 200, 16, False)
    c["free"][::2] = 1 << 20
    c["table"][3, :] = -9
    check(lib, c)


def test_long_context_places(lib):
    # places near 2^31: sums in 64 bits
    c = case(10, 2, 4, 10, 256, False)
    width = 1 << 23
    c.update(ctx=np.array([2**31 - 3, 5], dtype=np.int32), new=np.array([1, 3], dtype=np.int32), owned=np.array([1 << 23, 1], dtype=np.int32))
    o = dict(table=np.full((2, width), 3, dtype=np.int32), blocks=8, cap=6)
    c.update(o)
    got, status = run(lib, c)
    assert got["slots"].tolist()[:4] == [3 * 256 + 253] + [3 * 256 + x for x in (5, 6, 7)] and status == 0
    assert got["positions"].tolist()[0] == 2**31 - 3


def test_steps_in_a_graph_follow_their_inputs(lib):
    """Captured once, replayed with other lengths; the cursor and page counts go from step to step."""
    reqs, page, width = 5, 16, 40
    d = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ctx, new, owned, cur = d([0] * reqs), d([7] * reqs), d([0] * reqs), d([0])
    table = torch.full((reqs, width), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(500, dtype=torch.int32, device="cuda")
    cu, seq, pages, cur2 = d([0] * (reqs + 1)), d([0] * reqs), d([0] * reqs), d([0])
    pos, slots = d([0] * 50), torch.zeros(50, dtype=torch.int64, device="cuda")
    call = lambda: lib.idx_build_slots(ctx, new, owned, table, free, cur, 500, page, cu, seq, pages, cur2, pos, slots)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
            ctx.copy_(seq)
            owned.copy_(pages)
            cur.copy_(cur2)
    torch.cuda.synchronize()
    want_table, want_cur, lens, own = np.full((reqs, width), -1), 0, np.zeros(reqs, int), np.zeros(reqs, int)
    for k in range(4):
        add = np.array([k, 2 * k, 9, 0, 1])
        new.copy_(d(add.tolist()))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        ref = step.build_slots(lens, add, own, want_table, list(range(500)), want_cur, 500, page, 50)
        want_table, want_cur, lens, own = ref["block_table"], ref["cursor_out"], ref["seq_lens"], ref["pages_out"]
        assert np.array_equal(table.cpu().numpy(), want_table) and np.array_equal(slots.cpu().numpy(), ref["slots"])
