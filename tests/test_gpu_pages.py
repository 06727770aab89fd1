"""idx_settle_drafts, idx_fork_pages and idx_release_pages: equal to the oracle in every byte and entry."""

import numpy as np
import pytest
import torch

from oracle import serve

pytestmark = pytest.mark.gpu


def dev(x, kind=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(kind).cuda()


def np_(t):
    return t.cpu().numpy()


ROWS = [((2, 64), torch.bfloat16), ((3, 5), torch.uint8), ((4,), torch.float32), ((1, 7), torch.float16), ((576,), torch.bfloat16), ((2, 3, 8), torch.int64)]


def caches_of(blocks, page, rows, planes=3, layout="plain"):
    """Caches of several row sizes, as bytes compared later; layouts: planes first, blocks before planes, heads before tokens."""
    out = []
    for row, kind in rows:
        shape = (blocks, planes, page, *row) if layout == "blocks" else (planes, blocks, page, *row)
        raw = torch.randint(0, 256, (*shape[:-1], shape[-1] * kind.itemsize), dtype=torch.uint8, device="cuda")
        c = raw.view(kind) if kind != torch.uint8 else raw
        out.append(c.transpose(0, 1) if layout == "blocks" else c)
    return out


def as_bytes(c):
    return c.contiguous().view(torch.uint8).cpu().numpy()


def walk(rng, n):
    """A path through a tree of n nodes: ascending node numbers."""
    return sorted(rng.choice(np.arange(1, n), size=rng.integers(0, n), replace=False).tolist()) if n > 1 else []


class Settle:
    def __init__(self, ns, page=16, rows=ROWS[:3], planes=3, layout="plain", vocab=50, max_out=None, seed=0, paths=None):
        rng = np.random.default_rng(seed)
        self.ns, total = ns, sum(ns)
        blocks = -(-total // page) + 5
        self.caches = caches_of(blocks, page, rows, planes, layout)
        self.slots = rng.permutation(blocks * page)[: max(total, 1)]
        self.cu = np.concatenate([[0], np.cumsum(ns)])
        paths = [walk(rng, n) for n in ns] if paths is None else paths
        self.max_out = max_out or max(max(ns, default=1), 1)
        self.nodes = np.full((len(ns), self.max_out), -1)
        self.accepted = np.zeros(len(ns), dtype=np.int64)
        for r, p in enumerate(paths):
            p = p[: self.max_out - 1]
            self.nodes[r, : len(p)], self.accepted[r] = p, len(p)
        self.tokens = rng.integers(0, vocab, self.nodes.shape)
        self.ctx = rng.integers(0, 1000, len(ns))
        self.counts = rng.integers(0, 4, (len(ns), vocab)).astype(np.int32)
        self.counts[:, ::7] |= -(2**31)

    def check(self, lib, status=0, counts=True):
        want, ctx, cnt = serve.settle([as_bytes(c) for c in self.caches], self.slots, self.cu, self.tokens, self.nodes, self.accepted, self.ctx,
                                      self.counts if counts else None)
        ctx_in = dev(self.ctx)
        ctx_out, cd, st = torch.zeros_like(ctx_in), dev(self.counts) if counts else None, dev([0])
        lib.idx_settle_drafts(self.caches, dev(self.slots, torch.int64), dev(self.cu), dev(self.tokens), dev(self.nodes), dev(self.accepted), ctx_in, ctx_out,
                              counts=cd, status=st)
        assert st.item() == status
        for c, w in zip(self.caches, want):
            assert np.array_equal(as_bytes(c), w)
        assert np.array_equal(np_(ctx_out), ctx)
        if counts:
            assert np.array_equal(np_(cd), cnt)
        return self


@pytest.mark.parametrize("layout", ["plain", "blocks"])
@pytest.mark.parametrize("row", range(len(ROWS)))
def test_settle_row_sizes(lib, row, layout):
    Settle([5, 1, 8, 0, 3], rows=[ROWS[row]], layout=layout, seed=row).check(lib)


@pytest.mark.parametrize("ns", [[1], [0], [2, 0, 0, 9], [64] * 3, [300, 5], [8] * 700, []])
def test_settle_sizes(lib, ns):
    Settle(ns, page=16, rows=ROWS[:2], seed=len(ns)).check(lib)


def test_settle_long_paths_overwrite_nothing_unread(lib):
    Settle([200, 130], paths=[list(range(2, 200, 1))[:150], list(range(1, 130))], seed=1).check(lib)  # every row one place on; every row at its place
    Settle([200], paths=[list(range(3, 200, 2))], seed=2).check(lib)


def test_settle_without_caches_or_counts(lib):
    s = Settle([4, 4])
    s.check(lib, counts=False)
    s.caches = []
    s.check(lib)


def test_settle_bad_nodes_and_slots(lib):
    s = Settle([6, 6, 6, 6], paths=[[2, 4], [1, 3, 5], [2, 3], [3, 4, 5]])
    s.nodes[0, 1], s.nodes[1, 1] = 6, 1  # past the request's end; before its place
    s.check(lib, status=lib.ST_BAD_TREE)
    s = Settle([6, 6], paths=[[2, 4], [3, 5]])
    s.slots[4], s.slots[6 + 1] = -1, -1  # a source and a target without a slot
    s.check(lib)
    s = Settle([6, 6], paths=[[2, 4], [3, 5]])
    s.slots[2] = 10**9
    s.check(lib, status=lib.ST_BLOCK_OOR)
    s = Settle([4, 3], paths=[[1, 2, 3], [2]], max_out=7)
    s.accepted[:] = [9, -3]  # more than there are; fewer than none
    s.check(lib)
    s = Settle([4], paths=[[2, 3]])
    s.tokens[0, :2] = [-1, 50]  # tokens outside the vocabulary are not counted
    s.check(lib)


def test_settle_in_place_context_and_index_pages(lib):
    pages = torch.randint(0, 256, (6, 128, 72), dtype=torch.uint8, device="cuda")
    flat = pages.flatten(1).clone()
    slots = torch.tensor([126, 127, 128, 300, 301], device="cuda")
    ctx = dev([40])
    lib.idx_settle_drafts(lib.index_caches(pages), slots, dev([0, 5]), dev([[1, 1, 1]]), dev([[2, 4, -1]]), dev([2]), ctx, ctx)
    want = flat.clone()
    for src, dst in ((128, 127), (301, 128)):
        (b, o), (c, p) = divmod(src, 128), divmod(dst, 128)
        want[c, p * 64 : p * 64 + 64], want[c, 8192 + p * 8 : 8192 + p * 8 + 8] = flat[b, o * 64 : o * 64 + 64], flat[b, 8192 + o * 8 : 8192 + o * 8 + 8]
    assert torch.equal(pages.flatten(1), want) and ctx.item() == 43


def test_settle_offsets_past_32_bits(lib):
    """Planes that lie more than 4 GB apart."""
    raw = torch.zeros(3, 300, 128, 57600, dtype=torch.uint8, device="cuda")  # 6.6 GB
    raw[2, 299, 126:], raw[1, 298, 5] = 7, 9
    slots = torch.tensor([0, 299 * 128 + 1, 299 * 128 + 127, 298 * 128 + 5], device="cuda")
    ctx = dev([0])
    lib.idx_settle_drafts([raw], slots, dev([0, 4]), dev([[1, 1, 1]]), dev([[2, 3, -1]]), dev([2]), ctx, ctx)
    assert raw[2, 299, 1].eq(7).all() and not raw[0, 299, 1].any() and raw[1, 299, 127].eq(9).all() and not raw[2, 299, 127].any()
    del raw
    torch.cuda.empty_cache()


class Pool:
    """Requests with pages, some shared already."""

    def __init__(self, lens, page=4, width=12, extra=20, rows=ROWS[:2], planes=2, reqs=None, seed=0, free=None):
        rng = np.random.default_rng(seed)
        reqs = reqs or len(lens) * 2
        self.page = page
        self.ctx, self.owned = np.zeros(reqs, dtype=np.int64), np.zeros(reqs, dtype=np.int64)
        need = [-(-n // page) for n in lens]
        blocks = sum(need) + extra
        perm = rng.permutation(blocks)
        self.table = rng.integers(0, blocks, (reqs, width))
        at = 0
        for r, n in enumerate(lens):
            self.ctx[r], self.owned[r] = n, need[r]
            self.table[r, : need[r]] = perm[at : at + need[r]]
            at += need[r]
        self.free, self.cursor, self.blocks = perm[: at + (extra if free is None else free)].copy(), at, blocks
        self.refs = np.zeros(blocks, dtype=np.int32)
        self.caches = caches_of(blocks, page, rows, planes)

    def fork(self, lib, parents, children, status=0):
        want = serve.fork([as_bytes(c) for c in self.caches], parents, children, self.ctx, self.owned, self.table, self.refs, self.free, self.cursor, self.page,
                          self.blocks)
        ctx, owned, table, refs, st, out = dev(self.ctx), dev(self.owned), dev(self.table), dev(self.refs), dev([0]), dev([-5])
        lib.idx_fork_pages(self.caches, dev(parents), dev(children), ctx, owned, table, refs, dev(self.free), dev([self.cursor]), out,
                           page_tokens=self.page, status=st)
        assert st.item() == want[6] == status
        for c, w in zip(self.caches, want[0]):
            assert np.array_equal(as_bytes(c), w)
        for got, w in zip((ctx, owned, table, refs), want[1:5]):
            assert np.array_equal(np_(got), w)
        assert out.item() == want[5]
        _, self.ctx, self.owned, self.table, self.refs, self.cursor, _ = want
        return self

    def release(self, lib, keep, status=0):
        want = serve.release(keep, self.owned, self.table, self.refs, self.free, self.cursor, self.page)
        refs, free, st, out = dev(self.refs), dev(self.free), dev([0]), dev([-5])
        pages = torch.zeros(len(keep), dtype=torch.int32, device="cuda")
        lib.idx_release_pages(dev(keep), dev(self.owned), dev(self.table), refs, free, dev([self.cursor]), out, pages, self.page, status=st)
        assert st.item() == want[4] == status
        assert np.array_equal(np_(refs), want[0]) and np.array_equal(np_(free), want[1]) and out.item() == want[2] and np.array_equal(np_(pages), want[3])
        self.refs, self.free, self.cursor, self.owned, _ = want
        return self


@pytest.mark.parametrize("page", [1, 4, 16, 128])
def test_forks_then_releases(lib, page):
    p = Pool([3 * page + 1, 2 * page, 0, 1, 5 * page - 1], page=page, seed=page)
    p.fork(lib, [0, 0, 1, 2, 4], [5, 6, 7, 8, 9])
    keep = p.ctx.copy()
    keep[[0, 5, 4]], keep[9] = 0, page
    p.release(lib, keep)
    p.release(lib, np.zeros(len(keep), dtype=np.int64))
    assert p.cursor == 0 and not p.refs.any() and sorted(p.free[: p.blocks]) == sorted(set(p.free))


@pytest.mark.parametrize("row", range(len(ROWS)))
def test_fork_row_sizes(lib, row):
    Pool([9, 14, 3], rows=[ROWS[row]], seed=row).fork(lib, [0, 1, 2], [3, 4, 5])


def test_fork_many(lib):
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 47, 300).tolist()
    p = Pool(lens, extra=2000, reqs=1300, rows=ROWS[1:2], planes=1)
    p.fork(lib, rng.integers(0, 300, 1000), rng.permutation(np.arange(300, 1300)))
    p.release(lib, rng.integers(-3, 47, 1300))
    p.release(lib, np.zeros(1300, dtype=np.int64))
    assert p.cursor == 0


def test_fork_without_room(lib):
    p = Pool([5, 6, 8, 7], free=2, reqs=9)
    p.fork(lib, [0, 2, 1, 3, 0], [4, 5, 6, 7, 8], status=lib.ST_NO_BLOCKS)  # whole pages need no block
    assert p.owned[5] == 2 and p.owned[7] == p.owned[8] == 0


def test_forks_that_are_refused(lib):
    for parents, children in (([0, 1], [4, 4]), ([0, 4], [4, 5]), ([0], [0]), ([-1, 0], [4, 5]), ([0, 1], [4, 6]), ([6, 0], [4, 5]), ([0, 1, 2], [-2, 4, 5])):
        Pool([5, 6, 7], reqs=6).fork(lib, parents, children, status=lib.ST_BAD_FORK)


def test_forks_that_are_none(lib):
    """Empty places of a call, and a call of none: the cursor is passed on."""
    Pool([5, 6, 7], reqs=6).fork(lib, [0, 7, 2], [3, -1, 5])
    Pool([5, 6, 7], reqs=6).fork(lib, [0], [-1])
    p = Pool([5, 6, 7], reqs=6)
    p.fork(lib, [0, 4, -9], [4, -1, -1])  # whatever the parent there
    assert p.owned[4] == p.owned[0] > 0
    Pool([5, 6, 7], reqs=6).fork(lib, np.zeros(0, dtype=np.int32), np.zeros(0, dtype=np.int32))


def test_fork_of_bad_tables(lib):
    p = Pool([9, 6])
    p.table[0, 1], p.table[1, 1] = -1, 10**6
    p.fork(lib, [0, 1], [2, 3], status=lib.ST_BLOCK_OOR)
    p = Pool([9, 6])
    p.ctx[0] = 100  # more than its pages hold
    p.fork(lib, [0, 1], [2, 3], status=lib.ST_LEN_CLAMPED)


def test_fork_without_caches(lib):
    p = Pool([9, 6, 0], rows=[])
    p.fork(lib, [0, 1, 2], [3, 4, 5])


def test_release_sizes(lib):
    Pool([0, 0, 0]).release(lib, np.zeros(6, dtype=np.int64))
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 3000, 50).tolist()
    p = Pool(lens, width=800, extra=70_000, rows=[], free=10)
    p.release(lib, np.maximum(0, np.concatenate([lens, lens]) - rng.integers(0, 2000, 100)))
    p.release(lib, np.zeros(100, dtype=np.int64))
    assert p.cursor == 0


def test_release_with_bad_entries(lib):
    p = Pool([9, 6, 12])
    p.table[0, 2], p.table[1, 0] = -1, 10**6
    p.release(lib, np.zeros(6, dtype=np.int64), status=lib.ST_BLOCK_OOR)
    p = Pool([9, 6], width=3)
    p.owned[1] = 50  # more than the table is wide
    p.table[1, 2] = -1
    p.release(lib, np.zeros(4, dtype=np.int64))


def test_a_block_released_twice_goes_back_once(lib):
    p = Pool([8, 8])
    p.table[1, :2] = p.table[0, :2]  # the same pages, not counted as shared
    p.release(lib, np.zeros(4, dtype=np.int64))


def test_release_of_more_than_was_taken(lib):
    p = Pool([8, 8])
    p.cursor = 2
    p.release(lib, np.zeros(4, dtype=np.int64), status=lib.ST_BAD_OUTPUT)


def test_graphs_and_streams(lib):
    """Fork, settle and release captured into one graph on another stream's pool, replayed twice."""
    p = Pool([9, 14, 3], reqs=6)
    ctx, owned, table, refs, free = dev(p.ctx), dev(p.owned), dev(p.table), dev(p.refs), dev(p.free)
    cur, out, back, pages, keep = dev([p.cursor]), dev([0]), dev([0]), torch.zeros(6, dtype=torch.int32, device="cuda"), dev([9, 14, 3, 0, 0, 0])
    parents, children, st = dev([0, 1, 2]), dev([3, 4, 5]), dev([0])

    def steps():
        lib.idx_fork_pages(p.caches, parents, children, ctx, owned, table, refs, free, cur, out, status=st)
        lib.idx_release_pages(keep, owned, table, refs, free, out, back, pages, p.page, status=st)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        steps()
    s.synchronize()
    first = [x.clone() for x in (ctx, owned, table, refs, free, back, pages)]
    assert st.item() == 0 and back.item() == p.cursor and not refs.any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert st.item() == 0 and back.item() == p.cursor and not refs.any()
        assert torch.equal(pages, first[6]) and torch.equal(ctx, first[0]) and torch.equal(owned, first[1])
