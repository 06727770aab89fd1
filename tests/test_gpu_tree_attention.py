"""idx_tree_attention against the softmax in 64 bits.

Tolerance, per output element, with A = sum p |v| / sum p and n keys seen:
a score is off by at most ds = 2^-20 * scale * sum |q d| |k d| (fp32 products
and sums of head_dim terms), so a weight by a factor within exp(2 ds), plus
2^-20 for the exponential; a weight is rounded to the type (eps / 2); n + 16
additions in fp32 lose at most 2^-23 each; the quotient is rounded to the type:
    eps / 2 |out| + (eps / 2 + 2 ds + 2^-20 + (n + 16) 2^-23) A (1 + eps)
The logarithm L is off by at most ds + 2^-20 + (n + 16) 2^-23 + 2^-22 |L|.
"""

import numpy as np
import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def make(seed, ctx, new, hq, hk, dim, page, dtype, tree="tree", layout="tokens", blocks_extra=3, q_gap=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = TYPES[dtype]
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    blocks, width = sum(need) + blocks_extra, max(max(need), 1)
    shape = (2, blocks, hk, page, dim) if layout == "heads" else (2, blocks, page, hk, dim)
    cache = torch.randn(shape, device="cuda", generator=g).to(dt)
    if layout == "heads":
        cache = cache.transpose(2, 3)
    table = np.full((len(ctx), width), -1, dtype=np.int32)
    ids = rng.permutation(blocks)
    at = 0
    for r, m in enumerate(need):
        table[r, :m] = ids[at : at + m]
        at += m
    tokens = sum(new)
    q = torch.randn(tokens, hq * dim + q_gap, device="cuda", generator=g).to(dt)[:, : hq * dim].unflatten(1, (hq, dim))
    mask = None
    if tree == "tree":
        mask = np.zeros(tokens, dtype=np.uint64)
        t = 0
        for n in new:
            for i in range(n):
                par = int(rng.integers(-1, i)) if i else -1
                mask[t + i] = np.uint64((1 << i) | (int(mask[t + par]) if par >= 0 else 0)) if i < 64 else np.uint64(0)
            t += n
    elif tree == "random":
        mask = rng.integers(0, 2**64, tokens, dtype=np.uint64)
    return dict(q=q, cache=cache, table=table, seq=np.array([c + n for c, n in zip(ctx, new)], dtype=np.int32),
                cu=np.concatenate([[0], np.cumsum(new)]).astype(np.int32), mask=mask, dt=dt, pages=None, scale=dim**-0.5)


def run(lib, c, out=None, lse=True, stream=None, workspace=None):
    d = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
    q = c["q"]
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda") if out is None else out
    L = torch.full(q.shape[:2], 9.0, device="cuda") if lse else None
    hk = c["cache"].shape[3]
    lists, per = (0, 0) if c["pages"] is None else c["pages"].shape[1:]
    size = lib.idx_tree_attention_workspace_bytes(len(c["seq"]), q.shape[0], q.shape[1], hk, q.shape[2], lists, per)
    ws = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mask = None if c["mask"] is None else d(c["mask"].view(np.int64))
    lib.idx_tree_attention(q, c["cache"][0], c["cache"][1], d(c["table"]), d(c["seq"]), d(c["cu"]), out, c["scale"], tree_mask=mask,
                           pages=d(c["pages"]), lse=L, workspace=ws, status=status, stream=stream)
    torch.cuda.synchronize()
    return out, L, int(status.item())


def reference(c, clean=None):
    cache = c["cache"].double().cpu().numpy() if clean is None else clean
    return step.tree_attention(c["q"].double().cpu().numpy(), cache[0], cache[1], c["table"], c["seq"], c["cu"], c["scale"],
                               c["mask"], c["pages"])


def compare(c, out, L, ref):
    want, lse, mag, big, n = ref
    eps = torch.finfo(c["dt"]).eps
    ds = 2.0**-20 * big
    add = (n[:, None] + 16) * 2.0**-23
    tol = eps / 2 * np.abs(want) + (eps / 2 + 2 * ds + 2.0**-20 + add)[..., None] * mag * (1 + eps)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    err = np.abs(got - want) - tol - float(torch.finfo(c["dt"]).smallest_normal) * eps
    assert err.max() <= 0, (err.max(), np.unravel_index(err.argmax(), err.shape))
    if L is not None:
        gl = L.double().cpu().numpy()
        empty = np.isneginf(lse)
        assert np.array_equal(np.isneginf(gl), empty)
        off = np.abs(gl[~empty] - lse[~empty]) - (ds + 2.0**-20 + add)[~empty] - 2.0**-22 * np.abs(lse[~empty])
        assert off.size == 0 or off.max() <= 0


def check(lib, c, status=0):
    out, L, st = run(lib, c)
    assert st == status
    compare(c, out, L, reference(c))
    return out


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("hq,hk,dim", [(64, 4, 128), (32, 8, 64), (8, 8, 128), (12, 1, 64), (40, 10, 128), (1, 1, 128), (100, 1, 64)])
def test_heads_and_types(lib, dtype, hq, hk, dim):
    check(lib, make(hq + dim, [300, 0, 127, 1000], [8, 3, 1, 11], hq, hk, dim, 128, dtype))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 384])
@pytest.mark.parametrize("dim", [64, 128])
def test_pages(lib, page, dim):
    check(lib, make(page, [page * 2 - 3, 5, page - 1, 700, 2 * page], [6, 1, 2, 9, 1], 16, 2, dim, page, "bf16"))


@pytest.mark.parametrize("ctx,new", [([0], [1]), ([1], [1]), ([127], [1]), ([128], [1]), ([129], [2]), ([0], [64]), ([5000], [1]),
                                     ([100] * 30, [4] * 30), ([0] * 9, [1] * 9), ([4095, 0, 64], [64, 1, 33])])
def test_lengths(lib, ctx, new):
    check(lib, make(sum(ctx) + sum(new), ctx, new, 32, 2, 128, 64, "bf16"))
    check(lib, make(sum(ctx) + sum(new), ctx, new, 6, 2, 64, 128, "fp16", tree="chain"))


@pytest.mark.parametrize("tree", ["random", "chain"])
def test_masks(lib, tree):
    check(lib, make(5, [200, 0, 77], [64, 40, 7], 16, 2, 128, 32, "bf16", tree=tree))


def test_long_chains_are_causal_prompts(lib):
    check(lib, make(6, [0, 300], [400, 131], 8, 2, 64, 16, "bf16", tree="chain"))
    check(lib, make(7, [60], [300], 64, 4, 128, 128, "fp16", tree="chain"))


def test_rows_that_see_nothing(lib):
    c = make(8, [0, 0, 40], [5, 3, 2], 16, 2, 128, 16, "bf16")
    c["mask"][:] = [0, 1, 0, 2, 0, 0, 0, 0, 0, 0]
    out = check(lib, c)
    assert not out[0].any() and not out[5:8].any()
    # requests without tokens, without keys, and a batch of such alone
    c = make(9, [0, 50, 0], [0, 2, 0], 16, 2, 64, 16, "fp16")
    check(lib, c)


def test_large_scores_do_not_overflow(lib):
    c = make(10, [500, 900], [8, 8], 16, 2, 128, 128, "bf16")
    c["q"].mul_(30)
    check(lib, c)
    c["scale"] = -0.2
    check(lib, c)


def test_rising_and_falling_scores(lib):
    """The running maximum moves at every tile, up and down."""
    c = make(11, [2000], [8], 16, 2, 128, 128, "bf16")
    k = c["cache"][0]
    for j, b in enumerate(c["table"][0]):
        k[int(b)] *= 0.2 + (j if j < 8 else 16 - j) * 0.7
    check(lib, c)


def test_what_no_token_sees_has_no_effect(lib):
    """NaN and infinities in unwritten slots, in unused blocks and in drafted tokens that a token does not see."""
    c = make(12, [130, 20, 0], [5, 3, 6], 16, 2, 128, 64, "bf16")
    clean = c["cache"].double().cpu().numpy()
    want = reference(c, clean)
    used = np.zeros(c["cache"].shape[1:3], dtype=bool)
    for r, s in enumerate(c["seq"]):
        for place in range(s):
            used[c["table"][r, place // 64], place % 64] = True
    bad = torch.from_numpy(~used).cuda()
    c["cache"][0][bad] = float("nan")
    c["cache"][1][bad] = float("inf")
    out, L, st = run(lib, c)
    compare(c, out, L, want)
    # a drafted token of a branch: its key and value reach its own branch only
    place = int(c["seq"][0]) - 5 + 3
    b, o = c["table"][0, place // 64], place % 64
    c["cache"][0, b, o, :, :] = float("nan")
    c["cache"][1, b, o, :, 0::2] = float("inf")
    c["cache"][1, b, o, :, 1::2] = float("nan")
    c["mask"][:5] = [1, 3, 5, 8 | 1, 16 | 8 | 1]
    clean2 = clean.copy()
    c2 = dict(c, mask=c["mask"].copy())
    want = step.tree_attention(c["q"].double().cpu().numpy(), clean2[0], clean2[1], c["table"], c["seq"], c["cu"], c["scale"], c["mask"])
    out, L, _ = run(lib, c2)
    touched = [3, 4]
    keep = [i for i in range(out.shape[0]) if i not in touched]
    assert out[touched].isnan().all()
    sub = lambda x: x[keep]
    compare(dict(c), out[keep], L[keep], tuple(sub(x) for x in want))


def test_infinite_values_keep_their_sign(lib):
    c = make(13, [140], [3], 4, 1, 64, 128, "fp16")
    c["mask"][:] = [1, 3, 5]
    b, o = c["table"][0, 141 // 128], 141 % 128  # drafted token 1
    c["cache"][1, b, o, 0, 5], c["cache"][1, b, o, 0, 6] = float("inf"), float("-inf")
    out, _, _ = run(lib, c)
    assert out[1, :, 5].isposinf().all() and out[1, :, 6].isneginf().all()
    out[1, :, 5:7] = 0
    assert out.isfinite().all()


def test_strided_tensors_and_caches(lib):
    check(lib, make(14, [333, 50], [4, 7], 16, 4, 128, 32, "bf16", layout="heads", q_gap=8))
    c = make(15, [333, 50], [4, 7], 16, 4, 64, 128, "fp16")
    wide = torch.zeros(11, 20, 64, device="cuda", dtype=torch.float16)
    out, L, st = run(lib, c, out=wide[:, 2:18])
    compare(c, out, L, reference(c))
    assert not wide[:, :2].any() and not wide[:, 18:].any()


def test_blocks_outside_the_pool_are_not_seen(lib):
    c = make(16, [700, 300], [4, 4], 16, 2, 128, 128, "bf16")
    c["table"][0, 2] = 10_000
    c["table"][1, 0] = -4
    check(lib, c, status=lib.ST_BLOCK_OOR)
    c = make(16, [700, 300], [4, 4], 16, 2, 128, 16, "bf16")
    c["table"][0, 2:9] = 10_000
    c["table"][1, :] = -1
    check(lib, c, status=lib.ST_BLOCK_OOR)


def test_lengths_past_the_table_are_clamped(lib):
    c = make(17, [700], [4], 16, 2, 128, 128, "bf16")
    c["table"] = c["table"][:, :4].copy()
    check(lib, c, status=lib.ST_LEN_CLAMPED)


def lists_of(c, rng, lists, per, page):
    """Random lists: some short, with gaps, repetitions, pages past the request's, and each token's own page at the end."""
    tokens = c["q"].shape[0]
    pages = np.full((tokens, lists, per), -1, dtype=np.int32)
    for r in range(len(c["seq"])):
        used = -(-int(c["seq"][r]) // page)
        n = int(c["cu"][r + 1] - c["cu"][r])
        for i in range(n):
            t = int(c["cu"][r]) + i
            own = (int(c["seq"][r]) - n + i) // page
            for h in range(lists):
                m = int(rng.integers(0, per))
                pages[t, h, :m] = rng.integers(0, used + 2, m)
                if rng.random() < 0.3:
                    pages[t, h, rng.integers(0, per)] = -1
                if rng.random() < 0.9:
                    pages[t, h, per - 1] = own
    return pages


@pytest.mark.parametrize("page", [16, 64, 128, 256])
@pytest.mark.parametrize("hq,hk,lists,dim", [(64, 4, 4, 128), (16, 4, 2, 64), (8, 8, 1, 128)])
def test_chosen_pages(lib, page, hq, hk, lists, dim):
    c = make(page + hq, [page * 30, 10, page * 3 + 5, 0], [8, 2, 1, 5], hq, hk, dim, page, "bf16")
    c["pages"] = lists_of(c, np.random.default_rng(page), lists, 16, page)
    check(lib, c)


def test_chosen_pages_of_many_requests(lib):
    c = make(18, [1500] * 40, [8] * 40, 64, 4, 128, 128, "bf16")
    c["pages"] = lists_of(c, np.random.default_rng(1), 4, 16, 128)
    check(lib, c)
    c = make(19, [3000] * 3, [40, 64, 1], 4, 1, 128, 16, "fp16")
    c["pages"] = lists_of(c, np.random.default_rng(2), 1, 64, 16)
    check(lib, c)


def test_all_pages_listed_is_the_dense_call(lib):
    c = make(20, [900, 100], [8, 8], 64, 4, 128, 128, "bf16", tree="chain")
    dense, _, _ = run(lib, c)
    c["pages"] = np.tile(np.r_[np.arange(8), -1].astype(np.int32), (16, 4, 1))
    listed, _, _ = run(lib, c)
    assert (dense.float() - listed.float()).abs().max() < 0.02


def test_many_keys_split_over_the_gpu(lib):
    c = make(21, [70_000], [2], 16, 2, 128, 128, "bf16")
    check(lib, c)
    c = make(22, [30_000, 100, 9_000], [8, 64, 1], 16, 2, 128, 16, "fp16")
    check(lib, c)


def test_repeats_and_streams_give_the_same_bits(lib):
    c = make(23, [9000, 500, 3000, 10], [8, 5, 1, 8], 64, 4, 128, 128, "bf16")
    first, l0, _ = run(lib, c)
    s = torch.cuda.Stream()
    for k in range(6):
        torch.cuda.synchronize()
        out, L, _ = run(lib, c, stream=s if k % 2 else None)
        assert torch.equal(out, first) and torch.equal(L, l0)


def test_graph_replays_follow_new_inputs(lib):
    a, b = make(24, [800, 100], [4, 4], 16, 2, 128, 64, "bf16"), make(25, [700, 180], [4, 4], 16, 2, 128, 64, "bf16")
    width = max(a["table"].shape[1], b["table"].shape[1])
    pad = lambda t: np.pad(t, ((0, 0), (0, width - t.shape[1])), constant_values=-1)
    blocks = max(a["cache"].shape[1], b["cache"].shape[1])
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    cache = torch.zeros((2, blocks, *a["cache"].shape[2:]), dtype=a["dt"], device="cuda")
    q, table, seq, cu, mask = torch.empty_like(a["q"]), d(pad(a["table"])), d(a["seq"]), d(a["cu"]), d(a["mask"].view(np.int64))
    out = torch.empty_like(q)
    size = lib.idx_tree_attention_workspace_bytes(2, 8, 16, 2, 128)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        lib.idx_tree_attention(q, cache[0], cache[1], table, seq, cu, out, a["scale"], tree_mask=mask, workspace=ws)
    for c in (a, b, a):
        cache[:, : c["cache"].shape[1]].copy_(c["cache"])
        q.copy_(c["q"]), table.copy_(d(pad(c["table"]))), seq.copy_(d(c["seq"])), mask.copy_(d(c["mask"].view(np.int64)))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        compare(c, out, None, reference(c))


def test_offsets_past_32_bits(lib):
    """A cache of more than 2^31 elements, the request's blocks at its end."""
    hk, dim, page = 8, 128, 128
    blocks = 2**31 // (page * hk * dim) + 40
    cache = torch.empty(2, blocks, page, hk, dim, dtype=torch.bfloat16, device="cuda")
    c = make(26, [600], [4], 16, hk, dim, page, "bf16")
    small = c["cache"]
    n = small.shape[1]
    cache[:, blocks - n :].copy_(small)
    want = reference(c)
    c["cache"] = cache
    c["table"] = np.where(c["table"] >= 0, c["table"] + blocks - n, -1).astype(np.int32)
    out, L, st = run(lib, c)
    compare(c, out, L, want)


def test_times_out_then_recovers(lib):
    """With a budget of zero polls a wait is a single test, so the launch gives up, reports it and ends; the next is right."""
    c = make(27, [9000, 500, 3000, 10], [8, 5, 1, 8], 64, 4, 128, 128, "bf16")
    ref = reference(c)
    for _ in range(3):
        prev = lib.idx_set_wait_limit(0)
        try:
            _, _, st = run(lib, c)
        finally:
            assert lib.idx_set_wait_limit(prev) == 0
        assert st & lib.ST_TIMEOUT
        out, L, st = run(lib, c)
        assert st == 0
        compare(c, out, L, ref)


@pytest.mark.parametrize("tree", ["tree", "none"])
@pytest.mark.parametrize("ctx,new,hq,hk", [([3000], [64], 64, 4), ([0], [64], 64, 4), ([1500] * 4, [16] * 4, 64, 4),
                                           ([2000, 900, 2500, 10], [16, 24, 8, 40], 64, 4), ([1200, 700], [56, 48], 64, 4),
                                           ([2500, 0, 1800], [61, 1, 33], 32, 8), ([700], [11], 100, 1), ([600, 600], [9, 10], 128, 1),
                                           ([5000, 130], [2, 64], 128, 2)])
def test_requests_of_several_blocks(lib, ctx, new, hq, hk, tree):
    """Two to eight blocks of rows a request, and numbers that only single CTAs take; requests of one size and of several."""
    c = make(sum(ctx) + sum(new), ctx, new, hq, hk, 128, 128, "bf16", tree=tree)
    first = check(lib, c)
    again, _, _ = run(lib, c)
    assert torch.equal(first, again)


def test_long_chain_in_blocks(lib):
    """A prompt's chunk: 300 tokens, 38 blocks of 8, each seeing less than the next."""
    check(lib, make(5, [513, 0], [300, 17], 64, 4, 64, 32, "fp16", tree="none"))
