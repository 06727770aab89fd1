"""idx_tree_attention with infinities and NaN among the values.

Where a row sees such a value in a column, the column is what the weighted sum
gives (weights are positive): the infinity, or NaN for NaN or infinities of both
signs.  Everything else is as if the value were not there, within the main
tests' tolerances; and the call's time stays near that of finite values.
"""

import numpy as np
import pytest
import torch

from oracle import step
from test_gpu_tree_attention import compare, lists_of, make, run

pytestmark = pytest.mark.gpu


def plant(c, rng, count, drafted_only=False):
    """`count` values that are not finite, at places in use (a third of them drafted tokens') and in unwritten slots."""
    page, hk, dim = c["cache"].shape[2:]
    kinds = [float("inf"), float("-inf"), float("nan")]
    for _ in range(count):
        r = int(rng.integers(0, len(c["seq"])))
        n = int(c["cu"][r + 1] - c["cu"][r])
        s = int(c["seq"][r])
        if n == 0:
            continue
        place = s - 1 - int(rng.integers(0, n)) if drafted_only or rng.random() < 0.33 else int(rng.integers(0, s))
        h, col = int(rng.integers(0, hk)), int(rng.integers(0, dim))
        c["cache"][1, int(c["table"][r, place // page]), place % page, h, col] = kinds[int(rng.integers(0, 3))]
        if s % page:
            c["cache"][1, int(c["table"][r, (s - 1) // page]), s % page :] = kinds[int(rng.integers(0, 3))]


def check(lib, c):
    out, L, st = run(lib, c)
    assert st == 0
    cache = c["cache"].double().cpu().numpy()
    # (unwritten slots may hold anything and are not read)
    ref = lambda v: step.tree_attention(c["q"].double().cpu().numpy(), cache[0], v, c["table"], c["seq"], c["cu"], c["scale"], c["mask"],
                                        c["pages"])
    with np.errstate(invalid="ignore"):
        want = ref(cache[1])[0]
    clean = ref(np.nan_to_num(cache[1], nan=0.0, posinf=0.0, neginf=0.0))
    got = out.double().cpu().numpy()
    for kind in (np.isnan, np.isposinf, np.isneginf):
        assert np.array_equal(kind(got), kind(want)), (kind, np.argwhere(kind(got) != kind(want))[:4])
    bad = ~np.isfinite(want)
    fixed = torch.where(torch.from_numpy(bad).cuda(), torch.from_numpy(clean[0]).cuda(), out.double())
    compare(c, fixed, L, clean)
    return int(bad.sum()), out


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hk,dim", [(64, 4, 128), (32, 8, 64), (12, 1, 64), (100, 1, 128), (64, 2, 64), (40, 10, 128)])
def test_heads_and_types(lib, dtype, hq, hk, dim):
    rng = np.random.default_rng(hq + dim)
    c = make(hq + dim, [300, 0, 127, 1000, 9000], [8, 3, 1, 11, 4], hq, hk, dim, 128, dtype)
    plant(c, rng, 30)
    assert check(lib, c)[0] > 0


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("tree", ["tree", "random", "chain"])
def test_values_that_only_some_rows_see(lib, page, tree):
    rng = np.random.default_rng(page)
    c = make(page, [page * 2 - 3, 5, 20_000, 700], [30, 1, 17, 9], 16, 2, 128, page, "bf16", tree=tree)
    plant(c, rng, 12, drafted_only=True)
    check(lib, c)


@pytest.mark.parametrize("page", [16, 64, 128])
def test_chosen_pages(lib, page):
    rng = np.random.default_rng(page)
    c = make(page + 1, [page * 30, 10, page * 3 + 5, 0] * 6, [8, 2, 1, 5] * 6, 16, 4, 128, page, "fp16")
    c["pages"] = lists_of(c, rng, 2, 16, page)
    plant(c, rng, 60)
    check(lib, c)


def test_every_place_bad(lib):
    c = make(40, [700, 3], [5, 2], 16, 2, 64, 16, "fp16")
    c["cache"][1, :, :, 0, 3] = float("inf")
    c["cache"][1, :, :, 1, :] = float("nan")
    c["cache"][1, ::2, :, 0, 4] = float("-inf")
    c["cache"][1, 1::2, :, 0, 4] = float("inf")
    check(lib, c)


def test_scores_that_are_not_finite_stay_in_their_rows(lib):
    c = make(41, [3000, 40], [6, 3], 16, 2, 128, 128, "bf16")
    want, l0, _ = run(lib, c)
    c["q"][2, 5, 7] = float("nan")
    c["q"][7, 9, 1] = float("inf")
    out, L, st = run(lib, c)
    assert st == 0 and out[2, 5].isnan().all() and out[7, 9].isnan().all()
    out[2, 5], out[7, 9] = want[2, 5], want[7, 9]
    assert torch.equal(out, want)


@pytest.mark.parametrize("ctx", [0, 1, 128, 143, 1000, 20_000])
@pytest.mark.parametrize("hq,hk,dim,lists", [(4, 1, 128, 0), (64, 4, 64, 0), (64, 1, 128, 0), (8, 2, 64, 2)])
def test_a_key_that_is_nan_reaches_the_rows_that_see_it(lib, ctx, hq, hk, dim, lists):
    """The first and the last place in turn: in short contexts and at a tile's begin the only place that a part of a row sees."""
    for place in (0, ctx):
        c = make(44 + ctx, [ctx, 50], [1, 2], hq, hk, dim, 128, "bf16")
        if lists:
            c["pages"] = np.tile(np.array([0, ctx // 128, -1], dtype=np.int32), (3, lists, 1))
        want, l0, _ = run(lib, c)
        c["cache"][0, int(c["table"][0, place // 128]), place % 128, 0, 3] = float("nan")
        out, L, st = run(lib, c)
        g = hq // hk
        assert st == 0 and out[0, :g].isnan().all() and L[0, :g].isnan().all()
        out[0, :g], L[0, :g] = want[0, :g], l0[0, :g]
        assert torch.equal(out, want) and torch.equal(L, l0)


def test_an_infinity_far_below_the_largest_weight(lib):
    """Seen with a weight that fp32 cannot hold, in a stretch of its own."""
    c = make(42, [40_000], [2], 4, 1, 64, 128, "bf16")
    c["q"].fill_(1.0)
    c["cache"][0].mul_(0.01)
    b = int(c["table"][0, 200])
    c["cache"][0, b, 7] = 20.0  # one score above the others by 160
    first = int(c["table"][0, 3])
    c["cache"][1, first, 5, 0, 9] = float("-inf")
    check(lib, c)


def events(fn, n=5):
    took = []
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        fn()
        b.record()
        b.synchronize()
        took.append(a.elapsed_time(b))
    return sorted(took)[n // 2]


@pytest.mark.parametrize("seen", [True, False])
@pytest.mark.parametrize("reqs,ctx,hq,hk", [(1, 100_000, 64, 4), (40, 20_000, 16, 4)])
def test_long_contexts_take_about_as_long(lib, reqs, ctx, hq, hk, seen):
    """One value in a context of 100,000 places, or in one of 40 requests, seen by all of its rows or by one."""
    c = make(43, [ctx] * reqs, [8] * reqs, hq, hk, 128, 128, "bf16")
    out = torch.empty_like(c["q"])
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    table, seq, cu, mask = d(c["table"]), d(c["seq"]), d(c["cu"]), d(c["mask"].view(np.int64))
    size = lib.idx_tree_attention_workspace_bytes(reqs, 8 * reqs, hq, hk, 128)
    ws, status = torch.zeros(size, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: lib.idx_tree_attention(c["q"], c["cache"][0], c["cache"][1], table, seq, cu, out, c["scale"], tree_mask=mask,
                                          workspace=ws, status=status)
    call()
    clean, want = events(call), out.clone()
    place = 777 if seen else ctx + 7  # the last drafted token: its own row sees it
    c["cache"][1, int(c["table"][0, place // 128]), place % 128, 1, 70] = float("inf")
    call()
    took = events(call)
    assert int(status.item()) == 0
    assert took < 6 * clean + 0.1, (took, clean)
    g = hq // hk
    rows = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    rows[:8, g : 2 * g] = (d(c["mask"].view(np.int64))[:8, None] >> 7 & 1 == 1) if not seen else True
    assert out[..., 70][rows].isposinf().all()
    out[..., 70] = torch.where(rows, want[..., 70], out[..., 70])
    assert torch.equal(out, want)
