"""idx_tree_attention: weights far below the largest, padded batches, many requests.

Tolerances are those of the main tests; where weights below fp16's smallest
normal number carry the result, each adds half of their step, 2^-32 of the
row's largest weight, times |v|.
"""

import numpy as np
import pytest
import torch

from test_gpu_tree_attention import check, compare, lists_of, make, reference, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("where", [0, 9001, 16383])
def test_one_key_above_a_long_tail(lib, where, dtype):
    """16,383 keys of 2^-27 to 2^-24 of the largest weight, which has the value 0: the output is the tail's alone.

    So many requests (of the same blocks) that each is one CTA's, and so many heads that each half row is one thread's."""
    places, reqs, hq, dim, page = 16384, 160, 128, 64, 128
    dt = torch.float16 if dtype == "fp16" else torch.bfloat16
    rng = np.random.default_rng(where)
    k = np.zeros((places, 1, dim))
    k[:, 0, 0] = rng.uniform(-27, -24, places)
    v = 0.5 + 0.5 * rng.random((places, 1, dim))
    k[where], v[where] = 0, 0
    cache = torch.from_numpy(np.stack([k, v]).reshape(2, places // page, page, 1, dim)).cuda().to(dt)
    q = torch.zeros(reqs, hq, dim, device="cuda", dtype=dt)
    q[..., 0] = 1
    q[..., 1:] = torch.randn(reqs, hq, dim - 1, device="cuda").to(dt)  # meets zeros
    table = np.tile(np.arange(places // page, dtype=np.int32), (reqs, 1))
    c = dict(q=q, cache=cache, table=table, seq=np.full(reqs, places, dtype=np.int32), cu=np.arange(reqs + 1, dtype=np.int32), mask=None,
             dt=dt, pages=None, scale=float(np.log(2)))
    out, L, st = run(lib, c)
    assert st == 0
    one = dict(c, q=q[:1, :1], table=table[:1], seq=c["seq"][:1], cu=c["cu"][:2])
    want, lse, mag, big, n = reference(one)
    tile = lambda x: np.broadcast_to(x, (reqs, hq, *x.shape[2:]))
    # what numbers below the normal ones may lose, as a part of `mag`'s bound
    eps = torch.finfo(dt).eps
    small = places * 2.0**-32 / (eps / 2) if dtype == "fp16" else 0.0
    compare(c, out, L, (tile(want), tile(lse), tile(mag + small), tile(big), np.tile(n, reqs)))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("top", [1e3, 1e5, 1.6e7])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("ctx,hq,hk,dim", [(700, 4, 1, 64), (700, 64, 1, 64), (30_000, 16, 2, 128)])
def test_a_largest_score_far_above_the_others(lib, ctx, hq, hk, dim, sign, top, dtype):
    """Products of small whole numbers are exact, and all other scores are hundreds below: the output is one key's value to
    the roundings of its weight and of the output, L its score."""
    c = make(ctx + hq, [ctx], [3], hq, hk, dim, 128, dtype, tree="chain")
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    c["q"].copy_(torch.randint(-1, 2, c["q"].shape, device="cuda", generator=g))
    c["q"][:, :, 0] = 3 * sign
    c["cache"][0].copy_(torch.randint(-1, 2, c["cache"][0].shape, device="cuda", generator=g))
    place = ctx // 2
    b, o = int(c["table"][0, place // 128]), place % 128
    c["cache"][0, b, o, :, 0] = 64  # all others: at most 3 + dim - 1 of 192 - dim + 1
    if dim == 128:
        c["cache"][0, b, o, :, 0] = 120
    k = c["cache"][0, b, o].double().repeat_interleave(hq // hk, 0)
    raw = (c["q"].double() * k).sum(-1)
    c["scale"] = float(np.float32(top / float(raw.abs().max())))
    if sign < 0:
        c["scale"] = -c["scale"]
    out, L, st = run(lib, c)
    assert st == 0
    best = c["cache"][1, b, o].double().repeat_interleave(hq // hk, 0)
    assert ((out.double() - best).abs() <= torch.finfo(c["dt"]).eps * (1 + 2.0**-8) * best.abs()).all()
    assert ((L.double() - raw * c["scale"]).abs() <= 2.0**-21 * (raw * c["scale"]).abs()).all()


@pytest.mark.parametrize("lists", [0, 2])
@pytest.mark.parametrize("pad", [1, 7, 300])
def test_rows_past_the_last_request_are_empty(lib, pad, lists):
    c = make(30 + pad, [300, 0, 90], [5, 0, 3], 16, 2, 128, 16, "bf16")
    extra = torch.randn(pad, 16, 128, device="cuda").bfloat16()
    c["q"] = torch.cat([c["q"], extra])
    c["mask"] = np.concatenate([c["mask"], np.full(pad, 2**64 - 1, dtype=np.uint64)])
    if lists:
        c["pages"] = lists_of(c, np.random.default_rng(pad), lists, 16, 16)
    out, L, st = run(lib, c)  # out and L hold 9 before
    assert st == 0
    compare(c, out, L, reference(c))
    assert not out[8:].any() and L[8:].isneginf().all()
    # rows of a wider tensor: what lies between them stays
    wide = torch.full((8 + pad, 20, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    again, _, _ = run(lib, c, out=wide[:, 2:18])
    assert torch.equal(again, out) and wide[:, :2].eq(7).all() and wide[:, 18:].eq(7).all()


def test_a_padded_batch_of_slots_feeds_the_attention(lib):
    """idx_build_slots with room for more tokens than there are, then the attention over its lengths."""
    reqs, page, cap, hq, hk, dim = 4, 16, 40, 8, 2, 64
    d = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ctx, new = [37, 0, 64, 5], [3, 6, 0, 8]
    width, blocks = 8, 30
    e = lambda n, t=torch.int32: torch.full((n,), -77, dtype=t, device="cuda")
    table = torch.full((reqs, width), -1, dtype=torch.int32, device="cuda")
    cu, seq, pages, cur, pos, slots, mask = e(reqs + 1), e(reqs), e(reqs), e(1), e(cap), e(cap, torch.int64), e(cap, torch.int64)
    parents = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    lib.idx_build_slots(d(ctx), d(new), d([0] * reqs), table, torch.randperm(blocks, device="cuda").to(torch.int32), d([0]), blocks, page,
                        cu, seq, pages, cur, pos, slots, parents=parents, tree_mask=mask)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    cache = torch.randn(2, blocks, page, hk, dim, device="cuda", generator=g).bfloat16()
    q = torch.randn(cap, hq, dim, device="cuda", generator=g).bfloat16()
    np_ = lambda t: t.cpu().numpy()
    c = dict(q=q, cache=cache, table=np_(table), seq=np_(seq), cu=np_(cu), mask=np_(mask).view(np.uint64), dt=torch.bfloat16, pages=None,
             scale=dim**-0.5)
    assert c["cu"].tolist() == [0, 3, 9, 9, 17]
    out = check(lib, c)
    assert not out[17:].any()


@pytest.mark.parametrize("reqs", [417, 1300])
@pytest.mark.parametrize("lists", [0, 2])
def test_many_requests(lib, reqs, lists):
    """More requests than a CTA has threads, some without tokens, some of several blocks of rows."""
    rng = np.random.default_rng(reqs)
    ctx = rng.integers(0, 60, reqs)
    new = rng.choice([0, 0, 1, 1, 2, 3, 17], reqs)
    new[rng.integers(0, reqs, 5)] = 40
    ctx[rng.integers(0, reqs, 5)] = 900
    c = make(reqs, ctx.tolist(), new.tolist(), 16, 2, 64, 16, "bf16")
    if lists:
        c["pages"] = lists_of(c, rng, lists, 16, 16)
    check(lib, c)
    first = [0] * 500  # runs without a token before the first and after the last
    c = make(reqs + 1, first + [70, 3] + first, first + [3, 0] + first, 16, 2, 64, 16, "fp16")
    check(lib, c)
