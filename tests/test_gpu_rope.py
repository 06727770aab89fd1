"""idx_rope_append against the rotation in 64 bits.

Tolerance: the angle is exact to 2^-33 turns, its sine and cosine are fp32
values (an error below 2 units in the last place, times mscale and a rounding),
and two products and a sum round in fp32: below 8 * 2^-24 * mscale (|x1| +
|x2|); then one rounding to the type, at most eps / 2 of the value (and half
the smallest subnormal).
"""

import numpy as np
import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def bound(x, want, half, inter, mscale, dtype):
    one = np.arange(0, 2 * half, 2) if inter else np.arange(half)
    two = one + 1 if inter else one + half
    fi = torch.finfo(dtype)
    b = np.abs(want) * fi.eps / 2 + fi.smallest_normal * fi.eps
    mag = 8 * 2.0**-24 * abs(mscale) * (np.abs(x[..., one]) + np.abs(x[..., two]))
    for ix in (one, two):
        b[..., ix] += mag * (1 + fi.eps)
    return b


def check(lib, tokens, hq, hk, dim, rd, inter, dtype, page, mscale=1.0, start=0, layout="fused", kind=0, with_v=True, gap=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens * 7 + dim + rd)
    dt = TYPES[dtype]
    wide = (hq + 2 * hk) * dim + gap
    qkv = torch.randn(tokens, wide, device="cuda", generator=g).to(dt)
    q = qkv[:, : hq * dim].unflatten(1, (hq, dim)) if hq else None
    k = qkv[:, hq * dim : (hq + hk) * dim].unflatten(1, (hk, dim)) if hk else None
    v = qkv[:, (hq + hk) * dim : (hq + 2 * hk) * dim].unflatten(1, (hk, dim)) if hk and with_v else None
    blocks = -(-tokens // page) + 2
    shape = (2, blocks, hk, page, dim) if layout == "heads" else (2, blocks, page, hk, dim)
    cache = torch.randn(shape, device="cuda", generator=g).to(dt)
    if layout == "heads":
        cache = cache.transpose(2, 3)
    before = cache.double().cpu().numpy()
    slots = torch.randperm(blocks * page, device="cuda", generator=g)[:tokens]
    if tokens > 3:
        slots[2] = -1
    pos = (start + torch.arange(tokens, device="cuda") * 3).to(torch.int32)
    f, m = lib.idx_rope_frequencies(rd, 10000.0, kind, 8.0, 4096.0) if rd else (torch.zeros(0, dtype=torch.float64), 1.0)
    m = mscale if kind == 0 else m
    q_out = torch.full((tokens, hq, dim), 7.0, device="cuda", dtype=dt) if hq else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.idx_rope_append(q, k, v, pos, f.cuda(), q_out, cache[0] if hk else None, cache[1] if v is not None else None, slots if hk else None,
                        mscale=m, interleaved=inter, status=status)
    p, fr = pos.cpu().numpy(), f.numpy()
    assert status.item() == 0
    m32 = float(np.float32(m))
    if hq:
        x = q.double().cpu().numpy()
        want = step.rotate(x, p, fr, m32, inter)
        assert np.all(np.abs(q_out.double().cpu().numpy() - want) <= bound(x, want, rd // 2, inter, m, dt))
    if hk:
        x = k.double().cpu().numpy()
        turned = step.rotate(x, p, fr, m32, inter)
        want, tol = before.copy(), np.zeros(before.shape[1:])
        b = bound(x, turned, rd // 2, inter, m, dt)
        for t, s in enumerate(slots.tolist()):
            if s >= 0:
                want[0, s // page, s % page], tol[s // page, s % page] = turned[t], b[t]
                if v is not None:
                    want[1, s // page, s % page] = v[t].double().cpu().numpy()
        after = cache.double().cpu().numpy()
        assert np.all(np.abs(after[0] - want[0]) <= tol) and np.array_equal(after[1], want[1])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rd", [(128, 128), (128, 64), (64, 32), (96, 96), (80, 20), (6, 2), (7, 6), (40, 0), (256, 128)])
def test_layouts_and_parts(lib, dtype, inter, dim, rd):
    check(lib, 19, 5, 3, dim, rd, inter, dtype, 16, mscale=1.25)


@pytest.mark.parametrize("tokens,hq,hk", [(1, 64, 4), (1, 1, 1), (2, 0, 4), (700, 8, 0), (3001, 16, 2), (77, 40, 10)])
def test_sizes(lib, tokens, hq, hk):
    check(lib, tokens, hq, hk, 128, 128, False, "bf16", 128)
    check(lib, tokens, hq, hk, 64, 64, True, "fp16", 64, kind=2)


@pytest.mark.parametrize("start", [1_000_000, 2**31 - 1 - 300, -50])
def test_far_positions_keep_full_precision(lib, start):
    check(lib, 90, 2, 1, 128, 128, False, "fp32", 16, start=start)


def test_strides_and_alignment(lib):
    for gap in (1, 2, 4, 6):  # rows of the projection that start at any element
        check(lib, 33, 3, 2, 64, 64, False, "bf16", 16, gap=gap)
        check(lib, 33, 3, 2, 64, 64, True, "fp16", 16, gap=gap)
    check(lib, 33, 4, 2, 64, 32, False, "fp32", 16, layout="heads", kind=1)
    check(lib, 33, 4, 2, 64, 32, True, "bf16", 16, with_v=False)


def test_in_place_and_packed_keys(lib):
    x = torch.randn(50, 4, 64, device="cuda")
    f, _ = lib.idx_rope_frequencies(64, 10000.0)
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    want = torch.empty_like(x)
    lib.idx_rope_append(x, None, None, pos, f.cuda(), want, None, None)
    packed = torch.zeros(50, 1, 4, 64, device="cuda")  # slots None: token t in slot t
    lib.idx_rope_append(None, x, None, pos, f.cuda(), None, packed, None)
    assert torch.equal(packed[:, 0], want)
    lib.idx_rope_append(x, None, None, pos, f.cuda(), x, None, None)
    assert torch.equal(x, want)


def test_slots_past_the_cache_are_skipped(lib):
    k = torch.ones(3, 1, 8, device="cuda")
    cache = torch.zeros(2, 4, 1, 8, device="cuda")
    f, _ = lib.idx_rope_frequencies(8, 10000.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.idx_rope_append(None, k, None, torch.zeros(3, dtype=torch.int32, device="cuda"), f.cuda(), None, cache, None,
                        torch.tensor([8, -1, 7], device="cuda"), status=status)
    assert status.item() == lib.ST_BLOCK_OOR
    assert cache[1, 3].eq(1).all() and cache.sum().item() == 8


def test_other_stream(lib):
    x = torch.randn(4000, 8, 128, device="cuda").bfloat16()
    f = lib.idx_rope_frequencies(128, 10000.0)[0].cuda()
    pos = torch.arange(4000, dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    lib.idx_rope_append(x, None, None, pos, f, a, None, None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.idx_rope_append(x, None, None, pos, f, b, None, None)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(a, b)
