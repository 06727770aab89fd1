"""idx_norm_rope_append against the norm and the rotation in 64 bits.

Tolerance, in units of 2^-24: a row's sum of squares goes through at most 16
additions a lane and 5 between lanes, halved by the root, and the root itself is
off by 4: 16 units of the element; weights (their sum with the offset, the
products with sine and cosine) 3 more, the turn 8 of |n1| + |n2| as in the tests
of idx_rope_append.  32 units of m (|n1| + |n2|), or of |n|, cover them; then one
rounding to the type, at most eps / 2 of the value (and half the smallest
subnormal).
"""

import numpy as np
import pytest
import torch

from oracle import serve

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def bound(n, want, half, inter, mscale, dtype):
    """n: the normed rows before the turn."""
    one = np.arange(0, 2 * half, 2) if inter else np.arange(half)
    two = one + 1 if inter else one + half
    mag = np.abs(n)
    both = abs(mscale) * (mag[..., one] + mag[..., two])
    mag[..., one], mag[..., two] = both, both
    fi = torch.finfo(dtype)
    return np.abs(want) * fi.eps / 2 + fi.smallest_normal * fi.eps + 32 * 2.0**-24 * mag * (1 + fi.eps)


def check(lib, tokens, hq, hk, dim, rd, inter, dtype, page, mscale=1.0, offset=0.0, start=0, layout="fused", with_v=True, gap=0, weigh=(True, True), size=1.0,
          eps=1e-5):
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens * 7 + dim + rd)
    dt = TYPES[dtype]
    qkv = (size * torch.randn(tokens, (hq + 2 * hk) * dim + gap, device="cuda", generator=g)).to(dt)
    q = qkv[:, : hq * dim].unflatten(1, (hq, dim)) if hq else None
    k = qkv[:, hq * dim : (hq + hk) * dim].unflatten(1, (hk, dim)) if hk else None
    v = qkv[:, (hq + hk) * dim : (hq + 2 * hk) * dim].unflatten(1, (hk, dim)) if hk and with_v else None
    w = (1.0 - offset + 0.3 * torch.randn(2, dim, device="cuda", generator=g)).to(dt)
    qw, kw = (w[i] if weigh[i] else None for i in (0, 1))
    blocks = -(-tokens // page) + 2
    cache = torch.randn((2, blocks, hk, page, dim) if layout == "heads" else (2, blocks, page, hk, dim), device="cuda", generator=g).to(dt)
    if layout == "heads":
        cache = cache.transpose(2, 3)
    before = cache.double().cpu().numpy()
    slots = torch.randperm(blocks * page, device="cuda", generator=g)[:tokens]
    if tokens > 3:
        slots[2] = -1
    pos = (start + torch.arange(tokens, device="cuda") * 3).to(torch.int32)
    f = lib.idx_rope_frequencies(rd, 10000.0)[0] if rd else torch.zeros(0, dtype=torch.float64)
    q_out = torch.full((tokens, hq, dim), 7.0, device="cuda", dtype=dt) if hq else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.idx_norm_rope_append(q, k, v, qw, kw, eps, pos, f.cuda(), q_out, cache[0] if hk else None, cache[1] if v is not None else None,
                             slots if hk else None, mscale=mscale, offset=offset, interleaved=inter, status=status)
    assert status.item() == 0
    p, fr, m32, e32, o32 = pos.cpu().numpy(), f.numpy(), float(np.float32(mscale)), float(np.float32(eps)), float(np.float32(offset))
    weight = lambda w: None if w is None else w.double().cpu().numpy()
    rows = lambda x, w: (serve.norm_rotate(x, weight(w), e32, o32, p, fr[:0], 1.0, inter), serve.norm_rotate(x, weight(w), e32, o32, p, fr, m32, inter))
    if hq:
        n, want = rows(q.double().cpu().numpy(), qw)
        assert np.all(np.abs(q_out.double().cpu().numpy() - want) <= bound(n, want, rd // 2, inter, mscale, dt))
    if hk:
        n, turned = rows(k.double().cpu().numpy(), kw)
        want, tol = before.copy(), np.zeros(before.shape[1:])
        b = bound(n, turned, rd // 2, inter, mscale, dt)
        for t, s in enumerate(slots.tolist()):
            if s >= 0:
                want[0, s // page, s % page], tol[s // page, s % page] = turned[t], b[t]
                if v is not None:
                    want[1, s // page, s % page] = v[t].double().cpu().numpy()
        after = cache.double().cpu().numpy()
        assert np.all(np.abs(after[0] - want[0]) <= tol) and np.array_equal(after[1], want[1])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rd", [(128, 128), (128, 64), (64, 32), (96, 96), (80, 20), (6, 2), (7, 6), (40, 0), (256, 128), (512, 64), (8, 8)])
def test_layouts_and_parts(lib, dtype, inter, dim, rd):
    check(lib, 19, 5, 3, dim, rd, inter, dtype, 16, mscale=1.25)


@pytest.mark.parametrize("tokens,hq,hk", [(1, 64, 4), (1, 1, 1), (2, 0, 4), (700, 8, 0), (3001, 16, 2), (77, 40, 10), (0, 4, 4)])
def test_sizes(lib, tokens, hq, hk):
    check(lib, tokens, hq, hk, 128, 128, False, "bf16", 128)
    check(lib, tokens, hq, hk, 64, 64, True, "fp16", 64, offset=1.0)


@pytest.mark.parametrize("weigh", [(False, True), (True, False), (False, False)])
def test_a_side_without_weights_is_turned_only(lib, weigh):
    for dim, rd in ((128, 64), (40, 40), (7, 6)):
        check(lib, 21, 4, 2, dim, rd, False, "bf16", 16, weigh=weigh)


def test_without_weights_it_is_idx_rope_append(lib):
    x = torch.randn(90, 4, 128, device="cuda").bfloat16()
    x[3, 1, 100], x[4, 2, 3] = float("inf"), float("nan")
    f = lib.idx_rope_frequencies(64, 10000.0)[0].cuda()
    pos = torch.arange(90, dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    lib.idx_rope_append(x, None, None, pos, f, a, None, None)
    lib.idx_norm_rope_append(x, None, None, None, None, 1e-6, pos, f, b, None, None)
    assert torch.equal(a.nan_to_num(77.0), b.nan_to_num(77.0))


@pytest.mark.parametrize("start", [1_000_000, 2**31 - 1 - 300, -50])
def test_far_positions_keep_full_precision(lib, start):
    check(lib, 90, 2, 1, 128, 128, False, "fp32", 16, start=start)


@pytest.mark.parametrize("size", [1e-18, 1e-4, 1e6, 1e16])
def test_magnitudes(lib, size):
    check(lib, 40, 3, 2, 128, 64, False, "fp32", 16, size=size, eps=1e-30 if size < 1e-9 else 1e-5)
    check(lib, 40, 3, 2, 128, 64, True, "bf16", 16, size=size)


def test_strides_and_alignment(lib):
    for gap in (1, 2, 4, 6):  # rows of the projection that start at any element
        check(lib, 33, 3, 2, 64, 64, False, "bf16", 16, gap=gap)
        check(lib, 33, 3, 2, 64, 64, True, "fp16", 16, gap=gap)
    check(lib, 33, 4, 2, 64, 32, False, "fp32", 16, layout="heads")
    check(lib, 33, 4, 2, 64, 32, True, "bf16", 16, with_v=False)


def test_rows_without_a_norm_of_their_own(lib):
    """A row of zeros stays one; infinities and NaN stay in their row."""
    x = torch.randn(6, 4, 128, device="cuda").bfloat16()
    w = torch.ones(128, device="cuda").bfloat16()
    f = lib.idx_rope_frequencies(128, 10000.0)[0].cuda()
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    clean, out = torch.empty_like(x), torch.empty_like(x)
    lib.idx_norm_rope_append(x, None, None, w, None, 1e-6, pos, f, clean, None, None)
    x[0, 1], x[1, 2, 5], x[2, 3, 77] = 0.0, float("inf"), float("nan")
    lib.idx_norm_rope_append(x, None, None, w, None, 1e-6, pos, f, out, None, None)
    assert not out[0, 1].any() and not torch.isfinite(out[1, 2]).all() and not torch.isfinite(out[2, 3]).any()
    same = torch.ones(6, 4, dtype=torch.bool, device="cuda")
    same[0, 1] = same[1, 2] = same[2, 3] = False
    assert torch.equal(out[same], clean[same])


def test_in_place_other_streams_and_graphs(lib):
    x = torch.randn(4000, 8, 128, device="cuda").bfloat16()
    w = torch.rand(128, device="cuda").bfloat16()
    f = lib.idx_rope_frequencies(128, 10000.0)[0].cuda()
    pos = torch.arange(4000, dtype=torch.int32, device="cuda")
    want = torch.empty_like(x)
    lib.idx_norm_rope_append(x, None, None, w, None, 1e-6, pos, f, want, None, None)
    packed = torch.zeros(4000, 1, 8, 128, device="cuda", dtype=torch.bfloat16)  # slots None: token t in slot t
    lib.idx_norm_rope_append(None, x, None, None, w, 1e-6, pos, f, None, packed, None)
    assert torch.equal(packed[:, 0], want)
    s, y, z = torch.cuda.Stream(), x.clone(), torch.empty_like(x)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.idx_norm_rope_append(y, None, None, w, None, 1e-6, pos, f, y, None, None)
    s.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.idx_norm_rope_append(x, None, None, w, None, 1e-6, pos, f, z, None, None)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(z, want)


def test_slots_past_the_cache_are_skipped(lib):
    for dim in (8, 7):
        k = torch.ones(3, 1, dim, device="cuda")
        cache = torch.zeros(2, 4, 1, dim, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lib.idx_norm_rope_append(None, k, None, None, torch.ones(dim, device="cuda"), 0.0, torch.zeros(3, dtype=torch.int32, device="cuda"),
                                 torch.zeros(0, dtype=torch.float64, device="cuda"), None, cache, None, torch.tensor([8, -1, 7], device="cuda"), status=status)
        assert status.item() == lib.ST_BLOCK_OOR
        assert (cache[1, 3] - 1).abs().max() < 1e-6 and (cache.sum() - dim).abs() < 1e-5
