"""idx_index_append against the definition in 64 bits where fp32 falls short: sums of weights and offset, squares of small rows."""

import numpy as np
import pytest
import torch

from oracle import serve

pytestmark = pytest.mark.gpu


def dev(x, kind=torch.float32):
    return torch.from_numpy(np.asarray(x)).to(kind).cuda()


def run(lib, q, k, qw, kw, offset, eps, inter=False, freq=None):
    """q [T, H, 128] and k [T, 128] at positions 5, 6, ..., without rotation unless there are frequencies."""
    tokens, heads, _ = q.shape
    out, scale = torch.zeros(tokens, heads, 128, dtype=torch.uint8, device="cuda"), torch.zeros(tokens, heads, device="cuda")
    pages = torch.zeros(-(-tokens // 128), 128, 72, dtype=torch.uint8, device="cuda")
    freq = np.zeros(0) if freq is None else freq
    pos, status = 5 + torch.arange(tokens, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.idx_index_append(q, k, qw, kw, eps, pos, dev(freq, torch.float64), out, scale, pages, offset=offset, interleaved=inter, status=status)
    assert status.item() == 0
    wide = lambda t: t.double().cpu().numpy()
    p, e = pos.cpu().numpy(), float(np.float32(eps))
    codes, scales = serve.index_queries(wide(q), wide(qw), e, offset, p, freq, 1.0, inter, 1.0, None)
    key_codes, key_scales = serve.index_keys(wide(k), wide(kw), e, offset, p, freq, 1.0, inter)
    flat = pages.view(-1, 128 * 72).cpu().numpy()
    got_codes = flat[:, : 128 * 64].reshape(-1, 64)[:tokens]
    got_scales = flat[:, 128 * 64 :].reshape(-1, 8)[:tokens]
    got, want = out.cpu().numpy(), codes
    assert np.array_equal(np.where(got & 0x7F, got, 0), np.where(want & 0x7F, want, 0)), np.argwhere(got != want)[:5]
    assert np.array_equal(got_scales, key_scales), np.argwhere(got_scales != key_scales)[:5]
    for sh in (0, 4):
        x, y = got_codes >> sh & 15, key_codes >> sh & 15
        assert np.array_equal(np.where(x & 7, x, 0), np.where(y & 7, y, 0)), np.argwhere(x != y)[:5]
    # units of 2^-24: 7 sqrt 2 and one for the weight's sum of the largest element, 16 for the norm, 4 for the products
    assert np.all(np.abs(wide(scale) - scales) <= 32 * 2.0**-24 * np.abs(scales))


def test_sums_of_weights_and_offset_that_fp32_rounds(lib):
    """1 + w with w below half a step of fp32: with the sum rounded, each of the elements here gets another code."""
    w = np.zeros(128, dtype=np.float32)
    w[1::2] = 5.9e-8
    assert np.float32(1) + w[1] == 1
    rng = np.random.default_rng(0)
    zero = np.zeros(128)
    pos, none = np.zeros(1, dtype=np.int64), np.zeros(0)

    # queries: the largest element is 1; the others just below a middle between two codes, which 1 + w takes them over
    middles = (serve.E4M3[60:126] + serve.E4M3[61:127]) / 2 / 448.0
    x = middles.astype(np.float32)
    x = np.where(x >= middles, np.nextafter(x, np.float32(0)), x)
    x = x[(x < middles) & (x.astype(np.float64) * (1 + w[1].astype(np.float64)) > middles)]
    assert len(x) >= 10
    q = np.zeros((4, 1, 128), dtype=np.float32)
    q[:, 0, 0] = 1.0
    for t in range(4):
        q[t, 0, 1::2] = rng.choice(x, 64)
    codes = lambda weight: serve.index_queries(q, weight, 1e-6, 1.0, pos, none, 1.0, False, 1.0, None)[0]
    assert (codes(w) != codes(zero)).sum() == 4 * 64

    # keys: blocks whose scale, or whose second element's code, lies as near
    keys = []
    while len(keys) < 40:
        k = rng.standard_normal(128).astype(np.float32)
        e = 2 * rng.integers(0, 64) + 1
        r = serve._inverse_rms(k[None], w, 1e-6)[0]
        block = k[e // 16 * 16 : e // 16 * 16 + 16]
        s = serve.E4M3[serve.nearest_code(np.abs(block).max() * r / 6.0, serve.E4M3)]
        code = int(rng.integers(0, 7))
        k[e] = (serve.E2M1[code] + serve.E2M1[code + 1]) / 2 * s / r
        for _ in range(12):  # (r moves with the element)
            r = serve._inverse_rms(k[None], w, 1e-6)[0]
            k[e] = np.float32((serve.E2M1[code] + serve.E2M1[code + 1]) / 2 * s / r)
        for step in range(3):
            both = [np.concatenate(serve.index_keys(k[None], weight, 1e-6, 1.0, pos, none, 1.0, False), 1) for weight in (w, zero)]
            if not np.array_equal(*both):
                keys.append(k.copy())
                break
            k[e] = np.nextafter(k[e], np.float32(0))
    k = np.stack(keys)
    q = np.repeat(q, 10, 0)
    run(lib, dev(q), dev(k), dev(w), dev(w), 1.0, 1e-6)


@pytest.mark.parametrize("inter", [False, True])
def test_random_weights_with_an_offset(lib, inter):
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    freq = lib.idx_rope_frequencies(64, 10000.0)[0].numpy()
    run(lib, rand(3000, 8, 128), rand(3000, 128), 0.1 * rand(128), 0.1 * rand(128), 1.0, 1e-6, inter, freq)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-36])
def test_small_rows(lib, dtype, eps):
    """Rows whose squares are subnormal or 0 in fp32, with an eps that does not cover them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    size = torch.logspace(-29, -14, 61, base=10.0, device="cuda")
    q = (size[:, None, None] * torch.randn(61, 5, 128, device="cuda", generator=g)).to(dtype)
    k = (size[:, None] * torch.randn(61, 128, device="cuda", generator=g)).to(dtype)
    w = (1 + 0.2 * torch.randn(2, 128, device="cuda", generator=g)).to(dtype)
    freq = lib.idx_rope_frequencies(32, 10000.0)[0].numpy()
    run(lib, q, k, w[0], w[1], 0.0, eps, False, freq)


def test_rows_of_zeros_without_eps(lib):
    """0 / 0: scales are NaN, codes 0."""
    q, k = torch.zeros(1, 1, 128, device="cuda"), torch.zeros(1, 128, device="cuda")
    w, out, scale = torch.ones(128, device="cuda"), torch.ones(1, 1, 128, dtype=torch.uint8, device="cuda"), torch.zeros(1, 1, device="cuda")
    pages = torch.ones(1, 128, 72, dtype=torch.uint8, device="cuda")
    lib.idx_index_append(q, k, w, w, 0.0, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.float64, device="cuda"), out, scale, pages)
    flat = pages.view(-1)
    assert not out.any() and scale.isnan().all() and not flat[:64].any() and flat[128 * 64 : 128 * 64 + 8].eq(0x7F).all()


def test_small_rows_in_request_slots(lib):
    """With request slots and head weights: the flat call's scales at the requests' last slots, the others as they were; captured too."""
    g = torch.Generator(device="cuda")
    g.manual_seed(13)
    q = 1e-22 * torch.randn(9, 3, 128, device="cuda", generator=g)
    q[2] *= 1e22  # a row of ordinary size among them
    w, hw = 1 + 0.2 * torch.randn(128, device="cuda", generator=g), torch.randn(9, 3, device="cuda", generator=g)
    pos, freq = torch.arange(9, dtype=torch.int32, device="cuda"), lib.idx_rope_frequencies(32, 10000.0)[0].cuda()
    flat, flat_scale = torch.zeros(9, 3, 128, dtype=torch.uint8, device="cuda"), torch.zeros(9, 3, device="cuda")
    lib.idx_index_append(q, None, w, None, 0.0, pos, freq, flat, flat_scale, None, head_weights=hw, scale=0.5)
    _, want = serve.index_queries(q.double().cpu().numpy(), w.double().cpu().numpy(), 0.0, 0.0, np.arange(9), freq.cpu().numpy(), 1.0, False, 0.5,
                                  hw.double().cpu().numpy())
    assert np.all(np.abs(flat_scale.double().cpu().numpy() - want) <= 32 * 2.0**-24 * np.abs(want))
    cu = torch.tensor([0, 2, 2, 8], dtype=torch.int32, device="cuda")  # the last token is behind the requests, and the third has one too many
    out, scale = torch.full((3, 5, 3, 128), 0xAB, dtype=torch.uint8, device="cuda"), torch.full((3, 5, 3), -7.0, device="cuda")

    def call():
        lib.idx_index_append(q, None, w, None, 0.0, pos, freq, out, scale, None, cu_tokens=cu, head_weights=hw, scale=0.5)

    call()
    for _ in range(2):
        assert scale[0, :3].eq(-7).all() and scale[1].eq(-7).all()
        assert torch.equal(scale[0, 3:], flat_scale[:2]) and torch.equal(scale[2], flat_scale[3:8]) and torch.equal(out[2], flat[3:8])
        scale.fill_(-7.0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graph.replay()
        torch.cuda.synchronize()
