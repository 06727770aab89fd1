"""idx_index_append against the definition in 64 bits where fp32 falls short: sums of weights and offset."""

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
