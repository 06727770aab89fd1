"""idx_norm_rope_append on rows whose squares' sum passes fp32's range: they become 0, unless they hold an infinity or NaN."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def run(lib, x, weight, rd, inter):
    """The same rows as queries and as keys."""
    tokens, heads, dim = x.shape
    w = torch.full((dim,), weight, device="cuda", dtype=x.dtype)
    f = lib.idx_rope_frequencies(rd, 10000.0)[0].cuda() if rd else torch.zeros(0, dtype=torch.float64, device="cuda")
    pos = 1000 + torch.arange(tokens, dtype=torch.int32, device="cuda")
    out, cache = torch.full_like(x, 7.0), torch.full((tokens, 1, heads, dim), 7.0, device="cuda", dtype=x.dtype)
    lib.idx_norm_rope_append(x, x, None, w, w, 1e-6, pos, f, out, cache, None, interleaved=inter)
    return out, cache[:, 0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rd", [(128, 128), (128, 64), (7, 6), (512, 512), (40, 0)])
@pytest.mark.parametrize("size", [1e20, 1.6e38, 3e38])
def test_large_rows(lib, dtype, inter, dim, rd, size):
    g = torch.Generator(device="cuda")
    g.manual_seed(dim)
    x = (size * torch.where(torch.rand(9, 3, dim, device="cuda", generator=g) < 0.5, -1.0, 1.0)).to(dtype)
    small = torch.randn(dim, device="cuda", generator=g).to(dtype)
    x[4, 1] = small
    for weight in (2.0, 1.0, 0.25):
        alone = run(lib, x[4:5, 1:2].expand(9, 3, dim).contiguous(), weight, rd, inter)
        for got, want in zip(run(lib, x, weight, rd, inter), alone):
            zero = torch.ones(9, 3, dtype=torch.bool, device="cuda")
            zero[4, 1] = False
            assert not got[zero].any()
            assert torch.equal(got[4, 1], want[4, 1])  # the row beside them is as ever
    bad = x.clone()
    bad[2, 0, 5], bad[3, 2, 1] = float("inf"), float("nan")
    for got in run(lib, bad, 2.0, rd, inter):
        assert not torch.isfinite(got[2, 0]).all() and not torch.isfinite(got[3, 2]).any()
        assert not got[:2].any() and not got[5:].any()
