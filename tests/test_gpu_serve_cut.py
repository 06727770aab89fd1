"""The serving example: forked requests cut back into pages that they share, then served on."""

import numpy as np
import pytest
import torch
from test_gpu_serve_steps import as_bytes, check_step, load, np_

pytestmark = pytest.mark.gpu


def rows_of(s, r, n):
    """The first n tokens of request r in every cache, as bytes."""
    b = s.table[r, torch.arange(n, device="cuda") // 128].long()
    o = torch.arange(n, device="cuda") % 128
    return [as_bytes(c[:, b, o]) for c in s.caches]


def same(a, b):
    return all(np.array_equal(x, y) for x, y in zip(a, b))


def test_a_request_cut_back_into_a_shared_page(lib):
    ex = load()
    s = ex.Server(8, 700, q_heads=8, kv_heads=4, vocab=1000)
    s.admit(3, 500)
    check_step(ex, s)
    s.fork([0, 0, 1])
    check_step(ex, s)
    length = np_(s.ctx).tolist()
    keep = length[:6]
    keep[0], keep[4], keep[5] = 130, 256, 300  # inside a page of three, at the end of one, inside a page of two
    before = [rows_of(s, r, min(keep[r], 500)) for r in range(6)]
    s.release(keep)
    assert s.active == 6 and np_(s.ctx)[:6].tolist() == keep and np_(s.owned)[:6].tolist() == [-(-n // 128) for n in keep]
    # no request's next token has a place in a page of others
    for r in range(6):
        if keep[r] % 128:
            assert s.refs[s.table[r, keep[r] // 128].long()] == 0
    for _ in range(3):
        for r in range(6):
            assert same(rows_of(s, r, min(keep[r], 500)), before[r]), r
        check_step(ex, s)
    for r in range(6):
        assert same(rows_of(s, r, min(keep[r], 500)), before[r]), r
    s.release([0] * s.active)
    torch.cuda.synchronize()
    assert int(s.cursor.item()) == 0 and not s.refs.any() and int(s.status.item()) == 0
    assert torch.equal(s.free.sort().values, torch.arange(s.blocks, dtype=torch.int32, device="cuda"))


def test_a_cut_without_a_row_to_spare(lib):
    ex = load()
    s = ex.Server(2, 500, q_heads=8, kv_heads=4, vocab=1000)
    s.admit(1, 300)
    check_step(ex, s)
    s.fork([0])
    with pytest.raises(ValueError, match="row"):
        s.release([130, 309])
