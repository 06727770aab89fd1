"""idx_logit_probs at its largest sizes within bounds counted from them, and waits that do run out.

The tolerance of p, in units of 2^-24 of p, with d = (m - x) / T (m the largest x): x - m, its product with log2(e) / T and
the factor's rounding 4 d; 2^x 4, and as many for the sum's terms; A additions on a term's way into the sum; 10 for two
rescalings to a larger maximum; the reciprocal and last product 2: 4 d + A + 20.  A row of these sizes is 8 CTAs', whose 256
threads add pairs of entries of 16-byte vectors into two sums, one after another; then the two, up to 4 changed entries and a
token of a path, or (many changed entries) one of each of a warp's words of 32; and 12 times between lanes, warps and CTAs.
An x that is changed rounds at most 5 times, at no more than the largest magnitude X on its way: 12 X / T, as in the other
tests of the call.  L is off by as much in absolute terms (d = 0), and by 4 units of |m| / T.
"""

import numpy as np
import pytest
import torch

from oracle import serve

pytestmark = pytest.mark.gpu
U = 2.0**-24


def additions(vocab, size, many):
    stretch = -(-vocab // 8 // 32) * 32 + 32
    vectors = -(-(stretch + 16 // size) * size // 16)
    return -(-vectors // 256) * (8 // size) + 1 + 5 + (-(-stretch // 32 // 8) if many else 0) + 12


def check(lib, x, temperature=None, big=0.0, many=False, **args):
    rows, vocab = x.shape
    cu = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    probs, lse = torch.empty(rows, vocab, device="cuda"), torch.empty(rows, device="cuda")
    heat = None if temperature is None else torch.tensor([temperature], device="cuda")
    lib.idx_logit_probs(x, probs, cu, temperature=heat, lse=lse, **args)
    want, want_lse = serve.logit_probs(x.double().cpu().numpy(), [0, rows], None if heat is None else heat.cpu().numpy(),
                                       **{k: v.cpu().numpy() for k, v in args.items()})
    a, t = additions(vocab, x.element_size(), many), 1.0 if heat is None else float(heat.cpu())
    d = np.log(want.max(1, keepdims=True)) - np.log(want)
    tol = want * U * (4 * d + a + 20 + 12 * big / t) + 2.0**-126
    assert np.all(np.abs(probs.double().cpu().numpy() - want) <= tol)
    m = x.double().abs().max(1).values.cpu().numpy() + big
    assert np.all(np.abs(lse.double().cpu().numpy() - want_lse) <= U * (a + 20 + 12 * big / t + 4 * m / t))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("vocab", [131_072, 200_003, 262_144])
def test_sums_of_the_longest_rows(lib, dtype, vocab):
    g = torch.Generator(device="cuda")
    g.manual_seed(vocab)
    x = torch.stack([torch.zeros(vocab, device="cuda"), torch.rand(vocab, device="cuda", generator=g), 2 * torch.randn(vocab, device="cuda", generator=g)])
    x[0, 7] = -1.0
    check(lib, x.to(dtype))
    check(lib, x.to(dtype), temperature=0.37)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sums_of_changed_entries(lib, dtype):
    """Every entry counted: each is formed by itself."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.rand(2, 262_144, device="cuda", generator=g).to(dtype)
    one = lambda v: torch.tensor([v], device="cuda")
    check(lib, x, 0.9, big=4.0, many=True, counts=torch.ones(1, 262_144, dtype=torch.int32, device="cuda"), repetition=one(1.3), presence=one(0.2),
          frequency=one(0.3))


def test_waits_run_out_and_say_so(lib):
    """Rows of 1 MB asked for just before they are waited for, with a budget of 0: a call that gives up is seen within 20."""
    x = torch.randn(600, 262_144, device="cuda")
    cu = torch.arange(601, dtype=torch.int32, device="cuda")
    probs, status = torch.empty_like(x), torch.zeros(1, dtype=torch.int32, device="cuda")
    before = lib.idx_set_wait_limit(0)
    try:
        for _ in range(20):
            lib.idx_logit_probs(x, probs, cu, status=status)
            if status.item() != 0:
                break
    finally:
        assert lib.idx_set_wait_limit(before) == 0
    assert status.item() == lib.ST_TIMEOUT
    status.zero_()
    lib.idx_logit_probs(x, probs, cu, status=status)
    assert status.item() == 0
    want = torch.softmax(x[::97].double(), 1)
    # d at most 12 between normal values of a row
    assert ((probs[::97].double() - want).abs() <= want * U * (4 * 12 + additions(262_144, 4, False) + 20)).all()
