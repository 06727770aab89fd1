"""idx_logit_probs against the definition in 64 bits.

Tolerance of p, in units of 2^-24 of p, with d = (m - x) / T (m the largest x):
x - m, its product with log2(e) / T and the factor's own rounding 4 d; 2^x 4 and
as many again for the sum's terms, its additions (at most 32 a thread in a row,
9 between threads, 8 between CTAs, and a rescaling for each) 96, the reciprocal
and last product 2: 4 d + 106, for which 4 d + 128 is taken.  An x that is
changed rounds at most 5 times (products, division, sums, biases) at no more
than the largest magnitude X on its way: 5 X / T, for the entry and for the sum:
12 X / T.  Results below 2^-126 may be 0.  L is off by as much in absolute terms
(T d = 0), and by 4 units of |m| / T for its own terms.
"""

import numpy as np
import pytest
import torch

from oracle import serve

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0**-24


def np_(t):
    return None if t is None else t.cpu().numpy()


def wide(t):
    return t.double().cpu().numpy()


class Case:
    def __init__(self, cu, vocab, dtype="bf16", pad=0, gap=0, seed=0, penalties=True, tree=None, biases=0, grammar=False, heat=True, drafts=True, seen=0.05):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + vocab)
        rand = lambda *s: torch.rand(*s, device="cuda", generator=g)
        reqs, rows = len(cu) - 1, cu[-1] + pad
        self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        store = (3.0 * torch.randn(rows, vocab + gap, device="cuda", generator=g)).to(TYPES[dtype])
        self.logits = store[:, gap:]
        self.args = {}
        if heat:
            self.args["temperature"] = 0.4 + rand(reqs)
        if penalties:
            counts = torch.where(rand(reqs, vocab) < seen, (1 + 5 * rand(reqs, vocab)).int(), 0)
            counts = torch.where(rand(reqs, vocab) < seen, counts | -(2**31), counts)
            self.args |= dict(repetition=0.7 + 0.8 * rand(reqs), presence=rand(reqs) - 0.3, frequency=0.6 * rand(reqs), counts=counts.to(torch.int32))
            if drafts:
                self.args["tokens"] = (rand(rows) * vocab * 1.01).to(torch.int32) - 1
        if tree is not None:
            self.args["tree_mask"] = tree
        self.biases = None
        if biases:
            n = torch.randint(0, biases + 1, (reqs,), device="cuda", generator=g).tolist()
            tok, val = (rand(sum(n)) * vocab).to(torch.int32), 5.0 * torch.randn(sum(n), device="cuda", generator=g)
            at = np.concatenate([[0], np.cumsum(n)])
            self.args |= dict(bias_cu=torch.tensor(at, dtype=torch.int32, device="cuda"), bias_tokens=tok, bias_values=val)
            self.biases = [list(zip(tok[a:b].tolist(), val[a:b].tolist())) for a, b in zip(at, at[1:])]
        if grammar:
            self.args["allowed"] = torch.randint(0, 2**32, (rows, (vocab + 31) // 32), device="cuda", generator=g).to(torch.int32)
        self.probs = torch.full((rows, vocab + 3), 9.0, device="cuda")
        self.lse = torch.full((rows,), 9.0, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, lib, **more):
        lib.idx_logit_probs(self.logits, self.probs[:, : self.logits.shape[1]], self.cu, **(self.args | dict(lse=self.lse, status=self.status) | more))
        return self

    def check(self, lib, status=0):
        self.run(lib)
        assert self.status.item() == status
        a = {k: np_(v) for k, v in self.args.items() if not k.startswith("bias")}
        x = wide(self.logits)
        want, lse = serve.logit_probs(x, self.cu.tolist(), biases=self.biases, **a)
        got, vocab = wide(self.probs), x.shape[1]
        assert np.array_equal(got[:, vocab:], np.full((len(x), 3), 9.0))  # columns past the row stay as they are
        got = got[:, :vocab]
        assert np.array_equal(np.isnan(got), np.isnan(want))
        heat = np.ones(len(x))
        for r in range(len(self.cu) - 1):
            if "temperature" in a:
                heat[self.cu[r] : self.cu[r + 1]] = a["temperature"][r] if a["temperature"][r] > 2.0**-60 else 1.0
        finite = np.where(np.isfinite(x), np.abs(x), 0.0)
        big = 1.5 * finite.max(1) + 12 + sum(abs(b) for row in self.biases or [] for _, b in row)
        top = np.nan_to_num(want).max(1, keepdims=True)
        with np.errstate(divide="ignore", invalid="ignore"):
            d = np.where(want > 0, np.log(top) - np.log(want), 0.0)
        tol = want * U * (4 * d + 128 + 12 * (big / heat)[:, None]) + 2.0**-126
        ok = ~np.isnan(want)
        assert np.all(np.abs(got - want)[ok] <= tol[ok]), np.max((np.abs(got - want) / tol)[ok])
        got = wide(self.lse)
        assert np.array_equal(np.isnan(got), np.isnan(lse)) and np.array_equal(got == -np.inf, lse == -np.inf)
        ok = np.isfinite(lse)
        assert np.all(np.abs(got[ok] - lse[ok]) <= U * (128 + 16 * big / heat)[ok])
        return self


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [1, 2, 31, 33, 1000, 4099, 32000])
def test_sizes_and_types(lib, dtype, vocab):
    Case([0, 1, 1, 4, 9], vocab, dtype, pad=2, biases=5, grammar=vocab > 1000).check(lib)
    Case([0, 1], vocab, dtype, penalties=False, heat=False).check(lib)


@pytest.mark.parametrize("vocab", [65_537, 200_003, 262_144])
def test_large_vocabularies(lib, vocab):
    Case([0, 2, 3], vocab, "bf16", biases=50, grammar=True).check(lib)
    Case([0, 1], vocab, "fp32").check(lib)


def test_many_rows(lib):
    Case(list(range(0, 1201, 3)), 130, "fp16", biases=3).check(lib)
    Case([0, 700], 5000, "bf16").check(lib)
    Case(list(range(0, 331, 11)), 9001, "fp32", grammar=True, pad=5).check(lib)


def test_alignment(lib):
    for gap in (1, 2, 3, 5):
        for dtype in TYPES:
            Case([0, 3, 7], 777, dtype, gap=gap, grammar=True).check(lib)


@pytest.mark.parametrize("seen", [0.0, 0.5, 1.0])
def test_tokens_seen(lib, seen):
    Case([0, 4, 8], 3001, seen=seen, biases=2).check(lib)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_more_special_entries_than_a_list_holds(lib, dtype):
    """Most tokens of a stretch seen, with and without biases, masks, a greedy row; and written in place.

    Of 600 biases over these vocabularies some tokens have several, whose sums round more often than the tolerance's 5 times,
    but at far less than the largest magnitude, which the sum of all biases is part of.
    """
    for cu, vocab in (([0, 2, 3, 7], 70_001), ([0, 30, 300], 9001)):
        for biases in (0, 100, 600):
            c = Case(cu, vocab, dtype, seen=0.7, biases=biases, grammar=biases != 100)
            c.args["temperature"][1] = 0.0
            c.check(lib)
            if dtype == "fp32":
                x = c.logits.clone()
                lib.idx_logit_probs(x, x, c.cu, **c.args)
                assert torch.equal(x, c.probs[:, :vocab])


def test_only_one_penalty(lib):
    for name in ("repetition", "presence", "frequency"):
        c = Case([0, 3, 5], 501)
        for other in {"repetition", "presence", "frequency"} - {name}:
            del c.args[other]
        c.check(lib)
    c = Case([0, 3, 5], 501)
    del c.args["counts"]  # the drafted tokens alone
    c.check(lib)
    c = Case([0, 3, 5], 501)  # without any, counts are not looked at
    for name in ("repetition", "presence", "frequency"):
        del c.args[name]
    c.check(lib)


def test_trees(lib):
    bits = [1, 3, 5, 9, 19, 35, 69, 147]  # of nodes 0 .. 7, parents -1 0 0 0 1 1 2 4
    tree = torch.tensor(bits * 3, dtype=torch.int64, device="cuda")
    c = Case([0, 8, 16, 24], 90, tree=tree)
    c.args["tokens"][:] = torch.tensor([5, 7, 7, 8, 7, 9, 7, 7] * 3)  # repeated along paths and beside them
    c.check(lib)
    # masks with bits past the request's end and a tree of 64
    c = Case([0, 3, 67], 200, tree=torch.full((67,), -1, dtype=torch.int64, device="cuda"))
    c.check(lib)


def test_trees_of_more_nodes_than_a_mask_has_bits(lib):
    """Nodes from 64 on have the mask that is given, over the first 64."""
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    masks = torch.randint(-(2**62), 2**62, (150,), device="cuda", generator=g)
    masks[70:75] = 0
    Case([0, 75, 150], 130, tree=masks).check(lib)


def test_waits_that_run_out(lib):
    """With a budget of 0 a row that is not there yet is given up; the call returns, and the next one is right."""
    c = Case([0, 40, 80], 30_001, grammar=True)
    want = c.run(lib).probs.clone()
    before = lib.idx_set_wait_limit(0)
    try:
        c.run(lib)
        torch.cuda.synchronize()
    finally:
        lib.idx_set_wait_limit(before)
    assert c.status.item() in (0, lib.ST_TIMEOUT)
    c.status.zero_()
    assert torch.equal(c.run(lib).probs, want) and c.status.item() == 0


def test_long_chains(lib):
    Case([0, 300], 1000).check(lib)
    c = Case([0, 1027], 64)
    c.run(lib)
    assert c.status.item() == lib.ST_BAD_TREE  # node 1,026's path has 1,026 tokens


def test_masks_that_leave_little(lib):
    c = Case([0, 3, 6], 5000, grammar=True, biases=9)
    a = c.args["allowed"]
    a[0] = 0  # nothing
    a[1], a[1, 77] = 0, 1 << 5  # one entry
    a[2] = -1  # everything
    a[4] = 0
    c.logits[1, 77 * 32 + 5] = -1000.0
    c.logits[5, :] = float("-inf")  # nothing left though all is allowed
    a[5] = -1
    c.check(lib)
    assert not c.probs[0, :5000].any() and c.lse[0].item() == float("-inf") and c.probs[1, 77 * 32 + 5].item() == 1.0


def test_what_is_masked_has_no_effect(lib):
    c = Case([0, 2, 5], 4001, "fp32", grammar=True)
    v = torch.arange(4001, device="cuda")
    out = (c.args["allowed"][:, v >> 5] >> (v & 31)) & 1 == 0
    c.run(lib)
    clean = c.probs.clone()
    for bad in (float("nan"), float("inf"), float("-inf"), torch.finfo(torch.float32).max, torch.finfo(torch.float32).min):
        c.logits[out] = bad
        assert torch.equal(c.run(lib).probs, clean)


def test_values_that_are_not_finite(lib):
    for dtype in TYPES:
        c = Case([0, 3, 6], 300, dtype, penalties=False)
        c.logits[0, 7], c.logits[1, 9], c.logits[3, :250] = float("nan"), float("inf"), float("-inf")
        c.logits[4, 11], c.logits[4, 12] = torch.finfo(c.logits.dtype).min, float("-inf")
        c.check(lib)
        c = Case([0, 3, 6], 300, dtype, penalties=False)
        c.args["temperature"].zero_()
        c.logits[0, 7], c.logits[1, 9], c.logits[3, :250], c.logits[5] = float("nan"), float("inf"), float("-inf"), float("-inf")
        c.check(lib)
    c = Case([0, 1], 300, "fp32", penalties=False, heat=False)
    c.logits[:] = torch.finfo(torch.float32).min  # the type's lowest value everywhere: even chances
    c.check(lib)


def test_temperature_zero(lib):
    for vocab in (40, 9000, 70_001):
        c = Case([0, 4, 9], vocab, "bf16", biases=4, grammar=True)
        c.args["temperature"] = torch.tensor([0.0, 1e-30], device="cuda")
        c.check(lib)
        c.logits[:] = 1.5  # the lowest of equal ones that are left
        c.args = {"temperature": c.args["temperature"], "allowed": c.args["allowed"]}
        c.biases = None
        c.check(lib)


def test_temperatures(lib):
    c = Case([0, 1, 2, 3, 4], 2000, "fp32")
    c.args["temperature"] = torch.tensor([1e-3, 0.03, 30.0, 1e6], device="cuda")
    c.check(lib)


def test_in_place_strides_and_repeats(lib):
    c = Case([0, 3, 6], 7001, "fp32", biases=5)
    want = c.run(lib).probs[:, :7001].clone()
    x = c.logits.clone()
    lib.idx_logit_probs(x, x, c.cu, **c.args)
    assert torch.equal(x, want)
    wide_counts = torch.zeros(2, 9000, dtype=torch.int32, device="cuda")
    wide_counts[:, :7001] = c.args["counts"]
    for _ in range(5):
        c.probs.fill_(9.0)
        assert torch.equal(c.run(lib, counts=wide_counts[:, :7001]).probs[:, :7001], want)  # the same to the bit


def test_other_streams_and_graphs(lib):
    cases = [Case([0, 8, 16], 50_001, seed=s, grammar=True, biases=9) for s in (1, 2)]
    want = [c.run(lib).probs.clone() for c in cases]
    for c in cases:
        c.probs.fill_(9.0)
    streams = [torch.cuda.Stream() for _ in cases]
    for s, c in zip(streams, cases):  # two at once
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            c.run(lib)
    torch.cuda.synchronize()
    assert all(torch.equal(c.probs, w) for c, w in zip(cases, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cases[0].run(lib)
    cases[0].logits.copy_(cases[1].logits)
    for k in ("temperature", "repetition", "presence", "frequency", "counts", "tokens", "allowed"):
        cases[0].args[k].copy_(cases[1].args[k])
    graph.replay()
    torch.cuda.synchronize()
    fresh = Case([0, 8, 16], 50_001, seed=1, grammar=True, biases=9)
    fresh.logits, fresh.args = cases[0].logits, cases[0].args
    assert torch.equal(cases[0].probs, fresh.run(lib).probs)


def test_the_rows_feed_the_verification(lib):
    c = Case([0, 4, 8], 3000).run(lib)
    out = [torch.zeros(2, 4, dtype=torch.int32, device="cuda") for _ in range(2)]
    acc = torch.zeros(2, dtype=torch.int32, device="cuda")
    u = torch.rand(8, device="cuda")
    target = c.probs[:, :3000].contiguous()
    lib.idx_verify_drafts(target, None, c.args["tokens"].clamp(min=0), c.cu, u, u[:2], out[0], out[1], acc)
    from oracle import step

    a, toks, nodes = step.verify(target.cpu().numpy(), None, np_(c.args["tokens"].clamp(min=0)), np.array([-1, 0, 1, 2] * 2), np_(c.cu), np_(u), np_(u[:2]), 4)
    assert np.array_equal(np_(acc), a) and np.array_equal(np_(out[0]), toks) and np.array_equal(np_(out[1]), nodes)
