"""idx_index_append against the definition in 64 bits.

Codes and key scales are equal to the oracle's in every entry (its angles are
off by less than 2^-35 at these positions, so that an entry which its own
rounding decides has to lie that near a border between codes; with the seeds here none does).  A
query's scale is fp32: 2^-24 times 7 sqrt 2 for the largest element, 16 for the
norm, 4 for the products with the scales; 32 of them are allowed.
"""

import numpy as np
import pytest
import torch

from oracle import serve

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def np_(t):
    return None if t is None else t.double().cpu().numpy()


class Case:
    def __init__(self, lib, tokens, heads, rd=64, inter=False, dtype="bf16", page=128, gap=0, weigh=(True, True), offset=0.0, mscale=1.0, start=100000,
                 cu=None, slots_per=8, hw=False, keys=True, size=1.0, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + tokens * 31 + heads + rd)
        dt = TYPES[dtype]
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
        self.lib, self.tokens, self.heads, self.inter, self.page, self.offset, self.mscale = lib, tokens, heads, inter, page, offset, mscale
        x = (size * rand(tokens, (heads + 1) * 128 + gap)).to(dt)
        self.q = x[:, : heads * 128].unflatten(1, (heads, 128)) if heads else None
        self.k = x[:, heads * 128 : (heads + 1) * 128] if keys else None
        w = (1.0 - offset + 0.3 * rand(2, 128)).to(dt)
        self.qw, self.kw = (w[i] if weigh[i] else None for i in (0, 1))
        self.pos = (start + 7 * torch.arange(tokens, device="cuda")).to(torch.int32)
        self.f = lib.idx_rope_frequencies(rd, 500000.0)[0] if rd else torch.zeros(0, dtype=torch.float64)
        blocks = -(-tokens // page) + 2
        self.index_k = torch.randint(0, 256, (blocks, page, 72), device="cuda", dtype=torch.uint8, generator=g)
        self.slots = torch.randperm(blocks * page, device="cuda", generator=g)[:tokens]
        if tokens > 5:
            self.slots[3] = -1
        self.cu = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
        shape = (tokens, heads) if cu is None else (len(cu) - 1, slots_per, heads)
        self.q_out = torch.full((*shape, 128), 0xAB, dtype=torch.uint8, device="cuda")
        self.q_scale = torch.full(shape, -7.0, device="cuda")
        self.hw = rand(tokens, heads) if hw else None
        self.scale = 0.125
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, **more):
        q = self.heads > 0
        self.lib.idx_index_append(self.q, self.k, self.qw, self.kw, 1e-6, self.pos, self.f.cuda(), self.q_out if q else None, self.q_scale if q else None,
                                  self.index_k if self.k is not None else None, **(dict(
                                      slots=self.slots, cu_tokens=self.cu, head_weights=self.hw, scale=self.scale, mscale=self.mscale, offset=self.offset,
                                      interleaved=self.inter, status=self.status) | more))
        return self

    def check(self, status=0):
        codes, scales, before = self.q_out.clone(), self.q_scale.clone(), self.index_k.flatten(1).cpu().numpy()
        self.run()
        assert self.status.item() == status
        eps, p, f, m = float(np.float32(1e-6)), self.pos.cpu().numpy(), self.f.numpy(), float(np.float32(self.mscale))
        if self.heads:
            want, s = serve.index_queries(np_(self.q), np_(self.qw), eps, self.offset, p, f, m, self.inter, self.scale, np_(self.hw))
            codes, scales = codes.cpu().numpy(), scales.double().cpu().numpy()
            if self.cu is None:
                codes, scales = want, s
            else:
                cu = self.cu.tolist()
                for r in range(len(cu) - 1):
                    n = min(cu[r + 1] - cu[r], codes.shape[1])
                    if n > 0:
                        codes[r, -n:], scales[r, -n:] = want[cu[r + 1] - n : cu[r + 1]], s[cu[r + 1] - n : cu[r + 1]]
            got = self.q_out.cpu().numpy()
            same = (got == codes) | ((got & 0x7F) + (codes & 0x7F) == 0)  # zeros of either sign
            assert same.all(), (np.argwhere(~same)[:5], got[~same][:5], codes[~same][:5])
            got = self.q_scale.double().cpu().numpy()
            assert np.array_equal(np.isnan(got), np.isnan(scales))
            ok = ~np.isnan(got)
            assert np.all(np.abs(got - scales)[ok] <= 32 * 2.0**-24 * np.abs(scales[ok]))
        if self.k is not None:
            code, scale = serve.index_keys(np_(self.k), np_(self.kw), eps, self.offset, p, f, m, self.inter)
            want, page = before.copy(), self.page
            for t, slot in enumerate(self.slots.tolist()):
                if 0 <= slot < before.shape[0] * page:
                    b, o = divmod(slot, page)
                    want[b, o * 64 : o * 64 + 64], want[b, page * 64 + o * 8 : page * 64 + o * 8 + 8] = code[t], scale[t]
            got = self.index_k.flatten(1).cpu().numpy()
            bad = got != want
            # a code of either zero
            codes_part = bad[:, : page * 64]
            gc, wc = got[:, : page * 64], want[:, : page * 64]
            for sh in (0, 4):
                x, y = gc >> sh & 15, wc >> sh & 15
                assert np.all((x == y) | ((x | y) == 8)), np.argwhere(codes_part)[:5]
            assert not bad[:, page * 64 :].any()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rd", [0, 16, 64, 128])
def test_types_and_parts(lib, dtype, inter, rd):
    Case(lib, 77, 5, rd=rd, inter=inter, dtype=dtype).check()
    Case(lib, 77, 5, rd=rd, inter=inter, dtype=dtype, weigh=(False, False), mscale=1.25).check()


@pytest.mark.parametrize("power", [119, 40, -40, -90])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_queries_near_the_ends_of_the_range(lib, dtype, power):
    """Weights that make rows large or small: enough rows that some have elements near a border between codes."""
    for inter in (False, True):
        c = Case(lib, 1500, 8, inter=inter, dtype=dtype, keys=False, seed=power)
        c.qw = (c.qw.double() * 2.0**power).to(c.qw.dtype)
        c.check()


@pytest.mark.parametrize("tokens,heads", [(1, 4), (1, 1), (513, 4), (300, 64), (19, 128), (40, 3), (0, 4), (9, 0)])
def test_sizes(lib, tokens, heads):
    Case(lib, tokens, heads, hw=heads > 0).check()
    Case(lib, tokens, heads, keys=heads == 0, page=256, inter=True, rd=24 if heads != 3 else 8, dtype="fp16").check()


def test_many_rows_are_exact(lib):
    """A million query elements, of which some hundred lie within fp32's errors of a border."""
    Case(lib, 1500, 8, rd=128, dtype="bf16", seed=1).check()
    Case(lib, 900, 8, rd=32, dtype="fp32", seed=2).check()


def test_values_on_borders(lib):
    """Small whole numbers at position 0: many quotients are exactly half way between two codes."""
    c = Case(lib, 200, 4, rd=64, dtype="bf16", weigh=(False, False), start=0)
    c.pos.zero_()
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    c.q.copy_(torch.randint(-28, 29, c.q.shape, device="cuda", generator=g))
    c.q[:, :, 5] = 28.0
    c.k.copy_(torch.randint(-24, 25, c.k.shape, device="cuda", generator=g).float() / 4)
    c.k[:, ::16] = 6.0  # a scale of 1: quarters are half way between halves
    c.check()
    c.k[:, ::16] = 6.75  # 6.75 / 6 is half way between two scales
    c.check()


@pytest.mark.parametrize("cu,per", [([0, 8, 16, 24], 8), ([0, 1, 1, 6, 11], 8), ([0, 3, 14], 8), ([0, 4], 8), ([0] + [2] * 70 + [9], 8), ([0, 5, 9], 3), ([0, 0, 0], 8)])
def test_slots_of_requests(lib, cu, per):
    tokens = max(cu[-1], 1) + 2  # two behind the last request
    over = any(b - a > per for a, b in zip(cu, cu[1:]))
    Case(lib, tokens, 4, cu=cu, slots_per=per).check(status=lib.ST_BAD_OUTPUT if over else 0)


def test_strides_and_alignment(lib):
    for gap in (0, 1, 4, 8):
        for dtype in TYPES:
            Case(lib, 33, 3, gap=gap, dtype=dtype).check()
            Case(lib, 33, 2, gap=gap, dtype=dtype, rd=128, inter=True).check()


def test_offsets_and_magnitudes(lib):
    Case(lib, 50, 4, offset=1.0).check()
    for size in (1e-12, 1e-3, 1e5, 1e15):
        Case(lib, 50, 4, dtype="fp32", size=size).check()
        Case(lib, 50, 4, dtype="bf16", size=size, weigh=(False, False)).check()


def test_rows_that_are_not_finite(lib):
    c = Case(lib, 40, 4)
    c.q[3, 1, 7], c.q[4, 2, 100], c.k[5, 9], c.k[6, 100] = float("inf"), float("nan"), float("-inf"), float("nan")
    c.q[7, 0] = 0.0
    c.k[8] = 0.0
    c.check()
    assert c.q_out[3, 1].eq(0x7F).all() and c.q_scale[4, 2].isnan() and c.q_scale[7, 0] == 0 and not c.q_out[7, 0].any()


def test_slots_past_the_pages_are_skipped(lib):
    c = Case(lib, 9, 2)
    c.slots[4], c.slots[5] = c.index_k.shape[0] * 128, 2**40
    c.check(status=lib.ST_BLOCK_OOR)
    c = Case(lib, 200, 0)
    c.slots = torch.arange(200, device="cuda")
    c.check()
    d = Case(lib, 200, 0).run(slots=None)
    assert torch.equal(c.index_k, d.index_k)


def test_the_scorer_reads_what_is_written(lib):
    """Queries and keys through the decode step's scores: those of the rows themselves, within the codes' steps."""
    r, n, page = 2, 3, 128
    keys = Case(lib, r * 300, 0, start=0)
    table = torch.randperm(2 * 3, device="cuda").view(2, 3).to(torch.int32)
    place = torch.arange(300, device="cuda")
    keys.slots = (table[:, :, None].long() * page + torch.arange(page, device="cuda")).flatten(1)[:, :300].flatten()
    keys.index_k = torch.zeros(6, page, 72, dtype=torch.uint8, device="cuda")
    keys.pos = torch.cat([place, place]).to(torch.int32)
    keys.check()
    queries = Case(lib, r * n, 4, cu=[0, n, 2 * n], keys=False, start=0)
    queries.pos = torch.tensor([297, 298, 299] * 2, dtype=torch.int32, device="cuda")
    queries.q_out.zero_(), queries.q_scale.zero_()
    queries.run()
    seq = torch.tensor([300, 300], dtype=torch.int32, device="cuda")
    scores = torch.zeros(r, 32, 3, device="cuda")
    pages = torch.zeros(r, n, 4, 16, dtype=torch.int32, device="cuda")
    lib.idx_decode_step(queries.q_out, queries.q_scale, keys.index_k, table, seq, n, scores, pages, None, queries.status)
    assert queries.status.item() == 0
    eps, f = float(np.float32(1e-6)), keys.f.numpy()
    kr = serve.norm_rotate(np_(keys.k)[:, None], np_(keys.kw), eps, 0.0, keys.pos.cpu().numpy(), f, 1.0, False)[:, 0].reshape(r, 300, 128)
    qr = serve.norm_rotate(np_(queries.q), np_(queries.qw), eps, 0.0, queries.pos.cpu().numpy(), f, 1.0, False).reshape(r, n, 4, 128)
    dots = np.einsum("rnhd,rkd->rnhk", qr, kr)[..., :256].reshape(r, n, 4, 2, 128).max(-1) * queries.scale
    # an element is off by at most 2^-4 of itself (E4M3) and, with the block's scale, a quarter of its block's largest (E2M1)
    got = scores.view(r, 8, 4, 3)[:, 8 - n :, :, :2].double().cpu().numpy()
    block = np.abs(kr).reshape(r, 300, 8, 16).max(-1).repeat(16, -1)
    slack = queries.scale * (np.einsum("rnhd,rkd->rnhk", np.abs(qr), 0.0625 * np.abs(kr) + 1.0625 * 0.26 * block)[..., :256].reshape(r, n, 4, 2, 128).max(-1))
    assert np.all(np.abs(got - dots) <= slack)


def test_other_streams_and_graphs(lib):
    a, b, c = (Case(lib, 2000, 4, hw=True) for _ in range(3))
    a.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.run()
    s.synchronize()
    f = c.f.cuda()
    c.f = f
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    graph.replay()
    torch.cuda.synchronize()
    for x in (b, c):
        assert torch.equal(a.q_out, x.q_out) and torch.equal(a.q_scale, x.q_scale) and torch.equal(a.index_k, x.index_k)
