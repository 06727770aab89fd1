"""What the operators around the indexer refuse: answered on the host, before any CUDA call."""

import numpy as np
import pytest
import torch

from oracle import step

E_NULL, E_SHAPE, E_MIS, E_LARGE, E_WS, E_DEVICE = -1, -2, -3, -5, -7, -8
A = 1 << 20  # a stand-in address; no call below touches it


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_nvfp4_gb300 import build

    build.build()
    import sparse_attention_indexer_nvfp4_gb300 as idx

    return idx


def refuse(fn, good, changes):
    """Each change (position, value) of good arguments gives its code; the good ones pass every check of arguments."""
    for where, value, want in changes:
        args = list(good)
        for i, v in zip(where, value) if isinstance(where, tuple) else ((where, value),):
            args[i] = v
        assert fn(*args) == want, (where, value)
    if not torch.cuda.is_available():
        assert fn(*good) == E_DEVICE


def test_build_slots(lib):
    #        ctx new own R  bt  str maxb free nf cur     nb  P  par  T   cu seq pages curo pos slots mask st stream
    good = [A, A + 64, A + 128, 4, A, 10, 10, A, 20, A + 4, 100, 16, A, 30, A, A + 8, A + 16, A + 12, A, A, A, None, None]
    refuse(lib.load_library().idx_build_slots, good, [
        (3, -1, E_SHAPE), (3, 65536, E_LARGE), (5, 9, E_SHAPE), (6, -1, E_SHAPE), (8, -1, E_SHAPE), (10, -1, E_SHAPE),
        (11, 0, E_SHAPE), (13, -1, E_SHAPE), (0, None, E_NULL), (1, None, E_NULL), (2, None, E_NULL), (4, None, E_NULL),
        (7, None, E_NULL), (9, None, E_NULL), (14, None, E_NULL), (15, None, E_NULL), (16, None, E_NULL), (17, None, E_NULL),
        (18, None, E_NULL), (19, None, E_NULL), (20, None, E_NULL), (12, None, E_NULL),  # parents and masks go together
        (17, A + 4, E_SHAPE), (16, A + 128, E_SHAPE), (15, A, E_SHAPE),  # inputs must not be overwritten
        (0, A + 2, E_MIS), (19, A + 4, E_MIS), (20, A + 4, E_MIS), (21, A + 1, E_MIS)])


def test_rope_append(lib):
    #        q qts qhs qo ots ohs hq k kts khs v vts vhs hk T  D   rd pos f  m    slots kc vc nb P  cbs   cts cht dt fl st stream
    good = [A, 640, 64, A, 256, 64, 4, A, 640, 64, A, 640, 64, 3, 9, 64, 32, A, A, 1.0, A, A, A, 5, 16, 3072, 192, 64, 0, 1, None, None]
    fn = lib.load_library().idx_rope_append
    refuse(fn, good, [
        (14, -1, E_SHAPE), (6, -1, E_SHAPE), (13, -1, E_SHAPE), (15, 0, E_SHAPE), (15, 513, E_LARGE), (16, 31, E_SHAPE), (16, 66, E_SHAPE),
        (16, -2, E_SHAPE), (23, -1, E_SHAPE), (24, 0, E_SHAPE), (28, 3, E_SHAPE), (28, -1, E_SHAPE), (29, 2, E_SHAPE), (1, -1, E_SHAPE),
        (4, 32, E_SHAPE), (5, 32, E_SHAPE), (27, 32, E_SHAPE), (26, 32, E_SHAPE), (25, 32, E_SHAPE), (0, None, E_NULL), (3, None, E_NULL),
        (7, None, E_NULL), (21, None, E_NULL), (22, None, E_NULL), (10, None, E_NULL), (17, None, E_NULL), (18, None, E_NULL),
        (0, A + 1, E_MIS), (21, A + 1, E_MIS), (18, A + 4, E_MIS), (20, A + 4, E_MIS), (14, 0, 0), ((6, 13), (0, 0), 0)])


def test_rope_frequencies(lib):
    for kind, args in ((0, {}), (1, dict(factor=4.0)), (2, dict(factor=8.0, orig_len=4096.0)), (2, dict(factor=0.5, orig_len=100.0)),
                       (2, dict(factor=40.0, orig_len=32768.0, beta_fast=16.0, beta_slow=2.0))):
        for rd, base in ((128, 10000.0), (64, 500000.0), (2, 100.0), (32, 1.5)):
            f, m = lib.idx_rope_frequencies(rd, base, kind, **args)
            want, wm = step.rope_frequencies(rd, base, kind, **args)
            np.testing.assert_allclose(f.numpy(), want, rtol=1e-14)
            assert abs(m - wm) < 1e-15
    assert lib.idx_rope_frequencies(0)[0].numel() == 0
    for bad in (dict(rotary_dim=3), dict(rotary_dim=-2), dict(rotary_dim=8, base=1.0), dict(rotary_dim=8, base=float("nan")),
                dict(rotary_dim=8, kind=3), dict(rotary_dim=8, kind=1, factor=0.0), dict(rotary_dim=8, kind=2, factor=2.0)):
        with pytest.raises(lib.IdxError) as e:
            lib.idx_rope_frequencies(**bad)
        assert e.value.code == E_SHAPE


def test_tree_attention(lib):
    need = lib.idx_tree_attention_workspace_bytes(3, 9, 16, 4, 128, 2, 16)
    assert need > 0
    for bad in ((0, 9, 16, 4, 128), (3, 0, 16, 4, 128), (3, 9, -1, 4, 128), (3, 9, 16, 0, 128), (3, 9, 16, 4, 0), (3, 9, 16, 4, 128, -1, 0)):
        assert lib.idx_tree_attention_workspace_bytes(*bad) == 0
    #        q ts    hs  kc vc nb P   cbs    cts  chs bt bts mb seq cu R T hq  hk D    mask pages li per sc  dt out ots   ohs lse ws ws_b st stream
    good = [A, 2048, 128, A, A, 50, 128, 65536, 512, 128, A, 20, 20, A, A, 3, 9, 16, 4, 128, A, A, 2, 16, 0.1, 0, A, 2048, 128, A, A, need, None, None]
    refuse(lib.load_library().idx_tree_attention, good, [
        (15, -1, E_SHAPE), (15, 65536, E_LARGE), (16, -1, E_SHAPE), (17, 15, E_SHAPE), (17, 0, E_SHAPE), (18, 0, E_SHAPE), (19, 96, E_SHAPE),
        (19, 256, E_SHAPE), (6, 48, E_SHAPE), (6, 8, E_SHAPE), (6, 0, E_SHAPE), (6, 192, E_SHAPE), (25, 2, E_SHAPE), (25, -1, E_SHAPE),
        (22, 3, E_SHAPE), (22, 0, E_SHAPE), (23, 0, E_SHAPE), (23, 65, E_LARGE), (5, -1, E_SHAPE), (5, 1 << 31, E_LARGE), (11, 19, E_SHAPE),
        (12, -1, E_SHAPE), (1, 2044, E_SHAPE), (7, -8, E_SHAPE), (8, 12, E_SHAPE), (27, 120, E_SHAPE), (28, 64, E_SHAPE), (0, None, E_NULL),
        (3, None, E_NULL), (4, None, E_NULL), (10, None, E_NULL), (13, None, E_NULL), (14, None, E_NULL), (26, None, E_NULL),
        (0, A + 8, E_MIS), (3, A + 8, E_MIS), (26, A + 2, E_MIS), (20, A + 4, E_MIS), (30, A + 16, E_MIS), (30, None, E_WS),
        (31, need - 1, E_WS), (16, 0, 0), ((17, 18), (258, 2), E_LARGE)])


def test_verify_drafts(lib):
    #        p  ps  q  qs  V   tok par cu R T  au su ot on mo na st stream
    good = [A, 100, A, 100, 100, A, A, A, 4, 20, A, A, A, A, 5, A, None, None]
    refuse(lib.load_library().idx_verify_drafts, good, [
        (1, 99, E_SHAPE), (3, 99, E_SHAPE), (4, 0, E_SHAPE), ((1, 3, 4), (2**31 - 1,) * 3, E_LARGE), (8, -1, E_SHAPE), (8, 65536, E_LARGE),
        (9, -1, E_SHAPE), (14, 0, E_SHAPE), (0, None, E_NULL), (5, None, E_NULL), (7, None, E_NULL), (10, None, E_NULL), (11, None, E_NULL),
        (12, None, E_NULL), (13, None, E_NULL), (15, None, E_NULL), (0, A + 2, E_MIS), (2, A + 2, E_MIS), (15, A + 2, E_MIS), (8, 0, 0)])


def test_the_binding_checks_tensors(lib):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    f32 = lambda *s: torch.zeros(s)
    q, cache = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    att = lambda **k: lib.idx_tree_attention(**(dict(q=q, k_cache=cache, v_cache=cache, block_table=i32(1, 2), seq_lens=i32(1), cu_tokens=i32(2),
                                                     out=torch.zeros_like(q), scale=1.0, stream=1) | k))
    for bad in (dict(q=q.half()), dict(out=torch.zeros(2, 4, 32, dtype=torch.bfloat16)), dict(cu_tokens=i32(3)), dict(seq_lens=torch.zeros(1)),
                dict(v_cache=torch.zeros(3, 16, 2, 128, dtype=torch.bfloat16)[..., ::2]), dict(lse=torch.zeros(2, 3)),
                dict(tree_mask=i32(2)), dict(pages=i32(3, 1, 4)), dict(v_cache=torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16).transpose(1, 2))):
        with pytest.raises(ValueError):
            att(**bad)
    ver = lambda **k: lib.idx_verify_drafts(**(dict(target=f32(4, 9), draft=f32(4, 9), tokens=i32(4), cu_tokens=i32(2), accept_u=f32(4), sample_u=f32(1),
                                                    out_tokens=i32(1, 3), out_nodes=i32(1, 3), num_accepted=i32(1), stream=1) | k))
    for bad in (dict(draft=f32(4, 8)), dict(target=f32(9, 4).T), dict(tokens=f32(4)), dict(sample_u=f32(2)), dict(out_nodes=i32(1, 2)),
                dict(accept_u=f32(8)[::2])):
        with pytest.raises(ValueError):
            ver(**bad)
    x = torch.zeros(5, 2, 8)
    rope = lambda **k: lib.idx_rope_append(**(dict(q=x, k=x, v=x, positions=i32(5), inv_freq=torch.zeros(4, dtype=torch.float64), q_out=x,
                                                   k_cache=f32(2, 4, 2, 8), v_cache=f32(2, 4, 2, 8), stream=1) | k))
    for bad in (dict(q_out=None), dict(k=None), dict(v_cache=None), dict(q=None, q_out=None, k=None, k_cache=None), dict(v=x.half()),
                dict(positions=i32(4)), dict(inv_freq=f32(4)), dict(v_cache=f32(2, 2, 4, 8).transpose(1, 2)), dict(q=x[:, :1]),
                dict(q=x.double(), k=x.double(), v=x.double())):
        with pytest.raises(ValueError):
            rope(**bad)
    slots = lambda **k: lib.idx_build_slots(**(dict(ctx_lens=i32(2), new_lens=i32(2), owned_pages=i32(2), block_table=i32(2, 3), free_blocks=i32(4),
                                                    free_cursor=i32(1), num_blocks=9, page_tokens=4, cu_tokens=i32(3), seq_lens=i32(2), pages_out=i32(2),
                                                    cursor_out=i32(1), positions=i32(6), slots=torch.zeros(6, dtype=torch.int64), stream=1) | k))
    for bad in (dict(new_lens=i32(3)), dict(slots=i32(6)), dict(cu_tokens=i32(2)), dict(block_table=i32(3, 2).T), dict(tree_mask=i32(6)),
                dict(parents=i32(5)), dict(free_cursor=i32(2))):
        with pytest.raises(ValueError):
            slots(**bad)
