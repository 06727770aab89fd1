"""What the calls between a decoding step's own refuse: answered on the host, before any CUDA call."""

import struct

import pytest
import torch

E_NULL, E_SHAPE, E_MIS, E_LARGE, E_DEVICE = -1, -2, -3, -5, -8
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


def test_norm_rope_append(lib):
    #        q qts qhs qo ots ohs hq k kts khs v vts vhs hk T  D   rd qw kw eps   off  pos f  m    slots kc vc nb P  cbs   cts cht dt fl st stream
    good = [A, 640, 64, A, 256, 64, 4, A, 640, 64, A, 640, 64, 3, 9, 64, 32, A, A, 1e-6, 0.0, A, A, 1.0, A, A, A, 5, 16, 3200, 192, 64, 0, 1, None, None]
    refuse(lib.load_library().idx_norm_rope_append, good, [
        (14, -1, E_SHAPE), (6, -1, E_SHAPE), (13, -1, E_SHAPE), (15, 0, E_SHAPE), (15, 513, E_LARGE), (16, 31, E_SHAPE), (16, 66, E_SHAPE),
        (19, -1.0, E_SHAPE), (19, float("nan"), E_SHAPE), (27, -1, E_SHAPE), (28, 0, E_SHAPE), (32, 3, E_SHAPE), (33, 2, E_SHAPE), (1, -1, E_SHAPE),
        (4, 32, E_SHAPE), (5, 32, E_SHAPE), (31, 32, E_SHAPE), (30, 32, E_SHAPE), (29, 32, E_SHAPE), (0, None, E_NULL), (3, None, E_NULL),
        (7, None, E_NULL), (25, None, E_NULL), (26, None, E_NULL), (10, None, E_NULL), (21, None, E_NULL), (22, None, E_NULL),
        (0, A + 1, E_MIS), (17, A + 1, E_MIS), (22, A + 4, E_MIS), (24, A + 4, E_MIS), (14, 0, 0), ((6, 13), (0, 0), 0)])


def test_index_append(lib):
    #        q qts  qhs H k kts T  rd  qw kw eps   off  pos f m    hw scale cu R S  qo qs slots ik nb P   dt fl st stream
    good = [A, 640, 128, 4, A, 640, 9, 64, A, A, 1e-6, 0.0, A, A, 1.0, A, 1.0, A, 3, 8, A, A, A, A, 5, 128, 0, 0, None, None]
    refuse(lib.load_library().idx_index_append, good, [
        (3, -1, E_SHAPE), (3, 129, E_LARGE), (6, -1, E_SHAPE), (7, 8, E_SHAPE), (7, 144, E_SHAPE), ((7, 27), (12, 1), E_SHAPE), (10, -1.0, E_SHAPE),
        (18, -1, E_SHAPE), (18, 65536, E_LARGE), (19, 0, E_SHAPE), (24, -1, E_SHAPE), (25, 64, E_SHAPE), (26, 3, E_SHAPE), (27, 2, E_SHAPE),
        (1, -1, E_SHAPE), (5, -1, E_SHAPE), (0, None, E_NULL), (20, None, E_NULL), (21, None, E_NULL), (23, None, E_NULL), (4, None, E_NULL),
        (12, None, E_NULL), (13, None, E_NULL), (0, A + 1, E_MIS), (20, A + 8, E_MIS), (23, A + 8, E_MIS), (22, A + 4, E_MIS), (21, A + 2, E_MIS),
        (6, 0, 0), ((3, 4, 23), (0, None, None), 0)])


def test_logit_probs(lib):
    #        x  xs  dt V   T  cu R heat rep pre fre cnt cs  tok mask bcu bt bv nb al as p  ps  lse st stream
    good = [A, 100, 0, 100, 9, A, 3, A, A, A, A, A, 100, A, A, A, A, A, 7, A, 4, A, 100, A, None, None]
    refuse(lib.load_library().idx_logit_probs, good, [
        (3, 0, E_SHAPE), ((1, 3, 12, 20, 22), (270_000, 270_000, 270_000, 8_500, 270_000), E_LARGE), (4, -1, E_SHAPE), (6, -1, E_SHAPE), (6, 65536, E_LARGE),
        (2, 3, E_SHAPE), (18, -1, E_SHAPE), (1, 99, E_SHAPE), (22, 99, E_SHAPE), (12, 99, E_SHAPE), (20, 3, E_SHAPE), (0, None, E_NULL),
        (5, None, E_NULL), (21, None, E_NULL), (13, None, E_NULL), (16, None, E_NULL), (17, None, E_NULL), (0, A + 1, E_MIS), (21, A + 2, E_MIS),
        (14, A + 4, E_MIS), (11, A + 2, E_MIS), (4, 0, 0)])


def cache(base=A, plane=4096, block=1024, token=64, planes=2, row=64):
    return struct.pack("Pqqqii", base, plane, block, token, planes, row)


BAD_CACHES = [(cache(plane=32), E_SHAPE), (cache(block=-1), E_SHAPE), (cache(token=48), E_SHAPE), (cache(planes=-1), E_SHAPE),
              (cache(row=-4), E_SHAPE), (cache(base=0), E_NULL), (None, E_NULL)]


def test_settle_drafts(lib):
    #        caches n nb P  slots cu R T  ot on mo acc ctx out cnt cs  V  st stream
    good = [cache(), 1, 4, 16, A, A, 3, 9, A, A, 4, A, A, A, A, 50, 50, None, None]
    refuse(lib.load_library().idx_settle_drafts, good, [(0, c, want) for c, want in BAD_CACHES] + [
        (1, -1, E_SHAPE), (1, 9, E_LARGE), (2, -1, E_SHAPE), (3, 0, E_SHAPE), (6, -1, E_SHAPE), (6, 65536, E_LARGE), (7, -1, E_SHAPE), (10, 0, E_SHAPE),
        (15, 49, E_SHAPE), (16, 0, E_SHAPE), (4, None, E_NULL), (5, None, E_NULL), (8, None, E_NULL), (9, None, E_NULL), (11, None, E_NULL),
        (12, None, E_NULL), (13, None, E_NULL), (4, A + 4, E_MIS), (9, A + 2, E_MIS), (6, 0, 0)])


def test_fork_pages(lib):
    #        caches n nb P  par ch F ctx own R bt bs mb refs free nf cur curo st stream
    good = [cache(), 1, 4, 16, A, A, 2, A, A, 5, A, 10, 10, A, A, 7, A, A + 4, None, None]
    refuse(lib.load_library().idx_fork_pages, good, [(0, c, want) for c, want in BAD_CACHES] + [
        (6, -1, E_SHAPE), (6, 4097, E_LARGE), (9, -1, E_SHAPE), (9, 65536, E_LARGE), (11, 9, E_SHAPE), (12, -1, E_SHAPE), (15, -1, E_SHAPE),
        (17, A, E_SHAPE), (4, None, E_NULL), (5, None, E_NULL), (7, None, E_NULL), (8, None, E_NULL), (10, None, E_NULL), (13, None, E_NULL),
        (14, None, E_NULL), (16, None, E_NULL), (17, None, E_NULL), (13, A + 2, E_MIS)])


def test_release_pages(lib):
    #        keep own     R bt bs mb refs nb free nf cur curo pages P  st stream
    good = [A, A + 64, 5, A, 10, 10, A, 30, A, 7, A, A + 4, A + 128, 16, None, None]
    refuse(lib.load_library().idx_release_pages, good, [
        (2, -1, E_SHAPE), (2, 65536, E_LARGE), (4, 9, E_SHAPE), (5, -1, E_SHAPE), (7, -1, E_SHAPE), (7, 1 << 31, E_LARGE), (9, -1, E_SHAPE),
        (13, 0, E_SHAPE), (11, A, E_SHAPE), (12, A + 64, E_SHAPE), (0, None, E_NULL), (1, None, E_NULL), (3, None, E_NULL), (6, None, E_NULL),
        (8, None, E_NULL), (10, None, E_NULL), (11, None, E_NULL), (12, None, E_NULL), (6, A + 2, E_MIS)])


def test_release_pages_writes_no_input(lib):
    good = [A, A + 64, 5, A, 10, 10, A, 30, A, 7, A, A + 4, A + 128, 16, None, None]
    refuse(lib.load_library().idx_release_pages, good, [(12, A, E_SHAPE)])


def calls(idx, device):
    """Each function with arguments that pass every check but, perhaps, that of the device."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)
    i64 = lambda *s: torch.zeros(s, dtype=torch.int64, device=device)
    f32 = lambda *s: torch.zeros(s, device=device)
    f64 = lambda *s: torch.zeros(s, dtype=torch.float64, device=device)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=device)
    return {
        idx.idx_norm_rope_append: dict(q=f32(5, 2, 8), k=f32(5, 2, 8), v=f32(5, 2, 8), q_weight=f32(8), k_weight=f32(8), eps=1e-6, positions=i32(5),
                                       inv_freq=f64(4), slots=torch.arange(5, device=device), q_out=f32(5, 2, 8), k_cache=f32(2, 4, 2, 8),
                                       v_cache=f32(2, 4, 2, 8), status=i32(1)),
        idx.idx_index_append: dict(q=f32(5, 2, 128), k=f32(5, 128), q_weight=f32(128), k_weight=f32(128), eps=1e-6, positions=i32(5), inv_freq=f64(32),
                                   q_out=u8(1, 8, 2, 128), q_scale=f32(1, 8, 2), index_k=u8(2, 128, 72), slots=torch.arange(5, device=device),
                                   cu_tokens=i32(2), head_weights=f32(5, 2), status=i32(1)),
        idx.idx_logit_probs: dict(logits=f32(4, 9), probs=f32(4, 9), cu_tokens=i32(3), temperature=f32(2), repetition=f32(2), presence=f32(2),
                                  frequency=f32(2), counts=i32(2, 9), tokens=i32(4), tree_mask=i64(4), bias_cu=i32(3), bias_tokens=i32(2),
                                  bias_values=f32(2), allowed=i32(4, 1), lse=f32(4), status=i32(1)),
        idx.idx_settle_drafts: dict(caches=[f32(2, 3, 4, 5)], slots=i64(6), cu_tokens=i32(3), out_tokens=i32(2, 3), out_nodes=i32(2, 3),
                                    num_accepted=i32(2), ctx_lens=i32(2), ctx_out=i32(2), counts=i32(2, 7), status=i32(1)),
        idx.idx_fork_pages: dict(caches=[f32(2, 3, 4, 5)], parents=i32(1), children=torch.ones(1, dtype=torch.int32, device=device), ctx_lens=i32(2),
                                 owned_pages=i32(2), block_table=i32(2, 3), refs=i32(3), free_blocks=i32(4), free_cursor=i32(1), cursor_out=i32(1),
                                 status=i32(1)),
        idx.idx_release_pages: dict(keep_lens=i32(2), owned_pages=i32(2), block_table=i32(2, 3), refs=i32(9), free_blocks=i32(4), free_cursor=i32(1),
                                    cursor_out=i32(1), pages_out=i32(2), page_tokens=4, status=i32(1)),
    }


def test_host_tensors_and_statuses_are_refused(lib):
    for fn, args in calls(lib, "cpu").items():
        with pytest.raises(ValueError, match="is on cpu"):
            fn(**args, stream=1)
        for bad, what in ((torch.zeros(1), "status has type"), (torch.zeros(0, dtype=torch.int32), "status has no element")):
            with pytest.raises(ValueError, match=what):
                fn(**(args | dict(status=bad)), stream=1)


def test_the_binding_checks_tensors(lib):
    good = {fn.__name__: (fn, args) for fn, args in calls(lib, "cpu").items()}
    i32, half = lambda *s: torch.zeros(s, dtype=torch.int32), lambda *s: torch.zeros(s, dtype=torch.float16)
    for name, what in [
        ("idx_norm_rope_append", [dict(q_out=None), dict(k=None), dict(v_cache=None), dict(q=None, q_out=None, k=None, k_cache=None), dict(q_weight=torch.zeros(7)),
                                  dict(k_weight=half(8)), dict(positions=i32(4)), dict(v=half(5, 2, 8)), dict(slots=i32(5)),
                                  dict(v_cache=torch.zeros(2, 2, 4, 8).transpose(1, 2))]),
        ("idx_index_append", [dict(q_out=None), dict(index_k=None), dict(q=None, q_out=None, q_scale=None, k=None, index_k=None), dict(q_scale=torch.zeros(1, 8, 3)),
                              dict(q=torch.zeros(5, 2, 64)), dict(index_k=torch.zeros(2, 128, 64, dtype=torch.uint8)), dict(head_weights=torch.zeros(5, 3)),
                              dict(cu_tokens=i32(4)), dict(cu_tokens=None), dict(k=half(5, 128)), dict(q_weight=torch.zeros(64))]),
        ("idx_logit_probs", [dict(probs=half(4, 9)), dict(probs=torch.zeros(4, 8)), dict(cu_tokens=i32(4)), dict(temperature=torch.zeros(3)), dict(counts=i32(2, 8)),
                             dict(counts=torch.zeros(2, 9)), dict(tokens=None), dict(tree_mask=i32(4)), dict(bias_tokens=None), dict(bias_values=torch.zeros(3)),
                             dict(allowed=i32(4, 2)), dict(lse=torch.zeros(3)), dict(logits=torch.zeros(4, 9, dtype=torch.int64)),
                             dict(logits=torch.zeros(9, 4).T)]),
        ("idx_settle_drafts", [dict(caches=[torch.zeros(3, 4, 5)]), dict(caches=[torch.zeros(2, 3, 4, 5), torch.zeros(2, 3, 5, 5)]), dict(slots=i32(6)),
                               dict(out_tokens=i32(2, 4)), dict(ctx_out=i32(3)), dict(counts=i32(3, 7))]),
        ("idx_fork_pages", [dict(caches=[torch.zeros(2, 4, 4, 5)]), dict(children=i32(2)), dict(owned_pages=i32(3)), dict(page_tokens=8), dict(caches=[]),
                            dict(cursor_out=i32(2)), dict(block_table=i32(3, 2).T)]),
        ("idx_release_pages", [dict(keep_lens=i32(3)), dict(refs=torch.zeros(9)), dict(pages_out=i32(1)), dict(free_cursor=i32(2)), dict(owned_pages=torch.zeros(2))]),
    ]:
        fn, args = good[name]
        for bad in what:
            with pytest.raises(ValueError):
                fn(**(args | bad), stream=1)


def test_index_caches(lib):
    pages = torch.arange(2 * 128 * 72).to(torch.uint8).view(2, 128, 72)
    codes, scales = lib.index_caches(pages)
    assert codes.shape == (1, 2, 128, 64) and scales.shape == (1, 2, 128, 8)
    flat = pages.flatten(1)
    assert torch.equal(codes[0, 1, 5], flat[1, 5 * 64 : 6 * 64]) and torch.equal(scales[0, 1, 5], flat[1, 8192 + 40 : 8192 + 48])
    with pytest.raises(ValueError):
        lib.index_caches(pages[:, :, :64])


@pytest.mark.gpu
def test_one_host_tensor_is_refused_by_name(lib):
    """Among tensors of the GPU: answered before anything is launched."""
    for fn, args in calls(lib, "cuda").items():
        for name, t in args.items():
            if torch.is_tensor(t):
                with pytest.raises(ValueError, match=f"{name} is on cpu"):
                    fn(**(args | {name: t.cpu()}))
        if "caches" in args:
            with pytest.raises(ValueError, match="a cache is on cpu"):
                fn(**(args | {"caches": [args["caches"][0].cpu()]}))


@pytest.mark.gpu
def test_tensors_of_the_gpu_pass(lib):
    for fn, args in calls(lib, "cuda").items():
        assert fn(**args) == 0
        assert fn(**(args | dict(status=None))) == 0
    torch.cuda.synchronize()
