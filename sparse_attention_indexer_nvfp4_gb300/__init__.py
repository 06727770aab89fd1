"""Python binding of libidx.so, the GB300 sparse-attention indexer library.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Functions take torch CUDA tensors (device memory and streams are
PyTorch's), read their data pointers and shapes, and call the C entry point
of the same name declared in include/idx.h.  A negative return code raises
IdxError.  The library is loaded on first use; if it has not been built the
call fails loudly (there is no fallback).
"""

from __future__ import annotations

import ctypes
import os

__all__ = [
    "IdxError",
    "load_library",
    "library_path",
    "idx_strerror",
    "idx_have_qmul4",
    "idx_workspace_bytes",
    "idx_decode_workspace_bytes",
    "idx_decode_fused_workspace_bytes",
    "idx_set_wait_limit",
    "DEFAULT_WAIT_POLLS",
    "idx_dequant_nvfp4_pages",
    "idx_score_pages",
    "idx_topk16_select",
    "idx_topk16_select_noalloc",
    "NOALLOC_SCRATCH_BYTES",
    "idx_decode_step",
    "RANK_16BIT",
    "PAGE_256",
    "FUSED_SELECT",
    "idx_mtp_score_fp8",
    "idx_prefill_workspace_bytes",
    "idx_prefill_index_step",
    "idx_mxfp8_quantize",
    "idx_fp8_mma_probe",
    "idx_build_slots",
    "idx_rope_frequencies",
    "ROPE_PLAIN",
    "ROPE_LINEAR",
    "ROPE_RAMP",
    "idx_rope_append",
    "idx_tree_attention_workspace_bytes",
    "idx_tree_attention",
    "idx_verify_drafts",
    "VERIFY_MAX_NODES",
    "SYMBOLS",
    "ST_BLOCK_OOR",
    "ST_LEN_CLAMPED",
    "ST_BAD_OUTPUT",
    "ST_TIMEOUT",
    "ST_NO_BLOCKS",
    "ST_BAD_TREE",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "_lib", "libidx.so")
_LIB = None

ST_BLOCK_OOR = 1
ST_LEN_CLAMPED = 2
ST_BAD_OUTPUT = 4
ST_TIMEOUT = 8
ST_NO_BLOCKS = 16
ST_BAD_TREE = 32
NOALLOC_SCRATCH_BYTES = 4 << 20  # scratch inside the library used by idx_topk16_select_noalloc
DEFAULT_WAIT_POLLS = 100_000  # pipeline-wait budget of the tensor-core kernels (about 2 s)

_p = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t
_f32 = ctypes.c_float
_f64 = ctypes.c_double

# name -> (restype, argtypes); mirrors include/idx.h
SYMBOLS = {
    "idx_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "idx_have_qmul4": (ctypes.c_int, []),
    "idx_workspace_bytes": (_sz, [_i32, _i32]),
    "idx_decode_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "idx_decode_fused_workspace_bytes": (_sz, [_i32]),
    "idx_set_wait_limit": (ctypes.c_uint32, [ctypes.c_uint32]),
    "idx_dequant_nvfp4_pages": (ctypes.c_int, [_p, _i64, _p, _i64, _i32, _p, _p, _i32, _i32, _p, _i64, _p, _p]),
    "idx_score_pages": (ctypes.c_int, [_p, _p, _p, _i64, _p, _i64, _i32, _p, _i32, _i32, _i32, _p, _p, _p]),
    "idx_topk16_select": (ctypes.c_int, [_p, _i64, _i32, _i32, _p, _i32, _i32, _p, _p, _p, _sz, _p]),
    "idx_topk16_select_noalloc": (ctypes.c_int, [_p, _i64, _i32, _i32, _p, _i32, _i32, _p, _p, _p]),
    "idx_decode_step": (ctypes.c_int, [_p, _p, _p, _i64, _p, _i64, _i32, _p, _i32, _i32, _i32, _p, _p, _p, _sz, _i32, _p,
                                       _p]),
    "idx_mtp_score_fp8": (ctypes.c_int, [_p, _p, _i32, _i32, _p, _p, _i64, _p, _i64, _i32, _p, _p, _i32, _i32, _p, _p, _p]),
    "idx_prefill_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "idx_prefill_index_step": (ctypes.c_int, [_p, _i64, _p, _i64, _i32, _p, _p, _i32, _p, _p, _i32, _i32, _i32, _p, _p,
                                              _p, _sz, _p, _p]),
    "idx_mxfp8_quantize": (ctypes.c_int, [_p, _i64, _i64, _i64, _p, _i64, _p, _i64, _p]),
    "idx_fp8_mma_probe": (ctypes.c_int, [_i32, _p, ctypes.POINTER(ctypes.c_double), _p, _p]),
    "idx_build_slots": (ctypes.c_int, [_p, _p, _p, _i32, _p, _i64, _i32, _p, _i32, _p, _i64, _i32, _p, _i32, _p, _p, _p, _p,
                                       _p, _p, _p, _p, _p]),
    "idx_rope_frequencies": (ctypes.c_int, [_i32, _f64, _i32, _f64, _f64, _f64, _f64, _p, _p]),
    "idx_rope_append": (ctypes.c_int, [_p, _i64, _i64, _p, _i64, _i64, _i32, _p, _i64, _i64, _p, _i64, _i64, _i32, _i32,
                                       _i32, _i32, _p, _p, _f32, _p, _p, _p, _i64, _i32, _i64, _i64, _i64, _i32, _i32, _p,
                                       _p]),
    "idx_tree_attention_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32]),
    "idx_tree_attention": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _i64, _i32, _i64, _i64, _i64, _p, _i64, _i32, _p, _p, _i32,
                                          _i32, _i32, _i32, _i32, _p, _p, _i32, _i32, _f32, _i32, _p, _i64, _i64, _p, _p,
                                          _sz, _p, _p]),
    "idx_verify_drafts": (ctypes.c_int, [_p, _i64, _p, _i64, _i32, _p, _p, _p, _i32, _i32, _p, _p, _p, _p, _i32, _p, _p,
                                         _p]),
}


class IdxError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {code} ({idx_strerror(code)})")


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libidx.so (built by sparse_attention_indexer_nvfp4_gb300.build)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(
                f"{_LIB_PATH} is missing: build it with `python -m sparse_attention_indexer_nvfp4_gb300.build` "
                "(there is no CPU fallback)"
            )
        lib = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in SYMBOLS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _row_stride(t) -> int:
    """Elements between rows; a single-row tensor's stride is its width."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _width(scores, width) -> int:
    """Columns to rank: the tensor's width, or a narrower override (never wider)."""
    if width is None:
        return scores.shape[1]
    width = int(width)
    if width > scores.shape[-1]:
        raise ValueError(f"width {width} exceeds the score tensor's {scores.shape[-1]} columns")
    return width


def _stream(stream) -> int | None:
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, rc: int) -> int:
    if rc < 0:
        raise IdxError(fn, rc)
    return rc


def idx_strerror(code: int) -> str:
    return load_library().idx_strerror(code).decode()


def idx_have_qmul4() -> bool:
    return bool(load_library().idx_have_qmul4())


def idx_workspace_bytes(rows: int, width: int) -> int:
    return int(load_library().idx_workspace_bytes(rows, width))


def idx_decode_workspace_bytes(num_reqs: int, query_len: int, width: int) -> int:
    return int(load_library().idx_decode_workspace_bytes(num_reqs, query_len, width))


def idx_decode_fused_workspace_bytes(num_reqs: int) -> int:
    """Workspace of a decode step with FUSED_SELECT (zero-filled before its first use)."""
    return int(load_library().idx_decode_fused_workspace_bytes(num_reqs))


def idx_set_wait_limit(polls: int) -> int:
    """Set the tensor-core kernels' pipeline-wait budget (suspended polls); returns the previous one."""
    return int(load_library().idx_set_wait_limit(int(polls)))


def idx_dequant_nvfp4_pages(kv, block_table, num_pages, page_offsets, max_num_pages: int, out, status=None,
                            stream=None) -> int:
    """kv [num_blocks,128,72] u8; block_table [R, maxb] i32; out [>=sum,128,128] u8/e4m3."""
    lib = load_library()
    return _check("idx_dequant_nvfp4_pages", lib.idx_dequant_nvfp4_pages(
        _ptr(kv), kv.shape[0], _ptr(block_table), _row_stride(block_table), block_table.shape[1], _ptr(num_pages),
        _ptr(page_offsets), block_table.shape[0], int(max_num_pages), _ptr(out), out.shape[0], _ptr(status),
        _stream(stream)))


def idx_score_pages(q, q_scale, kv, block_table, seq_lens, query_len: int, scores, status=None, stream=None) -> int:
    """q [B,8,4,128] e4m3; q_scale [B,8,4] f32; scores [B,32,width] f32."""
    lib = load_library()
    return _check("idx_score_pages", lib.idx_score_pages(
        _ptr(q), _ptr(q_scale), _ptr(kv), kv.shape[0], _ptr(block_table), _row_stride(block_table),
        block_table.shape[1], _ptr(seq_lens), seq_lens.shape[0], int(query_len), scores.shape[-1], _ptr(scores),
        _ptr(status), _stream(stream)))


def idx_topk16_select(scores, out_idx, valid_n=None, force_begin: int = 0, force_end: int = 0, out_keys=None,
                      workspace=None, width: int | None = None, stream=None) -> int:
    """scores [rows, >=width] f32 -> out_idx [rows,16] i32 (+ out_keys [rows,16] u64/i64)."""
    lib = load_library()
    rows = scores.shape[0]
    width = _width(scores, width)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return _check("idx_topk16_select", lib.idx_topk16_select(
        _ptr(scores), _row_stride(scores), rows, width, _ptr(valid_n), int(force_begin), int(force_end), _ptr(out_idx),
        _ptr(out_keys), _ptr(workspace), ws_bytes, _stream(stream)))


def idx_topk16_select_noalloc(scores, out_idx, valid_n=None, force_begin: int = 0, force_end: int = 0,
                              out_keys=None, width: int | None = None, stream=None) -> int:
    """idx_topk16_select for callers that cannot allocate: the split-row scratch
    is the library's own device array (at most NOALLOC_SCRATCH_BYTES)."""
    lib = load_library()
    rows = scores.shape[0]
    width = _width(scores, width)
    return _check("idx_topk16_select_noalloc", lib.idx_topk16_select_noalloc(
        _ptr(scores), _row_stride(scores), rows, width, _ptr(valid_n), int(force_begin), int(force_end),
        _ptr(out_idx), _ptr(out_keys), _stream(stream)))


RANK_16BIT = 1  # idx_decode_step flag: rank the scores rounded to binary16
PAGE_256 = 2  # idx_decode_step flag: P256 pages (scores_ws [B, 32, 2 * width], a page the max of a column pair)
FUSED_SELECT = 4  # idx_decode_step flag: selection inside the scorer's CTAs (zero-filled fused workspace)


def idx_decode_step(q, q_scale, kv, block_table, seq_lens, query_len: int, scores_ws, out, workspace=None,
                    status=None, stream=None, flags: int = 0) -> int:
    """One decode step: scores into scores_ws [B,32,width] ([B,32,2*width] with PAGE_256), rows into
    out [B,query_len,4,16] i32."""
    lib = load_library()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    width = scores_ws.shape[-1] // (2 if flags & PAGE_256 else 1)
    return _check("idx_decode_step", lib.idx_decode_step(
        _ptr(q), _ptr(q_scale), _ptr(kv), kv.shape[0], _ptr(block_table), _row_stride(block_table),
        block_table.shape[1], _ptr(seq_lens), seq_lens.shape[0], int(query_len), width,
        _ptr(scores_ws), _ptr(out), _ptr(workspace), ws_bytes, int(flags), _ptr(status), _stream(stream)))


def idx_mtp_score_fp8(q, q_scale, k, k_scale, block_table, num_keys, cu_tokens, max_keys: int, out, status=None,
                      stream=None) -> int:
    """q [T,H,128] e4m3; k [nb,128,128] e4m3; k_scale [nb,128] f32; out [T,max_keys] f32."""
    lib = load_library()
    return _check("idx_mtp_score_fp8", lib.idx_mtp_score_fp8(
        _ptr(q), _ptr(q_scale), q.shape[0], q.shape[1], _ptr(k), _ptr(k_scale), k.shape[0], _ptr(block_table),
        _row_stride(block_table), block_table.shape[1], _ptr(num_keys), _ptr(cu_tokens), num_keys.shape[0],
        int(max_keys), _ptr(out), _ptr(status), _stream(stream)))


def idx_prefill_workspace_bytes(num_reqs: int, max_blocks: int, num_tokens: int, max_keys: int) -> int:
    return int(load_library().idx_prefill_workspace_bytes(num_reqs, max_blocks, num_tokens, max_keys))


def idx_prefill_index_step(kv, block_table, num_keys, cu_tokens, q, q_scale, max_keys: int, scores, out, workspace,
                           status=None, stream=None) -> int:
    """Prefill chain: kv [nb,128,72] u8 NVFP4 pages; q [T,H,128] e4m3; scores [T,max_keys] f32; out [T,16] i32;
    workspace of idx_prefill_workspace_bytes(...) bytes."""
    lib = load_library()
    ws_bytes = workspace.numel() * workspace.element_size()
    return _check("idx_prefill_index_step", lib.idx_prefill_index_step(
        _ptr(kv), kv.shape[0], _ptr(block_table), _row_stride(block_table), block_table.shape[1], _ptr(num_keys),
        _ptr(cu_tokens), num_keys.shape[0], _ptr(q), _ptr(q_scale), q.shape[0], q.shape[1], int(max_keys),
        _ptr(scores), _ptr(out), _ptr(workspace), ws_bytes, _ptr(status), _stream(stream)))


def idx_mxfp8_quantize(x, out, scales, stream=None) -> int:
    """x [rows, cols] bf16 -> out [rows, cols] E4M3 bytes (uint8), scales [rows, cols // 32] E8M0 bytes (uint8)."""
    lib = load_library()
    return _check("idx_mxfp8_quantize", lib.idx_mxfp8_quantize(
        _ptr(x), x.shape[0], x.shape[1], x.stride(0), _ptr(out), out.stride(0), _ptr(scales), scales.stride(0),
        _stream(stream)))


def idx_fp8_mma_probe(iters: int, check=None, status=None, stream=None) -> float:
    """Launch the dense FP8 tensor-core probe; returns the launch's floating-point operations."""
    lib = load_library()
    flops = ctypes.c_double(0.0)
    _check("idx_fp8_mma_probe", lib.idx_fp8_mma_probe(int(iters), _ptr(check), ctypes.byref(flops), _ptr(status),
                                                        _stream(stream)))
    return float(flops.value)


# ---------------------------------------------------------------------------
# One step of decoding with drafted tokens, around the indexer
# ---------------------------------------------------------------------------

ROPE_PLAIN, ROPE_LINEAR, ROPE_RAMP = 0, 1, 2  # idx_rope_frequencies kinds
VERIFY_MAX_NODES = 1024  # tokens a request of idx_verify_drafts
_ROPE_INTERLEAVED = 1
_DTYPES = {"torch.bfloat16": 0, "torch.float16": 1, "torch.float32": 2}
_code_of: dict = {}  # dtype object -> code


def _dtype_code(name: str, *tensors) -> int:
    """The element type's code; all given tensors (None left out) must share it."""
    first = None
    for t in tensors:
        if t is None:
            continue
        if first is None:
            first = t.dtype
        elif t.dtype != first:
            raise ValueError(f"{name}: tensors of one element type are needed, got {first} and {t.dtype}")
    code = _code_of.get(first)
    if code is None:
        code = _DTYPES.get(str(first))
        if code is None:
            raise ValueError(f"{name}: bfloat16, float16 or float32 is needed, got {first}")
        _code_of[first] = code
    return code


def _want(name: str, **tensors) -> None:
    """Each given tensor contiguous along its rows: (tensor, dtype name, dimensions, first sizes or None)."""
    for arg, (t, dtype, shape) in tensors.items():
        if t is None:
            continue
        if _names.setdefault(t.dtype, str(t.dtype)) not in dtype:
            raise ValueError(f"{name}: {arg} has type {t.dtype}, {' or '.join(dtype)} is needed")
        have = t.shape
        if len(have) != len(shape) or any(w is not None and w != h for w, h in zip(shape, have)):
            raise ValueError(f"{name}: {arg} has shape {tuple(have)}, {tuple('any' if w is None else w for w in shape)} is needed")


_names: dict = {}  # dtype object -> its name
_I32, _I64, _F32 = ("torch.int32",), ("torch.int64", "torch.uint64"), ("torch.float32",)
_F64 = ("torch.float64",)


def _packed(name: str, **tensors) -> None:
    for arg, t in tensors.items():
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name}: {arg} must be contiguous")


def _inner(name: str, **tensors) -> None:
    for arg, t in tensors.items():
        if t is not None and t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError(f"{name}: the last dimension of {arg} must be contiguous")


def idx_build_slots(ctx_lens, new_lens, owned_pages, block_table, free_blocks, free_cursor, num_blocks: int,
                    page_tokens: int, cu_tokens, seq_lens, pages_out, cursor_out, positions, slots, parents=None,
                    tree_mask=None, status=None, stream=None) -> int:
    """Block tables (block_table [R, maxb] i32, in place), slots [T] i64 and positions [T] i32 of a step's tokens
    from ctx_lens / new_lens / owned_pages [R] i32 and the free list; with parents [T] i32 also tree_mask [T] i64."""
    lib = load_library()
    fn = "idx_build_slots"
    reqs, tokens = ctx_lens.shape[0], positions.shape[0]
    _want(fn, ctx_lens=(ctx_lens, _I32, (reqs,)), new_lens=(new_lens, _I32, (reqs,)), owned_pages=(owned_pages, _I32, (reqs,)),
          block_table=(block_table, _I32, (reqs, None)), free_blocks=(free_blocks, _I32, (None,)),
          free_cursor=(free_cursor, _I32, (1,)), cu_tokens=(cu_tokens, _I32, (reqs + 1,)), seq_lens=(seq_lens, _I32, (reqs,)),
          pages_out=(pages_out, _I32, (reqs,)), cursor_out=(cursor_out, _I32, (1,)), positions=(positions, _I32, (tokens,)),
          slots=(slots, _I64, (tokens,)), parents=(parents, _I32, (tokens,)), tree_mask=(tree_mask, _I64, (tokens,)))
    _packed(fn, ctx_lens=ctx_lens, new_lens=new_lens, owned_pages=owned_pages, free_blocks=free_blocks, cu_tokens=cu_tokens,
            seq_lens=seq_lens, pages_out=pages_out, positions=positions, slots=slots, parents=parents, tree_mask=tree_mask)
    _inner(fn, block_table=block_table)
    return _check(fn, lib.idx_build_slots(
        _ptr(ctx_lens), _ptr(new_lens), _ptr(owned_pages), reqs, _ptr(block_table), _row_stride(block_table),
        block_table.shape[1], _ptr(free_blocks), free_blocks.shape[0], _ptr(free_cursor), int(num_blocks),
        int(page_tokens), _ptr(parents), tokens, _ptr(cu_tokens), _ptr(seq_lens), _ptr(pages_out), _ptr(cursor_out),
        _ptr(positions), _ptr(slots), _ptr(tree_mask), _ptr(status), _stream(stream)))


def idx_rope_frequencies(rotary_dim: int, base: float = 10000.0, kind: int = ROPE_PLAIN, factor: float = 1.0,
                         orig_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """Rotary frequencies as a float64 host tensor [rotary_dim // 2] (move it to the GPU once) and the mscale to pass."""
    import torch

    f = torch.zeros(max(0, int(rotary_dim)) // 2, dtype=torch.float64)
    m = ctypes.c_double(1.0)
    _check("idx_rope_frequencies", load_library().idx_rope_frequencies(
        int(rotary_dim), float(base), int(kind), float(factor), float(orig_len), float(beta_fast), float(beta_slow),
        f.data_ptr() if f.numel() else None, ctypes.addressof(m)))
    return f, float(m.value)


def idx_rope_append(q, k, v, positions, inv_freq, q_out, k_cache, v_cache, slots=None, mscale: float = 1.0,
                    interleaved: bool = False, status=None, stream=None) -> int:
    """Rotate q [T,Hq,D] into q_out and k [T,Hk,D] into the cache [nb,P,Hk,D], v beside it, at slots [T] i64 (None:
    slot t).  q and q_out, or k, v and the caches, or v and v_cache may be None."""
    lib = load_library()
    fn = "idx_rope_append"
    code = _dtype_code(fn, q, q_out, k, v, k_cache, v_cache)
    for pair, x, y in (("q and q_out", q, q_out), ("k and k_cache", k, k_cache), ("v and v_cache", v, v_cache)):
        if (x is None) != (y is None):
            raise ValueError(f"{fn}: {pair} go together")
    some = q if q is not None else k
    if some is None or (v is not None and k is None):
        raise ValueError(f"{fn}: q, or k (with or without v), is needed")
    tokens, dim = some.shape[0], some.shape[-1]
    hq = 0 if q is None else q.shape[1]
    hk = 0 if k is None else k.shape[1]
    kind = (str(some.dtype),)
    _want(fn, q=(q, kind, (tokens, hq, dim)), q_out=(q_out, kind, (tokens, hq, dim)), k=(k, kind, (tokens, hk, dim)),
          v=(v, kind, (tokens, hk, dim)), k_cache=(k_cache, kind, (None, None, hk, dim)),
          v_cache=(v_cache, kind, (None, None, hk, dim)), positions=(positions, _I32, (tokens,)),
          inv_freq=(inv_freq, _F64, (None,)), slots=(slots, _I64, (tokens,)))
    _inner(fn, q=q, q_out=q_out, k=k, v=v, k_cache=k_cache, v_cache=v_cache)
    _packed(fn, positions=positions, inv_freq=inv_freq, slots=slots)
    if v_cache is not None and (v_cache.shape != k_cache.shape or v_cache.stride() != k_cache.stride()):
        raise ValueError(f"{fn}: k_cache and v_cache must have the same shape and strides")
    qs = (0, 0, 0) if q is None else q.stride()
    os_ = (0, 0, 0) if q is None else q_out.stride()
    ks = (0, 0, 0) if k is None else k.stride()
    vs = (0, 0, 0) if v is None else v.stride()
    cs = (0, 0, 0, 0) if k is None else k_cache.stride()
    nb, page = (0, 1) if k is None else k_cache.shape[:2]
    return _check(fn, lib.idx_rope_append(
        _ptr(q), qs[0], qs[1], _ptr(q_out), os_[0], os_[1], hq, _ptr(k), ks[0], ks[1], _ptr(v), vs[0], vs[1], hk, tokens, dim,
        2 * inv_freq.shape[0], _ptr(positions), _ptr(inv_freq), float(mscale), _ptr(slots), _ptr(k_cache), _ptr(v_cache), nb,
        page, cs[0], cs[1], cs[2], code, _ROPE_INTERLEAVED if interleaved else 0, _ptr(status), _stream(stream)))


def idx_tree_attention_workspace_bytes(num_reqs: int, num_tokens: int, q_heads: int, kv_heads: int, head_dim: int,
                                       page_lists: int = 0, pages_per_list: int = 0) -> int:
    return int(load_library().idx_tree_attention_workspace_bytes(num_reqs, num_tokens, q_heads, kv_heads, head_dim,
                                                                 page_lists, pages_per_list))


def idx_tree_attention(q, k_cache, v_cache, block_table, seq_lens, cu_tokens, out, scale: float, tree_mask=None, pages=None,
                       lse=None, workspace=None, status=None, stream=None) -> int:
    """q [T,Hq,D] over the cache [nb,P,Hk,D] of each token's request -> out [T,Hq,D] (+ lse [T,Hq] f32); tree_mask [T] i64
    (None: a chain); pages [T,lists,per] i32 (or idx_decode_step's [R,query_len,lists,per]): only those pages."""
    lib = load_library()
    fn = "idx_tree_attention"
    code = _dtype_code(fn, q, k_cache, v_cache, out)
    tokens, hq, dim = q.shape
    nb, page, hk = k_cache.shape[:3]
    reqs = seq_lens.shape[0]
    kind = (str(q.dtype),)
    lists = per = 0
    if pages is not None:
        lists, per = pages.shape[-2:]
        _want(fn, pages=(pages, _I32, (tokens, lists, per) if pages.dim() == 3 else (None, None, lists, per)))
        if pages.numel() != tokens * lists * per:
            raise ValueError(f"{fn}: pages has {pages.numel()} entries, {tokens * lists * per} are needed")
    _want(fn, out=(out, kind, (tokens, hq, dim)), k_cache=(k_cache, kind, (nb, page, hk, dim)),
          v_cache=(v_cache, kind, (nb, page, hk, dim)), block_table=(block_table, _I32, (reqs, None)),
          seq_lens=(seq_lens, _I32, (reqs,)), cu_tokens=(cu_tokens, _I32, (reqs + 1,)), tree_mask=(tree_mask, _I64, (tokens,)),
          lse=(lse, _F32, (tokens, hq)))
    _inner(fn, q=q, k_cache=k_cache, v_cache=v_cache, out=out, block_table=block_table)
    _packed(fn, seq_lens=seq_lens, cu_tokens=cu_tokens, tree_mask=tree_mask, lse=lse, pages=pages)
    cs = k_cache.stride()
    if v_cache.stride() != cs:
        raise ValueError(f"{fn}: k_cache and v_cache must have the same strides")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    qs, os_ = q.stride(), out.stride()
    return _check(fn, lib.idx_tree_attention(
        _ptr(q), qs[0], qs[1], _ptr(k_cache), _ptr(v_cache), nb, page, cs[0], cs[1], cs[2], _ptr(block_table),
        _row_stride(block_table), block_table.shape[1], _ptr(seq_lens), _ptr(cu_tokens), reqs, tokens, hq, hk, dim,
        _ptr(tree_mask), _ptr(pages), lists, per, float(scale), code, _ptr(out), os_[0], os_[1], _ptr(lse), _ptr(workspace),
        ws_bytes, _ptr(status), _stream(stream)))


def idx_verify_drafts(target, draft, tokens, cu_tokens, accept_u, sample_u, out_tokens, out_nodes, num_accepted,
                      parents=None, status=None, stream=None) -> int:
    """Which of the drafted tokens [T] i32 stand: target [T,V] f32, draft [T,V] f32 (None: drafts without randomness),
    accept_u [T], sample_u [R] f32 -> out_tokens, out_nodes [R,max_out] i32, num_accepted [R] i32."""
    lib = load_library()
    fn = "idx_verify_drafts"
    total, vocab = target.shape
    reqs, max_out = out_tokens.shape
    _want(fn, target=(target, _F32, (total, vocab)), draft=(draft, _F32, (total, vocab)), tokens=(tokens, _I32, (total,)),
          parents=(parents, _I32, (total,)), cu_tokens=(cu_tokens, _I32, (reqs + 1,)), accept_u=(accept_u, _F32, (total,)),
          sample_u=(sample_u, _F32, (reqs,)), out_tokens=(out_tokens, _I32, (reqs, max_out)),
          out_nodes=(out_nodes, _I32, (reqs, max_out)), num_accepted=(num_accepted, _I32, (reqs,)))
    _inner(fn, target=target, draft=draft)
    _packed(fn, tokens=tokens, parents=parents, cu_tokens=cu_tokens, accept_u=accept_u, sample_u=sample_u,
            out_tokens=out_tokens, out_nodes=out_nodes, num_accepted=num_accepted)
    return _check(fn, lib.idx_verify_drafts(
        _ptr(target), _row_stride(target), _ptr(draft), 0 if draft is None else _row_stride(draft), vocab, _ptr(tokens),
        _ptr(parents), _ptr(cu_tokens), reqs, total, _ptr(accept_u), _ptr(sample_u), _ptr(out_tokens), _ptr(out_nodes),
        max_out, _ptr(num_accepted), _ptr(status), _stream(stream)))
