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
_T = None  # torch's types and the raw stream getter, bound at the first call


class _Torch:
    def __init__(self):
        import torch

        self.i32, self.i64, self.f32, self.f64 = torch.int32, torch.int64, torch.float32, torch.float64
        self.words = (torch.int64, torch.uint64)
        self.codes = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
        self.many = torch.cuda.device_count() > 1
        self.device = torch.cuda.current_device
        # the current stream's handle without a Stream object (3 us less a call)
        self.raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)


def _torch() -> _Torch:
    global _T
    if _T is None:
        _T = _Torch()
    return _T


def _stream_on(stream, t) -> int | None:
    """The given stream, or the current one of t's device."""
    if stream is None:
        return _T.raw(t.get_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _are(dtype, shape, *tensors) -> bool:
    """Whether every given tensor (None left out) is on a GPU, has the type and the sizes and is contiguous."""
    for t in tensors:
        if t is not None and (not t.is_cuda or t.dtype is not dtype or t.shape != shape or not t.is_contiguous()):
            return False
    return True


def _here(*tensors) -> bool:
    """Whether all are on the current device.  Asked only where there are several: it costs as much as the other checks."""
    dev = _T.device()
    return all(t is None or t.get_device() == dev for t in tensors)


# The checks below run as one expression a call; only where it fails does
# _explain go through the tensors again to name the one that is wrong.
def _explain(name: str, dense=(), **tensors) -> None:
    """Raise for the first tensor that is not what is needed: each is (tensor, types or None, sizes with None for any, or
    None: not empty); those named in `dense` must be contiguous, the others in their last dimension.  The device comes last."""
    for arg, (t, dtypes, shape) in tensors.items():
        if t is None:
            continue
        dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
        if dtypes != (None,) and t.dtype not in dtypes:
            raise ValueError(f"{name}: {arg} has type {t.dtype}, {' or '.join(map(str, dtypes))} is needed")
        if shape is None:
            if t.numel() == 0 and dtypes != (None,):
                raise ValueError(f"{name}: {arg} has no element")
            continue
        if t.dim() != len(shape) or any(w is not None and w != h for w, h in zip(shape, t.shape)):
            need = tuple("any" if w is None else w for w in shape)
            raise ValueError(f"{name}: {arg} has shape {tuple(t.shape)}, {need} is needed")
        if arg in dense:
            if not t.is_contiguous():
                raise ValueError(f"{name}: {arg} must be contiguous")
        elif t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError(f"{name}: the last dimension of {arg} must be contiguous")
    for arg, (t, *_) in tensors.items():
        if t is not None and not (t.is_cuda and _here(t)):
            raise ValueError(f"{name}: {arg} is on {t.device}, the current CUDA device is needed")
    raise ValueError(f"{name}: a tensor has the wrong type, shape or strides")


def _rows_ok(dtype, shape, *tensors) -> bool:
    """On a GPU, type and sizes, and the last dimension contiguous (the others may have any strides)."""
    for t in tensors:
        if t is not None and (not t.is_cuda or t.dtype is not dtype or t.shape != shape or (t.stride(-1) != 1 and shape[-1] > 1)):
            return False
    return True


def idx_build_slots(ctx_lens, new_lens, owned_pages, block_table, free_blocks, free_cursor, num_blocks: int,
                    page_tokens: int, cu_tokens, seq_lens, pages_out, cursor_out, positions, slots, parents=None,
                    tree_mask=None, status=None, stream=None) -> int:
    """Block tables (block_table [R, maxb] i32, in place), slots [T] i64 and positions [T] i32 of a step's tokens
    from ctx_lens / new_lens / owned_pages [R] i32 and the free list; with parents [T] i32 also tree_mask [T] i64."""
    lib, T, fn = load_library(), _torch(), "idx_build_slots"
    i32 = T.i32
    per_req, per_token = ctx_lens.shape, positions.shape
    reqs, width, tokens, free = per_req[0], block_table.shape[-1], per_token[0], free_blocks.shape[0]
    if not (_are(i32, (reqs,), ctx_lens, new_lens, owned_pages, seq_lens, pages_out) and _are(i32, (reqs + 1,), cu_tokens)
            and _are(i32, (1,), free_cursor, cursor_out) and _are(i32, (free,), free_blocks)
            and _are(i32, (tokens,), positions, parents) and slots.is_cuda and slots.shape == per_token and slots.dtype in T.words
            and slots.is_contiguous() and _rows_ok(i32, (reqs, width), block_table)
            and (tree_mask is None or (tree_mask.is_cuda and tree_mask.shape == per_token and tree_mask.dtype in T.words
                                       and tree_mask.is_contiguous()))
            and (status is None or (status.is_cuda and status.dtype is i32 and status.numel() > 0))
            and (not T.many or _here(ctx_lens, new_lens, owned_pages, block_table, free_blocks, free_cursor, cu_tokens, seq_lens, pages_out,
                                     cursor_out, positions, slots, parents, tree_mask, status))):
        r, t, one = (reqs,), (tokens,), (1,)
        _explain(fn, ("ctx_lens", "new_lens", "owned_pages", "free_blocks", "cu_tokens", "seq_lens", "pages_out", "positions", "slots",
                      "parents", "tree_mask"), ctx_lens=(ctx_lens, i32, r), new_lens=(new_lens, i32, r),
                 owned_pages=(owned_pages, i32, r), block_table=(block_table, i32, (reqs, None)), free_blocks=(free_blocks, i32, (None,)),
                 free_cursor=(free_cursor, i32, one), cu_tokens=(cu_tokens, i32, (reqs + 1,)), seq_lens=(seq_lens, i32, r),
                 pages_out=(pages_out, i32, r), cursor_out=(cursor_out, i32, one), positions=(positions, i32, t),
                 slots=(slots, T.words, t), parents=(parents, i32, t), tree_mask=(tree_mask, T.words, t), status=(status, i32, None))
    rc = lib.idx_build_slots(
        ctx_lens.data_ptr(), new_lens.data_ptr(), owned_pages.data_ptr(), reqs, block_table.data_ptr(), _row_stride(block_table),
        width, free_blocks.data_ptr(), free, free_cursor.data_ptr(), num_blocks, page_tokens, None if parents is None else parents.data_ptr(), tokens,
        cu_tokens.data_ptr(), seq_lens.data_ptr(), pages_out.data_ptr(), cursor_out.data_ptr(), positions.data_ptr(),
        slots.data_ptr(), None if tree_mask is None else tree_mask.data_ptr(), None if status is None else status.data_ptr(), _stream_on(stream, positions))
    return rc if rc >= 0 else _check(fn, rc)


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
    lib, T, fn = load_library(), _torch(), "idx_rope_append"
    some = q if q is not None else k
    if some is None or (v is not None and k is None):
        raise ValueError(f"{fn}: q, or k (with or without v), is needed")
    if (q is None) != (q_out is None) or (k is None) != (k_cache is None) or (v is None) != (v_cache is None):
        raise ValueError(f"{fn}: q and q_out, k and k_cache, v and v_cache go together")
    kind = some.dtype
    code = T.codes.get(kind)
    if code is None:
        raise ValueError(f"{fn}: bfloat16, float16 or float32 is needed, got {kind}")
    tokens, dim = some.shape[0], some.shape[-1]
    hq = 0 if q is None else q.shape[1]
    nb, page, hk = (0, 1, 0) if k is None else (k_cache.shape[0], k_cache.shape[1], k.shape[1])
    qshape, kshape, cshape = (tokens, hq, dim), (tokens, hk, dim), (nb, page, hk, dim)
    if not (_rows_ok(kind, qshape, q, q_out) and _rows_ok(kind, kshape, k, v) and _rows_ok(kind, cshape, k_cache, v_cache)
            and _are(T.i32, (tokens,), positions) and _are(T.f64, inv_freq.shape[:1], inv_freq)
            and (slots is None or (slots.is_cuda and slots.dtype in T.words and slots.shape == positions.shape and slots.is_contiguous()))
            and (status is None or (status.is_cuda and status.dtype is T.i32 and status.numel() > 0))
            and (not T.many or _here(q, q_out, k, v, k_cache, v_cache, positions, inv_freq, slots, status))):
        _explain(fn, ("positions", "inv_freq", "slots"), q=(q, kind, qshape), q_out=(q_out, kind, qshape), k=(k, kind, kshape),
                 v=(v, kind, kshape), k_cache=(k_cache, kind, (None, None, hk, dim)), v_cache=(v_cache, kind, cshape),
                 positions=(positions, T.i32, (tokens,)), inv_freq=(inv_freq, T.f64, (None,)), slots=(slots, T.words, (tokens,)),
                 status=(status, T.i32, None))
    cs = (0, 0, 0, 0) if k is None else k_cache.stride()
    if v_cache is not None and v_cache.stride() != cs:
        raise ValueError(f"{fn}: k_cache and v_cache must have the same strides")
    none = (0, 0, 0)
    qs, os_ = (none, none) if q is None else (q.stride(), q_out.stride())
    ks = none if k is None else k.stride()
    vs = none if v is None else v.stride()
    rc = lib.idx_rope_append(
        None if q is None else q.data_ptr(), qs[0], qs[1], None if q_out is None else q_out.data_ptr(), os_[0], os_[1], hq, None if k is None else k.data_ptr(), ks[0], ks[1], None if v is None else v.data_ptr(), vs[0], vs[1], hk, tokens, dim,
        2 * inv_freq.shape[0], positions.data_ptr(), inv_freq.data_ptr(), mscale, None if slots is None else slots.data_ptr(), None if k_cache is None else k_cache.data_ptr(), None if v_cache is None else v_cache.data_ptr(), nb,
        page, cs[0], cs[1], cs[2], code, _ROPE_INTERLEAVED if interleaved else 0, None if status is None else status.data_ptr(), _stream_on(stream, some))
    return rc if rc >= 0 else _check(fn, rc)


def idx_tree_attention_workspace_bytes(num_reqs: int, num_tokens: int, q_heads: int, kv_heads: int, head_dim: int,
                                       page_lists: int = 0, pages_per_list: int = 0) -> int:
    return int(load_library().idx_tree_attention_workspace_bytes(num_reqs, num_tokens, q_heads, kv_heads, head_dim,
                                                                 page_lists, pages_per_list))


def idx_tree_attention(q, k_cache, v_cache, block_table, seq_lens, cu_tokens, out, scale: float, tree_mask=None, pages=None,
                       lse=None, workspace=None, status=None, stream=None) -> int:
    """q [T,Hq,D] over the cache [nb,P,Hk,D] of each token's request -> out [T,Hq,D] (+ lse [T,Hq] f32); tree_mask [T] i64
    (None: a chain); pages [T,lists,per] i32 (or idx_decode_step's [R,query_len,lists,per]): only those pages."""
    lib, T, fn = load_library(), _torch(), "idx_tree_attention"
    kind, shape, cshape = q.dtype, q.shape, k_cache.shape
    code = T.codes.get(kind, 2)
    if code == 2:
        raise ValueError(f"{fn}: bfloat16 or float16 is needed, got {kind}")
    tokens, hq, dim = shape
    nb, page, hk, _ = cshape
    reqs, width = block_table.shape
    lists = per = 0
    if pages is not None:
        lists, per = pages.shape[-2:]
    if not (_rows_ok(kind, shape, q, out) and cshape[3] == dim and _rows_ok(kind, cshape, k_cache, v_cache)
            and _rows_ok(T.i32, (reqs, width), block_table) and _are(T.i32, (reqs,), seq_lens)
            and _are(T.i32, (reqs + 1,), cu_tokens) and _are(T.f32, (tokens, hq), lse)
            and (tree_mask is None or (tree_mask.is_cuda and tree_mask.dtype in T.words and tree_mask.shape == (tokens,)
                                       and tree_mask.is_contiguous()))
            and (pages is None or (pages.is_cuda and pages.dtype is T.i32 and pages.is_contiguous()
                                   and pages.numel() == tokens * lists * per))
            and (status is None or (status.is_cuda and status.dtype is T.i32 and status.numel() > 0))
            and (workspace is None or workspace.is_cuda)
            and (not T.many or _here(q, k_cache, v_cache, block_table, seq_lens, cu_tokens, out, tree_mask, pages, lse, workspace, status))):
        _explain(fn, ("seq_lens", "cu_tokens", "tree_mask", "lse", "pages"), q=(q, kind, shape), out=(out, kind, shape),
                 k_cache=(k_cache, kind, (nb, page, hk, dim)), v_cache=(v_cache, kind, (nb, page, hk, dim)),
                 block_table=(block_table, T.i32, (reqs, None)), seq_lens=(seq_lens, T.i32, (reqs,)),
                 cu_tokens=(cu_tokens, T.i32, (reqs + 1,)), tree_mask=(tree_mask, T.words, (tokens,)), lse=(lse, T.f32, (tokens, hq)),
                 pages=(pages if pages is None or pages.dim() < 4 else pages.flatten(0, -3), T.i32, (tokens, lists, per)),
                 workspace=(workspace, None, None), status=(status, T.i32, None))
    cs = k_cache.stride()
    if v_cache.stride() != cs:
        raise ValueError(f"{fn}: k_cache and v_cache must have the same strides")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    qs, os_ = q.stride(), out.stride()
    rc = lib.idx_tree_attention(
        q.data_ptr(), qs[0], qs[1], k_cache.data_ptr(), v_cache.data_ptr(), nb, page, cs[0], cs[1], cs[2], block_table.data_ptr(),
        _row_stride(block_table), width, seq_lens.data_ptr(), cu_tokens.data_ptr(), reqs, tokens, hq, hk, dim, None if tree_mask is None else tree_mask.data_ptr(),
        None if pages is None else pages.data_ptr(), lists, per, scale, code, out.data_ptr(), os_[0], os_[1], None if lse is None else lse.data_ptr(), None if workspace is None else workspace.data_ptr(), ws_bytes, None if status is None else status.data_ptr(),
        _stream_on(stream, q))
    return rc if rc >= 0 else _check(fn, rc)


def idx_verify_drafts(target, draft, tokens, cu_tokens, accept_u, sample_u, out_tokens, out_nodes, num_accepted,
                      parents=None, status=None, stream=None) -> int:
    """Which of the drafted tokens [T] i32 stand: target [T,V] f32, draft [T,V] f32 (None: drafts without randomness),
    accept_u [T], sample_u [R] f32 -> out_tokens, out_nodes [R,max_out] i32, num_accepted [R] i32."""
    lib, T, fn = load_library(), _torch(), "idx_verify_drafts"
    i32, f32 = T.i32, T.f32
    total, vocab = rows = target.shape
    reqs, max_out = out_shape = out_tokens.shape
    if not (_rows_ok(f32, rows, target, draft) and _are(i32, (total,), tokens, parents)
            and _are(i32, (reqs + 1,), cu_tokens) and _are(f32, (total,), accept_u) and _are(f32, (reqs,), sample_u)
            and _are(i32, out_shape, out_tokens, out_nodes) and _are(i32, (reqs,), num_accepted)
            and (status is None or (status.is_cuda and status.dtype is i32 and status.numel() > 0))
            and (not T.many or _here(target, draft, tokens, parents, cu_tokens, accept_u, sample_u, out_tokens, out_nodes, num_accepted,
                                     status))):
        _explain(fn, ("tokens", "parents", "cu_tokens", "accept_u", "sample_u", "out_tokens", "out_nodes", "num_accepted"),
                 target=(target, f32, rows), draft=(draft, f32, rows), tokens=(tokens, i32, (total,)), parents=(parents, i32, (total,)),
                 cu_tokens=(cu_tokens, i32, (reqs + 1,)), accept_u=(accept_u, f32, (total,)), sample_u=(sample_u, f32, (reqs,)),
                 out_tokens=(out_tokens, i32, out_shape), out_nodes=(out_nodes, i32, out_shape), num_accepted=(num_accepted, i32, (reqs,)),
                 status=(status, i32, None))
    rc = lib.idx_verify_drafts(
        target.data_ptr(), _row_stride(target), None if draft is None else draft.data_ptr(), 0 if draft is None else _row_stride(draft), vocab, tokens.data_ptr(),
        None if parents is None else parents.data_ptr(), cu_tokens.data_ptr(), reqs, total, accept_u.data_ptr(), sample_u.data_ptr(), out_tokens.data_ptr(),
        out_nodes.data_ptr(), max_out, num_accepted.data_ptr(), None if status is None else status.data_ptr(), _stream_on(stream, target))
    return rc if rc >= 0 else _check(fn, rc)
