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
import struct

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
    "idx_norm_rope_append",
    "idx_index_append",
    "idx_logit_probs",
    "PROBS_MAX_VOCAB",
    "index_caches",
    "idx_settle_drafts",
    "idx_fork_pages",
    "idx_release_pages",
    "MAX_CACHES",
    "MAX_FORKS",
    "SYMBOLS",
    "ST_BLOCK_OOR",
    "ST_LEN_CLAMPED",
    "ST_BAD_OUTPUT",
    "ST_TIMEOUT",
    "ST_NO_BLOCKS",
    "ST_BAD_TREE",
    "ST_BAD_FORK",
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
ST_BAD_FORK = 64
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
    "idx_norm_rope_append": (ctypes.c_int, [_p, _i64, _i64, _p, _i64, _i64, _i32, _p, _i64, _i64, _p, _i64, _i64, _i32, _i32,
                                            _i32, _i32, _p, _p, _f32, _f32, _p, _p, _f32, _p, _p, _p, _i64, _i32, _i64, _i64,
                                            _i64, _i32, _i32, _p, _p]),
    "idx_index_append": (ctypes.c_int, [_p, _i64, _i64, _i32, _p, _i64, _i32, _i32, _p, _p, _f32, _f32, _p, _p, _f32, _p, _f32,
                                        _p, _i32, _i32, _p, _p, _p, _p, _i64, _i32, _i32, _i32, _p, _p]),
    "idx_logit_probs": (ctypes.c_int, [_p, _i64, _i32, _i32, _i32, _p, _i32, _p, _p, _p, _p, _p, _i64, _p, _p, _p, _p, _p, _i32,
                                       _p, _i64, _p, _i64, _p, _p, _p]),
    "idx_settle_drafts": (ctypes.c_int, [_p, _i32, _i64, _i32, _p, _p, _i32, _i32, _p, _p, _i32, _p, _p, _p, _p, _i64, _i32, _p,
                                         _p]),
    "idx_fork_pages": (ctypes.c_int, [_p, _i32, _i64, _i32, _p, _p, _i32, _p, _p, _i32, _p, _i64, _i32, _p, _p, _i32, _p, _p, _p,
                                      _p]),
    "idx_release_pages": (ctypes.c_int, [_p, _p, _i32, _p, _i64, _i32, _p, _i64, _p, _i32, _p, _p, _p, _i32, _p, _p]),
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

        self.i32, self.i64, self.f32, self.f64, self.u8 = torch.int32, torch.int64, torch.float32, torch.float64, torch.uint8
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


# ---------------------------------------------------------------------------
# Between those calls: norms, the indexer's inputs, probabilities, caches
# ---------------------------------------------------------------------------

PROBS_MAX_VOCAB = 262144  # entries of a row of idx_logit_probs
MAX_CACHES = 8  # caches of one call of idx_settle_drafts and idx_fork_pages
MAX_FORKS = 4096  # forks of one call
_CACHE = "Pqqqii"  # idx_cache


def idx_norm_rope_append(q, k, v, q_weight, k_weight, eps: float, positions, inv_freq, q_out, k_cache, v_cache, slots=None,
                         mscale: float = 1.0, offset: float = 0.0, interleaved: bool = False, status=None, stream=None) -> int:
    """idx_rope_append after a norm of each head with q_weight, k_weight [D] (None: that side is turned only)."""
    lib, T, fn = load_library(), _torch(), "idx_norm_rope_append"
    some = q if q is not None else k
    if some is None or (v is not None and k is None):
        raise ValueError(f"{fn}: q, or k (with or without v), is needed")
    if (q is None) != (q_out is None) or (k is None) != (k_cache is None) or (v is None) != (v_cache is None):
        raise ValueError(f"{fn}: q and q_out, k and k_cache, v and v_cache go together")
    kind = some.dtype
    code = T.codes.get(kind)
    if code is None:
        raise ValueError(f"{fn}: bfloat16, float16 or float32 is needed, got {kind}")
    tokens, _, dim = shape = some.shape
    none = (0, 0, 1, 1)
    qs = os_ = ks = vs = cs = none
    hq = hk = nb = 0
    page, one, per_dim = 1, (tokens,), (dim,)
    qshape = kshape = cshape = shape
    if q is not None:
        qshape, qs, os_ = q.shape, q.stride(), q_out.stride()
        hq = qshape[1]
    if k is not None:
        hk, ks, cs = k.shape[1], k.stride(), k_cache.stride()
        nb, page = k_cache.shape[:2]
        kshape, cshape = (tokens, hk, dim), (nb, page, hk, dim)
        vs = none if v is None else v.stride()
    # (the checks stand in one expression: a call each would cost as much as the launch)
    if not (some.is_cuda and (q is None or (q_out.is_cuda and q_out.dtype is kind and q_out.shape == qshape))
            and (k is None or (k.is_cuda and k.dtype is kind and k.shape == kshape and k_cache.is_cuda and k_cache.dtype is kind and k_cache.shape == cshape
                               and (v is None or (v.is_cuda and v.dtype is kind and v.shape == kshape and v_cache.is_cuda and v_cache.dtype is kind
                                                  and v_cache.shape == cshape))))
            and ((qs[2] == 1 and os_[2] == 1 and ks[2] == 1 and vs[2] == 1 and cs[3] == 1) or dim == 1)
            and (q_weight is None or (q_weight.is_cuda and q_weight.dtype is kind and q_weight.shape == per_dim and q_weight.is_contiguous()))
            and (k_weight is None or (k_weight.is_cuda and k_weight.dtype is kind and k_weight.shape == per_dim and k_weight.is_contiguous()))
            and positions.is_cuda and positions.dtype is T.i32 and positions.shape == one and positions.is_contiguous()
            and inv_freq.is_cuda and inv_freq.dtype is T.f64 and inv_freq.dim() == 1 and inv_freq.is_contiguous()
            and (slots is None or (slots.is_cuda and slots.dtype in T.words and slots.shape == one and slots.is_contiguous()))
            and (status is None or (status.is_cuda and status.dtype is T.i32 and status.numel() > 0))
            and (not T.many or _here(q, q_out, k, v, k_cache, v_cache, q_weight, k_weight, positions, inv_freq, slots, status))):
        _explain(fn, ("positions", "inv_freq", "slots", "q_weight", "k_weight"), q=(q, kind, qshape), q_out=(q_out, kind, qshape),
                 k=(k, kind, kshape), v=(v, kind, kshape), k_cache=(k_cache, kind, (None, None, hk, dim)), v_cache=(v_cache, kind, cshape),
                 q_weight=(q_weight, kind, (dim,)), k_weight=(k_weight, kind, (dim,)), positions=(positions, T.i32, one),
                 inv_freq=(inv_freq, T.f64, (None,)), slots=(slots, T.words, one), status=(status, T.i32, None))
    if v_cache is not None and v_cache.stride() != cs:
        raise ValueError(f"{fn}: k_cache and v_cache must have the same strides")
    rc = lib.idx_norm_rope_append(
        None if q is None else q.data_ptr(), qs[0], qs[1], None if q is None else q_out.data_ptr(), os_[0], os_[1], hq, None if k is None else k.data_ptr(),
        ks[0], ks[1], None if v is None else v.data_ptr(), vs[0], vs[1], hk, tokens, dim, 2 * inv_freq.shape[0],
        None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(), eps, offset, positions.data_ptr(),
        inv_freq.data_ptr(), mscale, None if slots is None else slots.data_ptr(), None if k is None else k_cache.data_ptr(),
        None if v is None else v_cache.data_ptr(), nb, page, cs[0], cs[1], cs[2], code, _ROPE_INTERLEAVED if interleaved else 0,
        None if status is None else status.data_ptr(), _stream_on(stream, some))
    return rc if rc >= 0 else _check(fn, rc)


def idx_index_append(q, k, q_weight, k_weight, eps: float, positions, inv_freq, q_out, q_scale, index_k, slots=None, cu_tokens=None,
                     head_weights=None, scale: float = 1.0, mscale: float = 1.0, offset: float = 0.0, interleaved: bool = False, status=None,
                     stream=None) -> int:
    """The indexer's inputs: q [T,H,128] -> q_out E4M3 bytes and q_scale f32, [T,H,128] and [T,H], or with cu_tokens [R+1] i32
    [R,S,H,128] and [R,S,H] (a request's tokens in its last slots); k [T,128] -> index_k [nb,P,72] u8 pages at slots [T] i64
    (None: slot t).  q, q_out and q_scale, or k and index_k may be None; weights [128] (None: no norm); head_weights [T,H] f32."""
    lib, T, fn = load_library(), _torch(), "idx_index_append"
    some = q if q is not None else k
    if some is None:
        raise ValueError(f"{fn}: q or k is needed")
    if (q is None) != (q_out is None) or (q is None) != (q_scale is None) or (k is None) != (index_k is None):
        raise ValueError(f"{fn}: q, q_out and q_scale, k and index_k go together")
    kind = some.dtype
    code = T.codes.get(kind)
    if code is None:
        raise ValueError(f"{fn}: bfloat16, float16 or float32 is needed, got {kind}")
    tokens, u8, f32, i32 = some.shape[0], T.u8, T.f32, T.i32
    heads = reqs = per = nb = 0
    page, one, wide, out = 128, (tokens,), (128,), ()
    qs, ks = (0, 0, 1), (0, 1)
    if q is not None:
        tokens, heads, _ = qshape = q.shape
        qs, out = q.stride(), qshape[:2]
        if cu_tokens is not None:
            reqs, per = cu_tokens.shape[0] - 1, q_out.shape[1]
            out = (reqs, per, heads)
    if k is not None:
        ks = k.stride()
        nb, page, _ = index_k.shape
    if not (some.is_cuda and (q is None or (qshape[2] == 128 and qs[2] == 1 and q_out.is_cuda and q_out.dtype is u8 and q_out.shape == (*out, 128)
                                            and q_out.is_contiguous() and q_scale.is_cuda and q_scale.dtype is f32 and q_scale.shape == out
                                            and q_scale.is_contiguous()))
            and (k is None or (k.is_cuda and k.dtype is kind and k.shape == (tokens, 128) and ks[1] == 1 and index_k.is_cuda and index_k.dtype is u8
                               and index_k.shape[2] == 72 and index_k.is_contiguous()))
            and (q_weight is None or (q_weight.is_cuda and q_weight.dtype is kind and q_weight.shape == wide and q_weight.is_contiguous()))
            and (k_weight is None or (k_weight.is_cuda and k_weight.dtype is kind and k_weight.shape == wide and k_weight.is_contiguous()))
            and positions.is_cuda and positions.dtype is i32 and positions.shape == one and positions.is_contiguous()
            and inv_freq.is_cuda and inv_freq.dtype is T.f64 and inv_freq.dim() == 1 and inv_freq.is_contiguous()
            and (slots is None or (slots.is_cuda and slots.dtype in T.words and slots.shape == one and slots.is_contiguous()))
            and (cu_tokens is None or (cu_tokens.is_cuda and cu_tokens.dtype is i32 and cu_tokens.dim() == 1 and cu_tokens.is_contiguous()))
            and (head_weights is None or _are(f32, (tokens, heads), head_weights))
            and (status is None or (status.is_cuda and status.dtype is i32 and status.numel() > 0))
            and (not T.many or _here(q, k, q_out, q_scale, index_k, q_weight, k_weight, positions, inv_freq, slots, cu_tokens, head_weights, status))):
        _explain(fn, ("q_out", "q_scale", "index_k", "q_weight", "k_weight", "positions", "inv_freq", "slots", "head_weights", "cu_tokens"),
                 q=(q, kind, (tokens, heads, 128)), k=(k, kind, (tokens, 128)), q_out=(q_out, u8, (*out, 128)), q_scale=(q_scale, f32, tuple(out)),
                 index_k=(index_k, u8, (None, None, 72)), q_weight=(q_weight, kind, wide),
                 k_weight=(k_weight, kind, wide), positions=(positions, T.i32, one), inv_freq=(inv_freq, T.f64, (None,)),
                 slots=(slots, T.words, one), cu_tokens=(cu_tokens, T.i32, (None,)), head_weights=(head_weights, T.f32, (tokens, heads)),
                 status=(status, T.i32, None))
    rc = lib.idx_index_append(
        None if q is None else q.data_ptr(), qs[0], qs[1], heads, None if k is None else k.data_ptr(), ks[0], tokens, 2 * inv_freq.shape[0],
        None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(), eps, offset, positions.data_ptr(),
        inv_freq.data_ptr(), mscale, None if head_weights is None else head_weights.data_ptr(), scale,
        None if q is None or cu_tokens is None else cu_tokens.data_ptr(), reqs, per, None if q is None else q_out.data_ptr(),
        None if q is None else q_scale.data_ptr(), None if slots is None else slots.data_ptr(), None if k is None else index_k.data_ptr(), nb, page, code,
        _ROPE_INTERLEAVED if interleaved else 0, None if status is None else status.data_ptr(), _stream_on(stream, some))
    return rc if rc >= 0 else _check(fn, rc)


def idx_logit_probs(logits, probs, cu_tokens, temperature=None, repetition=None, presence=None, frequency=None, counts=None, tokens=None,
                    tree_mask=None, bias_cu=None, bias_tokens=None, bias_values=None, allowed=None, lse=None, status=None, stream=None) -> int:
    """logits [T,V] -> probs [T,V] f32 (+ lse [T] f32); temperature, repetition, presence, frequency [R] f32; counts [R,V] i32 (highest
    bit: in the prompt); tokens [T] i32 and tree_mask [T] i64 (None: a chain) of the drafts; biases bias_cu [R+1] i32, bias_tokens i32,
    bias_values f32; allowed [T,ceil(V/32)] i32 bits."""
    lib, T, fn = load_library(), _torch(), "idx_logit_probs"
    i32, f32, kind = T.i32, T.f32, logits.dtype
    code = T.codes.get(kind)
    if code is None:
        raise ValueError(f"{fn}: bfloat16, float16 or float32 is needed, got {kind}")
    if (bias_cu is None) != (bias_tokens is None) or (bias_cu is None) != (bias_values is None):
        raise ValueError(f"{fn}: bias_cu, bias_tokens and bias_values go together")
    if tree_mask is not None and tokens is None:
        raise ValueError(f"{fn}: tree_mask goes with tokens")
    total, vocab = shape = logits.shape
    reqs = cu_tokens.shape[0] - 1
    one, per_req, words = (total,), (reqs,), (total, (vocab + 31) // 32)
    biases = 0 if bias_tokens is None else bias_tokens.shape[0]
    per_cu, ls, ps = (reqs + 1,), logits.stride(), probs.stride()
    if not (logits.is_cuda and probs.is_cuda and probs.dtype is f32 and probs.shape == shape and ((ls[1] == 1 and ps[1] == 1) or vocab == 1)
            and cu_tokens.is_cuda and cu_tokens.dtype is i32 and cu_tokens.dim() == 1 and cu_tokens.is_contiguous()
            and _are(f32, per_req, temperature, repetition, presence, frequency) and (counts is None or reqs == 0 or _rows_ok(i32, (reqs, vocab), counts))
            and (tokens is None or (tokens.is_cuda and tokens.dtype is i32 and tokens.shape == one and tokens.is_contiguous()))
            and (tree_mask is None or (tree_mask.is_cuda and tree_mask.dtype in T.words and tree_mask.shape == one and tree_mask.is_contiguous()))
            and (bias_cu is None or (_are(i32, per_cu, bias_cu) and _are(i32, (biases,), bias_tokens) and _are(f32, (biases,), bias_values)))
            and (allowed is None or _rows_ok(i32, words, allowed))
            and (lse is None or (lse.is_cuda and lse.dtype is f32 and lse.shape == one and lse.is_contiguous()))
            and (status is None or (status.is_cuda and status.dtype is i32 and status.numel() > 0))
            and (not T.many or _here(logits, probs, cu_tokens, temperature, repetition, presence, frequency, counts, tokens, tree_mask, bias_cu,
                                     bias_tokens, bias_values, allowed, lse, status))):
        _explain(fn, ("cu_tokens", "temperature", "repetition", "presence", "frequency", "tokens", "tree_mask", "bias_cu", "bias_tokens",
                      "bias_values", "lse"), logits=(logits, kind, shape), probs=(probs, f32, shape), cu_tokens=(cu_tokens, i32, (None,)),
                 temperature=(temperature, f32, per_req), repetition=(repetition, f32, per_req), presence=(presence, f32, per_req),
                 frequency=(frequency, f32, per_req), counts=(counts, i32, (reqs, vocab)), tokens=(tokens, i32, one),
                 tree_mask=(tree_mask, T.words, one), bias_cu=(bias_cu, i32, (reqs + 1,)), bias_tokens=(bias_tokens, i32, (biases,)),
                 bias_values=(bias_values, f32, (biases,)), allowed=(allowed, i32, words), lse=(lse, f32, one), status=(status, i32, None))
    rc = lib.idx_logit_probs(
        logits.data_ptr(), ls[0] if total > 1 else vocab, code, vocab, total, cu_tokens.data_ptr(), reqs,
        None if temperature is None else temperature.data_ptr(), None if repetition is None else repetition.data_ptr(),
        None if presence is None else presence.data_ptr(), None if frequency is None else frequency.data_ptr(),
        None if counts is None else counts.data_ptr(), 0 if counts is None else _row_stride(counts), None if tokens is None else tokens.data_ptr(),
        None if tree_mask is None else tree_mask.data_ptr(), None if bias_cu is None else bias_cu.data_ptr(),
        None if bias_cu is None else bias_tokens.data_ptr(), None if bias_cu is None else bias_values.data_ptr(), biases,
        None if allowed is None else allowed.data_ptr(), 0 if allowed is None else _row_stride(allowed), probs.data_ptr(), ps[0] if total > 1 else vocab,
        None if lse is None else lse.data_ptr(), None if status is None else status.data_ptr(), _stream_on(stream, logits))
    return rc if rc >= 0 else _check(fn, rc)


def index_caches(index_k):
    """The two caches that NVFP4 index-K pages [nb,P,72] u8 are to idx_settle_drafts and idx_fork_pages: codes and scales."""
    blocks, page, width = index_k.shape
    if width != 72 or not index_k.is_contiguous():
        raise ValueError("index_caches: contiguous pages [num_blocks, page_tokens, 72] are needed")
    flat = index_k.view(1, blocks, page * 72)
    return flat[:, :, : page * 64].unflatten(2, (page, 64)), flat[:, :, page * 64 :].unflatten(2, (page, 8))


def _pack_caches(fn: str, T, caches):
    """idx_cache entries of tensors [planes, blocks, page_tokens, row...] (the row contiguous), and the blocks and page they share."""
    blocks, page = caches[0].shape[1:3] if caches and caches[0].dim() > 3 else (0, 1)
    fields = []
    for c in caches:
        shape, strides, size = c.shape, c.stride(), c.element_size()
        row, fine, n = 1, len(shape) > 3 and shape[1] == blocks and shape[2] == page and c.is_cuda and (not T.many or _here(c)), len(shape) - 1
        while n > 2:
            m = shape[n]
            if m != 1 and strides[n] != row:
                fine = False
            row *= m
            n -= 1
        if not fine:
            if len(shape) < 4 or shape[1] != blocks or shape[2] != page:
                raise ValueError(f"{fn}: a cache has shape {tuple(shape)}, (any, {blocks}, {page}, any...) is needed")
            if not (c.is_cuda and (not T.many or _here(c))):
                raise ValueError(f"{fn}: a cache is on {c.device}, the current CUDA device is needed")
            raise ValueError(f"{fn}: a token's row of a cache must be contiguous")
        fields += (c.data_ptr(), strides[0] * size, strides[1] * size, strides[2] * size, shape[0], row * size)
    return struct.pack(_CACHE * len(caches), *fields), blocks, page


def idx_settle_drafts(caches, slots, cu_tokens, out_tokens, out_nodes, num_accepted, ctx_lens, ctx_out, counts=None, status=None,
                      stream=None) -> int:
    """After idx_verify_drafts: rows of the nodes that stand moved together in caches (tensors [planes,nb,P,row...]; index_caches gives
    those of index-K pages), ctx_out [R] i32 from ctx_lens (may be the same), counts [R,V] i32 with the step's tokens."""
    lib, T, fn = load_library(), _torch(), "idx_settle_drafts"
    i32 = T.i32
    reqs, max_out = out_shape = out_nodes.shape
    per_req, tokens = (reqs,), slots.shape[0]
    vocab = 0 if counts is None else counts.shape[-1]
    if not (slots.is_cuda and slots.dtype in T.words and slots.dim() == 1 and slots.is_contiguous()
            and cu_tokens.is_cuda and cu_tokens.dtype is i32 and cu_tokens.shape == (reqs + 1,) and cu_tokens.is_contiguous()
            and out_tokens.is_cuda and out_tokens.dtype is i32 and out_tokens.shape == out_shape and out_tokens.is_contiguous()
            and out_nodes.is_cuda and out_nodes.dtype is i32 and out_nodes.is_contiguous()
            and num_accepted.is_cuda and num_accepted.dtype is i32 and num_accepted.shape == per_req and num_accepted.is_contiguous()
            and ctx_lens.is_cuda and ctx_lens.dtype is i32 and ctx_lens.shape == per_req and ctx_lens.is_contiguous()
            and ctx_out.is_cuda and ctx_out.dtype is i32 and ctx_out.shape == per_req and ctx_out.is_contiguous()
            and (counts is None or reqs == 0 or _rows_ok(i32, (reqs, vocab), counts))
            and (status is None or (status.is_cuda and status.dtype is i32 and status.numel() > 0))
            and (not T.many or _here(slots, cu_tokens, out_tokens, out_nodes, num_accepted, ctx_lens, ctx_out, counts, status))):
        _explain(fn, ("slots", "cu_tokens", "out_tokens", "out_nodes", "num_accepted", "ctx_lens", "ctx_out"), slots=(slots, T.words, (tokens,)),
                 cu_tokens=(cu_tokens, i32, (reqs + 1,)), out_tokens=(out_tokens, i32, out_shape), out_nodes=(out_nodes, i32, out_shape),
                 num_accepted=(num_accepted, i32, per_req), ctx_lens=(ctx_lens, i32, per_req), ctx_out=(ctx_out, i32, per_req),
                 counts=(counts, i32, (reqs, vocab)), status=(status, i32, None))
    packed, blocks, page = _pack_caches(fn, T, caches)
    rc = lib.idx_settle_drafts(
        packed, len(caches), blocks, page, slots.data_ptr(), cu_tokens.data_ptr(), reqs, tokens, out_tokens.data_ptr(), out_nodes.data_ptr(), max_out,
        num_accepted.data_ptr(), ctx_lens.data_ptr(), ctx_out.data_ptr(), None if counts is None else counts.data_ptr(),
        0 if counts is None else _row_stride(counts), vocab, None if status is None else status.data_ptr(), _stream_on(stream, out_nodes))
    return rc if rc >= 0 else _check(fn, rc)


def idx_fork_pages(caches, parents, children, ctx_lens, owned_pages, block_table, refs, free_blocks, free_cursor, cursor_out, page_tokens=None,
                   status=None, stream=None) -> int:
    """Requests children [F] i32 forked off parents [F] i32: ctx_lens and owned_pages [R] i32 and block_table [R,maxb] i32 in place, full
    pages shared (refs [nb] i32), the last one copied in caches (as in idx_settle_drafts; page_tokens where there are none)."""
    lib, T, fn = load_library(), _torch(), "idx_fork_pages"
    i32 = T.i32
    forks, free = parents.shape[0], free_blocks.shape[0]
    reqs, width = block_table.shape
    some, per_req, nb = (forks,), (reqs,), refs.shape[0]
    if not (_are(i32, some, parents, children) and _are(i32, per_req, ctx_lens, owned_pages) and _rows_ok(i32, (reqs, width), block_table)
            and _are(i32, (nb,), refs) and _are(i32, (free,), free_blocks) and _are(i32, (1,), free_cursor, cursor_out) and (status is None or (status.is_cuda and status.dtype is i32 and status.numel() > 0))
            and (not T.many or _here(parents, children, ctx_lens, owned_pages, block_table, refs, free_blocks, free_cursor, cursor_out, status))):
        _explain(fn, ("parents", "children", "ctx_lens", "owned_pages", "refs", "free_blocks", "free_cursor", "cursor_out"),
                 parents=(parents, i32, some), children=(children, i32, some), ctx_lens=(ctx_lens, i32, per_req),
                 owned_pages=(owned_pages, i32, per_req), block_table=(block_table, i32, (reqs, None)), refs=(refs, i32, (None,)),
                 free_blocks=(free_blocks, i32, (None,)), free_cursor=(free_cursor, i32, (1,)), cursor_out=(cursor_out, i32, (1,)),
                 status=(status, i32, None))
    packed, blocks, page = _pack_caches(fn, T, caches)
    if caches and blocks != nb:
        raise ValueError(f"{fn}: refs has {nb} entries, the caches have {blocks} blocks")
    if caches and page_tokens is not None and page_tokens != page:
        raise ValueError(f"{fn}: page_tokens is {page_tokens}, the caches have pages of {page}")
    if not caches:
        if page_tokens is None:
            raise ValueError(f"{fn}: page_tokens is needed where there are no caches")
        page = page_tokens
    rc = lib.idx_fork_pages(
        packed, len(caches), nb, page, parents.data_ptr(), children.data_ptr(), forks, ctx_lens.data_ptr(), owned_pages.data_ptr(), reqs,
        block_table.data_ptr(), _row_stride(block_table), width, refs.data_ptr(), free_blocks.data_ptr(), free, free_cursor.data_ptr(),
        cursor_out.data_ptr(), None if status is None else status.data_ptr(), _stream_on(stream, parents))
    return rc if rc >= 0 else _check(fn, rc)


def idx_release_pages(keep_lens, owned_pages, block_table, refs, free_blocks, free_cursor, cursor_out, pages_out, page_tokens: int, status=None,
                      stream=None) -> int:
    """Pages past keep_lens [R] i32 given back: refs [nb] i32 less one each, the blocks that nobody holds into free_blocks before the
    cursor by ascending id; cursor_out, and pages_out [R] i32, the pages that are left.  A length that ends inside a page with refs
    above 0 afterwards must not be written on from: such a request is forked there, which copies the page, and given up."""
    lib, T, fn = load_library(), _torch(), "idx_release_pages"
    i32 = T.i32
    reqs, width = block_table.shape
    per_req, nb, free = (reqs,), refs.shape[0], free_blocks.shape[0]
    if not (_are(i32, per_req, keep_lens, owned_pages, pages_out) and _rows_ok(i32, (reqs, width), block_table) and _are(i32, (nb,), refs)
            and _are(i32, (free,), free_blocks) and _are(i32, (1,), free_cursor, cursor_out) and (status is None or (status.is_cuda and status.dtype is i32 and status.numel() > 0))
            and (not T.many or _here(keep_lens, owned_pages, pages_out, block_table, refs, free_blocks, free_cursor, cursor_out, status))):
        _explain(fn, ("keep_lens", "owned_pages", "pages_out", "refs", "free_blocks", "free_cursor", "cursor_out"),
                 keep_lens=(keep_lens, i32, per_req), owned_pages=(owned_pages, i32, per_req), pages_out=(pages_out, i32, per_req),
                 block_table=(block_table, i32, (reqs, None)), refs=(refs, i32, (None,)), free_blocks=(free_blocks, i32, (None,)),
                 free_cursor=(free_cursor, i32, (1,)), cursor_out=(cursor_out, i32, (1,)), status=(status, i32, None))
    rc = lib.idx_release_pages(
        keep_lens.data_ptr(), owned_pages.data_ptr(), reqs, block_table.data_ptr(), _row_stride(block_table), width, refs.data_ptr(), nb,
        free_blocks.data_ptr(), free, free_cursor.data_ptr(), cursor_out.data_ptr(), pages_out.data_ptr(), page_tokens, None if status is None else status.data_ptr(),
        _stream_on(stream, refs))
    return rc if rc >= 0 else _check(fn, rc)
