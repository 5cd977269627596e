"""Python binding of libdsa.so, the B200 (sm_100a) DSA sparse-attention prefill library.

Argument marshalling only: each function below passes its arguments to the C
entry point of the same name (declared in include/dsa.h) and returns its
status code. Every step of the layer runs in the library's CUDA kernels;
there is no other implementation to fall back to: the first call raises
RuntimeError when libdsa.so has not been built.

Tensors may be given as torch tensors (their data_ptr() is passed) or as raw
integer device addresses. ``stream`` defaults to torch's current CUDA stream.

DSA_LIBRARY=check in the environment loads libdsa_check.so instead: the same
kernels built with bounds checks that report a bad index in the workspace
status (DSA_ERR_CUDA from dsa_device_status, site 1000 + n in the header)
rather than making the access.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsa_check.so" if os.environ.get("DSA_LIBRARY") == "check"
                        else "libdsa.so")

_lib = None

DSA_OK = 0
DSA_ERR_NULL = -1
DSA_ERR_ALIGN = -2
DSA_ERR_DIMS = -3
DSA_ERR_CAUSAL = -4
DSA_ERR_WORKSPACE = -5
DSA_ERR_TIMEOUT = -6
DSA_ERR_CUDA = -7
DSA_ERR_DEVICE = -8
DSA_ERR_RANGE = -9
DSA_ERR_SCRATCH_LIMIT = -10
DSA_ERR_LAYOUT = -11
DSA_NOALLOC_SCRATCH_BYTES = 32 << 20

DSA_WS_INDEX_SCORES = 0
DSA_WS_TOPK = 1
DSA_WS_ATTN = 2
DSA_WS_LAYER = 3
DSA_WS_DECODE_ATTN = 4
DSA_WS_DECODE_LAYER = 5
DSA_WS_BLOCK_ATTN = 6
DSA_FLAG_FP8_INDEXER = 1
DSA_FLAG_ATTN_PAIR = 2
DSA_FLAG_HOST_UNORDERED = 4
DSA_FLAG_L2_SCORES = 8
DSA_MAX_BLOCK_QUERIES = 2

DSA_ROPE_INTERLEAVED = 0
DSA_ROPE_HALVES = 1

DSA_MAX_TOPK = 2048
DSA_MAX_CTX = 131072

EXPORTED = ("dsa_workspace_size", "dsa_index_scores", "dsa_topk_select",
            "dsa_sparse_attn_prefill", "dsa_prefill_layer", "dsa_device_status",
            "dsa_status_string", "dsa_prefill_layer_noalloc", "dsa_prefill_layer_host",
            "dsa_selftest_bounded_wait", "dsa_partition_queries", "dsa_sparse_attn_decode",
            "dsa_decode_layer", "dsa_sparse_attn_block", "dsa_quantize_fp8",
            "dsa_index_scores_fp8", "dsa_selftest_mma_layout", "dsa_cache_workspace_size",
            "dsa_cache_append", "dsa_cache_gather", "dsa_cache_attn", "dsa_selftest_cache_wait")


class dsa_dims(ctypes.Structure):
    _fields_ = [
        ("n_q", ctypes.c_int32),
        ("q_pos0", ctypes.c_int32),
        ("ctx_len", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
        ("d_latent", ctypes.c_int32),
        ("d_rope", ctypes.c_int32),
        ("n_idx_heads", ctypes.c_int32),
        ("d_idx", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float),
        ("flags", ctypes.c_uint32),
    ]


class dsa_device_tensors(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in
                ("q", "latent", "rope", "q_idx", "k_idx", "w_idx", "out", "lse", "idx")]


class dsa_cache(ctypes.Structure):
    _fields_ = [
        ("latent", ctypes.c_void_p),
        ("rope", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
        ("latent_page_stride", ctypes.c_int64),
        ("rope_page_stride", ctypes.c_int64),
        ("n_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("d_latent", ctypes.c_int32),
        ("d_rope", ctypes.c_int32),
    ]


class dsa_batch(ctypes.Structure):
    _fields_ = [
        ("page_table", ctypes.c_void_p),
        ("cu_seqlens", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p),
        ("n_seq", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("n_tok", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class DsaError(RuntimeError):
    def __init__(self, status: int):
        super().__init__(f"dsa status {status}: {dsa_status_string(status)}")
        self.status = status


_P = ctypes.c_void_p
_DP = ctypes.POINTER(dsa_dims)
_CP = ctypes.POINTER(dsa_cache)
_BP = ctypes.POINTER(dsa_batch)


def library():
    """The loaded ctypes library; raises RuntimeError if it was never built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: the DSA CUDA library has not been built "
            "(python -m sparse_attention_prefill_dsa_b200.build). There is no fallback.")
    lib = ctypes.CDLL(LIB_PATH)
    lib.dsa_workspace_size.argtypes = [_DP, ctypes.c_int32]
    lib.dsa_workspace_size.restype = ctypes.c_size_t
    lib.dsa_index_scores.argtypes = [_DP, _P, _P, _P, _P, ctypes.c_int64, _P, ctypes.c_size_t, _P]
    lib.dsa_topk_select.argtypes = [_DP, _P, ctypes.c_int64, _P, _P, _P, _P, _P, ctypes.c_size_t,
                                    _P]
    lib.dsa_sparse_attn_prefill.argtypes = [_DP, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
    lib.dsa_prefill_layer.argtypes = [_DP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                      ctypes.c_size_t, _P]
    lib.dsa_sparse_attn_decode.argtypes = [_DP, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
    lib.dsa_decode_layer.argtypes = [_DP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                     ctypes.c_size_t, _P]
    lib.dsa_sparse_attn_block.argtypes = [_DP, _P, _P, _P, _P, _P, _P, ctypes.c_int32, _P,
                                          ctypes.c_size_t, _P]
    lib.dsa_quantize_fp8.argtypes = [_P, ctypes.c_int64, ctypes.c_int32, _P, _P, _P, _P]
    lib.dsa_index_scores_fp8.argtypes = [_DP, _P, _P, _P, _P, _P, _P, ctypes.c_int64, _P,
                                         ctypes.c_size_t, _P]
    lib.dsa_prefill_layer_noalloc.argtypes = [_DP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]
    lib.dsa_prefill_layer_host.argtypes = [_DP, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                           ctypes.POINTER(dsa_device_tensors), _P, ctypes.c_size_t,
                                           ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.c_int32]
    lib.dsa_selftest_bounded_wait.argtypes = [_P, ctypes.c_size_t, _P, _P]
    lib.dsa_selftest_mma_layout.argtypes = [_P, ctypes.c_size_t, ctypes.POINTER(ctypes.c_int32),
                                            ctypes.POINTER(ctypes.c_float), _P]
    lib.dsa_partition_queries.argtypes = [_DP, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)]
    i32, i64, size = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.dsa_cache_workspace_size.argtypes = [_CP, _BP, i32]
    lib.dsa_cache_workspace_size.restype = size
    lib.dsa_cache_append.argtypes = [_CP, _BP, _P, i64, _P, i64, _P, i32, _P, i64, i64, _P, i32, _P,
                                     size, _P]
    lib.dsa_cache_gather.argtypes = [_CP, _BP, i32, i32, i32, _P, _P, _P, size, _P]
    lib.dsa_cache_attn.argtypes = [_CP, _BP, _P, i32, ctypes.c_float, i32, i32, _P, _P, _P, size,
                                   _P]
    lib.dsa_selftest_cache_wait.argtypes = [_CP, _BP, _P, i32, ctypes.c_float, i32, i32, _P, _P,
                                            i64, _P, size, _P]
    lib.dsa_device_status.argtypes = [_P, _P]
    lib.dsa_status_string.argtypes = [ctypes.c_int32]
    lib.dsa_status_string.restype = ctypes.c_char_p
    for f in ("dsa_index_scores", "dsa_topk_select", "dsa_sparse_attn_prefill",
              "dsa_prefill_layer", "dsa_device_status", "dsa_prefill_layer_noalloc",
              "dsa_prefill_layer_host", "dsa_selftest_bounded_wait", "dsa_partition_queries",
              "dsa_sparse_attn_decode", "dsa_decode_layer", "dsa_sparse_attn_block",
              "dsa_quantize_fp8", "dsa_index_scores_fp8", "dsa_selftest_mma_layout",
              "dsa_cache_append", "dsa_cache_gather", "dsa_cache_attn", "dsa_selftest_cache_wait"):
        getattr(lib, f).restype = ctypes.c_int32
    _lib = lib
    return lib


def make_dims(d) -> dsa_dims:
    """dsa_dims from any object with the same attribute names (flags default 0)."""
    return dsa_dims(int(d.n_q), int(d.q_pos0), int(d.ctx_len), int(d.n_heads),
                    int(d.d_latent), int(d.d_rope), int(d.n_idx_heads), int(d.d_idx),
                    int(d.top_k), float(d.softmax_scale), int(getattr(d, "flags", 0)))


def _dims(d):
    return ctypes.byref(d if isinstance(d, dsa_dims) else make_dims(d))


def _p(x):
    if x is None:
        return None
    if isinstance(x, int):
        return _P(x)
    return _P(x.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        return _P(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return _P(stream)
    return _P(stream.cuda_stream)


def _nbytes(ws, ws_bytes):
    if ws_bytes is not None:
        return int(ws_bytes)
    if ws is None or isinstance(ws, int):
        return 0
    return ws.numel() * ws.element_size()


def dsa_workspace_size(dims, which: int) -> int:
    return int(library().dsa_workspace_size(_dims(dims), int(which)))


def dsa_index_scores(dims, q_idx, k_idx, w_idx, scores, ld_scores, workspace, workspace_bytes=None,
                     stream=None) -> int:
    return library().dsa_index_scores(_dims(dims), _p(q_idx), _p(k_idx), _p(w_idx), _p(scores),
                                 int(ld_scores), _p(workspace),
                                 _nbytes(workspace, workspace_bytes), _stream(stream))


def dsa_topk_select(dims, scores, ld_scores, q_idx, k_idx, w_idx, idx, workspace,
                    workspace_bytes=None, stream=None) -> int:
    return library().dsa_topk_select(_dims(dims), _p(scores), int(ld_scores), _p(q_idx), _p(k_idx),
                                _p(w_idx), _p(idx), _p(workspace),
                                _nbytes(workspace, workspace_bytes), _stream(stream))


def dsa_sparse_attn_prefill(dims, q, latent, rope, idx, out, lse, workspace, workspace_bytes=None,
                            stream=None) -> int:
    return library().dsa_sparse_attn_prefill(_dims(dims), _p(q), _p(latent), _p(rope), _p(idx),
                                        _p(out), _p(lse), _p(workspace),
                                        _nbytes(workspace, workspace_bytes), _stream(stream))


def dsa_prefill_layer(dims, q, latent, rope, q_idx, k_idx, w_idx, out, lse, idx_out, workspace,
                      workspace_bytes=None, stream=None) -> int:
    return library().dsa_prefill_layer(_dims(dims), _p(q), _p(latent), _p(rope), _p(q_idx),
                                  _p(k_idx), _p(w_idx), _p(out), _p(lse), _p(idx_out),
                                  _p(workspace), _nbytes(workspace, workspace_bytes),
                                  _stream(stream))


def dsa_sparse_attn_decode(dims, q, latent, rope, idx, out, lse, workspace, workspace_bytes=None,
                           stream=None) -> int:
    return library().dsa_sparse_attn_decode(_dims(dims), _p(q), _p(latent), _p(rope), _p(idx),
                                            _p(out), _p(lse), _p(workspace),
                                            _nbytes(workspace, workspace_bytes), _stream(stream))


def dsa_sparse_attn_block(dims, q, latent, rope, idx, out, lse, block_queries, workspace,
                          workspace_bytes=None, stream=None) -> int:
    return library().dsa_sparse_attn_block(_dims(dims), _p(q), _p(latent), _p(rope), _p(idx),
                                           _p(out), _p(lse), int(block_queries), _p(workspace),
                                           _nbytes(workspace, workspace_bytes), _stream(stream))


def dsa_quantize_fp8(x, rows, cols, x8, scale, xhat, stream=None) -> int:
    return library().dsa_quantize_fp8(_p(x), int(rows), int(cols), _p(x8), _p(scale), _p(xhat),
                                      _stream(stream))


def dsa_index_scores_fp8(dims, q8, q_scale, k8, k_scale, w_idx, scores, ld_scores, workspace,
                         workspace_bytes=None, stream=None) -> int:
    return library().dsa_index_scores_fp8(_dims(dims), _p(q8), _p(q_scale), _p(k8), _p(k_scale),
                                          _p(w_idx), _p(scores), int(ld_scores), _p(workspace),
                                          _nbytes(workspace, workspace_bytes), _stream(stream))


def dsa_decode_layer(dims, q, latent, rope, q_idx, k_idx, w_idx, out, lse, idx_out, workspace,
                     workspace_bytes=None, stream=None) -> int:
    return library().dsa_decode_layer(_dims(dims), _p(q), _p(latent), _p(rope), _p(q_idx),
                                      _p(k_idx), _p(w_idx), _p(out), _p(lse), _p(idx_out),
                                      _p(workspace), _nbytes(workspace, workspace_bytes),
                                      _stream(stream))


def dsa_prefill_layer_noalloc(dims, q, latent, rope, q_idx, k_idx, w_idx, out, lse, idx_out,
                              device_status=None, stream=None) -> int:
    """The layer on the library's static scratch array (no workspace argument)."""
    return library().dsa_prefill_layer_noalloc(_dims(dims), _p(q), _p(latent), _p(rope),
                                               _p(q_idx), _p(k_idx), _p(w_idx), _p(out), _p(lse),
                                               _p(idx_out), _p(device_status), _stream(stream))


def dsa_prefill_layer_host(dims, q, latent, rope, q_idx, k_idx, w_idx, out, lse, idx_out, dev,
                           workspace, streams, events, n_sub=4, workspace_bytes=None) -> int:
    """The layer on host buffers (q .. idx_out: page-locked host tensors or
    addresses), copies overlapped with the compute over n_sub query
    sub-chunks. dev maps the names of dsa_device_tensors to device tensors or
    addresses; streams are three CUDA streams (copy in, compute, copy out),
    events two CUDA events (torch.cuda.Event or raw cudaEvent_t addresses)."""
    d = dsa_device_tensors(*[_p(dev.get(name)) for name, _ in dsa_device_tensors._fields_])
    st = (_P * 3)(*[_stream(x) for x in streams])
    ev = (_P * 2)(*[_P(x) if isinstance(x, int) else _P(x.cuda_event) for x in events])
    return library().dsa_prefill_layer_host(_dims(dims), _p(q), _p(latent), _p(rope), _p(q_idx),
                                            _p(k_idx), _p(w_idx), _p(out), _p(lse), _p(idx_out),
                                            ctypes.byref(d), _p(workspace),
                                            _nbytes(workspace, workspace_bytes), st, ev, int(n_sub))


def dsa_selftest_bounded_wait(workspace, cycles=None, workspace_bytes=None, stream=None) -> int:
    """One CTA whose bounded waits give up (see include/dsa.h); cycles is an
    optional device int64 tensor of 2 elements."""
    return library().dsa_selftest_bounded_wait(_p(workspace), _nbytes(workspace, workspace_bytes),
                                               _p(cycles), _stream(stream))


def dsa_selftest_mma_layout(workspace, workspace_bytes=None, stream=None):
    """The tensor-core layout self-test (see include/dsa.h): returns (status,
    [wrong elements of each of the four forms], [cycles per MMA of each form])."""
    counts = (ctypes.c_int32 * 4)()
    cycles = (ctypes.c_float * 4)()
    st = library().dsa_selftest_mma_layout(_p(workspace), _nbytes(workspace, workspace_bytes),
                                           counts, cycles, _stream(stream))
    return st, list(counts), list(cycles)


def dsa_device_status(workspace, stream=None) -> int:
    return library().dsa_device_status(_p(workspace), _stream(stream))


def dsa_status_string(status: int) -> str:
    return library().dsa_status_string(int(status)).decode()


def check(status: int) -> None:
    """Raises DsaError unless status is DSA_OK."""
    if status != DSA_OK:
        raise DsaError(status)



def dsa_partition_queries(dims, n_parts: int, starts=None):
    """Query ranges of one chunk over n_parts ranks (see include/dsa.h).
    Returns (status, starts) with starts a list of n_parts + 1 row offsets."""
    arr = (ctypes.c_int32 * (int(n_parts) + 1))() if n_parts >= 1 else (ctypes.c_int32 * 1)()
    st = library().dsa_partition_queries(_dims(dims), int(n_parts), arr)
    out = list(arr)
    if starts is not None:
        starts[:] = out
    return st, out


def make_cache(latent, rope, scale) -> dsa_cache:
    """dsa_cache of three device tensors: latent and rope, one byte an element,
    [n_pages, page_size, width] with dense pages (the stride between pages is
    taken from the tensor), and scale, float32 [n_pages]. The struct keeps the
    tensors alive."""
    for name, x in (("latent", latent), ("rope", rope)):
        if x.dim() != 3 or x.element_size() != 1 or (
                x.numel() and (x.stride(2) != 1 or x.stride(1) != x.shape[2])):
            raise ValueError(f"{name}: [n_pages, page_size, width] of one-byte elements with dense "
                             "pages is wanted")
    if latent.shape[:2] != rope.shape[:2] or tuple(scale.shape) != (latent.shape[0],) or \
            str(scale.dtype) != "torch.float32" or not scale.is_contiguous():
        raise ValueError("latent, rope and scale (float32 [n_pages]) do not belong together")
    pages, size, dc = latent.shape
    # a pool of one page may have any stride; the call checks the lower bound
    c = dsa_cache(latent.data_ptr(), rope.data_ptr(), scale.data_ptr(),
                  latent.stride(0) if pages > 1 else size * dc,
                  rope.stride(0) if pages > 1 else size * rope.shape[2], pages, size, dc,
                  rope.shape[2])
    c.tensors = (latent, rope, scale)
    return c


def make_batch(page_table, cu_seqlens, seq_lens, n_tok: int) -> dsa_batch:
    """dsa_batch of three int32 device tensors: page_table [n_seq, max_pages],
    cu_seqlens [n_seq + 1] and seq_lens [n_seq], all dense; n_tok is the number
    of rows of the calls' token tensors. The struct keeps the tensors alive."""
    n_seq = seq_lens.shape[0]
    for x in (page_table, cu_seqlens, seq_lens):
        if str(x.dtype) != "torch.int32" or not x.is_contiguous():
            raise ValueError("dense int32 tensors are wanted")
    if page_table.dim() != 2 or page_table.shape[0] != n_seq or cu_seqlens.shape != (n_seq + 1,) or \
            seq_lens.dim() != 1:
        raise ValueError("page_table [n_seq, max_pages], cu_seqlens [n_seq + 1] and seq_lens "
                         "[n_seq] do not belong together")
    b = dsa_batch(page_table.data_ptr(), cu_seqlens.data_ptr(), seq_lens.data_ptr(), n_seq,
                  page_table.shape[1], int(n_tok), 0)
    b.tensors = (page_table, cu_seqlens, seq_lens)
    return b


def _ld(ld, x, dim, default):
    """A stride in elements: the one given, else the tensor's, else the dense one."""
    if ld is not None:
        return int(ld)
    if x is None or isinstance(x, int):
        return default
    strides = x.stride()
    if strides[-1] != 1 and x.shape[-1] > 1:
        raise ValueError("rows have to be dense in their last dimension")
    # (a dimension of one may have any stride)
    return default if strides[dim] == default or x.shape[dim] == 1 else strides[dim]


def dsa_cache_workspace_size(cache, batch, n_heads: int) -> int:
    return int(library().dsa_cache_workspace_size(cache, batch, int(n_heads)))


def _at(x):
    """Address of a tensor or raw address (ctypes converts the int)."""
    return x if x is None or isinstance(x, int) else x.data_ptr()


_raw_stream = None


def _on(stream):
    """Raw stream: the one given, or torch's current one, without making a
    torch.cuda.Stream for it (these calls are made every step of a decode)."""
    global _raw_stream
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    if _raw_stream is None:
        import torch

        get, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
        _raw_stream = (lambda: get(device())) if get is not None else (
            lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def dsa_cache_append(cache, batch, latent, rope, inv_freq, rope_style, q_rope, q, n_heads,
                     workspace, workspace_bytes=None, stream=None, ld_latent=None, ld_rope=None,
                     ld_q_tok=None, ld_q_head=None) -> int:
    """Strides are taken from the tensors unless given (see include/dsa.h)."""
    dr = cache.d_rope
    return library().dsa_cache_append(
        cache, batch, _at(latent), _ld(ld_latent, latent, 0, cache.d_latent), _at(rope),
        _ld(ld_rope, rope, 0, dr), _at(inv_freq), rope_style, _at(q_rope),
        _ld(ld_q_tok, q_rope, 0, n_heads * dr), _ld(ld_q_head, q_rope, 1, dr), _at(q), n_heads,
        _at(workspace), _nbytes(workspace, workspace_bytes), _on(stream))


def dsa_cache_gather(cache, batch, seq, pos0, n_rows, latent, rope, workspace,
                     workspace_bytes=None, stream=None) -> int:
    return library().dsa_cache_gather(cache, batch, seq, pos0, n_rows, _at(latent), _at(rope),
                                      _at(workspace), _nbytes(workspace, workspace_bytes),
                                      _on(stream))


def dsa_cache_attn(cache, batch, q, n_heads, softmax_scale, window, n_sink, out, lse, workspace,
                   workspace_bytes=None, stream=None) -> int:
    return library().dsa_cache_attn(cache, batch, _at(q), n_heads, softmax_scale, window, n_sink,
                                    _at(out), _at(lse), _at(workspace),
                                    _nbytes(workspace, workspace_bytes), _on(stream))


def dsa_selftest_cache_wait(cache, batch, q, n_heads, softmax_scale, window, n_sink, out, lse,
                            wait_cycles, workspace, workspace_bytes=None, stream=None) -> int:
    """dsa_cache_attn with its waits limited to wait_cycles (see include/dsa.h)."""
    return library().dsa_selftest_cache_wait(cache, batch, _at(q), n_heads, softmax_scale, window,
                                             n_sink, _at(out), _at(lse), int(wait_cycles),
                                             _at(workspace), _nbytes(workspace, workspace_bytes),
                                             _on(stream))
