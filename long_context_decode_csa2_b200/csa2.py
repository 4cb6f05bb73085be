"""Thin Python binding of the CSA2 C ABI (``include/csa2.h``).

Argument marshalling only: every function below checks each tensor's element
type and size against the C declaration (the library sees only pointers),
forwards the torch CUDA tensors as raw device pointers to the function of the
same name in ``libcsa2.so`` and raises on a non-zero status.  All computation
happens in the library's CUDA kernels; there is no fallback of any kind.  Workspaces come from
``workspace(nbytes)`` (zero-filled, 256-byte aligned torch allocations).
"""
from __future__ import annotations

import ctypes as C
import os

import torch

from . import _build

MAIN_DIM, Q_HEADS, IDX_HEADS, IDX_DIM, BLOCK, WINDOW = 512, 16, 4, 128, 8, 128
DEV_FLAGS = {1: "INDEX_RANGE", 2: "ROW_LAYOUT", 4: "FP16_RANGE", 8: "LENGTH", 16: "TIMEOUT", 32: "NO_TOKEN"}

_lib = None


class Csa2Error(RuntimeError):
    def __init__(self, status, fn, msg):
        super().__init__(f"{fn}: status {status} ({msg})")
        self.status = status


class MXFP4Cache(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("rows", C.c_int64)]


class PageTable:
    """Paged cache layout: ``pages`` [B, max_pages] int32 CUDA tensor of page
    ids, ``page_rows`` rows per page (a power of two, >= 512).  Pass it where a
    call takes ``seq_row_off``; the ``*_paged`` entry point is used then."""

    def __init__(self, pages: torch.Tensor, page_rows: int):
        assert pages.dtype == torch.int32 and pages.dim() == 2
        self.pages, self.page_rows = pages, int(page_rows)

    @property
    def max_pages(self):
        return self.pages.shape[1]


def lib():
    """Load (building first if the sources are newer) the CUDA library."""
    global _lib
    if _lib is None:
        path = _build.LIB
        if _build.stale():
            path = _build.build()
        if not os.path.exists(path):
            raise RuntimeError("libcsa2.so is missing and could not be built")
        L = C.CDLL(path)
        P, I, I64, F, Z = C.c_void_p, C.c_int, C.c_int64, C.c_float, C.c_size_t
        Cache = MXFP4Cache
        sig = {
            "csa2_index_full_workspace_bytes": (Z, [I, I, I, I]),
            "csa2_index_full": (I, [Cache, P, P, P, P, P, I, I, I, I, P, P, P, P, Z, P]),
            "csa2_index_reindex_workspace_bytes": (Z, [I, I, I]),
            "csa2_index_reindex": (I, [Cache, P, P, P, P, P, P, I, I, I, P, P, Z, P]),
            "csa2_sparse_attn_decode_workspace_bytes": (Z, [I, I]),
            "csa2_sparse_attn_decode": (I, [P, Cache, P, P, P, I, P, P, P, F, P, P, I, P, Z, P]),
            "csa2_compress_append_workspace_bytes": (Z, [I]),
            "csa2_compress_append": (I, [Cache, Cache, P, P, P, P, P, P, P, P, I, I, I64, I64, P, Z, P]),
            "csa2_compress_stream_workspace_bytes": (Z, [I]),
            "csa2_compress_stream": (I, [Cache, Cache, P, P, P, P, P, P, P, P, P, P, P, P, I, I64, I64, P, Z, P]),
            "csa2_index_multi_workspace_bytes": (Z, [I, I, I64, I, I]),
            "csa2_index_multi": (I, [Cache, P, P, P, P, P, P, I, I, I64, I, I, P, P, P, P, Z, P]),
            "csa2_index_full_pool": (I, [Cache, P, P, P, P, P, I, I, I, I, P, P, P, Z, P]),
            "csa2_index_full_topk": (I, [Cache, P, P, P, P, P, I, I, I, I, P, P, P, P, Z, P]),
            "csa2_index_full_paged": (I, [Cache, P, P, P, P, I, I, P, I, I, I, I, P, P, P, P, Z, P]),
            "csa2_index_reindex_paged": (I, [Cache, P, P, P, P, I, I, P, P, I, I, I, P, P, Z, P]),
            "csa2_sparse_attn_decode_paged": (I, [P, Cache, P, I, I, P, P, I, P, P, P, F, P, P, I, P, Z, P]),
            "csa2_compress_stream_paged": (I, [Cache, Cache, P, P, P, P, P, P, I, I, P, P, P, P, P, P, I, I64, I64, P,
                                               Z, P]),
            "csa2_score_positions_workspace_bytes": (Z, [I]),
            "csa2_score_positions": (I, [Cache, P, P, P, P, P, P, I, I, I, P, P, Z, P]),
            "csa2_topk_merge_workspace_bytes": (Z, [I, I, I]),
            "csa2_topk_merge": (I, [P, P, P, I, I, I, I, P, P, P, P, P, Z, P]),
            "csa2_attn_combine": (I, [P, P, I, I, P, P, P]),
            "csa2_index_prefill_workspace_bytes": (Z, [I, I64, I, I]),
            "csa2_index_prefill": (I, [Cache, P, P, P, P, I, I64, I64, I, I, I, P, P, P, Z, P]),
            "csa2_sparse_attn_prefill_workspace_bytes": (Z, [I, I]),
            "csa2_sparse_attn_prefill": (I, [P, P, I, Cache, I64, I64, I, P, I, P, I64, F, F, P, P, P, Z, P]),
            "csa2_sparse_attn_decode_noalloc": (I, [P, Cache, P, P, P, I, P, P, P, F, P, P, P, I, P]),
            "csa2_verify_drafts_workspace_bytes": (Z, [I, I]),
            "csa2_verify_drafts": (I, [P, I, I64, P, I, I64, P, P, P, P, I, I, I, P, P, P, P, P, I, P, Z, P]),
            "csa2_attn_weights_workspace_bytes": (Z, [I, I, I]),
            "csa2_attn_weights": (I, [P, Cache, P, P, P, P, P, I, P, F, P, P, I, I, P, Z, P]),
            "csa2_attn_weights_paged": (I, [P, Cache, P, I, I, P, P, P, P, I, P, F, P, P, I, I, P, Z, P]),
            "csa2_acc_clear_workspace_bytes": (Z, [I]),
            "csa2_acc_clear": (I, [P, I64, P, P, P, I, P, Z, P]),
            "csa2_acc_clear_paged": (I, [P, I64, P, I, I, P, P, I, P, Z, P]),
            "csa2_cache_evict_workspace_bytes": (Z, [I, I]),
            "csa2_cache_evict": (I, [Cache, Cache, P, P, P, P, Cache, Cache, P, P, P, P, I, I, I, I, I, P, Z, P]),
            "csa2_cache_evict_paged": (I, [Cache, Cache, P, P, I, P, P, Cache, Cache, P, P, I, I, P, P, I, I, I, I, I,
                                           P, Z, P]),
            "csa2_cache_evict_layers": (I, [I, P, P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, P, Z, P]),
            "csa2_cache_evict_layers_paged": (I, [I, P, P, P, P, I, P, P, P, P, P, P, I, I, P, P, I, I, I, I, I, P, Z,
                                                  P]),
            "csa2_device_status": (I, [P, P, C.POINTER(C.c_uint32)]),
            "csa2_status_string": (C.c_char_p, [I]),
            "csa2_last_error": (C.c_char_p, []),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_cuda:
        raise ValueError("CSA2 arguments must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("CSA2 arguments must be contiguous")
    return t.data_ptr()


_Tensor = torch.Tensor

# Element types of the C ABI's pointer arguments and the torch dtypes that
# may carry them (same width, same kind of number).
_KINDS = {
    "u8": (torch.uint8, torch.int8, torch.float8_e4m3fn),   # E2M1 codes, E8M0 scales, E4M3 bytes
    "bf16": (torch.bfloat16, torch.int16, torch.uint16),    # bf16 bit patterns
    "i32": (torch.int32, torch.uint32),                     # int32 ids / lengths, uint32 keys and flags
    "f32": (torch.float32,),
    "i64": (torch.int64, torch.uint64),
    "prob": (torch.float32, torch.bfloat16, torch.float16),  # probabilities, with a type code beside the pointer
}


def _arg(fn, name, t, kind, numel=0):
    """Device pointer of an optional tensor argument, after checking that its
    elements have the C type's width and kind and that it holds at least
    `numel` of them (the library cannot see buffer sizes)."""
    if t is None:
        return None
    if not isinstance(t, _Tensor):
        raise Csa2Error(-1, fn, f"{name}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype not in _KINDS[kind]:
        raise Csa2Error(-1, fn, f"{name}: {kind} elements expected, got {t.dtype}")
    if t.numel() < numel:
        raise Csa2Error(-1, fn, f"{name}: at least {numel} elements expected, got {t.numel()}")
    return t.data_ptr() if t.is_cuda and t.is_contiguous() else _ptr(t)


def _queries(fn, n, q_codes, q_scales, w):
    """Pointers of n indexer queries: codes [n][4][64], scales [n][4][4], weights [n][4]."""
    return (_arg(fn, "q_codes", q_codes, "u8", n * IDX_HEADS * IDX_DIM // 2),
            _arg(fn, "q_scales", q_scales, "u8", n * IDX_HEADS * IDX_DIM // 32),
            _arg(fn, "w", w, "f32", n * IDX_HEADS))


def _window(fn, n, win, win_scale, win_len):
    return (_arg(fn, "win", win, "u8", n * WINDOW * MAIN_DIM), _arg(fn, "win_scale", win_scale, "f32", n),
            _arg(fn, "win_len", win_len, "i32", n))


def _attn_out(fn, n, out, lse):
    return _arg(fn, "out", out, "f32", n * Q_HEADS * MAIN_DIM), _arg(fn, "lse", lse, "f32", n * Q_HEADS)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _check(rc, fn):
    if rc != 0:
        L = lib()
        raise Csa2Error(rc, fn, L.csa2_last_error().decode() or L.csa2_status_string(rc).decode())


def cache(codes: torch.Tensor, scales: torch.Tensor) -> MXFP4Cache:
    """Describe an MXFP4 cache: codes uint8 [rows, n/2], scales uint8 [rows, n/32].

    The returned struct keeps references to both tensors, so the memory stays
    alive as long as the struct does."""
    assert codes.dtype == torch.uint8 and scales.dtype == torch.uint8 and codes.shape[0] == scales.shape[0]
    c = MXFP4Cache(_ptr(codes), _ptr(scales), codes.shape[0])
    c._keep = (codes, scales)
    return c


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """Zero-filled device scratch (torch allocations are 256-byte aligned)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


def _ws(ws):
    return _ptr(ws), ws.numel()


def device_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronise, return and clear the workspace's device status flags."""
    flags = C.c_uint32(0)
    rc = lib().csa2_device_status(_ptr(ws), _stream(stream), C.byref(flags))
    if rc not in (0, -5):
        _check(rc, "csa2_device_status")
    return int(flags.value)


# ----------------------------------------------------------------------------
# one wrapper per C entry point
# ----------------------------------------------------------------------------

def csa2_index_full_workspace_bytes(B, max_len, pool_blocks, k):
    return lib().csa2_index_full_workspace_bytes(B, max_len, pool_blocks, k)


def _full_args(fn, q_codes, q_scales, w, seq_len, max_len, pool_blocks, k, pool_out, topk_out, scores_out):
    B = seq_len.shape[0]
    return (B, *_queries(fn, B, q_codes, q_scales, w), _arg(fn, "seq_len", seq_len, "i32", B),
            _arg(fn, "pool_out", pool_out, "i32", B * pool_blocks), _arg(fn, "topk_out", topk_out, "i32", B * k),
            _arg(fn, "scores_out", scores_out, "f32", B * max_len))


def _row_off(fn, seq_row_off, B):
    return _arg(fn, "seq_row_off", seq_row_off, "i64", B)


def _pages(fn, pt, B):
    return _arg(fn, "pages", pt.pages, "i32", B * pt.max_pages)


def csa2_index_full(idx_k, q_codes, q_scales, w, seq_row_off, seq_len, max_len, pool_blocks, k, pool_out, topk_out,
                    ws, scores_out=None, stream=None):
    wp, wn = _ws(ws)
    if isinstance(seq_row_off, PageTable):
        fn, pt = "csa2_index_full_paged", seq_row_off
        B, qc, qs, wv, sl, po, to, so = _full_args(fn, q_codes, q_scales, w, seq_len, max_len, pool_blocks, k,
                                                   pool_out, topk_out, scores_out)
        rc = lib().csa2_index_full_paged(idx_k, qc, qs, wv, _pages(fn, pt, B), pt.page_rows, pt.max_pages, sl, B,
                                         max_len, pool_blocks, k, po, to, so, wp, wn, _stream(stream))
        _check(rc, fn)
        return
    fn = "csa2_index_full"
    B, qc, qs, wv, sl, po, to, so = _full_args(fn, q_codes, q_scales, w, seq_len, max_len, pool_blocks, k, pool_out,
                                               topk_out, scores_out)
    rc = lib().csa2_index_full(idx_k, qc, qs, wv, _row_off(fn, seq_row_off, B), sl, B, max_len, pool_blocks, k, po,
                               to, so, wp, wn, _stream(stream))
    _check(rc, fn)


def csa2_index_full_pool(idx_k, q_codes, q_scales, w, seq_row_off, seq_len, max_len, pool_blocks, k, pool_out, ws,
                         scores_out=None, stream=None):
    fn = "csa2_index_full_pool"
    wp, wn = _ws(ws)
    B, qc, qs, wv, sl, po, _, so = _full_args(fn, q_codes, q_scales, w, seq_len, max_len, pool_blocks, k, pool_out,
                                              None, scores_out)
    rc = lib().csa2_index_full_pool(idx_k, qc, qs, wv, _row_off(fn, seq_row_off, B), sl, B, max_len, pool_blocks, k,
                                    po, so, wp, wn, _stream(stream))
    _check(rc, fn)


def csa2_index_full_topk(idx_k, q_codes, q_scales, w, seq_row_off, seq_len, max_len, pool_blocks, k, pool, topk_out,
                         ws, scores_out=None, stream=None):
    fn = "csa2_index_full_topk"
    wp, wn = _ws(ws)
    B, qc, qs, wv, sl, po, to, so = _full_args(fn, q_codes, q_scales, w, seq_len, max_len, pool_blocks, k, pool,
                                               topk_out, scores_out)
    rc = lib().csa2_index_full_topk(idx_k, qc, qs, wv, _row_off(fn, seq_row_off, B), sl, B, max_len, pool_blocks, k,
                                    po, to, so, wp, wn, _stream(stream))
    _check(rc, fn)


def csa2_index_reindex_workspace_bytes(B, pool_blocks, k):
    return lib().csa2_index_reindex_workspace_bytes(B, pool_blocks, k)


def csa2_index_reindex(idx_k, q_codes, q_scales, w, seq_row_off, seq_len, pool, k, topk_out, ws, stream=None):
    B, P = pool.shape
    wp, wn = _ws(ws)
    paged = isinstance(seq_row_off, PageTable)
    fn = "csa2_index_reindex_paged" if paged else "csa2_index_reindex"
    qc, qs, wv = _queries(fn, B, q_codes, q_scales, w)
    sl, pp = _arg(fn, "seq_len", seq_len, "i32", B), _arg(fn, "pool", pool, "i32", B * P)
    to = _arg(fn, "topk_out", topk_out, "i32", B * k)
    if paged:
        pt = seq_row_off
        rc = lib().csa2_index_reindex_paged(idx_k, qc, qs, wv, _pages(fn, pt, B), pt.page_rows, pt.max_pages, sl, pp,
                                            B, P, k, to, wp, wn, _stream(stream))
    else:
        rc = lib().csa2_index_reindex(idx_k, qc, qs, wv, _row_off(fn, seq_row_off, B), sl, pp, B, P, k, to, wp, wn,
                                      _stream(stream))
    _check(rc, fn)


def csa2_sparse_attn_decode_workspace_bytes(B, k):
    return lib().csa2_sparse_attn_decode_workspace_bytes(B, k)


def _decode_args(fn, q, seq_len, topk, win, win_scale, win_len, out, lse):
    B, k = topk.shape
    return (B, k, _arg(fn, "q", q, "bf16", B * Q_HEADS * MAIN_DIM), _arg(fn, "seq_len", seq_len, "i32", B),
            _arg(fn, "topk", topk, "i32", B * k), *_window(fn, B, win, win_scale, win_len), *_attn_out(fn, B, out, lse))


def csa2_sparse_attn_decode(q, main_kv, seq_row_off, seq_len, topk, win, win_scale, win_len, sm_scale, out, ws,
                            lse=None, stream=None):
    wp, wn = _ws(ws)
    paged = isinstance(seq_row_off, PageTable)
    fn = "csa2_sparse_attn_decode_paged" if paged else "csa2_sparse_attn_decode"
    B, k, qp, sl, tp, wi, wsc, wl, op, lp = _decode_args(fn, q, seq_len, topk, win, win_scale, win_len, out, lse)
    if paged:
        pt = seq_row_off
        rc = lib().csa2_sparse_attn_decode_paged(qp, main_kv, _pages(fn, pt, B), pt.page_rows, pt.max_pages, sl, tp,
                                                 k, wi, wsc, wl, float(sm_scale), op, lp, B, wp, wn, _stream(stream))
    else:
        rc = lib().csa2_sparse_attn_decode(qp, main_kv, _row_off(fn, seq_row_off, B), sl, tp, k, wi, wsc, wl,
                                           float(sm_scale), op, lp, B, wp, wn, _stream(stream))
    _check(rc, fn)


def csa2_compress_append_workspace_bytes(B):
    return lib().csa2_compress_append_workspace_bytes(B)


def _append_args(fn, raw, logits, w_idx, idx_raw, tok_off, seq_len_in, seq_len_out):
    """Pointers of the token inputs and lengths shared by the append calls."""
    B = seq_len_in.shape[0]
    n_tok = raw.shape[0] if raw is not None else 0
    return (B, n_tok, _arg(fn, "raw", raw, "bf16", n_tok * MAIN_DIM), _arg(fn, "logits", logits, "f32", n_tok),
            _arg(fn, "w_idx", w_idx, "f32", MAIN_DIM * IDX_DIM), _arg(fn, "idx_raw", idx_raw, "bf16", n_tok * IDX_DIM),
            _arg(fn, "tok_off", tok_off, "i64", B + 1), _arg(fn, "seq_len_in", seq_len_in, "i32", B),
            _arg(fn, "seq_len_out", seq_len_out, "i32", B))


def csa2_compress_append(main_kv, idx_k, raw, logits, tok_off, seq_row_off, seq_len_in, seq_len_out, ratio, max_new,
                         ws, w_idx=None, idx_raw=None, stream=None):
    fn = "csa2_compress_append"
    wp, wn = _ws(ws)
    B, n_tok, rp, lg, wi, ir, to, li, lo = _append_args(fn, raw, logits, w_idx, idx_raw, tok_off, seq_len_in,
                                                        seq_len_out)
    rc = lib().csa2_compress_append(main_kv, idx_k, rp, lg, wi, ir, to, _row_off(fn, seq_row_off, B), li, lo, B,
                                    ratio, n_tok, int(max_new), wp, wn, _stream(stream))
    _check(rc, fn)


def csa2_compress_stream_workspace_bytes(B):
    return lib().csa2_compress_stream_workspace_bytes(B)


def csa2_compress_stream(main_kv, idx_k, raw, logits, tok_off, seq_row_off, seq_len_in, seq_len_out, pend_n, pend_raw,
                         pend_logit, max_new, ws, w_idx=None, idx_raw=None, pend_idx=None, stream=None):
    """seq_len_out may be seq_len_in (in place) or None; raw may be None when no token is appended."""
    wp, wn = _ws(ws)
    paged = isinstance(seq_row_off, PageTable)
    fn = "csa2_compress_stream_paged" if paged else "csa2_compress_stream"
    B, n_tok, rp, lg, wi, ir, to, li, lo = _append_args(fn, raw, logits, w_idx, idx_raw, tok_off, seq_len_in,
                                                        seq_len_out)
    pend = (_arg(fn, "pend_n", pend_n, "i32", B), _arg(fn, "pend_raw", pend_raw, "bf16", B * MAIN_DIM),
            _arg(fn, "pend_logit", pend_logit, "f32", B), _arg(fn, "pend_idx", pend_idx, "bf16", B * IDX_DIM))
    if paged:
        pt = seq_row_off
        rc = lib().csa2_compress_stream_paged(main_kv, idx_k, rp, lg, wi, ir, to, _pages(fn, pt, B), pt.page_rows,
                                              pt.max_pages, li, lo, *pend, B, n_tok, int(max_new), wp, wn,
                                              _stream(stream))
    else:
        rc = lib().csa2_compress_stream(main_kv, idx_k, rp, lg, wi, ir, to, _row_off(fn, seq_row_off, B), li, lo,
                                        *pend, B, n_tok, int(max_new), wp, wn, _stream(stream))
    _check(rc, fn)


def csa2_index_multi_workspace_bytes(B, Q, max_vis, pool_blocks, k):
    return lib().csa2_index_multi_workspace_bytes(B, Q, max_vis, pool_blocks, k)


def csa2_index_multi(idx_k, q_codes, q_scales, w, seq_row_off, q_off, q_vis, max_vis, pool_blocks, k, pool_out,
                     topk_out, ws, q_row_off_out=None, stream=None):
    fn = "csa2_index_multi"
    B, Q = seq_row_off.shape[0], q_vis.shape[0]
    wp, wn = _ws(ws)
    rc = lib().csa2_index_multi(idx_k, *_queries(fn, Q, q_codes, q_scales, w), _row_off(fn, seq_row_off, B),
                                _arg(fn, "q_off", q_off, "i32", B + 1), _arg(fn, "q_vis", q_vis, "i32", Q), B, Q,
                                int(max_vis), pool_blocks, k, _arg(fn, "pool_out", pool_out, "i32", Q * pool_blocks),
                                _arg(fn, "topk_out", topk_out, "i32", Q * k),
                                _arg(fn, "q_row_off_out", q_row_off_out, "i64", Q), wp, wn, _stream(stream))
    _check(rc, fn)


def csa2_score_positions_workspace_bytes(B):
    return lib().csa2_score_positions_workspace_bytes(B)


def csa2_score_positions(idx_k, q_codes, q_scales, w, seq_row_off, seq_len, ids, block, keys_out, ws, stream=None):
    """keys_out [B, n] uint32 (int32 tensors carry the bits) <- rank keys of ids [B, n] (block 1 or 8)."""
    fn = "csa2_score_positions"
    B, n = ids.shape
    wp, wn = _ws(ws)
    rc = lib().csa2_score_positions(idx_k, *_queries(fn, B, q_codes, q_scales, w), _row_off(fn, seq_row_off, B),
                                    _arg(fn, "seq_len", seq_len, "i32", B), _arg(fn, "ids", ids, "i32", B * n), B, n,
                                    int(block), _arg(fn, "keys_out", keys_out, "i32", B * n), wp, wn, _stream(stream))
    _check(rc, fn)


def csa2_topk_merge_workspace_bytes(G, B, n):
    return lib().csa2_topk_merge_workspace_bytes(G, B, n)


def csa2_topk_merge(keys, ids, src_off, k, out, ws, lo=None, hi=None, out_local=None, stream=None):
    """keys / ids [G, B, n] from the shards -> out [B, k] (and out_local [B, k] for [lo, hi))."""
    fn = "csa2_topk_merge"
    G, B, n = ids.shape
    wp, wn = _ws(ws)
    rc = lib().csa2_topk_merge(_arg(fn, "keys", keys, "i32", G * B * n), _arg(fn, "ids", ids, "i32", G * B * n),
                               _arg(fn, "src_off", src_off, "i64", G * B), G, B, n, k, _arg(fn, "lo", lo, "i64", B),
                               _arg(fn, "hi", hi, "i64", B), _arg(fn, "out", out, "i32", B * k),
                               _arg(fn, "out_local", out_local, "i32", B * k), wp, wn, _stream(stream))
    _check(rc, fn)


def csa2_attn_combine(out_parts, lse_parts, out, lse=None, stream=None):
    """out_parts [G, B, 16, 512], lse_parts [G, B, 16] -> out [B, 16, 512], lse [B, 16]."""
    fn = "csa2_attn_combine"
    G, B = lse_parts.shape[0], lse_parts.shape[1]
    rc = lib().csa2_attn_combine(_arg(fn, "out_parts", out_parts, "f32", G * B * Q_HEADS * MAIN_DIM),
                                 _arg(fn, "lse_parts", lse_parts, "f32", G * B * Q_HEADS), G, B,
                                 *_attn_out(fn, B, out, lse), _stream(stream))
    _check(rc, fn)


def csa2_index_prefill_workspace_bytes(T, n_entries, pool_blocks, k):
    return lib().csa2_index_prefill_workspace_bytes(T, n_entries, pool_blocks, k)


def csa2_index_prefill(idx_k, q_codes, q_scales, w, q_pos, row0, n_entries, ratio, pool_blocks, k, pool_out,
                       topk_out, ws, stream=None):
    fn = "csa2_index_prefill"
    T = q_pos.shape[0]
    wp, wn = _ws(ws)
    rc = lib().csa2_index_prefill(idx_k, *_queries(fn, T, q_codes, q_scales, w), _arg(fn, "q_pos", q_pos, "i32", T), T,
                                  row0, n_entries, ratio, pool_blocks, k,
                                  _arg(fn, "pool_out", pool_out, "i32", T * pool_blocks),
                                  _arg(fn, "topk_out", topk_out, "i32", T * k), wp, wn, _stream(stream))
    _check(rc, fn)


def csa2_sparse_attn_prefill_workspace_bytes(T, k):
    return lib().csa2_sparse_attn_prefill_workspace_bytes(T, k)


def csa2_sparse_attn_prefill(q, q_pos, main_kv, row0, n_entries, ratio, topk, raw_win, win_scale, sm_scale, out, ws,
                             lse=None, stream=None):
    fn = "csa2_sparse_attn_prefill"
    T, k = topk.shape
    wp, wn = _ws(ws)
    rc = lib().csa2_sparse_attn_prefill(_arg(fn, "q", q, "bf16", T * Q_HEADS * MAIN_DIM),
                                        _arg(fn, "q_pos", q_pos, "i32", T), T, main_kv, row0, n_entries, ratio,
                                        _arg(fn, "topk", topk, "i32", T * k), k,
                                        _arg(fn, "raw_win", raw_win, "u8", raw_win.shape[0] * MAIN_DIM),
                                        raw_win.shape[0], float(win_scale), float(sm_scale), *_attn_out(fn, T, out, lse),
                                        wp, wn, _stream(stream))
    _check(rc, fn)


def noalloc_setup(stream=None):
    """The B = 0 call of csa2_sparse_attn_decode_noalloc: loads the library's
    scratch array and the attention kernel on the current device (the one
    time that call may allocate device memory) and launches nothing."""
    fn = "csa2_sparse_attn_decode_noalloc"
    rc = lib().csa2_sparse_attn_decode_noalloc(None, MXFP4Cache(None, None, 0), None, None, None, 1, None, None, None,
                                               0.0, None, None, None, 0, _stream(stream))
    _check(rc, fn)


def csa2_sparse_attn_decode_noalloc(q, main_kv, seq_row_off, seq_len, topk, win, win_scale, win_len, sm_scale, out,
                                    lse=None, flags_out=None, stream=None):
    """csa2_sparse_attn_decode without a workspace (fixed library scratch; B <= 64, k <= 512).

    For callers that may not allocate device memory while they run.  All calls
    on one device share the scratch, so calls that overlap on the GPU race."""
    fn = "csa2_sparse_attn_decode_noalloc"
    B, k, qp, sl, tp, wi, wsc, wl, op, lp = _decode_args(fn, q, seq_len, topk, win, win_scale, win_len, out, lse)
    if B == 0:
        return noalloc_setup(stream)
    rc = lib().csa2_sparse_attn_decode_noalloc(qp, main_kv, _row_off(fn, seq_row_off, B), sl, tp, k, wi, wsc, wl,
                                               float(sm_scale), op, lp, _arg(fn, "flags_out", flags_out, "i32", 1), B,
                                               _stream(stream))
    _check(rc, fn)


# ----------------------------------------------------------------------------
# after a step: verification of drafts, attention weights, eviction
# ----------------------------------------------------------------------------

# (absent from a torch built without CUDA, where no call gets that far)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_PROB_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _launch(fn, tensors, stream, *args):
    """Calls `fn` on the device of its tensors (which must be one device, not
    necessarily the current one); stream None is that device's current stream."""
    devices = {t.get_device() for t in tensors if t is not None}  # (-1: a host tensor)
    if len(devices) != 1:
        raise Csa2Error(-1, fn, f"tensors on devices {sorted(devices)}")
    dev = devices.pop()
    f = getattr(_lib or lib(), fn)
    if dev < 0:
        rc = f(*args, _stream(stream))
    else:
        # (the raw handle: torch.cuda.current_stream() builds a Stream object, 3.7 us)
        st = stream.cuda_stream if stream is not None else _raw_stream(dev)
        if dev != _current_device():
            with torch.cuda.device(dev):
                rc = f(*args, st)
        else:
            rc = f(*args, st)
    if rc != 0:
        _check(rc, fn)


def _cache_tensors(*caches):
    out = []
    for c in caches:
        out.extend(getattr(c, "_keep", ()) if c is not None else ())
    return out


def _prob_rows(fn, name, t, Q, V):
    """(pointer, type code, row stride) of Q rows of V probabilities: fp32, bf16 or fp16, each row
    contiguous, rows any distance apart."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype not in _PROB_TYPES:
        raise Csa2Error(-1, fn, f"{name}: a 2-d fp32, bf16 or fp16 tensor expected")
    rows, cols = t.shape
    if rows < Q or cols != V:
        raise Csa2Error(-1, fn, f"{name}: [{Q}, {V}] expected, got [{rows}, {cols}]")
    if t.is_contiguous():
        return _arg(fn, name, t, "prob"), _PROB_TYPES[t.dtype], V
    if V > 1 and t.stride(1) != 1:
        raise Csa2Error(-1, fn, f"{name}: the probabilities of a row must be contiguous")
    return _arg(fn, name, t[0], "prob"), _PROB_TYPES[t.dtype], t.stride(0)


def _rows_out(fn, name, t, kind, rows, cols):
    """_arg of an output of `rows` rows of `cols` elements, one behind the other: a flat tensor, or one whose rows have
    exactly that many."""
    if isinstance(t, _Tensor) and t.dim() != 1 and (t.dim() != 2 or t.shape[1] != cols):
        raise Csa2Error(-1, fn, f"{name}: [{rows}, {cols}] expected, got {list(t.shape)}")
    return _arg(fn, name, t, kind, rows * cols)


def csa2_verify_drafts_workspace_bytes(B, V):
    return lib().csa2_verify_drafts_workspace_bytes(B, V)


def csa2_verify_drafts(target, tokens, q_off, u, r, n_accept, next_tok, ws, draft=None, out_tokens=None,
                       seq_len_in=None, seq_len_out=None, stream=None):
    """target / draft: [Q, V] probabilities (fp32, bf16 or fp16; rows may be strided); tokens [Q]; q_off [B+1];
    u [Q], r [B] random numbers; n_accept, next_tok [B]; out_tokens [B, M] or None."""
    fn = "csa2_verify_drafts"
    B, Q = n_accept.shape[0], tokens.shape[0]
    if not isinstance(target, torch.Tensor) or target.dim() != 2:
        raise Csa2Error(-1, fn, "target: a 2-d fp32, bf16 or fp16 tensor expected")
    V = target.shape[1]
    tp, tt, ts = _prob_rows(fn, "target", target, Q, V)
    dp, dt, ds = _prob_rows(fn, "draft", draft, Q, V) if draft is not None else (None, 0, 0)
    M = 0
    if out_tokens is not None:
        if out_tokens.dim() != 2 or out_tokens.shape[0] < B:
            raise Csa2Error(-1, fn, f"out_tokens: [{B}, M] expected, got {list(out_tokens.shape)}")
        M = out_tokens.shape[1]
    wp, wn = _ws(ws)
    _launch(fn, (target, draft, tokens, q_off, u, r, seq_len_in, seq_len_out, n_accept, next_tok, out_tokens, ws),
            stream, tp, tt, ts, dp, dt, ds, _arg(fn, "tokens", tokens, "i32", Q), _arg(fn, "q_off", q_off, "i32", B + 1),
            _arg(fn, "u", u, "f32", Q), _arg(fn, "r", r, "f32", B), B, Q, V,
            _arg(fn, "seq_len_in", seq_len_in, "i32", B), _arg(fn, "seq_len_out", seq_len_out, "i32", B),
            _arg(fn, "n_accept", n_accept, "i32", B), _arg(fn, "next_tok", next_tok, "i32", B),
            _arg(fn, "out_tokens", out_tokens, "i32", B * M), M, wp, wn)


def csa2_attn_weights_workspace_bytes(B, Q, k):
    return lib().csa2_attn_weights_workspace_bytes(B, Q, k)


def csa2_attn_weights(q, main_kv, seq_row_off, seq_len, topk, lse, sm_scale, acc, ws, q_off=None, n_accept=None,
                      weights=None, stream=None):
    """acc [main_kv.rows] fp32 += the attention weight of the selected entries; weights [Q, k] or None receives
    the weights.  seq_row_off: [B] offsets or a PageTable; q_off / n_accept as in a verification step."""
    paged = isinstance(seq_row_off, PageTable)
    fn = "csa2_attn_weights_paged" if paged else "csa2_attn_weights"
    Q, k = topk.shape
    B = seq_len.shape[0]
    wp, wn = _ws(ws)
    qp = _arg(fn, "q", q, "bf16", Q * Q_HEADS * MAIN_DIM)
    rest = (_arg(fn, "seq_len", seq_len, "i32", B), _arg(fn, "q_off", q_off, "i32", B + 1),
            _arg(fn, "n_accept", n_accept, "i32", B), _arg(fn, "topk", topk, "i32", Q * k), k,
            _arg(fn, "lse", lse, "f32", Q * Q_HEADS), float(sm_scale), _arg(fn, "acc", acc, "f32", main_kv.rows),
            _rows_out(fn, "weights", weights, "f32", Q, k), B, Q, wp, wn)
    where = seq_row_off.pages if paged else seq_row_off
    tensors = (q, seq_len, q_off, n_accept, topk, lse, acc, weights, ws, where, *_cache_tensors(main_kv))
    if paged:
        pt = seq_row_off
        _launch(fn, tensors, stream, qp, main_kv, _pages(fn, pt, B), pt.page_rows, pt.max_pages, *rest)
    else:
        _launch(fn, tensors, stream, qp, main_kv, _row_off(fn, seq_row_off, B), *rest)


def csa2_acc_clear_workspace_bytes(B):
    return lib().csa2_acc_clear_workspace_bytes(B)


def csa2_acc_clear(acc, seq_row_off, len_from, len_to, ws, rows=None, stream=None):
    """acc of positions len_from[b] .. len_to[b]-1 of every sequence = 0.  seq_row_off: [B] offsets or a PageTable;
    rows: capacity of the caches (None: acc has one element per row)."""
    paged = isinstance(seq_row_off, PageTable)
    fn = "csa2_acc_clear_paged" if paged else "csa2_acc_clear"
    B = len_to.shape[0]
    rows = acc.numel() if rows is None else int(rows)
    wp, wn = _ws(ws)
    ap = _arg(fn, "acc", acc, "f32", rows)
    rest = (_arg(fn, "len_from", len_from, "i32", B), _arg(fn, "len_to", len_to, "i32", B), B, wp, wn)
    tensors = (acc, seq_row_off.pages if paged else seq_row_off, len_from, len_to, ws)
    if paged:
        _launch(fn, tensors, stream, ap, rows, _pages(fn, seq_row_off, B), seq_row_off.page_rows, seq_row_off.max_pages,
                *rest)
    else:
        _launch(fn, tensors, stream, ap, rows, _row_off(fn, seq_row_off, B), *rest)


def csa2_cache_evict_workspace_bytes(B, max_len):
    return lib().csa2_cache_evict_workspace_bytes(B, max_len)


def csa2_cache_evict(main_src, idx_src, acc_src, src, seq_len, keep, max_len, max_keep, main_dst, idx_dst, acc_dst,
                     dst, kept, seq_len_out, ws, first=0, last=0, stream=None):
    """Keeps keep[b] entries of every sequence (the first `first`, the last `last`, the best others by acc_src) and
    copies their rows to the destination.  src / dst: [B] row offsets, or a PageTable each; idx_src / idx_dst may
    both be None; kept [B, max_keep] receives the source positions, seq_len_out [B] their number."""
    paged = isinstance(src, PageTable)
    fn = "csa2_cache_evict_paged" if paged else "csa2_cache_evict"
    if paged != isinstance(dst, PageTable) or (paged and src.page_rows != dst.page_rows):
        raise Csa2Error(-1, fn, "source and destination must both be row offsets, or page tables of one page size")
    if (idx_src is None) != (idx_dst is None):
        raise Csa2Error(-1, fn, "idx_src and idx_dst go together")
    none = MXFP4Cache(None, None, 0)
    i_src, i_dst = (none, none) if idx_src is None else (idx_src, idx_dst)
    B = seq_len.shape[0]
    wp, wn = _ws(ws)
    # an accumulator per row that the caches hold
    n_src = main_src.rows if idx_src is None else min(main_src.rows, idx_src.rows)
    n_dst = main_dst.rows if idx_dst is None else min(main_dst.rows, idx_dst.rows)
    ac, sl, kp = (_arg(fn, "acc_src", acc_src, "f32", n_src), _arg(fn, "seq_len", seq_len, "i32", B),
                  _arg(fn, "keep", keep, "i32", B))
    ad, ko, so = (_arg(fn, "acc_dst", acc_dst, "f32", n_dst), _rows_out(fn, "kept", kept, "i32", B, max_keep),
                  _arg(fn, "seq_len_out", seq_len_out, "i32", B))
    tensors = (acc_src, seq_len, keep, acc_dst, kept, seq_len_out, ws, src.pages if paged else src,
               dst.pages if paged else dst, *_cache_tensors(main_src, idx_src, main_dst, idx_dst))
    tail = (ko, so, B, int(max_len), int(max_keep), int(first), int(last), wp, wn)
    if paged:
        _launch(fn, tensors, stream, main_src, i_src, ac, _pages(fn, src, B), src.max_pages, sl, kp, main_dst, i_dst,
                ad, _pages(fn, dst, B), dst.max_pages, src.page_rows, *tail)
    else:
        _launch(fn, tensors, stream, main_src, i_src, ac, _row_off(fn, src, B), sl, kp, main_dst, i_dst, ad,
                _row_off(fn, dst, B), *tail)


def csa2_cache_evict_layers(main_src, idx_src, acc_src, src, seq_len, keep, max_len, max_keep, main_dst, idx_dst,
                            acc_dst, dst, kept, seq_len_out, ws, first=0, last=0, stream=None):
    """csa2_cache_evict of several layers, which keep the same entries: the best by the sum of their accumulators.
    main_src, idx_src, acc_src, main_dst, idx_dst, acc_dst: one per layer (idx_src / idx_dst: lists, or None)."""
    paged = isinstance(src, PageTable)
    fn = "csa2_cache_evict_layers_paged" if paged else "csa2_cache_evict_layers"
    if paged != isinstance(dst, PageTable) or (paged and src.page_rows != dst.page_rows):
        raise Csa2Error(-1, fn, "source and destination must both be row offsets, or page tables of one page size")
    n = len(main_src)
    idx_src, idx_dst = (x if x is not None else [None] * n for x in (idx_src, idx_dst))
    if n < 1 or any(len(x) != n for x in (idx_src, acc_src, main_dst, idx_dst, acc_dst)):
        raise Csa2Error(-1, fn, "one cache and one accumulator per layer on each side expected")
    if any((a is None) != (b is None) for a, b in zip(idx_src, idx_dst)):
        raise Csa2Error(-1, fn, "idx_src and idx_dst go together")
    B = seq_len.shape[0]
    wp, wn = _ws(ws)
    # an accumulator per row that all caches of a side hold
    n_src = min(c.rows for c in (*main_src, *idx_src) if c is not None)
    n_dst = min(c.rows for c in (*main_dst, *idx_dst) if c is not None)
    none = MXFP4Cache(None, None, 0)
    caches = lambda cs: (MXFP4Cache * n)(*(none if c is None else c for c in cs))  # noqa: E731
    accs = lambda name, ts, rows: (C.c_void_p * n)(*(_arg(fn, name, t, "f32", rows) for t in ts))  # noqa: E731
    head = (n, caches(main_src), caches(idx_src), accs("acc_src", acc_src, n_src))
    there = (caches(main_dst), caches(idx_dst), accs("acc_dst", acc_dst, n_dst))
    sl, kp = _arg(fn, "seq_len", seq_len, "i32", B), _arg(fn, "keep", keep, "i32", B)
    tail = (_rows_out(fn, "kept", kept, "i32", B, max_keep), _arg(fn, "seq_len_out", seq_len_out, "i32", B), B,
            int(max_len), int(max_keep), int(first), int(last), wp, wn)
    tensors = (*acc_src, seq_len, keep, *acc_dst, kept, seq_len_out, ws, src.pages if paged else src,
               dst.pages if paged else dst, *_cache_tensors(*main_src, *idx_src, *main_dst, *idx_dst))
    if paged:
        _launch(fn, tensors, stream, *head, _pages(fn, src, B), src.max_pages, sl, kp, *there, _pages(fn, dst, B),
                dst.max_pages, src.page_rows, *tail)
    else:
        _launch(fn, tensors, stream, *head, _row_off(fn, src, B), sl, kp, *there, _row_off(fn, dst, B), *tail)
