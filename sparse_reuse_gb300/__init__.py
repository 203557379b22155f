"""Python binding of libspecfold (the C ABI in include/specfold.h).

Argument marshalling only: every step of the verification pass runs in the
library's CUDA kernels.  The in-tree libspecfold.so is loaded on the first
call into the binding; if it is missing that call raises ImportError (build it with
``python -c "import __graft_entry__ as g; g.build()"`` or
``python sparse_reuse_gb300/build.py``).  PyTorch provides device memory and
streams only.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import List, Optional, Sequence

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libspecfold.so")

SF_OK, SF_ERR_INVALID_ARG, SF_ERR_SHAPE, SF_ERR_TREE, SF_ERR_UNSUPPORTED, SF_ERR_OOM, SF_ERR_CUDA, \
    SF_ERR_DEVICE_ASSERT = range(8)
SF_F32, SF_BF16 = 0, 1
FAMILIES = ["gate", "norm", "gemm_qkv", "attn_prefix", "attn_block", "gemm_o", "gemm_gateup", "gemm_down",
            "residual", "aux", "attn_correct"]
SF_ATTN_DIRECT, SF_ATTN_CORRECT, SF_ATTN_DIRECT_SPLIT = 0, 1, 2
SF_K_COUNT = len(FAMILIES)

# every symbol include/specfold.h declares
EXPORTS = ["sf_create", "sf_verify", "sf_set_debug", "sf_set_rho_dump", "sf_set_attention_mode", "sf_sync_status", "sf_destroy", "sf_status_str",
           "sf_last_error", "sf_get_stats", "sf_set_graphs", "sf_timing_begin", "sf_timing_read", "sf_timing_list",
           "sfk_gemm_bf16", "sfk_gate_noalloc", "sf_inject_stall",
           "sf_head_create", "sf_head_verify", "sf_head_last_error", "sf_head_destroy",
           "sf_cache_create", "sf_cache_append", "sf_cache_attend", "sf_cache_evict", "sf_cache_sync_status",
           "sf_cache_last_error", "sf_cache_destroy", "sf_cache_create_with", "sf_cache_reposition",
           "sf_cache_attend_rows", "sf_cache_attend_shared", "sf_cache_inject_stall"]
SF_ROTARY_HALVES, SF_ROTARY_NEIGHBOURS = 0, 1


class SfShapes(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("d_model", ctypes.c_int), ("n_q_heads", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("d_ffn", ctypes.c_int),
                ("dtype", ctypes.c_int), ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float),
                ("block_len", ctypes.c_int), ("max_requests", ctypes.c_int), ("max_branches", ctypes.c_int),
                ("max_prefix", ctypes.c_int)]


class SfLayerWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "w_gate", "w_up", "w_down")]


class SfHeadShapes(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int), ("vocab", ctypes.c_int), ("dtype", ctypes.c_int),
                ("rms_eps", ctypes.c_float), ("max_rows", ctypes.c_int)]


class SfCacheShapes(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("dtype", ctypes.c_int), ("page_size", ctypes.c_int), ("max_seqs", ctypes.c_int),
                ("max_len", ctypes.c_int), ("max_pos", ctypes.c_int), ("rms_eps", ctypes.c_float),
                ("rope_theta", ctypes.c_float), ("track_weights", ctypes.c_int)]


class SfCacheOptions(ctypes.Structure):
    _fields_ = [("rotary_layout", ctypes.c_int), ("rotary_dim", ctypes.c_int),
                ("inv_freq", ctypes.POINTER(ctypes.c_double)), ("rotary_magnitude", ctypes.c_double),
                ("max_rows", ctypes.c_int)]


class SfStats(ctypes.Structure):
    _fields_ = [("passes", ctypes.c_uint64), ("kernel_launches", ctypes.c_uint64),
                ("graph_replays", ctypes.c_uint64), ("family_launches", ctypes.c_uint64 * SF_K_COUNT)]


class SpecFoldError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libspecfold.so is not built ({LIB_PATH}); run sparse_reuse_gb300/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32p, c_int, c_float = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32), ctypes.c_int, ctypes.c_float
    lib.sf_create.argtypes = [ctypes.POINTER(SfShapes), ctypes.POINTER(SfLayerWeights), ctypes.POINTER(vp)]
    lib.sf_verify.argtypes = [vp, vp, vp, i32p, vp, vp, c_int, c_int, c_int, c_float, vp, vp, vp, vp]
    lib.sf_set_debug.argtypes = [vp, vp, vp]
    lib.sf_set_rho_dump.argtypes = [vp, vp]
    lib.sf_set_attention_mode.argtypes = [vp, c_int]
    lib.sf_sync_status.argtypes = [vp, vp]
    lib.sf_inject_stall.argtypes = [vp, c_int]
    lib.sf_destroy.argtypes = [vp]
    lib.sf_status_str.argtypes = [c_int]
    lib.sf_status_str.restype = ctypes.c_char_p
    lib.sf_last_error.argtypes = [vp]
    lib.sf_last_error.restype = ctypes.c_char_p
    lib.sf_get_stats.argtypes = [vp, ctypes.POINTER(SfStats)]
    lib.sf_set_graphs.argtypes = [vp, c_int]
    lib.sf_timing_begin.argtypes = [vp, ctypes.c_uint]
    lib.sf_timing_read.argtypes = [vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)]
    lib.sf_timing_list.argtypes = [vp, c_int, ctypes.POINTER(ctypes.c_double), c_int, ctypes.POINTER(c_int)]
    lib.sfk_gemm_bf16.argtypes = [vp, vp, c_int, vp, c_int, c_int, vp, c_int, vp, c_int, c_int, vp]
    lib.sfk_gate_noalloc.argtypes = [vp, vp, c_int, i32p, c_int, c_int, c_int, c_int, c_float, vp, vp, vp, vp, vp,
                                     vp]
    lib.sf_head_create.argtypes = [ctypes.POINTER(SfHeadShapes), vp, vp, ctypes.POINTER(vp)]
    lib.sf_head_verify.argtypes = [vp, vp, vp, vp, i32p, c_int, c_int, c_int, vp, vp, vp]
    lib.sf_head_last_error.argtypes = [vp]
    lib.sf_head_last_error.restype = ctypes.c_char_p
    lib.sf_head_destroy.argtypes = [vp]
    i64 = ctypes.c_int64
    lib.sf_cache_create.argtypes = [ctypes.POINTER(SfCacheShapes), ctypes.POINTER(vp)]
    lib.sf_cache_append.argtypes = [vp, vp, vp, i64, c_int, vp, vp, vp, vp, vp, vp, c_int, c_int, i64, vp, vp, i64,
                                    vp, i64]
    lib.sf_cache_attend.argtypes = [vp, vp, vp, i64, vp, vp, i64, vp, c_int, c_int, i64, vp, c_float, vp, i64, vp, vp,
                                    i64]
    lib.sf_cache_evict.argtypes = [vp, vp, vp, vp, i64, vp, c_int, c_int, i64, vp, vp, i64, c_int, c_int, c_int, vp,
                                   vp, i64, vp, c_int, i64, vp, vp, vp]
    lib.sf_cache_create_with.argtypes = [ctypes.POINTER(SfCacheShapes), ctypes.POINTER(SfCacheOptions),
                                         ctypes.POINTER(vp)]
    lib.sf_cache_reposition.argtypes = [vp, vp, vp, i64, vp, c_int, c_int, i64, vp, vp, vp, i64]
    lib.sf_cache_attend_rows.argtypes = [vp, vp, vp, i64, c_int, vp, vp, i64, vp, c_int, c_int, i64, vp, vp, c_float,
                                         vp, i64, vp]
    lib.sf_cache_attend_shared.argtypes = [vp, vp, vp, i64, vp, vp, i64, vp, c_int, c_int, i64, vp, vp, c_int, c_int,
                                           i64, vp, vp, c_float, vp, i64, vp]
    lib.sf_cache_inject_stall.argtypes = [vp, c_int]
    lib.sf_cache_sync_status.argtypes = [vp, vp]
    lib.sf_cache_last_error.argtypes = [vp]
    lib.sf_cache_last_error.restype = ctypes.c_char_p
    lib.sf_cache_destroy.argtypes = [vp]
    for name in EXPORTS:
        fn = getattr(lib, name)
        if name not in ("sf_status_str", "sf_last_error", "sf_head_last_error", "sf_cache_last_error"):
            fn.restype = c_int
    return lib


class _LazyLib:
    """Loads libspecfold.so on first use so that the build module inside this
    package can be imported on a machine where it is not built yet; any call
    into the binding without the library raises ImportError."""

    _cdll = None

    def __getattr__(self, name):
        if _LazyLib._cdll is None:
            _LazyLib._cdll = _load()
        return getattr(_LazyLib._cdll, name)


lib = _LazyLib()


def _marshal():
    """The compiled marshalling of the paged-cache calls (csrc/sf_torch.cpp); ImportError if it is not built."""
    import torch  # noqa: F401  (the module links against torch's libraries)
    if not os.path.exists(os.path.join(_PKG, "_sf_torch.so")):
        raise ImportError("_sf_torch.so is not built; run sparse_reuse_gb300/build.py with torch and Python's headers "
                          "installed")
    from . import _sf_torch
    return _sf_torch


def _check(st: int, ctx=None, what: str = "", head=None, cache=None):
    if st != SF_OK:
        msg = lib.sf_status_str(st).decode()
        if ctx or head or cache:
            extra = (lib.sf_last_error(ctx) if ctx else lib.sf_head_last_error(head) if head else
                     lib.sf_cache_last_error(cache)).decode()
            if extra:
                msg += f": {extra}"
        raise SpecFoldError(st, f"{what}: {msg}" if what else msg)


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _stream_handle(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    h = int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
    return h or None


def _empty(stream, device, shape, dtype):
    """A new output of a call on `stream` (a torch stream, its handle, or None for the current one), in memory of
    that stream's own pool: what was there before is done with in stream order when the call writes it, whatever the
    current stream still has to do.  It counts as used by the current stream too, so that a reader there need not
    record it."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.cuda_stream == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


# ---------------------------------------------------------------- C-ABI mirrors

def sf_create(shapes: SfShapes, layers: Sequence[SfLayerWeights]) -> int:
    arr = (SfLayerWeights * len(layers))(*layers)
    ctx = ctypes.c_void_p()
    _check(lib.sf_create(ctypes.byref(shapes), arr, ctypes.byref(ctx)), None, "sf_create")
    return ctx.value


def sf_verify(ctx, stream, hidden_in, parent, prefix_k, prefix_v, R, B, P, delta, hidden_out,
              fold_mask=None, src=None, rc_count=None) -> None:
    par = np.ascontiguousarray(parent, dtype=np.int32)
    _check(lib.sf_verify(ctx, stream, hidden_in, par.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), prefix_k,
                         prefix_v, int(R), int(B), int(P), float(delta), hidden_out, fold_mask, src, rc_count),
           ctx, "sf_verify")


def sf_set_debug(ctx, layer_hidden, rc_rows) -> None:
    _check(lib.sf_set_debug(ctx, layer_hidden, rc_rows), ctx, "sf_set_debug")


def sf_set_attention_mode(ctx, mode: int) -> None:
    _check(lib.sf_set_attention_mode(ctx, int(mode)), ctx, "sf_set_attention_mode")


def sf_set_rho_dump(ctx, rho) -> None:
    _check(lib.sf_set_rho_dump(ctx, rho), ctx, "sf_set_rho_dump")


def sf_sync_status(ctx, stream) -> None:
    _check(lib.sf_sync_status(ctx, stream), ctx, "sf_sync_status")


def sf_inject_stall(ctx, on: bool) -> None:
    _check(lib.sf_inject_stall(ctx, int(bool(on))), ctx, "sf_inject_stall")


def sf_destroy(ctx) -> None:
    _check(lib.sf_destroy(ctx), None, "sf_destroy")


def sf_get_stats(ctx) -> dict:
    s = SfStats()
    _check(lib.sf_get_stats(ctx, ctypes.byref(s)), ctx, "sf_get_stats")
    return {"passes": s.passes, "kernel_launches": s.kernel_launches, "graph_replays": s.graph_replays,
            "family_launches": {FAMILIES[i]: s.family_launches[i] for i in range(SF_K_COUNT)}}


def sf_set_graphs(ctx, on: bool) -> None:
    _check(lib.sf_set_graphs(ctx, int(bool(on))), ctx, "sf_set_graphs")


def sf_timing_begin(ctx, families: Sequence[str]) -> None:
    mask = 0
    for f in families:
        mask |= 1 << FAMILIES.index(f)
    _check(lib.sf_timing_begin(ctx, mask), ctx, "sf_timing_begin")


def sf_timing_read(ctx) -> dict:
    ms = (ctypes.c_double * SF_K_COUNT)()
    n = (ctypes.c_int64 * SF_K_COUNT)()
    _check(lib.sf_timing_read(ctx, ms, n), ctx, "sf_timing_read")
    return {FAMILIES[i]: (ms[i], n[i]) for i in range(SF_K_COUNT) if n[i] > 0}


def sf_timing_list(ctx, family: str) -> List[float]:
    """Durations (ms) of the timed launches of one family, in launch order."""
    n = ctypes.c_int(0)
    _check(lib.sf_timing_list(ctx, FAMILIES.index(family), None, 0, ctypes.byref(n)), ctx, "sf_timing_list")
    buf = (ctypes.c_double * max(1, n.value))()
    _check(lib.sf_timing_list(ctx, FAMILIES.index(family), buf, n.value, ctypes.byref(n)), ctx, "sf_timing_list")
    return [buf[i] for i in range(n.value)]


def sfk_gemm_bf16(stream, X, rows_cap, W, M, K, count, dense_count, Y, ldy, splits, err=None) -> None:
    _check(lib.sfk_gemm_bf16(stream, X, int(rows_cap), W, int(M), int(K), count, int(dense_count), Y, int(ldy),
                             int(splits), err), None, "sfk_gemm_bf16")


def sfk_gate_noalloc(stream, hidden, dtype, parent, R, B, L, d, delta, H_out, fold, rc, rcslot, src,
                     rc_count) -> None:
    par = np.ascontiguousarray(parent, dtype=np.int32)
    _check(lib.sfk_gate_noalloc(stream, hidden, int(dtype), par.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                int(R), int(B), int(L), int(d), float(delta), H_out, fold, rc, rcslot, src,
                                rc_count), None, "sfk_gate_noalloc")


def sf_head_create(shapes: SfHeadShapes, final_norm, w_lm) -> int:
    h = ctypes.c_void_p()
    _check(lib.sf_head_create(ctypes.byref(shapes), final_norm, w_lm, ctypes.byref(h)), None, "sf_head_create")
    return h.value


def sf_head_verify(head, stream, hidden, tokens, parent, R, B, L, pred, accepted=None, chosen=None) -> None:
    par = np.ascontiguousarray(parent, dtype=np.int32)
    _check(lib.sf_head_verify(head, stream, hidden, tokens, par.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                              int(R), int(B), int(L), pred, accepted, chosen), None, "sf_head_verify", head=head)


def sf_head_destroy(head) -> None:
    _check(lib.sf_head_destroy(head), None, "sf_head_destroy")


def sf_cache_create(shapes: SfCacheShapes) -> int:
    c = ctypes.c_void_p()
    _check(lib.sf_cache_create(ctypes.byref(shapes), ctypes.byref(c)), None, "sf_cache_create")
    return c.value


def sf_cache_create_with(shapes: SfCacheShapes, options: SfCacheOptions) -> int:
    c = ctypes.c_void_p()
    _check(lib.sf_cache_create_with(ctypes.byref(shapes), ctypes.byref(options), ctypes.byref(c)), None,
           "sf_cache_create_with")
    return c.value


def sf_cache_reposition(cache, stream, k_pages, n_pages, page_table, S, table_cols, ld_table, lens, pos_from, pos_to,
                        ld_pos) -> None:
    _check(lib.sf_cache_reposition(cache, stream, k_pages, n_pages, page_table, S, table_cols, ld_table, lens,
                                   pos_from, pos_to, ld_pos), None, "sf_cache_reposition", cache=cache)


def sf_cache_attend_rows(cache, stream, q, ld_q, T, k_pages, v_pages, n_pages, page_table, S, table_cols, ld_table,
                         lens, starts, scale, out, ld_out, lse=None) -> None:
    _check(lib.sf_cache_attend_rows(cache, stream, q, ld_q, T, k_pages, v_pages, n_pages, page_table, S, table_cols,
                                    ld_table, lens, starts, scale, out, ld_out, lse),
           None, "sf_cache_attend_rows", cache=cache)


def sf_cache_attend_shared(cache, stream, q, ld_q, k_pages, v_pages, n_pages, page_table, S, table_cols, ld_table,
                           lens, prefix_table, G, prefix_cols, ld_prefix, prefix_lens, starts, scale, out, ld_out,
                           lse=None) -> None:
    _check(lib.sf_cache_attend_shared(cache, stream, q, ld_q, k_pages, v_pages, n_pages, page_table, S, table_cols,
                                      ld_table, lens, prefix_table, G, prefix_cols, ld_prefix, prefix_lens, starts,
                                      scale, out, ld_out, lse),
           None, "sf_cache_attend_shared", cache=cache)


def sf_cache_inject_stall(cache, signal: int) -> None:
    _check(lib.sf_cache_inject_stall(cache, signal), None, "sf_cache_inject_stall", cache=cache)


def sf_cache_append(cache, stream, qkv, ld_qkv, T, q_gain, k_gain, index, pos, seq, page_table, S, table_cols,
                    ld_table, k_pages, v_pages, n_pages, q_out, ld_q) -> None:
    _check(lib.sf_cache_append(cache, stream, qkv, ld_qkv, T, q_gain, k_gain, index, pos, seq, page_table, S,
                               table_cols, ld_table, k_pages, v_pages, n_pages, q_out, ld_q),
           None, "sf_cache_append", cache=cache)


def sf_cache_attend(cache, stream, q, ld_q, k_pages, v_pages, n_pages, page_table, S, table_cols, ld_table, lens,
                    scale, out, ld_out, weights_in=None, weights_out=None, ld_w=0) -> None:
    _check(lib.sf_cache_attend(cache, stream, q, ld_q, k_pages, v_pages, n_pages, page_table, S, table_cols, ld_table,
                               lens, scale, out, ld_out, weights_in, weights_out, ld_w),
           None, "sf_cache_attend", cache=cache)


def sf_cache_evict(cache, stream, k_pages, v_pages, n_pages, page_table, S, table_cols, ld_table, lens, weights, ld_w,
                   budget, n_first, n_recent, k_out, v_out, n_pages_out, table_out, table_out_cols, ld_table_out,
                   weights_out, lens_out, kept) -> None:
    _check(lib.sf_cache_evict(cache, stream, k_pages, v_pages, n_pages, page_table, S, table_cols, ld_table, lens,
                              weights, ld_w, budget, n_first, n_recent, k_out, v_out, n_pages_out, table_out,
                              table_out_cols, ld_table_out, weights_out, lens_out, kept),
           None, "sf_cache_evict", cache=cache)


def sf_cache_sync_status(cache, stream) -> None:
    _check(lib.sf_cache_sync_status(cache, stream), None, "sf_cache_sync_status", cache=cache)


def sf_cache_destroy(cache) -> None:
    _check(lib.sf_cache_destroy(cache), None, "sf_cache_destroy")


# ---------------------------------------------------------------- torch convenience

class SpecFold:
    """A context over torch tensors.

    weights: per layer a dict with attn_norm, wq, wk, wv, wo, ffn_norm,
    w_gate, w_up, w_down (CUDA tensors, [in, out] row-major; gains fp32)."""

    def __init__(self, *, n_layers, d_model, n_q_heads, n_kv_heads, head_dim, d_ffn, dtype, block_len,
                 max_requests, max_branches, max_prefix, weights: List[dict], rms_eps=1e-6,
                 rope_theta=10000.0):
        self.shapes = SfShapes(n_layers, d_model, n_q_heads, n_kv_heads, head_dim, d_ffn,
                               SF_BF16 if dtype in ("bf16", SF_BF16) else SF_F32, rms_eps, rope_theta,
                               block_len, max_requests, max_branches, max_prefix)
        layers = []
        for w in weights:
            for k, t in w.items():
                if not t.is_cuda or not t.is_contiguous():
                    raise ValueError(f"weight {k} must be a contiguous CUDA tensor")
            layers.append(SfLayerWeights(*[_ptr(w[n]) for n in
                                           ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "w_gate",
                                            "w_up", "w_down")]))
        self.ctx = sf_create(self.shapes, layers)

    def close(self):
        if getattr(self, "ctx", None):
            sf_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def verify(self, hidden, parent, prefix_k, prefix_v, delta, *, out=None, fold=None, src=None,
               rc_count=None, stream=None, want_masks=True):
        """Enqueue one pass; returns (out, fold_mask, src, rc_count) tensors.  Those that the call makes belong to
        `stream`, as if made under torch.cuda.stream(stream)."""
        import torch
        parent = np.asarray(parent, dtype=np.int32)
        R, Bp = parent.shape
        L, nl = self.shapes.block_len, self.shapes.n_layers
        P = 0 if prefix_k is None else int(prefix_k.shape[2])
        row = self.shapes.n_kv_heads * self.shapes.head_dim
        for name, t in (("prefix_k", prefix_k), ("prefix_v", prefix_v)):
            if t is not None and prefix_k is not None:  # without keys there is no prefix
                # the heads may be flattened; layers behind the context's own are not read, nor, of one layer, requests
                requests = int(t.shape[1])
                if t.shape[0] < nl or requests < R or (requests > R and nl > 1) or t.shape[2] != P \
                        or t.shape[3:].numel() != row:
                    raise ValueError(f"{name} must be [n_layers, R, P, n_kv_heads, head_dim] = "
                                     f"{[nl, R, P, self.shapes.n_kv_heads, self.shapes.head_dim]} (P: prefix_k's): got "
                                     f"{list(t.shape)}")
        for name, t in (("hidden", hidden), ("prefix_k", prefix_k), ("prefix_v", prefix_v), ("out", out),
                        ("fold", fold), ("src", src), ("rc_count", rc_count)):
            # the pass reads and writes dense arrays: a slice of a longer prefix, say, has other strides
            if t is not None and not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous: got strides {list(t.stride())}")
        dev = hidden.device
        if out is None:
            out = _empty(stream, dev, hidden.shape, hidden.dtype)
        if want_masks:
            if fold is None:
                fold = _empty(stream, dev, (nl, R, Bp, L), torch.uint8)
            if src is None:
                src = _empty(stream, dev, (nl, R, Bp, L), torch.int32)
            if rc_count is None:
                rc_count = _empty(stream, dev, (nl,), torch.int32)
        sf_verify(self.ctx, _stream_handle(stream), _ptr(hidden), parent, _ptr(prefix_k), _ptr(prefix_v), R,
                  Bp - 1, P, delta, _ptr(out), _ptr(fold), _ptr(src), _ptr(rc_count))
        return out, fold, src, rc_count

    def set_debug(self, layer_hidden=None, rc_rows=None):
        sf_set_debug(self.ctx, _ptr(layer_hidden), _ptr(rc_rows))

    def set_attention_mode(self, mode: int):
        sf_set_attention_mode(self.ctx, mode)

    def set_rho_dump(self, rho=None):
        sf_set_rho_dump(self.ctx, _ptr(rho))

    def sync(self, stream=None):
        sf_sync_status(self.ctx, _stream_handle(stream))

    def stats(self):
        return sf_get_stats(self.ctx)

    def set_graphs(self, on: bool):
        sf_set_graphs(self.ctx, on)


class Head:
    """The verification head over torch tensors: final RMSNorm, LM head,
    greedy tokens and draft acceptance of a pass output.

    final_norm: fp32 CUDA tensor [d]; w_lm: CUDA tensor [d, vocab] in the
    context dtype."""

    def __init__(self, *, d_model, vocab, dtype, max_rows, final_norm, w_lm, rms_eps=1e-6):
        for name, t in (("final_norm", final_norm), ("w_lm", w_lm)):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous CUDA tensor")
        self.shapes = SfHeadShapes(d_model, vocab, SF_BF16 if dtype in ("bf16", SF_BF16) else SF_F32, rms_eps,
                                   max_rows)
        self.head = sf_head_create(self.shapes, _ptr(final_norm), _ptr(w_lm))

    def close(self):
        if getattr(self, "head", None):
            sf_head_destroy(self.head)
            self.head = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def verify(self, hidden, tokens, parent, *, pred=None, accepted=None, chosen=None, stream=None):
        """Enqueue the head for one pass output; returns (pred, accepted, chosen).  Those that the call makes belong
        to `stream`, as if made under torch.cuda.stream(stream)."""
        import torch
        parent = np.asarray(parent, dtype=np.int32)
        R, Bp = parent.shape
        L = int(hidden.shape[2])
        dev = hidden.device
        if pred is None:
            pred = _empty(stream, dev, (R, Bp, L), torch.int32)
        if accepted is None:
            accepted = _empty(stream, dev, (R, Bp), torch.uint8)
        if chosen is None:
            chosen = _empty(stream, dev, (R,), torch.int32)
        sf_head_verify(self.head, _stream_handle(stream), _ptr(hidden), _ptr(tokens), parent, R, Bp - 1, L,
                       _ptr(pred), _ptr(accepted), _ptr(chosen))
        return pred, accepted, chosen


def rotary_frequencies(dim, theta=10000.0, *, scaling="none", factor=1.0, original_len=None, fast=32.0, slow=1.0,
                       low=1.0, high=4.0):
    """Frequencies of the dim / 2 rotated pairs, scaled for contexts `factor` times longer than the original_len
    positions that a model was made for, and the magnitude that goes with them: PagedCache's inv_freq and
    rotary_magnitude.  With f_j = theta^(-2j/dim):

      "none"    f_j
      "linear"  f_j / factor
      "ntk"     f_j of theta * factor^(dim / (dim - 2)): the slowest pair is stretched by factor, the fastest stays
      "yarn"    f_j / factor * g + f_j * (1 - g), where g rises from 0 to 1 over the pairs j from floor(j(fast)) to
                ceil(j(slow)), kept within 0 .. dim - 1, and j(r) = dim ln(original_len / (2 pi r)) / (2 ln theta) is
                the pair that turns r times in original_len; magnitude 0.1 ln(factor) + 1 (1 for a factor up to 1)
      "bands"   the same with g = 1 for pairs that turn up to `low` times in original_len, 0 from `high` times on, and
                linear in the turns between; magnitude 1

    Returns (tuple of dim / 2 floats, magnitude)."""
    if dim < 2 or dim % 2:
        raise ValueError(f"dim must be even and positive: got {dim}")
    if not (math.isfinite(theta) and theta > 0) or not (math.isfinite(factor) and factor > 0):
        raise ValueError(f"theta and factor must be positive: got {theta}, {factor}")
    if scaling in ("yarn", "bands") and not (original_len and original_len > 0):
        raise ValueError(f"{scaling} needs original_len")
    if scaling == "ntk":
        if dim == 2:
            raise ValueError("ntk needs more than one pair")
        theta *= factor ** (dim / (dim - 2))
    freq = [theta ** (-2.0 * j / dim) for j in range(dim // 2)]
    magnitude = 1.0
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "yarn":
        if not 0 < slow < fast or theta == 1:
            raise ValueError(f"yarn needs 0 < slow < fast and a theta other than 1: got {slow}, {fast}, {theta}")
        a, b = (dim * math.log(original_len / (2 * math.pi * r)) / (2 * math.log(theta)) for r in (fast, slow))
        a, b = max(math.floor(a), 0), min(math.ceil(b), dim - 1)
        mix = [min(max((j - a) / max(b - a, 0.001), 0.0), 1.0) for j in range(dim // 2)]
        freq = [f / factor * g + f * (1 - g) for f, g in zip(freq, mix)]
        magnitude = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling == "bands":
        if not 0 < low < high:
            raise ValueError(f"bands need 0 < low < high: got {low}, {high}")
        mix = [min(max((original_len * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for f in freq]
        freq = [f / factor * (1 - g) + f * g for f, g in zip(freq, mix)]
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"scaling must be 'none', 'linear', 'ntk', 'yarn' or 'bands': got {scaling!r}")
    return tuple(freq), magnitude


class PagedCache:
    """Operators on a paged key-value cache over torch tensors (include/specfold_cache.h).

    Keys and values live in pools [n_pages, page_size, n_kv_heads, head_dim]
    that the caller owns, one pair per layer; table is int32 [S, columns],
    lens int32 [S].  A layer's prefix buffer of SpecFold.verify, viewed as
    [R * P / page_size, page_size, n_kv_heads, head_dim], is such a pool, so
    that append can write the prefix of a pass; what evict leaves keeps its
    keys' original positions, until reposition turns them to new ones.
    Rotation: the first rotary_dim dimensions of a head (default: all), in
    pairs (j, j + rotary_dim / 2), or (2j, 2j + 1) with
    rotary_layout="interleaved"; inv_freq and rotary_magnitude as
    rotary_frequencies returns them (default: rope_theta^(-2j / rotary_dim),
    1).  attend_rows and attend_shared take up to max_rows rows a call.  attend
    and evict plan for the longest sequence that the table's columns could hold: pass
    table[:, :columns in use] where the sequences are far shorter.
    Tensors must be on the object's device, of the documented type and shape
    with contiguous rows (ValueError otherwise).  Work runs on `stream` (a
    torch stream or its handle; default: the current one of the device); the
    caller orders the tensors it passes with that stream, and waits for it
    before another stream reads the results.  Outputs that a call makes belong
    to `stream`, as if made under torch.cuda.stream(stream)."""

    def __init__(self, *, n_q_heads, n_kv_heads, head_dim, dtype, page_size, max_seqs, max_len, max_pos=None,
                 rms_eps=1e-6, rope_theta=10000.0, track_weights=False, rotary_dim=None, rotary_layout="half",
                 inv_freq=None, rotary_magnitude=1.0, max_rows=0):
        import torch
        if rotary_layout not in ("half", "interleaved"):
            raise ValueError(f"rotary_layout must be 'half' or 'interleaved': got {rotary_layout!r}")
        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        if rotary_dim < 1 and head_dim > 0 or not rotary_magnitude > 0:  # the library's 0 is its default
            raise ValueError(f"rotary_dim and rotary_magnitude must be positive: got {rotary_dim}, {rotary_magnitude}")
        if inv_freq is not None:
            inv_freq = [float(f) for f in inv_freq]
            if len(inv_freq) != rotary_dim // 2:
                raise ValueError(f"inv_freq must hold rotary_dim / 2 = {rotary_dim // 2} numbers: got {len(inv_freq)}")
            inv_freq = (ctypes.c_double * len(inv_freq))(*inv_freq)
        if dtype not in ("bf16", "f32", SF_BF16, SF_F32):
            raise ValueError(f"dtype must be 'bf16' or 'f32': got {dtype!r}")
        bf16 = dtype in ("bf16", SF_BF16)
        self.shapes = SfCacheShapes(n_q_heads, n_kv_heads, head_dim, SF_BF16 if bf16 else SF_F32, page_size,
                                    max_seqs, max_len, max_len if max_pos is None else max_pos, rms_eps, rope_theta,
                                    int(bool(track_weights)))
        self.dtype = torch.bfloat16 if bf16 else torch.float32
        self.cache = sf_cache_create_with(self.shapes, SfCacheOptions(
            SF_ROTARY_NEIGHBOURS if rotary_layout == "interleaved" else SF_ROTARY_HALVES, rotary_dim, inv_freq,
            rotary_magnitude, max_rows))
        self.device = torch.device("cuda", torch.cuda.current_device())
        self._bind(self.cache, self.device.index)

    def _bind(self, cache, device):
        s = self.shapes
        self._call = _marshal()
        self._state = self._call.state(cache, device, int(s.dtype == SF_BF16), s.n_q_heads, s.n_kv_heads, s.head_dim,
                                       s.page_size)
        self._scale = s.head_dim ** -0.5

    def close(self):
        if getattr(self, "cache", None):
            self._state = None
            sf_cache_destroy(self.cache)
            self.cache = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _empty(self, stream, *shape, dtype):
        return _empty(stream, self.device, shape, dtype)

    def append(self, qkv, index, table, k_pages, v_pages, *, pos=None, seq=None, q_gain=None, k_gain=None, q=None,
               stream=None):
        """Norm (where a gain is given), rotate and store T new rows; returns the rotated queries [T, n_q_heads,
        head_dim].  qkv [T, n_q_heads + 2 n_kv_heads, head_dim] (or its two last dimensions flattened)."""
        if q is None:
            q = self._empty(stream, qkv.shape[0], self.shapes.n_q_heads, self.shapes.head_dim, dtype=self.dtype)
        st = self._call.append(self._state, qkv, index, table, k_pages, v_pages, pos, seq, q_gain, k_gain, q, stream)
        if st:
            _check(st, None, "sf_cache_append", cache=self.cache)
        return q

    def attend(self, q, k_pages, v_pages, table, lens, *, scale=None, out=None, weights=None, weights_out=None,
               stream=None):
        """Attention of one new token per sequence, q [S, n_q_heads, head_dim]; returns [S, n_q_heads, head_dim].
        weights (fp32 [S, n_kv_heads, at least max_len]) gets every position's attention weight added, in place
        or into weights_out; weights_out alone gets this call's weights."""
        if out is None:
            out = self._empty(stream, q.shape[0], self.shapes.n_q_heads, self.shapes.head_dim, dtype=self.dtype)
        st = self._call.attend(self._state, q, k_pages, v_pages, table, lens, self._scale if scale is None else scale,
                               out, weights, weights if weights_out is None else weights_out, stream)
        if st:
            _check(st, None, "sf_cache_attend", cache=self.cache)
        return out

    def attend_rows(self, q, k_pages, v_pages, table, lens, starts, *, scale=None, out=None, lse=None, stream=None):
        """Attention of blocks of rows, q [T, n_q_heads, head_dim]: rows starts[s] .. starts[s + 1] - 1 (int32
        [S + 1]) over all lens[s] positions of sequence s, with no mask among them; returns [T, n_q_heads, head_dim].
        lse (fp32 [T, n_q_heads]) gets the logarithm of every softmax's sum.  Rows of no sequence are left as they
        were in out and lse (undefined in an out that the call makes)."""
        if out is None:
            out = self._empty(stream, q.shape[0], self.shapes.n_q_heads, self.shapes.head_dim, dtype=self.dtype)
        st = self._call.attend_rows(self._state, q, k_pages, v_pages, table, lens, starts,
                                    self._scale if scale is None else scale, out, lse, stream)
        if st:
            _check(st, None, "sf_cache_attend_rows", cache=self.cache)
        return out

    def attend_shared(self, q, k_pages, v_pages, table, lens, prefix_table, prefix_lens, starts, *, scale=None,
                      out=None, lse=None, stream=None):
        """Attention of one new token per sequence, q [S, n_q_heads, head_dim], where sequences starts[g] ..
        starts[g + 1] - 1 (int32 [G + 1]) see the prefix_lens[g] positions of prefix g (prefix_table [G, columns])
        and then their own lens[s] positions (table); returns [S, n_q_heads, head_dim].  A group's prefix is read
        once.  lse (fp32 [S, n_q_heads]) gets the logarithm of every softmax's sum."""
        if out is None:
            out = self._empty(stream, q.shape[0], self.shapes.n_q_heads, self.shapes.head_dim, dtype=self.dtype)
        st = self._call.attend_shared(self._state, q, k_pages, v_pages, table, lens, prefix_table, prefix_lens,
                                      starts, self._scale if scale is None else scale, out, lse, stream)
        if st:
            _check(st, None, "sf_cache_attend_shared", cache=self.cache)
        return out

    def reposition(self, k_pages, table, lens, pos_from, *, pos_to=None, stream=None):
        """Turn the cached keys, in place, from the positions pos_from (int32 [S, n_kv_heads, n], n at least the
        longest length; evict's `kept` where positions were places) to pos_to (the same shape; default: their
        places).  Keys with a negative position stay as they are."""
        st = self._call.reposition(self._state, k_pages, table, lens, pos_from, pos_to, stream)
        if st:
            _check(st, None, "sf_cache_reposition", cache=self.cache)

    def evict(self, k_pages, v_pages, table, lens, weights, budget, *, n_first=0, n_recent=0, k_out=None, v_out=None,
              table_out=None, weights_out=None, lens_out=None, kept=None, stream=None):
        """Keep at most `budget` positions of every sequence and KV head: the first n_first, the last n_recent and
        the heaviest others, moved in order to the front of the same pages, or of k_out / v_out / table_out (given
        together).  weights moves along, in place or into weights_out.  Returns (lens_out [S], kept [S, n_kv_heads,
        budget])."""
        if k_out is None or v_out is None or table_out is None:
            if not (k_out is None and v_out is None and table_out is None):
                raise ValueError("k_out, v_out and table_out are given together")
            k_out, v_out, table_out = k_pages, v_pages, table
        if lens_out is None or kept is None:
            import torch
            S = lens.shape[0]
            if lens_out is None:
                lens_out = self._empty(stream, S, dtype=torch.int32)
            if kept is None:
                kept = self._empty(stream, S, self.shapes.n_kv_heads, max(int(budget), 0), dtype=torch.int32)
        st = self._call.evict(self._state, k_pages, v_pages, table, lens, weights, budget, n_first, n_recent, k_out,
                              v_out, table_out, weights if weights_out is None else weights_out, lens_out, kept,
                              stream)
        if st:
            _check(st, None, "sf_cache_evict", cache=self.cache)
        return lens_out, kept

    def sync(self, stream=None):
        sf_cache_sync_status(self.cache, _stream_handle(stream))


def from_config(cfg, weights, max_requests=None, max_branches=None, max_prefix=None) -> SpecFold:
    """Context for a workload description with the fields of synth.Config."""
    return SpecFold(n_layers=cfg.n_layers, d_model=cfg.d_model, n_q_heads=cfg.n_q_heads,
                    n_kv_heads=cfg.n_kv_heads, head_dim=cfg.head_dim, d_ffn=cfg.d_ffn, dtype=cfg.dtype,
                    block_len=cfg.block_len, max_requests=max_requests or cfg.n_requests,
                    max_branches=max_branches or cfg.n_branches, max_prefix=max_prefix or cfg.prefix_len,
                    weights=weights, rms_eps=cfg.rms_eps, rope_theta=cfg.rope_theta)
