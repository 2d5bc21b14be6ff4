"""Python binding of libpivot (ctypes).

The functions named ``pivot_*`` mirror the C ABI of ``include/pivot.h`` one
to one (argument marshalling only).  The lower-case helpers below them
(``dense_index``, ``proxy_reduce``, ...) allocate outputs and workspaces
with torch on the caller's device and stream and then call the same entry
points; every step of the indexer runs in the library's CUDA kernels.

There is no fallback: if ``libpivot.so`` is missing or cannot be loaded,
``load()`` raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpivot.so")

F32, BF16, E4M3 = 0, 1, 2
DENSE, REUSE, REFINE = 0, 1, 2
ORDER_POSITION, ORDER_RANK = 0, 1
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "workspace too small",
          4: "CUDA error", 5: "a kernel wait timed out", 6: "bad device-side data"}

ABI_SYMBOLS = [
    "pivot_dense_index", "pivot_dense_index_workspace_size", "pivot_proxy_reduce",
    "pivot_proxy_scan", "pivot_proxy_scan_workspace_size", "pivot_reuse", "pivot_refine",
    "pivot_refine_workspace_size", "pivot_decode", "pivot_decode_workspace_size",
    "pivot_get_device_error", "pivot_set_wait_limit_ns", "pivot_selftest_wait_timeout",
    "pivot_status_string", "pivot_version", "pivot_profile_enable", "pivot_profile_read",
    "pivot_launch_count", "pivot_decode_noalloc", "pivot_last_error_detail",
    "pivot_reuse_backfill", "pivot_window_union", "pivot_index_varlen",
    "pivot_index_varlen_workspace_size", "pivot_index_window_outside",
    "pivot_index_window_outside_workspace_size", "pivot_set_score_buffer_cap",
    "pivot_workspace_size", "pivot_set_fused_selection", "pivot_refine_adaptive",
    "pivot_refine_adaptive_workspace_size", "pivot_cache_append",
    "pivot_cache_append_workspace_size", "pivot_pages_fork", "pivot_pages_fork_workspace_size",
    "pivot_pages_free", "pivot_pages_copy", "pivot_pages_compact",
    "pivot_pages_compact_workspace_size", "pivot_paged_attention",
    "pivot_paged_attention_workspace_size", "pivot_selected_attention",
    "pivot_selected_attention_workspace_size",
]
KERNELS = {0: "scan", 1: "select", 2: "refine", 3: "reduce", 4: "reuse"}


class PivotError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} (status {status})")


class PivotSeq(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("L", ctypes.c_int32), ("H", ctypes.c_int32),
                ("D", ctypes.c_int32), ("q", ctypes.c_void_p), ("q_scale", ctypes.c_void_p),
                ("w", ctypes.c_void_p), ("k", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("t_begin", ctypes.c_int32), ("t_end", ctypes.c_int32),
                ("order", ctypes.c_int32)]


class PivotVarlen(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("nseq", ctypes.c_int32), ("H", ctypes.c_int32),
                ("D", ctypes.c_int32), ("cu_seqlens", ctypes.c_void_p), ("q", ctypes.c_void_p),
                ("q_scale", ctypes.c_void_p), ("w", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("order", ctypes.c_int32)]


class PivotDecode(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("B", ctypes.c_int32), ("Gm", ctypes.c_int32),
                ("H", ctypes.c_int32), ("D", ctypes.c_int32), ("maxlen", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("q_scale", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("kc", ctypes.c_void_p), ("kc_scale", ctypes.c_void_p),
                ("cache_len", ctypes.c_void_p), ("order", ctypes.c_int32)]


class PivotCache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("B", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("D", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("len", ctypes.c_void_p), ("refs", ctypes.c_void_p)]


class PivotAttend(ctypes.Structure):
    _fields_ = [("Hq", ctypes.c_int32), ("total", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("cu_new", ctypes.c_void_p), ("scale", ctypes.c_float),
                ("window", ctypes.c_int32), ("idx", ctypes.c_void_p), ("topk", ctypes.c_int32),
                ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


_lib = None


def load(path: str = LIB_PATH):
    """Load libpivot.so (raises if it is missing: there is no other path)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libpivot.so not built at {path}; run "
                          "`python -m top_token_selection_b200.build`")
    lib = ctypes.CDLL(path)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    sig = {
        "pivot_dense_index": ([P, I32, P, P, P, SZ, P], I32),
        "pivot_dense_index_workspace_size": ([P, I32], SZ),
        "pivot_proxy_reduce": ([P, I32, P, P, P, P], I32),
        "pivot_proxy_scan": ([P, I32, P, P, P, I32, I32, P, P, P, SZ, P], I32),
        "pivot_proxy_scan_workspace_size": ([P, I32, I32], SZ),
        "pivot_reuse": ([I32, I32, I32, P, I32, I32, P, P], I32),
        "pivot_refine": ([P, I32, P, I32, I32, P, P, P, SZ, P], I32),
        "pivot_refine_workspace_size": ([P, I32, I32, I32], SZ),
        "pivot_decode": ([P, I32, I32, I32, P, P, P, SZ, P], I32),
        "pivot_decode_workspace_size": ([P, I32, I32, I32], SZ),
        "pivot_get_device_error": ([P], I32),
        "pivot_set_wait_limit_ns": ([ctypes.c_uint64], I32),
        "pivot_set_score_buffer_cap": ([SZ], I32),
        "pivot_selftest_wait_timeout": ([P], I32),
        "pivot_status_string": ([I32], ctypes.c_char_p),
        "pivot_version": ([], I32),
        "pivot_profile_enable": ([I32], I32),
        "pivot_profile_read": ([I32, P, P, P], I32),
        "pivot_launch_count": ([], ctypes.c_int64),
        "pivot_decode_noalloc": ([P, I32, I32, I32, P, P, P], I32),
        "pivot_last_error_detail": ([], ctypes.c_char_p),
        "pivot_reuse_backfill": ([I32, I32, I32, P, P, I32, I32, P, P], I32),
        "pivot_window_union": ([P, I32, I32, I32, P, I32, P, P], I32),
        "pivot_index_varlen": ([P, I32, I32, I32, I32, P, P, SZ, P], I32),
        "pivot_index_varlen_workspace_size": ([P, I32, I32, I32, I32], SZ),
        "pivot_index_window_outside": ([P, I32, I32, I32, I32, I32, P, P, SZ, P], I32),
        "pivot_index_window_outside_workspace_size": ([P, I32, I32, I32, I32, I32], SZ),
        "pivot_workspace_size": ([I32, I32, I32, I32, I32, I32, I32, I32, I32], SZ),
        "pivot_set_fused_selection": ([I32, ctypes.c_float], I32),
        "pivot_refine_adaptive": ([P, I32, P, P, I32, I32, ctypes.c_float, P, P, P, P, SZ, P],
                                  I32),
        "pivot_refine_adaptive_workspace_size": ([P, I32, I32, I32], SZ),
        "pivot_cache_append": ([P, P, P, P, I32, I32, P, P, SZ, P], I32),
        "pivot_cache_append_workspace_size": ([P, I32], SZ),
        "pivot_pages_fork": ([P, P, P, I32, P, SZ, P], I32),
        "pivot_pages_fork_workspace_size": ([P, I32], SZ),
        "pivot_pages_free": ([P, P, P, I32, P], I32),
        "pivot_pages_copy": ([P, I32, P, I32, SZ, P, P, I32, P], I32),
        "pivot_pages_compact": ([P, P, P, P, SZ, P], I32),
        "pivot_pages_compact_workspace_size": ([P], SZ),
        "pivot_paged_attention": ([P, P, P, SZ, P], I32),
        "pivot_paged_attention_workspace_size": ([P, P], SZ),
        "pivot_selected_attention": ([P, P, P, SZ, P], I32),
        "pivot_selected_attention_workspace_size": ([P, P], SZ),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


# ---------------------------------------------------------------------------
# C ABI mirrors (same names, same arguments)
# ---------------------------------------------------------------------------

def pivot_dense_index(seq, topk, idx, score, ws, ws_bytes, stream):
    return load().pivot_dense_index(ctypes.byref(seq), topk, idx, score, ws, ws_bytes, stream)


def pivot_dense_index_workspace_size(seq, topk):
    return load().pivot_dense_index_workspace_size(ctypes.byref(seq), topk)


def pivot_proxy_reduce(seq, g, pq, pq_scale, pw, stream):
    return load().pivot_proxy_reduce(ctypes.byref(seq), g, pq, pq_scale, pw, stream)


def pivot_proxy_scan(seq, g, pq, pq_scale, pw, C, topk, cand, cand_score, ws, ws_bytes, stream):
    return load().pivot_proxy_scan(ctypes.byref(seq), g, pq, pq_scale, pw, C, topk, cand,
                                   cand_score, ws, ws_bytes, stream)


def pivot_proxy_scan_workspace_size(seq, g, C):
    return load().pivot_proxy_scan_workspace_size(ctypes.byref(seq), g, C)


def pivot_reuse(t_begin, t_end, g, cand, C, topk, idx, stream):
    return load().pivot_reuse(t_begin, t_end, g, cand, C, topk, idx, stream)


def pivot_reuse_backfill(t_begin, t_end, g, cand, cand_score, C, topk, idx, stream):
    return load().pivot_reuse_backfill(t_begin, t_end, g, cand, cand_score, C, topk, idx, stream)


def pivot_window_union(idx, rows, topk, t_begin, positions, window, out, stream):
    return load().pivot_window_union(idx, rows, topk, t_begin, positions, window, out, stream)


def pivot_refine(seq, g, cand, C, topk, idx, score, ws, ws_bytes, stream):
    return load().pivot_refine(ctypes.byref(seq), g, cand, C, topk, idx, score, ws, ws_bytes,
                               stream)


def pivot_refine_workspace_size(seq, g, C, topk):
    return load().pivot_refine_workspace_size(ctypes.byref(seq), g, C, topk)


def pivot_decode(batch, mode, C, topk, idx, cand, ws, ws_bytes, stream):
    return load().pivot_decode(ctypes.byref(batch), mode, C, topk, idx, cand, ws, ws_bytes,
                               stream)


def pivot_decode_workspace_size(batch, mode, C, topk):
    return load().pivot_decode_workspace_size(ctypes.byref(batch), mode, C, topk)


def pivot_workspace_size(mode, dtype, L_or_maxlen, B, H, D, g, C, topk):
    return load().pivot_workspace_size(mode, dtype, L_or_maxlen, B, H, D, g, C, topk)


def pivot_decode_noalloc(batch, mode, C, topk, idx, cand, stream):
    return load().pivot_decode_noalloc(ctypes.byref(batch), mode, C, topk, idx, cand, stream)


def pivot_get_device_error(stream):
    return load().pivot_get_device_error(stream)


def pivot_set_wait_limit_ns(ns):
    return load().pivot_set_wait_limit_ns(ns)


def pivot_set_score_buffer_cap(nbytes):
    return load().pivot_set_score_buffer_cap(nbytes)


def pivot_set_fused_selection(on, margin_sigmas=4.5):
    return load().pivot_set_fused_selection(on, margin_sigmas)


def pivot_selftest_wait_timeout(stream):
    return load().pivot_selftest_wait_timeout(stream)


def pivot_profile_enable(on):
    return load().pivot_profile_enable(on)


def pivot_profile_read(kernel, launches, total_ms, work):
    return load().pivot_profile_read(kernel, launches, total_ms, work)


def pivot_launch_count():
    return load().pivot_launch_count()


def profile_read(kernel):
    """(launches, total_ms, work) of one kernel class since profiling began."""
    n = ctypes.c_int64(0)
    ms = ctypes.c_double(0.0)
    wk = ctypes.c_double(0.0)
    _check(pivot_profile_read(kernel, ctypes.byref(n), ctypes.byref(ms), ctypes.byref(wk)),
           "pivot_profile_read")
    return n.value, ms.value, wk.value


def pivot_status_string(status):
    return load().pivot_status_string(status).decode()


def pivot_version():
    return load().pivot_version()


def pivot_last_error_detail():
    return load().pivot_last_error_detail().decode()


# ---------------------------------------------------------------------------
# torch marshalling helpers
# ---------------------------------------------------------------------------

def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype in (torch.float8_e4m3fn, torch.uint8):
        return E4M3
    raise TypeError(f"unsupported indexer dtype {t.dtype}")


def _p(t):
    if t is None:
        return None
    assert t.is_cuda and t.is_contiguous(), "libpivot takes contiguous CUDA tensors"
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status, what):
    if status != 0:
        if status == 4:
            what = f"{what} [{pivot_last_error_detail()}]"
        raise PivotError(status, what)


def _workspace(nbytes, device):
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def make_seq(q, q_scale, w, k, k_scale, t_begin=0, t_end=0, order=ORDER_POSITION) -> PivotSeq:
    """Describe one prefill sequence; the struct keeps the tensors alive."""
    L, H, D = q.shape
    s = PivotSeq(_dtype_code(q), L, H, D, _p(q), _p(q_scale), _p(w), _p(k), _p(k_scale),
                 t_begin, t_end, order)
    s._keep = (q, q_scale, w, k, k_scale)
    return s


def make_varlen(cu_seqlens, q, q_scale, w, k, k_scale, order=ORDER_POSITION) -> PivotVarlen:
    """Describe a ragged batch: cu_seqlens is a host sequence of nseq + 1
    row offsets; the struct keeps it and the tensors alive."""
    cu = (ctypes.c_int32 * len(cu_seqlens))(*[int(x) for x in cu_seqlens])
    _, H, D = q.shape
    s = PivotVarlen(_dtype_code(q), len(cu_seqlens) - 1, H, D, ctypes.addressof(cu), _p(q),
                    _p(q_scale), _p(w), _p(k), _p(k_scale), order)
    s._keep = (cu, q, q_scale, w, k, k_scale)
    return s


def pivot_index_varlen(batch, mode, g, C, topk, idx, ws, ws_bytes, stream):
    return load().pivot_index_varlen(ctypes.byref(batch), mode, g, C, topk, idx, ws, ws_bytes,
                                     stream)


def pivot_index_varlen_workspace_size(batch, mode, g, C, topk):
    return load().pivot_index_varlen_workspace_size(ctypes.byref(batch), mode, g, C, topk)


def pivot_index_window_outside(seq, mode, g, C, topk, window, idx, ws, ws_bytes, stream):
    return load().pivot_index_window_outside(ctypes.byref(seq), mode, g, C, topk, window, idx, ws,
                                             ws_bytes, stream)


def pivot_index_window_outside_workspace_size(seq, mode, g, C, topk, window):
    return load().pivot_index_window_outside_workspace_size(ctypes.byref(seq), mode, g, C, topk,
                                                            window)


def index_window_outside(seq: PivotSeq, mode, g, C, topk, window, ws=None, stream=None,
                         device="cuda"):
    idx = torch.empty(_rows(seq), topk + window, dtype=torch.int32, device=device)
    if ws is None:
        ws = _workspace(pivot_index_window_outside_workspace_size(seq, mode, g, C, topk, window),
                        device)
    _check(pivot_index_window_outside(seq, mode, g, C, topk, window, _p(idx), _p(ws), ws.numel(),
                                      _stream(stream)), "pivot_index_window_outside")
    return idx


def index_varlen(batch: PivotVarlen, mode, g, C, topk, ws=None, stream=None, device="cuda"):
    total = batch._keep[0][batch.nseq]
    idx = torch.empty(total, topk, dtype=torch.int32, device=device)
    if ws is None:
        ws = _workspace(pivot_index_varlen_workspace_size(batch, mode, g, C, topk), device)
    _check(pivot_index_varlen(batch, mode, g, C, topk, _p(idx), _p(ws), ws.numel(),
                              _stream(stream)), "pivot_index_varlen")
    return idx


def make_decode(q, q_scale, w, kc, kc_scale, cache_len, order=ORDER_POSITION) -> PivotDecode:
    """Describe one decode batch; the struct keeps the tensors alive."""
    B, Gm, H, D = q.shape
    s = PivotDecode(_dtype_code(q), B, Gm, H, D, kc.shape[1], _p(q), _p(q_scale), _p(w),
                    _p(kc), _p(kc_scale), _p(cache_len), order)
    s._keep = (q, q_scale, w, kc, kc_scale, cache_len)
    return s


def _rows(seq):
    return (seq.t_end or seq.L) - seq.t_begin


def dense_index(seq: PivotSeq, topk, with_score=False, ws=None, stream=None, device="cuda"):
    n = _rows(seq)
    idx = torch.empty(n, topk, dtype=torch.int32, device=device)
    score = torch.empty(n, topk, dtype=torch.float32, device=device) if with_score else None
    if ws is None:
        ws = _workspace(pivot_dense_index_workspace_size(seq, topk), device)
    _check(pivot_dense_index(seq, topk, _p(idx), _p(score), _p(ws), ws.numel(), _stream(stream)),
           "pivot_dense_index")
    return idx, score


def proxy_reduce(seq: PivotSeq, g, stream=None, device="cuda"):
    G = -(-_rows(seq) // g)
    store = {F32: torch.float32, BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn}[seq.dtype]
    pq = torch.empty(G, seq.H, seq.D, dtype=store, device=device)
    pqs = torch.empty(G, dtype=torch.float32, device=device) if seq.dtype == E4M3 else None
    pw = torch.empty(G, seq.H, dtype=torch.float32, device=device)
    _check(pivot_proxy_reduce(seq, g, _p(pq), _p(pqs), _p(pw), _stream(stream)),
           "pivot_proxy_reduce")
    return pq, pqs, pw


def proxy_scan(seq: PivotSeq, g, pq, pqs, pw, C, topk, with_score=False, ws=None, stream=None,
               device="cuda"):
    """Candidates [G, C]: each proxy's top-topk positions, then the rest of
    its top-C, each ascending (rank order throughout if seq.order asks)."""
    G = pq.shape[0]
    cand = torch.empty(G, C, dtype=torch.int32, device=device)
    cs = torch.empty(G, C, dtype=torch.float32, device=device) if with_score else None
    if ws is None:
        ws = _workspace(pivot_proxy_scan_workspace_size(seq, g, C), device)
    _check(pivot_proxy_scan(seq, g, _p(pq), _p(pqs), _p(pw), C, topk, _p(cand), _p(cs), _p(ws),
                            ws.numel(), _stream(stream)), "pivot_proxy_scan")
    return cand, cs


def reuse(t_begin, t_end, g, cand, topk, stream=None, device="cuda"):
    idx = torch.empty(t_end - t_begin, topk, dtype=torch.int32, device=device)
    _check(pivot_reuse(t_begin, t_end, g, _p(cand), cand.shape[1], topk, _p(idx),
                       _stream(stream)), "pivot_reuse")
    return idx


def reuse_backfill(t_begin, t_end, g, cand, cand_score, topk, stream=None, device="cuda"):
    idx = torch.empty(t_end - t_begin, topk, dtype=torch.int32, device=device)
    _check(pivot_reuse_backfill(t_begin, t_end, g, _p(cand), _p(cand_score), cand.shape[1], topk,
                                _p(idx), _stream(stream)), "pivot_reuse_backfill")
    return idx


def window_union(idx, window, t_begin=0, positions=None, stream=None):
    rows, topk = idx.shape
    out = torch.empty(rows, topk + window, dtype=torch.int32, device=idx.device)
    _check(pivot_window_union(_p(idx), rows, topk, t_begin, _p(positions), window, _p(out),
                              _stream(stream)), "pivot_window_union")
    return out


def refine(seq: PivotSeq, g, cand, topk, with_score=False, ws=None, stream=None, device="cuda"):
    n = _rows(seq)
    C = cand.shape[1]
    idx = torch.empty(n, topk, dtype=torch.int32, device=device)
    score = torch.empty(n, topk, dtype=torch.float32, device=device) if with_score else None
    if ws is None:
        ws = _workspace(pivot_refine_workspace_size(seq, g, C, topk), device)
    _check(pivot_refine(seq, g, _p(cand), C, topk, _p(idx), _p(score), _p(ws), ws.numel(),
                        _stream(stream)), "pivot_refine")
    return idx, score


def pivot_refine_adaptive(seq, g, cand, cand_score, C, topk, rho, cand_count, idx, score, ws,
                          ws_bytes, stream):
    return load().pivot_refine_adaptive(ctypes.byref(seq), g, cand, cand_score, C, topk, rho,
                                        cand_count, idx, score, ws, ws_bytes, stream)


def pivot_refine_adaptive_workspace_size(seq, g, C, topk):
    return load().pivot_refine_adaptive_workspace_size(ctypes.byref(seq), g, C, topk)


def refine_adaptive(seq: PivotSeq, g, cand, cand_score, topk, rho, ws=None, stream=None,
                    device="cuda"):
    """Refine over each group's adaptive count of rank-ordered candidates;
    returns (idx, counts)."""
    n = _rows(seq)
    C = cand.shape[1]
    idx = torch.empty(n, topk, dtype=torch.int32, device=device)
    counts = torch.empty(cand.shape[0], dtype=torch.int32, device=device)
    if ws is None:
        ws = _workspace(pivot_refine_adaptive_workspace_size(seq, g, C, topk), device)
    _check(pivot_refine_adaptive(seq, g, _p(cand), _p(cand_score), C, topk, rho, _p(counts),
                                 _p(idx), None, _p(ws), ws.numel(), _stream(stream)),
           "pivot_refine_adaptive")
    return idx, counts


def decode(batch: PivotDecode, mode, C, topk, want_cand=False, ws=None, stream=None,
           device="cuda"):
    idx = torch.empty(batch.B, batch.Gm, topk, dtype=torch.int32, device=device)
    cand = (torch.empty(batch.B, C, dtype=torch.int32, device=device)
            if (want_cand and mode != DENSE) else None)
    if ws is None:
        ws = _workspace(pivot_decode_workspace_size(batch, mode, C, topk), device)
    _check(pivot_decode(batch, mode, C, topk, _p(idx), _p(cand), _p(ws), ws.numel(),
                        _stream(stream)), "pivot_decode")
    return idx, cand


def device_error(stream=None) -> int:
    return pivot_get_device_error(_stream(stream))


# ---------------------------------------------------------------------------
# paged key/value cache: append, pages, attention
# ---------------------------------------------------------------------------

def pivot_cache_append(cache, k_new, v_new, cu_new, total, max_new, lack, ws, ws_bytes, stream):
    return load().pivot_cache_append(ctypes.byref(cache), k_new, v_new, cu_new, total, max_new,
                                     lack, ws, ws_bytes, stream)


def pivot_cache_append_workspace_size(cache, total):
    return load().pivot_cache_append_workspace_size(ctypes.byref(cache), total)


def pivot_pages_fork(cache, src, dst, n, ws, ws_bytes, stream):
    return load().pivot_pages_fork(ctypes.byref(cache), src, dst, n, ws, ws_bytes, stream)


def pivot_pages_fork_workspace_size(cache, n):
    return load().pivot_pages_fork_workspace_size(ctypes.byref(cache), n)


def pivot_pages_free(cache, seqs, keep, n, stream):
    return load().pivot_pages_free(ctypes.byref(cache), seqs, keep, n, stream)


def pivot_pages_copy(src, src_pages, dst, dst_pages, page_bytes, src_ids, dst_ids, n, stream):
    return load().pivot_pages_copy(src, src_pages, dst, dst_pages, page_bytes, src_ids, dst_ids, n,
                                   stream)


def pivot_pages_compact(cache, remap, used, ws, ws_bytes, stream):
    return load().pivot_pages_compact(ctypes.byref(cache), remap, used, ws, ws_bytes, stream)


def pivot_pages_compact_workspace_size(cache):
    return load().pivot_pages_compact_workspace_size(ctypes.byref(cache))


def pivot_paged_attention(cache, call, ws, ws_bytes, stream):
    return load().pivot_paged_attention(ctypes.byref(cache), ctypes.byref(call), ws, ws_bytes,
                                        stream)


def pivot_paged_attention_workspace_size(cache, call):
    return load().pivot_paged_attention_workspace_size(ctypes.byref(cache), ctypes.byref(call))


def pivot_selected_attention(cache, call, ws, ws_bytes, stream):
    return load().pivot_selected_attention(ctypes.byref(cache), ctypes.byref(call), ws, ws_bytes,
                                           stream)


def pivot_selected_attention_workspace_size(cache, call):
    return load().pivot_selected_attention_workspace_size(ctypes.byref(cache), ctypes.byref(call))


class _On:
    """The device of tensor `t` made current, and `stream` (None: that
    device's current stream), for the length of a call: what the helpers
    below allocate belongs to the stream that uses it."""

    def __init__(self, t, stream):
        self.ctx, self.index = [], t.device.index
        if self.index != torch.cuda.current_device():
            self.ctx.append(torch.cuda.device(t.device))
        if stream is not None:
            self.ctx.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.ctx:
            c.__enter__()
        return ctypes.c_void_p(torch.cuda.current_stream(self.index).cuda_stream)

    def __exit__(self, *exc):
        for c in reversed(self.ctx):
            c.__exit__(*exc)


def _arg(t, name, dtype, shape, device):
    """The address of `t` if it is a contiguous tensor of that type, shape and
    device; raises if not."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name}: a {dtype} tensor is wanted")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, wanted {tuple(shape)}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: wanted contiguous, on {device}")
    return t.data_ptr()


def make_cache(k, v, table, length, refs, k_scale=None, v_scale=None) -> PivotCache:
    """Describe a paged cache: k, v [num_pages, page_size, Hkv, D] bf16, or
    e4m3 with k_scale, v_scale [num_pages, page_size]; table [B, max_pages],
    length [B] and refs [num_pages] int32.  An empty cache has table -1,
    length 0 and refs 0.  The struct keeps the tensors alive."""
    if not k.is_cuda or k.dim() != 4 or table.dim() != 2:
        raise ValueError("k: [num_pages, page_size, Hkv, D] on a CUDA device; table: [B, max_pages]")
    n, page, Hkv, D = k.shape
    B, columns = table.shape
    dev, i32 = k.device, torch.int32
    code = _dtype_code(k)
    f32 = torch.float32
    c = PivotCache(code, B, Hkv, D, page, n, columns, _arg(k, "k", k.dtype, k.shape, dev),
                   _arg(v, "v", k.dtype, k.shape, dev),
                   None if k_scale is None else _arg(k_scale, "k_scale", f32, (n, page), dev),
                   None if v_scale is None else _arg(v_scale, "v_scale", f32, (n, page), dev),
                   _arg(table, "table", i32, (B, columns), dev),
                   _arg(length, "length", i32, (B,), dev), _arg(refs, "refs", i32, (n,), dev))
    c._keep = (k, v, k_scale, v_scale, table, length, refs)
    c.device = dev
    return c


def cache_append(cache: PivotCache, k_new, v_new, cu_new, max_new, ws=None, stream=None):
    """Append rows cu_new[b] .. cu_new[b + 1] of k_new, v_new (bf16
    [total, Hkv, D]) to sequence b; returns lack [1] int32 on the device: 0,
    or the free pages missing (then nothing was appended)."""
    dev, total = cache.device, k_new.shape[0]
    pk = _arg(k_new, "k_new", torch.bfloat16, (total, cache.Hkv, cache.D), dev)
    pv = _arg(v_new, "v_new", torch.bfloat16, k_new.shape, dev)
    pc = _arg(cu_new, "cu_new", torch.int32, (cache.B + 1,), dev)
    with _On(k_new, stream) as st:
        lack = torch.empty(1, dtype=torch.int32, device=dev)
        if ws is None:
            ws = _workspace(pivot_cache_append_workspace_size(cache, total), dev)
        _check(pivot_cache_append(cache, pk, pv, pc, total, max_new, lack.data_ptr(), _p(ws),
                                  ws.numel(), st), "pivot_cache_append")
    return lack


def pages_fork(cache: PivotCache, src, dst, ws=None, stream=None):
    """Make sequence dst[i] a copy of sequence src[i] as it stood before the
    call, its pages shared; src, dst [n] int32, dst distinct."""
    dev, n = cache.device, src.shape[0]
    ps = _arg(src, "src", torch.int32, (n,), dev)
    pd = _arg(dst, "dst", torch.int32, (n,), dev)
    with _On(src, stream) as st:
        if ws is None:
            ws = _workspace(pivot_pages_fork_workspace_size(cache, n), dev)
        _check(pivot_pages_fork(cache, ps, pd, n, _p(ws), ws.numel(), st),
               "pivot_pages_fork")


def pages_free(cache: PivotCache, seqs, keep, stream=None):
    """Cut sequence seqs[i] to its first keep[i] tokens (0: free it); seqs
    distinct."""
    dev, n = cache.device, seqs.shape[0]
    ps = _arg(seqs, "seqs", torch.int32, (n,), dev)
    pk = _arg(keep, "keep", torch.int32, (n,), dev)
    with _On(seqs, stream) as st:
        _check(pivot_pages_free(cache, ps, pk, n, st), "pivot_pages_free")


def pages_copy(src, dst, src_ids, dst_ids, stream=None):
    """dst[dst_ids[i]] = src[src_ids[i]] for planes whose first axis counts
    pages; ids [n] int32, no destination named twice or read in the same call."""
    dev, n = src.device, src_ids.shape[0]
    if src.dtype != dst.dtype or src.shape[1:] != dst.shape[1:]:
        raise ValueError("src and dst: pages of one type and shape")
    if not src.is_cuda or src.dim() < 1 or not src.shape[0]:
        raise ValueError("src: pages on a CUDA device")
    ps = _arg(src, "src", src.dtype, src.shape, dev)
    pd = _arg(dst, "dst", src.dtype, dst.shape, dev)
    pi = _arg(src_ids, "src_ids", torch.int32, (n,), dev)
    pj = _arg(dst_ids, "dst_ids", torch.int32, (n,), dev)
    page = src.numel() // src.shape[0] * src.element_size()
    with _On(src, stream) as st:
        _check(pivot_pages_copy(ps, src.shape[0], pd, dst.shape[0], page, pi, pj, n, st),
               "pivot_pages_copy")


def pages_compact(cache: PivotCache, ws=None, stream=None):
    """Move the pages in use to the lowest ids; returns (remap [num_pages]:
    each used page's new id, -1 for free ones; used [1])."""
    dev = cache.device
    with _On(cache._keep[0], stream) as st:
        remap = torch.empty(cache.num_pages, dtype=torch.int32, device=dev)
        used = torch.empty(1, dtype=torch.int32, device=dev)
        if ws is None:
            ws = _workspace(pivot_pages_compact_workspace_size(cache), dev)
        _check(pivot_pages_compact(cache, _p(remap), _p(used), _p(ws), ws.numel(), st),
               "pivot_pages_compact")
    return remap, used


def _attention(cache, q, cu_new, max_new, idx, scale, window, with_lse, o, ws, stream):
    dev = cache.device
    if q.dim() != 3:
        raise ValueError("q: [total, Hq, D]")
    total, Hq = q.shape[0], q.shape[1]
    pq = _arg(q, "q", torch.bfloat16, (total, Hq, cache.D), dev)
    pc = _arg(cu_new, "cu_new", torch.int32, (cache.B + 1,), dev)
    topk, pi = 0, None
    if idx is not None:
        topk = idx.shape[-1]
        pi = _arg(idx, "idx", torch.int32, (total, topk), dev)
    po = None if o is None else _arg(o, "o", torch.bfloat16, q.shape, dev)
    name = "pivot_paged_attention" if idx is None else "pivot_selected_attention"
    run, size = ((pivot_paged_attention, pivot_paged_attention_workspace_size) if idx is None else
                 (pivot_selected_attention, pivot_selected_attention_workspace_size))
    with _On(q, stream) as st:
        if o is None:
            o = torch.empty_like(q)
            po = o.data_ptr()
        lse = torch.empty(total, Hq, dtype=torch.float32, device=dev) if with_lse else None
        call = PivotAttend(Hq, total, max_new, pq, pc, cache.D ** -0.5 if scale is None else scale,
                           window, pi, topk, po, None if lse is None else lse.data_ptr())
        if ws is None:
            ws = _workspace(size(cache, call), dev)
        _check(run(cache, call, _p(ws), ws.numel(), st), name)
    return o, lse


def paged_attention(cache: PivotCache, q, cu_new, max_new, scale=None, window=0, with_lse=False,
                    o=None, ws=None, stream=None):
    """Causal attention of the batch's new tokens (q bf16 [total, Hq, D], rows
    cu_new[b] .. cu_new[b + 1] the last tokens of sequence b, already
    appended) over the cache; window > 0 keeps that many positions up to the
    token's own.  scale: 1 / sqrt(D) by default.  Returns (o, lse or None);
    rows behind cu_new[B] are left as they were."""
    return _attention(cache, q, cu_new, max_new, None, scale, window, with_lse, o, ws, stream)


def selected_attention(cache: PivotCache, q, cu_new, max_new, idx, scale=None, with_lse=False,
                       o=None, ws=None, stream=None):
    """paged_attention over the positions of idx [total, topk] (-1 padded), as
    dense_index, reuse, refine, decode ... return them."""
    return _attention(cache, q, cu_new, max_new, idx, scale, 0, with_lse, o, ws, stream)


def decode_attention(batch: PivotDecode, cache: PivotCache, q, k_new, v_new, mode, C, topk,
                     scale=None, with_lse=False, stream=None):
    """One sparse decode step of a model's layer: the Gm new tokens of every
    sequence are appended to the cache (k_new, v_new bf16
    [B, Gm, Hkv, D]), the indexer (`decode`, mode DENSE, REUSE or REFINE)
    names each token's positions, and attention (q bf16 [B, Gm, Hq, D])
    reads them.  batch.cache_len counts the new tokens: the lengths that the
    append leaves (it may be the cache's own length tensor).  Returns
    (o [B, Gm, Hq, D], lse or None, idx, lack); a lack other than 0 (on the
    device) says that nothing was appended: o and idx are then not to be used,
    and the error word may be set (a sequence shorter than Gm)."""
    B, Gm = batch.B, batch.Gm
    dev = cache.device
    if cache.B != B or tuple(q.shape[:2]) != (B, Gm):
        raise ValueError("batch, cache and q: one number of sequences and of new tokens")
    with _On(q, stream):
        cu = torch.arange(0, (B + 1) * Gm, Gm, dtype=torch.int32, device=dev)
        lack = cache_append(cache, k_new.reshape(B * Gm, cache.Hkv, cache.D),
                            v_new.reshape(B * Gm, cache.Hkv, cache.D), cu, Gm)
        idx, _ = decode(batch, mode, C, topk, device=dev)
        o, lse = selected_attention(cache, q.reshape(B * Gm, q.shape[2], cache.D), cu, Gm,
                                    idx.view(B * Gm, topk), scale=scale, with_lse=with_lse)
    return o.view(q.shape), None if lse is None else lse.view(B, Gm, -1), idx, lack


# ---------------------------------------------------------------------------
# cross-layer reuse of index rows
# ---------------------------------------------------------------------------

def layer_anchors(nlayers: int, period: int):
    """Which layer's index rows each of `nlayers` layers uses when every
    `period`-th layer runs the indexer and the layers after it reuse its rows
    (in the style of IndexCache, which the PIVOT blog post names as stacking
    with PIVOT; the pages give none of its method, so the schedule is a plain
    fixed period): anchors[l] = l - l % period."""
    if nlayers < 1 or period < 1:
        raise ValueError("nlayers and period must be >= 1")
    return [layer - layer % period for layer in range(nlayers)]


def index_layers(layer_seqs, mode, g, C, topk, period, stream=None, device="cuda"):
    """Index rows for every layer of a model's consecutive layers: the anchor
    layers (layer_anchors) run the indexer -- dense (mode DENSE) or PIVOT
    with Reuse or Refine -- through the library; every other layer is handed
    its anchor's rows (the same tensor: nothing is recomputed or copied).
    Returns one [rows, topk] int32 tensor per layer."""
    anchors = layer_anchors(len(layer_seqs), period)
    rows = {}
    for layer, seq in enumerate(layer_seqs):
        if anchors[layer] != layer:
            continue
        if mode == DENSE:
            rows[layer], _ = dense_index(seq, topk, stream=stream, device=device)
        else:
            pq, pqs, pw = proxy_reduce(seq, g, stream=stream, device=device)
            cand, _ = proxy_scan(seq, g, pq, pqs, pw, C, topk, stream=stream, device=device)
            t0 = seq.t_begin
            t1 = seq.t_end or seq.L
            rows[layer] = (reuse(t0, t1, g, cand, topk, stream=stream, device=device)
                           if mode == REUSE else
                           refine(seq, g, cand, topk, stream=stream, device=device)[0])
    return [rows[a] for a in anchors]
