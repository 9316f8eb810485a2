"""Thin ctypes binding of libds4a (include/ds4a.h): argument marshalling only.

Every function has the name of its C entry point and takes torch tensors
(device memory) where the C call takes device pointers; every step of the
path runs in the library's CUDA kernels.  A missing library raises; there is
no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os

__all__ = [
    "DS4A_OK", "DS4A_EINVAL", "DS4A_EUNSUPPORTED", "DS4A_ECUDA", "DS4A_EDEVICE", "DS4A_ETIMEOUT",
    "DS4A_ENOSPACE", "Ds4aError", "LayerCfg", "layer_cfg", "lib", "LIB_PATH", "ds4a_compress",
    "ds4a_compress_state_bytes", "ds4a_compress_append", "ds4a_index_topk_workspace", "ds4a_index_topk", "ds4a_index_topk_noalloc", "ds4a_attend_workspace", "ds4a_sparse_attend",
    "ds4a_hca_attend", "ds4a_check", "ds4a_strerror", "ds4a_trace_enable", "ds4a_trace_read",
    "ds4a_version", "ds4a_selftest_wait_timeout", "OprojCfg", "ds4a_out_proj_workspace", "ds4a_out_proj",
    "DS4A_MX_KV_FP8", "DS4A_MX_IDX_FP4", "ds4a_kv_fp8_row_bytes", "ds4a_quantize_kv_fp8", "ds4a_quantize_idx_fp4",
    "ds4a_compress_append_mx", "ds4a_index_topk_fp4", "ds4a_sparse_attend_fp8", "ds4a_hca_attend_fp8",
    "AppendJob", "append_job", "ds4a_compress_append_jobs",
    "PagedKv", "paged_kv", "ds4a_paged_attend_workspace", "ds4a_paged_attend", "ds4a_paged_append",
    "ds4a_paged_evict_workspace", "ds4a_paged_evict", "ds4a_mxfp4_scale_bytes", "ds4a_quantize_mxfp4",
    "ds4a_out_proj_mxfp4_workspace", "ds4a_out_proj_mxfp4",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libds4a.so")

DS4A_OK, DS4A_EINVAL, DS4A_EUNSUPPORTED, DS4A_ECUDA, DS4A_EDEVICE, DS4A_ETIMEOUT, DS4A_ENOSPACE = range(7)
DS4A_MX_KV_FP8, DS4A_MX_IDX_FP4 = 1, 2


class Ds4aError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {ds4a_strerror(code)} (code {code})")


class LayerCfg(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("window", ctypes.c_int32),
                ("idx_heads", ctypes.c_int32), ("idx_dim", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("ratio", ctypes.c_int32),
                ("sm_scale", ctypes.c_float), ("rope_base", ctypes.c_float),
                ("rms_eps", ctypes.c_float)]


class OprojCfg(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("group_rank", ctypes.c_int32), ("hidden", ctypes.c_int32)]


class AppendJob(ctypes.Structure):
    _fields_ = [("c", ctypes.c_int32), ("format", ctypes.c_int32),
                ("ca", ctypes.c_void_p), ("cb", ctypes.c_void_p), ("za", ctypes.c_void_p), ("zb", ctypes.c_void_p),
                ("bias_a", ctypes.c_void_p), ("bias_b", ctypes.c_void_p), ("norm_g", ctypes.c_void_p),
                ("state", ctypes.c_void_p), ("pool", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("pool_bstride", ctypes.c_int64)]


class PagedKv(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("format", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]
    # what paged_kv knows besides: the tensors, their device, the table's rows, elements of a page's row
    held = dev = rows = row_size = None


def layer_cfg(c) -> LayerCfg:
    """LayerCfg from any object with the fields of ds4a_layer_cfg
    (sm_scale defaults to 1/sqrt(head_dim))."""
    scale = getattr(c, "sm_scale", None) or 1.0 / math.sqrt(c.head_dim)
    return LayerCfg(c.n_heads, c.head_dim, c.rope_dim, c.window, c.idx_heads, c.idx_dim, c.topk,
                    c.ratio, scale, getattr(c, "rope_base", 10000.0), getattr(c, "rms_eps", 1e-6))


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_CFG = ctypes.POINTER(LayerCfg)
_KV = ctypes.POINTER(PagedKv)

_SIGS = {
    "ds4a_compress": (_I, [_CFG, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _I64, _P]),
    "ds4a_compress_state_bytes": (_SZ, [_CFG, _I, _I, _I]),
    "ds4a_compress_append": (_I, [_CFG, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _I64, _P]),
    "ds4a_index_topk_workspace": (_SZ, [_CFG, _I, _I, _I]),
    "ds4a_compress_append_jobs": (_I, [_CFG, _I, _P, _I, ctypes.POINTER(AppendJob), _I, _P]),
    "ds4a_kv_fp8_row_bytes": (_SZ, [_I, _I]),
    "ds4a_quantize_kv_fp8": (_I, [_I, _I, _I, _P, _I64, _P, _I64, _P]),
    "ds4a_quantize_idx_fp4": (_I, [_I, _I, _P, _I64, _P, _P, _P]),
    "ds4a_compress_append_mx": (_I, [_CFG, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _P, _I64, _P]),
    "ds4a_index_topk_fp4": (_I, [_CFG, _I, _I, _P, _P, _P, _P, _P, _I64, _I, _P, _P, _P, _SZ, _P]),
    "ds4a_sparse_attend_fp8": (_I, [_CFG, _I, _I, _P, _P, _P, _P, _I64, _I, _P, _P, _I, _I64, _P, _P, _P, _SZ, _P]),
    "ds4a_hca_attend_fp8": (_I, [_CFG, _I, _I, _P, _P, _P, _P, _I64, _I, _P, _I, _I64, _P, _P, _P, _SZ, _P]),
    "ds4a_index_topk": (_I, [_CFG, _I, _I, _P, _P, _P, _P, _I64, _I, _P, _P, _P, _SZ, _P]),
    "ds4a_index_topk_noalloc": (_I, [_CFG, _I, _I, _P, _P, _P, _P, _I64, _I, _P, _P, _P]),
    "ds4a_attend_workspace": (_SZ, [_CFG, _I, _I, _I, _I]),
    "ds4a_sparse_attend": (_I, [_CFG, _I, _I, _P, _P, _P, _P, _I64, _I, _P, _P, _I, _I64, _P, _P, _P, _SZ, _P]),
    "ds4a_hca_attend": (_I, [_CFG, _I, _I, _P, _P, _P, _P, _I64, _I, _P, _I, _I64, _P, _P, _P, _SZ, _P]),
    "ds4a_check": (_I, [_P, ctypes.POINTER(ctypes.c_uint32)]),
    "ds4a_out_proj_workspace": (_SZ, [ctypes.POINTER(OprojCfg), _I]),
    "ds4a_out_proj": (_I, [ctypes.POINTER(OprojCfg), _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "ds4a_selftest_wait_timeout": (_I, [_I64, _P, _P]),
    "ds4a_strerror": (ctypes.c_char_p, [_I]),
    "ds4a_trace_enable": (_I, [_I]),
    "ds4a_trace_read": (_I, [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float), _I]),
    "ds4a_version": (_I, []),
    "ds4a_paged_attend_workspace": (_SZ, [_CFG, _KV, _I, _I, _I]),
    "ds4a_paged_attend": (_I, [_CFG, _KV, _I, _P, _P, _P, _P, _P, _P, _I, _I64, _P, _P, _P, _I, _I64, _P, _SZ, _P]),
    "ds4a_paged_append": (_I, [_CFG, _KV, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "ds4a_paged_evict_workspace": (_SZ, [_KV, _I]),
    "ds4a_paged_evict": (_I, [_CFG, _KV, _I, _P, _P, _I64, _I, _I, _I, _P, _P, _I64, _P, _P, _SZ, _P]),
    "ds4a_mxfp4_scale_bytes": (_SZ, [_I, _I]),
    "ds4a_quantize_mxfp4": (_I, [_I, _I, _P, _I64, _P, _P, _P]),
    "ds4a_out_proj_mxfp4_workspace": (_SZ, [ctypes.POINTER(OprojCfg), _I]),
    "ds4a_out_proj_mxfp4": (_I, [ctypes.POINTER(OprojCfg), _I, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
}


def lib():
    """The loaded libds4a (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


# plain ints (or None) for pointer arguments: ctypes converts them through
# the c_void_p argtypes without a wrapper object per argument
def _ptr(t):
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        # torch.cuda.current_stream().cuda_stream without its Stream object (3 us a call), where torch offers it
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            return torch.cuda.current_stream().cuda_stream
        return raw(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ok(rc: int, where: str):
    if rc != DS4A_OK:
        raise Ds4aError(rc, where)


def _bf16(t, name):
    import torch
    if t is not None:
        if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
            raise TypeError(f"{name} must hold bfloat16 storage, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return t


def ds4a_strerror(code: int) -> str:
    return lib().ds4a_strerror(code).decode()


def ds4a_version() -> int:
    return lib().ds4a_version()


def ds4a_compress(cfg: LayerCfg, ca, za, bias_a, pool, *, entry_begin: int, entry_end: int,
                  cb=None, zb=None, bias_b=None, norm_g=None, tok_begin: int = 0, stream=None):
    """Streams [B, T_tok, c] (row r = token tok_begin + r) -> pool[b, i, :] for
    entry_begin <= i < entry_end.  cb None selects the single-stream HCA form;
    norm_g None stores the raw weighted sum (indexer keys)."""
    _bf16(ca, "ca"), _bf16(za, "za"), _bf16(cb, "cb"), _bf16(zb, "zb")
    B, T_tok, c = ca.shape
    rc = lib().ds4a_compress(ctypes.byref(cfg), B, T_tok, tok_begin, c, _ptr(ca), _ptr(cb), _ptr(za),
                             _ptr(zb), _ptr(bias_a), _ptr(bias_b), _ptr(norm_g), entry_begin,
                             entry_end, _ptr(pool), pool.stride(0), _stream(stream))
    _ok(rc, "ds4a_compress")


def ds4a_compress_state_bytes(cfg: LayerCfg, B: int, c: int, overlap: bool) -> int:
    return lib().ds4a_compress_state_bytes(ctypes.byref(cfg), B, c, int(bool(overlap)))


def ds4a_compress_append(cfg: LayerCfg, pos, ca, za, bias_a, state, pool, *, cb=None, zb=None, bias_b=None,
                         norm_g=None, stream=None):
    """New token rows ca/za (cb/zb) [B, c] at positions pos [B] into the
    ring state; entries that close go to pool [B, N_cap, c]."""
    _bf16(ca, "ca"), _bf16(za, "za"), _bf16(cb, "cb"), _bf16(zb, "zb")
    B, c = ca.shape
    rc = lib().ds4a_compress_append(ctypes.byref(cfg), B, c, _ptr(pos), _ptr(ca), _ptr(cb), _ptr(za), _ptr(zb),
                                    _ptr(bias_a), _ptr(bias_b), _ptr(norm_g), _ptr(state), pool.shape[1],
                                    _ptr(pool), pool.stride(0), _stream(stream))
    _ok(rc, "ds4a_compress_append")


def ds4a_kv_fp8_row_bytes(D: int, R: int) -> int:
    return lib().ds4a_kv_fp8_row_bytes(D, R)


def ds4a_quantize_kv_fp8(rows, R: int, out, *, stream=None):
    """bf16 K=V rows [n, D] -> FP8 / BF16 rows out [n, row_bytes] (uint8)."""
    _bf16(rows, "rows")
    n, D = rows.reshape(-1, rows.shape[-1]).shape
    rc = lib().ds4a_quantize_kv_fp8(n, D, R, _ptr(rows), D, _ptr(out), out.shape[-1], _stream(stream))
    _ok(rc, "ds4a_quantize_kv_fp8")


def ds4a_quantize_idx_fp4(keys, codes, scales, *, stream=None):
    """bf16 indexer keys [n, D] -> E2M1 codes [n, D/2] and E8M0 scales [n, D/32] (uint8)."""
    _bf16(keys, "keys")
    n, D = keys.reshape(-1, keys.shape[-1]).shape
    rc = lib().ds4a_quantize_idx_fp4(n, D, _ptr(keys), D, _ptr(codes), _ptr(scales), _stream(stream))
    _ok(rc, "ds4a_quantize_idx_fp4")


def ds4a_compress_append_mx(cfg: LayerCfg, pos, ca, za, bias_a, state, fmt: int, pool, *, scales=None, cb=None,
                            zb=None, bias_b=None, norm_g=None, stream=None):
    """ds4a_compress_append writing block-scaled entries: pool is uint8
    [B, N_cap, row_bytes] (FP8 K=V) or [B, N_cap, c/2] (FP4 keys, with
    scales [B, N_cap, c/32])."""
    _bf16(ca, "ca"), _bf16(za, "za"), _bf16(cb, "cb"), _bf16(zb, "zb")
    B, c = ca.shape
    rc = lib().ds4a_compress_append_mx(ctypes.byref(cfg), B, c, _ptr(pos), _ptr(ca), _ptr(cb), _ptr(za), _ptr(zb),
                                       _ptr(bias_a), _ptr(bias_b), _ptr(norm_g), _ptr(state), pool.shape[1], fmt,
                                       _ptr(pool), _ptr(scales), pool.shape[1], _stream(stream))
    _ok(rc, "ds4a_compress_append_mx")


def ds4a_index_topk_fp4(cfg: LayerCfg, q_pos, q_idx, w_idx, k_codes, k_scales, N_c: int, idx_out, ws, *,
                        score_out=None, stream=None):
    """ds4a_index_topk over FP4 keys: k_codes [B, >=N_c, D/2], k_scales [B, >=N_c, D/32]."""
    _bf16(q_idx, "q_idx"), _bf16(w_idx, "w_idx")
    B, T_q = q_pos.shape
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().ds4a_index_topk_fp4(ctypes.byref(cfg), B, T_q, _ptr(q_pos), _ptr(q_idx), _ptr(w_idx), _ptr(k_codes),
                                   _ptr(k_scales), 0 if k_codes is None else k_codes.shape[1], N_c, _ptr(idx_out),
                                   _ptr(score_out), _ptr(ws), ws_bytes, _stream(stream))
    _ok(rc, "ds4a_index_topk_fp4")


def ds4a_sparse_attend_fp8(cfg: LayerCfg, q_pos, q, q_norm_g, pool, N_c: int, idx, win, win_cap: int, sink, out,
                           ws=None, *, stream=None):
    """ds4a_sparse_attend over an FP8 / BF16 pool: uint8 [B, >=N_c, row_bytes]."""
    _bf16(q, "q")
    B, T_q = q_pos.shape
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().ds4a_sparse_attend_fp8(ctypes.byref(cfg), B, T_q, _ptr(q_pos), _ptr(q), _ptr(q_norm_g), _ptr(pool),
                                      0 if pool is None else pool.shape[1], N_c, _ptr(idx), _ptr(win), win_cap,
                                      0 if win is None else win.stride(0), _ptr(sink), _ptr(out), _ptr(ws), ws_bytes,
                                      _stream(stream))
    _ok(rc, "ds4a_sparse_attend_fp8")


def ds4a_hca_attend_fp8(cfg: LayerCfg, q_pos, q, q_norm_g, pool, N_c: int, win, win_cap: int, sink, out, ws=None,
                        *, stream=None):
    """ds4a_hca_attend over an FP8 / BF16 pool: uint8 [B, >=N_c, row_bytes]."""
    _bf16(q, "q")
    B, T_q = q_pos.shape
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().ds4a_hca_attend_fp8(ctypes.byref(cfg), B, T_q, _ptr(q_pos), _ptr(q), _ptr(q_norm_g), _ptr(pool),
                                   0 if pool is None else pool.shape[1], N_c, _ptr(win), win_cap,
                                   0 if win is None else win.stride(0), _ptr(sink), _ptr(out), _ptr(ws), ws_bytes,
                                   _stream(stream))
    _ok(rc, "ds4a_hca_attend_fp8")


def append_job(ca, za, bias_a, state, pool, *, cb=None, zb=None, bias_b=None, norm_g=None, fmt: int = 0,
               scales=None) -> AppendJob:
    """One job of ds4a_compress_append_jobs (pool: bf16 [B, N_cap, c], or the
    block-scaled uint8 rows of fmt)."""
    _bf16(ca, "ca"), _bf16(za, "za"), _bf16(cb, "cb"), _bf16(zb, "zb")
    bstride = pool.stride(0) if fmt == 0 else pool.shape[1]
    return AppendJob(ca.shape[1], fmt, _ptr(ca), _ptr(cb), _ptr(za), _ptr(zb), _ptr(bias_a), _ptr(bias_b),
                     _ptr(norm_g), _ptr(state), _ptr(pool), _ptr(scales), bstride)


def ds4a_compress_append_jobs(cfg: LayerCfg, pos, N_cap: int, jobs, *, stream=None):
    """Up to two compressors of one layer, one decode step, one launch when both are CSA-shaped."""
    arr = (AppendJob * len(jobs))(*jobs)
    rc = lib().ds4a_compress_append_jobs(ctypes.byref(cfg), pos.shape[0], _ptr(pos), N_cap, arr, len(jobs),
                                         _stream(stream))
    _ok(rc, "ds4a_compress_append_jobs")


def ds4a_index_topk_workspace(cfg: LayerCfg, B: int, T_q: int, N_c: int) -> int:
    return lib().ds4a_index_topk_workspace(ctypes.byref(cfg), B, T_q, N_c)


def ds4a_index_topk(cfg: LayerCfg, q_pos, q_idx, w_idx, k_idx, N_c: int, idx_out, ws, *,
                    score_out=None, stream=None):
    """q_idx [B,T_q,H_I,D_I], w_idx [B,T_q,H_I], k_idx [B,>=N_c,D_I] ->
    idx_out int32 [B,T_q,k] (ascending, -1 padded)."""
    _bf16(q_idx, "q_idx"), _bf16(w_idx, "w_idx")
    B, T_q = q_pos.shape
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().ds4a_index_topk(ctypes.byref(cfg), B, T_q, _ptr(q_pos), _ptr(q_idx), _ptr(w_idx),
                               _ptr(k_idx), 0 if k_idx is None else k_idx.stride(0), N_c,
                               _ptr(idx_out), _ptr(score_out), _ptr(ws), ws_bytes, _stream(stream))
    _ok(rc, "ds4a_index_topk")


def ds4a_index_topk_noalloc(cfg: LayerCfg, q_pos, q_idx, w_idx, k_idx, N_c: int, idx_out, *,
                            score_out=None, stream=None):
    """ds4a_index_topk without a workspace argument: the library's own
    fixed device scratch (up to 2**21 scores) serves every call, for
    callers that cannot allocate device memory."""
    _bf16(q_idx, "q_idx"), _bf16(w_idx, "w_idx")
    B, T_q = q_pos.shape
    rc = lib().ds4a_index_topk_noalloc(ctypes.byref(cfg), B, T_q, _ptr(q_pos), _ptr(q_idx), _ptr(w_idx),
                                       _ptr(k_idx), 0 if k_idx is None else k_idx.stride(0), N_c,
                                       _ptr(idx_out), _ptr(score_out), _stream(stream))
    _ok(rc, "ds4a_index_topk_noalloc")


def ds4a_attend_workspace(cfg: LayerCfg, B: int, T_q: int, N_c: int, sparse: bool) -> int:
    return lib().ds4a_attend_workspace(ctypes.byref(cfg), B, T_q, N_c, int(bool(sparse)))


def ds4a_sparse_attend(cfg: LayerCfg, q_pos, q, q_norm_g, pool, N_c: int, idx, win, win_cap: int,
                       sink, out, ws=None, *, stream=None):
    _bf16(q, "q")
    B, T_q = q_pos.shape
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().ds4a_sparse_attend(ctypes.byref(cfg), B, T_q, _ptr(q_pos), _ptr(q), _ptr(q_norm_g),
                                  _ptr(pool), 0 if pool is None else pool.stride(0), N_c, _ptr(idx),
                                  _ptr(win), win_cap, 0 if win is None else win.stride(0), _ptr(sink),
                                  _ptr(out), _ptr(ws), ws_bytes, _stream(stream))
    _ok(rc, "ds4a_sparse_attend")


def ds4a_hca_attend(cfg: LayerCfg, q_pos, q, q_norm_g, pool, N_c: int, win, win_cap: int, sink, out,
                    ws=None, *, stream=None):
    _bf16(q, "q")
    B, T_q = q_pos.shape
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().ds4a_hca_attend(ctypes.byref(cfg), B, T_q, _ptr(q_pos), _ptr(q), _ptr(q_norm_g),
                               _ptr(pool), 0 if pool is None else pool.stride(0), N_c, _ptr(win),
                               win_cap, 0 if win is None else win.stride(0), _ptr(sink), _ptr(out),
                               _ptr(ws), ws_bytes, _stream(stream))
    _ok(rc, "ds4a_hca_attend")


def ds4a_out_proj_workspace(cfg: OprojCfg, M: int) -> int:
    return lib().ds4a_out_proj_workspace(ctypes.byref(cfg), M)


def ds4a_out_proj(cfg: OprojCfg, o, w_a, w_b, mid, y, ws=None, *, stream=None):
    """o [M, H, D] -> mid [M, g*r] and y [M, hidden] (grouped projection)."""
    _bf16(o, "o"), _bf16(w_a, "w_a"), _bf16(w_b, "w_b")
    M = o.shape[0]
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = lib().ds4a_out_proj(ctypes.byref(cfg), M, _ptr(o), _ptr(w_a), _ptr(w_b), _ptr(mid), _ptr(y), _ptr(ws),
                             ws_bytes, _stream(stream))
    _ok(rc, "ds4a_out_proj")


_gpus = None


def _here() -> int:
    """The current device, where the paged and MXFP4 calls run and their
    tensors must be (-1 without one)."""
    import torch
    global _gpus
    if _gpus is None:
        _gpus = torch.cuda.is_available()
    return torch.cuda.current_device() if _gpus else -1


def _rows(t, dtype, name, B=None, dev=None):
    """A matrix of one row per sequence whose rows are contiguous: (width, stride)."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or (B is not None and t.shape[0] != B):
        raise ValueError(f"{name} must be [{'B' if B is None else B}, n] with contiguous rows")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} must be on the current device")
    return t.shape[1], (t.stride(0) if t.shape[0] > 1 else max(1, t.shape[1]))


def _flat(t, dtype, n, name, dev, least=False):
    """Address of a contiguous tensor of n elements (least: or more) on the current device."""
    if t.get_device() != dev or not t.is_contiguous() or (t.numel() < n if least else t.numel() != n) or \
            t.dtype != dtype:
        raise ValueError(f"{name} must be contiguous {dtype} of {n} elements on the current device")
    return t.data_ptr()


def _work(ws, dev):
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be contiguous and on the current device")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _kv_of(kv, B, dev):
    if kv.dev is not None and kv.dev != dev:
        raise ValueError("pages and table must be on the current device")
    if kv.rows is not None and kv.rows < B:
        raise ValueError(f"the page table must have {B} rows")


def paged_kv(pages, table, page_size: int, *, fmt: int = 0) -> PagedKv:
    """The paged cache of ds4a_paged_*: pages [n_pages, page_size, D] bf16, or
    uint8 [n_pages, page_size, row_bytes] with fmt DS4A_MX_KV_FP8; table int32
    [B, max_pages] (rows may lie apart).  It keeps both tensors alive."""
    import torch
    if fmt == 0:
        _bf16(pages, "pages")
    elif pages.dtype != torch.uint8 or not pages.is_contiguous():
        raise ValueError("pages of block-scaled rows must be contiguous uint8")
    if pages.dim() != 3 or pages.shape[1] != page_size:
        raise ValueError("pages must be [n_pages, page_size, row]")
    width, stride = _rows(table, torch.int32, "table")
    if table.get_device() != pages.get_device():
        raise ValueError("pages and table must be on one device")
    kv = PagedKv(pages.data_ptr(), table.data_ptr(), stride, fmt, pages.shape[0], page_size, width)
    kv.held, kv.dev, kv.rows, kv.row_size = (pages, table), pages.get_device(), table.shape[0], pages.shape[2]
    return kv


def _row_of(cfg, kv):
    if kv.row_size is None:
        return
    want = cfg.head_dim if kv.format == 0 else ds4a_kv_fp8_row_bytes(cfg.head_dim, cfg.rope_dim)
    if kv.row_size != want:
        raise ValueError(f"the pages' rows must have {want} elements")


def ds4a_paged_attend_workspace(cfg: LayerCfg, kv: PagedKv, B: int, sparse: bool = False, weights: bool = False) -> int:
    return lib().ds4a_paged_attend_workspace(ctypes.byref(cfg), ctypes.byref(kv), B, int(bool(sparse)),
                                             int(bool(weights)))


def ds4a_paged_attend(cfg: LayerCfg, kv: PagedKv, q_pos, q, q_norm_g, win, win_cap: int, sink, out, ws, *, drop=None,
                      idx=None, weights=None, stream=None):
    """One new token per sequence: q, out [B, H, D], q_pos [B]; idx int32
    [B, k] selects slots; weights bf16 [B, n] receives each slot's attention."""
    import torch
    bf, f32, i32, dev = torch.bfloat16, torch.float32, torch.int32, _here()
    B, H, D = q.shape[0], cfg.n_heads, cfg.head_dim
    _kv_of(kv, B, dev), _row_of(cfg, kv)
    w_len = w_stride = 0
    if weights is not None:
        w_len, w_stride = _rows(weights, bf, "weights", B, dev)
    if win is not None and (win.dtype != bf or win.get_device() != dev or win.dim() != 3 or win.shape[0] != B or
                            win.shape[1] < win_cap or win.shape[2] != D or win.stride(2) != 1 or win.stride(1) != D):
        raise ValueError("win must be bfloat16 [B, win_cap, head_dim] on the current device, its rows contiguous")
    n = B * H * D
    if not (q.get_device() == q_pos.get_device() == out.get_device() == sink.get_device() == q_norm_g.get_device() == dev
            and q.numel() == out.numel() == n and q_pos.numel() == B and sink.numel() == H and q_norm_g.numel() == D
            and q.dtype == out.dtype == bf and q_pos.dtype == i32 and sink.dtype == q_norm_g.dtype == f32
            and q.is_contiguous() and out.is_contiguous() and q_pos.is_contiguous() and sink.is_contiguous()
            and q_norm_g.is_contiguous()):  # (which one)
        _flat(q_pos, i32, B, "q_pos", dev), _flat(q, bf, n, "q", dev), _flat(q_norm_g, f32, D, "q_norm_g", dev)
        _flat(sink, f32, H, "sink", dev), _flat(out, bf, n, "out", dev)
    p_ws, n_ws = _work(ws, dev)
    rc = lib().ds4a_paged_attend(cfg, kv, B, q_pos.data_ptr(), q.data_ptr(), q_norm_g.data_ptr(),
                                 None if drop is None else _flat(drop, i32, B, "drop", dev),
                                 None if idx is None else _flat(idx, i32, B * cfg.topk, "idx", dev), _ptr(win), win_cap,
                                 0 if win is None else win.stride(0), sink.data_ptr(), out.data_ptr(), _ptr(weights),
                                 w_len, w_stride, p_ws, n_ws, _stream(stream))
    _ok(rc, "ds4a_paged_attend")


def ds4a_paged_append(cfg: LayerCfg, kv: PagedKv, pos, ca, za, bias_a, state, *, drop=None, cb=None, zb=None,
                      bias_b=None, norm_g=None, stream=None):
    """ds4a_compress_append of new rows [B, D] into a paged cache (slot = entry - drop)."""
    import torch
    bf, f32, i32, dev = torch.bfloat16, torch.float32, torch.int32, _here()
    B, c = ca.shape
    if c != cfg.head_dim:
        raise ValueError("a paged cache holds K=V entries of head_dim channels")
    _kv_of(kv, B, dev), _row_of(cfg, kv)
    some = lambda t, dtype, n, name: None if t is None else _flat(t, dtype, n, name, dev)  # noqa: E731
    need = ds4a_compress_state_bytes(cfg, B, c, cb is not None)
    if state.get_device() != dev or not state.is_contiguous() or state.numel() * state.element_size() < need:
        raise ValueError(f"state must be contiguous, of {need} bytes and on the current device")
    rc = lib().ds4a_paged_append(cfg, kv, B, _flat(pos, i32, B, "pos", dev), some(drop, i32, B, "drop"),
                                 _flat(ca, bf, B * c, "ca", dev), some(cb, bf, B * c, "cb"),
                                 _flat(za, bf, B * c, "za", dev), some(zb, bf, B * c, "zb"),
                                 _flat(bias_a, f32, cfg.ratio * c, "bias_a", dev),
                                 some(bias_b, f32, cfg.ratio * c, "bias_b"), some(norm_g, f32, c, "norm_g"),
                                 state.data_ptr(), _stream(stream))
    _ok(rc, "ds4a_paged_append")


def ds4a_paged_evict_workspace(kv: PagedKv, B: int) -> int:
    return lib().ds4a_paged_evict_workspace(ctypes.byref(kv), B)


def ds4a_paged_evict(cfg: LayerCfg, kv: PagedKv, q_pos, budget: int, recent: int, acc, entry, drop, ws, *,
                     weights=None, stream=None):
    """acc (float32) += weights (bf16), entry (int32), all [B, n_slots]; caches
    of more than budget entries are cut to it in place, drop [B] follows."""
    import torch
    i32, dev, B = torch.int32, _here(), q_pos.shape[0]
    _kv_of(kv, B, dev), _row_of(cfg, kv)
    if not (q_pos.get_device() == drop.get_device() == acc.get_device() == entry.get_device() == dev
            and q_pos.dtype == drop.dtype == entry.dtype == i32 and acc.dtype == torch.float32
            and q_pos.numel() == drop.numel() == B and acc.dim() == 2 and acc.shape == entry.shape and acc.shape[0] == B
            and q_pos.is_contiguous() and drop.is_contiguous() and acc.is_contiguous() and entry.is_contiguous()):
        _flat(q_pos, i32, B, "q_pos", dev), _flat(drop, i32, B, "drop", dev)
        n, stride = _rows(acc, torch.float32, "acc", B, dev)  # (rows may lie apart)
        if _rows(entry, i32, "entry", B, dev) != (n, stride):
            raise ValueError("acc and entry must have the same shape and stride")
    else:
        n = stride = acc.shape[1]
    w_stride = 0
    if weights is not None:
        w_len, w_stride = _rows(weights, torch.bfloat16, "weights", B, dev)
        if w_len < n:
            raise ValueError("weights must cover the slots of acc")
    p_ws, n_ws = _work(ws, dev)
    rc = lib().ds4a_paged_evict(cfg, kv, B, q_pos.data_ptr(), _ptr(weights), w_stride, budget, recent, n,
                                acc.data_ptr(), entry.data_ptr(), stride, drop.data_ptr(), p_ws, n_ws,
                                _stream(stream))
    _ok(rc, "ds4a_paged_evict")


def ds4a_mxfp4_scale_bytes(rows: int, K: int) -> int:
    return lib().ds4a_mxfp4_scale_bytes(rows, K)


def ds4a_quantize_mxfp4(rows, codes, scales, *, stream=None):
    """bf16 rows [n, K] (rows may lie apart) -> E2M1 codes [n, K/2] and E8M0
    scales in the products' order (ds4a_mxfp4_scale_bytes(n, K) bytes)."""
    import torch
    u8, dev, n = torch.uint8, _here(), rows.shape[0]
    K, stride = _rows(rows, torch.bfloat16, "rows", n, dev)
    rc = lib().ds4a_quantize_mxfp4(n, K, rows.data_ptr(), stride, _flat(codes, u8, n * K // 2, "codes", dev, True),
                                   _flat(scales, u8, ds4a_mxfp4_scale_bytes(n, K), "scales", dev, True),
                                   _stream(stream))
    _ok(rc, "ds4a_quantize_mxfp4")


def ds4a_out_proj_mxfp4_workspace(cfg: OprojCfg, M: int) -> int:
    return lib().ds4a_out_proj_mxfp4_workspace(ctypes.byref(cfg), M)


def ds4a_out_proj_mxfp4(cfg: OprojCfg, o, wa_codes, wa_scales, wb_codes, wb_scales, y, ws, *, stream=None):
    """o [M, H, D] -> y [M, hidden], weights and activations in MXFP4."""
    import torch
    bf, u8, dev, M = torch.bfloat16, torch.uint8, _here(), o.shape[0]
    n1, k1 = cfg.n_groups * cfg.group_rank, cfg.n_heads // max(1, cfg.n_groups) * cfg.head_dim
    p_ws, n_ws = _work(ws, dev)
    rc = lib().ds4a_out_proj_mxfp4(cfg, M, _flat(o, bf, M * cfg.n_heads * cfg.head_dim, "o", dev),
                                   _flat(wa_codes, u8, n1 * k1 // 2, "wa_codes", dev, True),
                                   _flat(wa_scales, u8, n1 * k1 // 32, "wa_scales", dev, True),
                                   _flat(wb_codes, u8, cfg.hidden * n1 // 2, "wb_codes", dev, True),
                                   _flat(wb_scales, u8, cfg.hidden * n1 // 32, "wb_scales", dev, True),
                                   _flat(y, bf, M * cfg.hidden, "y", dev), p_ws, n_ws, _stream(stream))
    _ok(rc, "ds4a_out_proj_mxfp4")


def ds4a_check(stream=None) -> tuple[int, int]:
    """Synchronise and read/clear the device error word -> (code, bits)."""
    bits = ctypes.c_uint32(0)
    rc = lib().ds4a_check(_stream(stream), ctypes.byref(bits))
    return rc, bits.value


def ds4a_selftest_wait_timeout(limit_cycles: int, status_out, *, stream=None):
    """One block waits on a barrier nothing arrives at, with a bound of
    limit_cycles SM cycles; status_out (int32 device tensor) gets 2 when the
    bound ran out.  ds4a_check then reports DS4A_ETIMEOUT."""
    rc = lib().ds4a_selftest_wait_timeout(int(limit_cycles), _ptr(status_out), _stream(stream))
    _ok(rc, "ds4a_selftest_wait_timeout")


def ds4a_trace_enable(on: bool = True):
    lib().ds4a_trace_enable(int(bool(on)))


def ds4a_trace_read(cap: int = 65536) -> list[tuple[str, float]]:
    names = (ctypes.c_char_p * cap)()
    ms = (ctypes.c_float * cap)()
    n = lib().ds4a_trace_read(names, ms, cap)
    if n < 0:
        raise Ds4aError(-n, "ds4a_trace_read")
    return [(names[i].decode(), ms[i]) for i in range(min(n, cap))]
