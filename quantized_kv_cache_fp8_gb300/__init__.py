"""Quantized MLA KV cache on GB300 — Python binding of the C ABI ``libkvq``.

Each function here has the name of the C entry point it wraps and only marshals its
arguments (torch tensors -> device pointers, the current CUDA stream): every step of
the path runs in the CUDA kernels of ``libkvq.so``.  There is no fallback: if the
library is missing or fails to load, importing :func:`lib` raises.

Layouts and semantics are documented once, in ``include/kvq.h``.
"""
from __future__ import annotations

import ctypes as C
import os
import threading

__all__ = [
    "KvqError", "lib", "kvq_version", "kvq_tq4_codebook", "kvq_set_fault",
    "kvq_encode_fp8", "kvq_encode_tq4", "kvq_append_q4", "kvq_project_append_q4",
    "kvq_gather_q4", "kvq_gather_rows", "WEIGHT_F32", "WEIGHT_BF16",
    "kvq_mla_decode", "kvq_mla_decode_workspace", "kvq_mla_decode_noalloc", "kvq_mla_decode_kernel",
    "MlaCache",
    "MlaProblem", "Q4Problem", "make_q4_problem", "kvq_q4_decode", "kvq_q4_decode_workspace",
    "FMT_FP8", "FMT_TQ4", "FMT_Q4_0", "FMT_TQ6", "FMT_TQ3", "TQ_FMT", "kvq_encode_tq", "kvq_encode_mla",
    "kvq_tq_codebook", "DEV_BAD_INDEX", "DEV_BAD_PAGE", "DEV_TIMEOUT",
    "DEV_BAD_FORMAT", "DEV_NO_PAGE",
    "PagePlan", "make_page_plan", "kvq_resize_pages", "kvq_append_mla",
    "TreeProblem", "make_tree_problem", "kvq_mla_tree_decode", "kvq_mla_tree_decode_workspace",
    "kvq_mla_tree_decode_kernel", "TREE_PACKED", "TREE_PER_QUERY",
    "AcceptDesc", "make_accept", "kvq_accept_mla",
    "Kv8Cache", "kvq_append_kv8", "Kv8Problem", "make_kv8_problem", "kvq_kv8_decode", "kvq_kv8_decode_workspace",
    "BeamProblem", "make_beam_problem", "kvq_beam_select", "kvq_beam_select_workspace", "DEV_BAD_VALUE",
    "ForkPlan", "make_fork_plan", "kvq_fork_pages", "kvq_fork_pages_workspace",
    "CompactPlan", "make_compact_plan", "kvq_compact_pages", "kvq_compact_pages_workspace",
    "PageCopy", "make_page_copy", "kvq_copy_pages",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libkvq.so")

FMT_FP8, FMT_TQ4, FMT_Q4_0, FMT_TQ6, FMT_TQ3 = 1, 2, 3, 4, 5
WEIGHT_F32, WEIGHT_BF16 = 0, 1
TQ_FMT = {3: FMT_TQ3, 4: FMT_TQ4, 6: FMT_TQ6}     # rotated tier of each code width
IMPL_AUTO, IMPL_SIMT, IMPL_TC, IMPL_MMA, IMPL_TC16, IMPL_TCF8 = 0, 1, 2, 3, 4, 5
IMPL_BY_FMT = 6   # kvq_mla_decode_kernel only: fp8 sequences on IMPL_TCF8, TQ4 ones on IMPL_TC
TREE_PACKED, TREE_PER_QUERY = 1, 2       # forms of kvq_mla_tree_decode
DEV_BAD_INDEX, DEV_BAD_PAGE, DEV_TIMEOUT, DEV_BAD_FORMAT, DEV_NO_PAGE = 1, 2, 4, 8, 16
DEV_BAD_VALUE = 32
STATUS = {0: "KVQ_OK", 1: "KVQ_EINVAL", 2: "KVQ_ENOTPOW2", 3: "KVQ_EFORMAT", 4: "KVQ_EALIGN",
          5: "KVQ_EWORKSPACE", 6: "KVQ_ECUDA", 7: "KVQ_EFAULT_INJECTED", 8: "KVQ_EMISMATCH",
          9: "KVQ_EIO"}

# every symbol include/kvq.h declares
EXPORTS = ["kvq_version", "kvq_status_string", "kvq_last_error", "kvq_set_fault",
           "kvq_set_wait_limit_ns",
           "kvq_tq4_codebook", "kvq_tq_codebook", "kvq_encode_fp8", "kvq_encode_tq4",
           "kvq_encode_tq", "kvq_encode_mla", "kvq_append_q4", "kvq_project_append_q4",
           "kvq_gather", "kvq_mla_decode_workspace", "kvq_mla_decode_kernel", "kvq_mla_decode",
           "kvq_mla_decode_noalloc", "kvq_q4_decode_workspace", "kvq_q4_decode",
           "kvq_cache_probe", "kvq_cache_save", "kvq_cache_save_f32", "kvq_cache_append",
           "kvq_cache_load_workspace", "kvq_cache_load",
           "kvq_resize_pages", "kvq_append_mla", "kvq_mla_tree_decode_kernel",
           "kvq_mla_tree_decode_workspace", "kvq_mla_tree_decode", "kvq_accept_mla",
           "kvq_append_kv8", "kvq_kv8_decode_workspace", "kvq_kv8_decode",
           "kvq_beam_select_workspace", "kvq_beam_select", "kvq_fork_pages_workspace", "kvq_fork_pages",
           "kvq_compact_pages_workspace", "kvq_compact_pages", "kvq_copy_pages"]


class KvqError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status


_p = C.c_void_p
_i32, _i64, _f32 = C.c_int32, C.c_int64, C.c_float


class MlaCache(C.Structure):
    _fields_ = [("lat", _p), ("lat_scale", _p), ("rope", _p), ("rope_scale", _p),
                ("n_rows", _i64)]


class GatherDesc(C.Structure):
    _fields_ = [("format", _i32),
                ("q4_pool", _p), ("n_seq", _i32), ("n_tok", _i32), ("n_heads", _i32),
                ("head_dim", _i32), ("pos0", _p), ("n_cells", _i64), ("q4_out", _p),
                ("page_table", _p), ("max_pages", _i32), ("page_size", _i32),
                ("mla_src", MlaCache), ("mla_src_rows", _i64), ("idx", _p), ("n_idx", _i64),
                ("dst_lat", _p), ("dst_lat_scale", _p), ("dst_rope", _p),
                ("dst_rope_scale", _p), ("dev_status", _p)]


class MlaProblem(C.Structure):
    _fields_ = [("n_seq", _i32), ("n_q", _i32), ("n_heads", _i32), ("d_lat", _i32),
                ("d_rope", _i32), ("causal", _i32), ("max_seq_len", _i32),
                ("seq_len", _p), ("seq_fmt", _p), ("fmt", _i32), ("block_table", _p),
                ("max_pages", _i32), ("page_size", _i32), ("seq_stride_rows", _i64),
                ("fp8", MlaCache), ("tq4", MlaCache), ("tq4_signs", _p),
                ("q_lat", _p), ("q_rope", _p), ("idx", _p), ("top_k", _i32),
                ("sm_scale", _f32), ("split_rows", _i32), ("impl", _i32),
                ("overlap_prior", _i32)]


class Q4Problem(C.Structure):
    _fields_ = [("n_seq", _i32), ("n_qh", _i32), ("n_kv", _i32), ("head_dim", _i32),
                ("seq_len", _p), ("max_seq_len", _i32), ("page_table", _p),
                ("max_pages", _i32), ("page_size", _i32), ("n_cells", _i64),
                ("k_pool", _p), ("v_pool", _p), ("q", _p), ("gate", _p),
                ("sm_scale", _f32), ("split_rows", _i32)]


class PagePlan(C.Structure):
    _fields_ = [("n_seq", _i32), ("max_pages", _i32), ("page_size", _i32), ("n_pages", _i32),
                ("max_tokens", _i32), ("keep_len", _p), ("n_new", _p), ("block_table", _p),
                ("n_held", _p), ("free_list", _p), ("n_free", _p), ("seq_len", _p),
                ("tok_start", _p), ("slot_map", _p), ("tok_pos", _p)]


class TreeProblem(C.Structure):
    _fields_ = [("n_seq", _i32), ("n_q", _i32), ("n_heads", _i32), ("d_lat", _i32),
                ("d_rope", _i32), ("fmt", _i32), ("max_seq_len", _i32), ("seq_len", _p),
                ("n_node", _p), ("mask", _p), ("block_table", _p), ("max_pages", _i32),
                ("page_size", _i32), ("seq_stride_rows", _i64), ("cache", MlaCache),
                ("signs", _p), ("q_lat", _p), ("q_rope", _p), ("ldq_lat", _i64),
                ("ldq_rope", _i64), ("sm_scale", _f32), ("impl", _i32)]


class AcceptDesc(C.Structure):
    _fields_ = [("n_seq", _i32), ("n_q", _i32), ("fmt", _i32), ("seq_len", _p), ("n_node", _p),
                ("path", _p), ("n_acc", _p), ("new_len", _p), ("block_table", _p),
                ("max_pages", _i32), ("page_size", _i32), ("seq_stride_rows", _i64),
                ("cache", MlaCache)]


class Kv8Cache(C.Structure):
    _fields_ = [("k", _p), ("k_scale", _p), ("v", _p), ("v_scale", _p), ("n_rows", _i64), ("n_kv", _i32),
                ("head_dim", _i32)]


class Kv8Problem(C.Structure):
    _fields_ = [("n_seq", _i32), ("n_qh", _i32), ("max_seq_len", _i32), ("window", _i32), ("seq_len", _p),
                ("block_table", _p), ("max_pages", _i32), ("page_size", _i32), ("seq_stride_rows", _i64),
                ("cache", Kv8Cache), ("q", _p), ("ldq", _i64), ("sm_scale", _f32)]


class BeamProblem(C.Structure):
    _fields_ = [("n_req", _i32), ("n_beam", _i32), ("vocab", _i32), ("n_out", _i32), ("x_type", _i32), ("eos", _i32),
                ("pad", _i32), ("logits", _p), ("ld", _i64), ("score", _p), ("finished", _p), ("out_score", _p),
                ("out_token", _p), ("out_parent", _p), ("out_finished", _p)]


class ForkPlan(C.Structure):
    _fields_ = [("n_seq", _i32), ("max_pages", _i32), ("page_size", _i32), ("n_pages", _i32), ("parent", _p),
                ("keep_len", _p), ("block_table", _p), ("n_held", _p), ("free_list", _p), ("n_free", _p),
                ("seq_len", _p), ("copy_src", _p), ("copy_dst", _p), ("copy_rows", _p), ("n_copy", _p)]


class CompactPlan(C.Structure):
    _fields_ = [("n_seq", _i32), ("max_pages", _i32), ("page_size", _i32), ("n_pages", _i32), ("max_copy", _i32),
                ("block_table", _p), ("n_held", _p), ("new_table", _p), ("free_list", _p), ("n_free", _p),
                ("n_used", _p), ("copy_src", _p), ("copy_dst", _p), ("copy_rows", _p), ("n_copy", _p)]


class Plane(C.Structure):
    _fields_ = [("base", _p), ("row_bytes", _i64), ("n_rows", _i64), ("n_outer", _i64), ("outer_stride", _i64)]


class PageCopy(C.Structure):
    _fields_ = [("planes", C.POINTER(Plane)), ("n_planes", _i32), ("page_size", _i32), ("max_copy", _i32),
                ("copy_src", _p), ("copy_dst", _p), ("copy_rows", _p), ("n_copy", _p)]


class CacheInfo(C.Structure):
    _fields_ = [("format", _i32), ("codec", _i32), ("bits", _i32), ("d_lat", _i32),
                ("d_rope", _i32), ("n_rows", _i64), ("record_bytes", _i64),
                ("trailing_bytes", _i64)]


_lock = threading.Lock()
_lib = None


def lib() -> C.CDLL:
    """Load libkvq.so (built by ``__graft_entry__.build()``); raise if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"libkvq.so not built ({LIB_PATH}); run __graft_entry__.build()")
            L = C.CDLL(LIB_PATH)
            _declare(L)
            _lib = L
    return _lib


def _declare(L):
    L.kvq_version.restype = C.c_int
    L.kvq_status_string.restype = C.c_char_p
    L.kvq_status_string.argtypes = [C.c_int]
    L.kvq_last_error.restype = C.c_char_p
    L.kvq_set_fault.restype = C.c_int
    L.kvq_set_fault.argtypes = [C.c_char_p]
    L.kvq_set_wait_limit_ns.restype = C.c_int
    L.kvq_set_wait_limit_ns.argtypes = [C.c_uint64]
    L.kvq_tq4_codebook.restype = C.c_int
    L.kvq_tq4_codebook.argtypes = [_p, _p]
    L.kvq_encode_fp8.restype = C.c_int
    L.kvq_encode_fp8.argtypes = [_p, _i64, C.c_int, _i64, _p, _i64, _p, _p]
    L.kvq_tq_codebook.restype = C.c_int
    L.kvq_tq_codebook.argtypes = [C.c_int, _p, _p]
    L.kvq_encode_tq.restype = C.c_int
    L.kvq_encode_tq.argtypes = [_p, _i64, C.c_int, _i64, C.c_int, _p, _p, _i64, _p, _p]
    L.kvq_encode_mla.restype = C.c_int
    L.kvq_encode_mla.argtypes = [_p, _i64, _p, _i64, _i64, C.c_int, _p, _p, _i64, _p, _p, _i64, _p, _p]
    L.kvq_encode_tq4.restype = C.c_int
    L.kvq_encode_tq4.argtypes = [_p, _i64, C.c_int, _i64, _p, _p, _i64, _p, _p]
    L.kvq_append_q4.restype = C.c_int
    L.kvq_append_q4.argtypes = [_p, _p, C.c_int, _p, C.c_int, C.c_int, C.c_int, _p, C.c_int,
                                C.c_int, _i64, _p, _p, _p, _p]
    L.kvq_project_append_q4.restype = C.c_int
    L.kvq_project_append_q4.argtypes = [_p, C.c_int, _p, C.c_int, C.c_int, _p, _p, C.c_int,
                                        C.c_int, C.c_int, _p, C.c_int, C.c_int, _i64, _p, _p,
                                        _p, _p]
    L.kvq_gather.restype = C.c_int
    L.kvq_gather.argtypes = [C.POINTER(GatherDesc), _p]
    L.kvq_mla_decode_workspace.restype = C.c_size_t
    L.kvq_mla_decode_workspace.argtypes = [C.POINTER(MlaProblem)]
    L.kvq_mla_decode_kernel.restype = C.c_int
    L.kvq_mla_decode_kernel.argtypes = [C.POINTER(MlaProblem)]
    L.kvq_mla_decode.restype = C.c_int
    L.kvq_mla_decode.argtypes = [C.POINTER(MlaProblem), _p, _p, _p, C.c_size_t, _p, _p]
    L.kvq_mla_decode_noalloc.restype = C.c_int
    L.kvq_mla_decode_noalloc.argtypes = [C.POINTER(MlaProblem), _p, _p, _p, _p]
    L.kvq_cache_probe.restype = C.c_int
    L.kvq_cache_probe.argtypes = [C.c_char_p, C.POINTER(CacheInfo)]
    L.kvq_cache_save.restype = C.c_int
    L.kvq_cache_save.argtypes = [C.c_char_p, C.c_int32, C.POINTER(MlaCache), _p, _i64, _p]
    L.kvq_cache_save_f32.restype = C.c_int
    L.kvq_cache_save_f32.argtypes = [C.c_char_p, _p, _p, _i64, _p]
    L.kvq_cache_append.restype = C.c_int
    L.kvq_cache_append.argtypes = [C.c_char_p, C.c_int32, C.POINTER(MlaCache), _i64, _i64, _p]
    L.kvq_cache_load_workspace.restype = C.c_size_t
    L.kvq_cache_load_workspace.argtypes = []
    L.kvq_cache_load.restype = C.c_int
    L.kvq_cache_load.argtypes = [C.c_char_p, C.c_int32, _p, C.POINTER(MlaCache), _i64,
                                 C.POINTER(_i64), _p, C.c_size_t, _p]
    L.kvq_resize_pages.restype = C.c_int
    L.kvq_resize_pages.argtypes = [C.POINTER(PagePlan), _p, _p]
    L.kvq_append_mla.restype = C.c_int
    L.kvq_append_mla.argtypes = [_p, _i64, _p, _i64, C.c_int, _i64, _p, C.c_int, _p, C.POINTER(MlaCache), _p, _p]
    L.kvq_mla_tree_decode_kernel.restype = C.c_int
    L.kvq_mla_tree_decode_kernel.argtypes = [C.POINTER(TreeProblem)]
    L.kvq_mla_tree_decode_workspace.restype = C.c_size_t
    L.kvq_mla_tree_decode_workspace.argtypes = [C.POINTER(TreeProblem)]
    L.kvq_mla_tree_decode.restype = C.c_int
    L.kvq_mla_tree_decode.argtypes = [C.POINTER(TreeProblem), _p, _p, _p, C.c_size_t, _p, _p]
    L.kvq_accept_mla.restype = C.c_int
    L.kvq_accept_mla.argtypes = [C.POINTER(AcceptDesc), _p, _p]
    L.kvq_append_kv8.restype = C.c_int
    L.kvq_append_kv8.argtypes = [_p, _i64, _i64, _p, _i64, _i64, C.c_int, _i64, _p, C.POINTER(Kv8Cache), _p, _p]
    L.kvq_kv8_decode_workspace.restype = C.c_size_t
    L.kvq_kv8_decode_workspace.argtypes = [C.POINTER(Kv8Problem)]
    L.kvq_kv8_decode.restype = C.c_int
    L.kvq_kv8_decode.argtypes = [C.POINTER(Kv8Problem), _p, _p, _p, C.c_size_t, _p, _p]
    for name, plan in (("kvq_beam_select", BeamProblem), ("kvq_fork_pages", ForkPlan), ("kvq_compact_pages", CompactPlan)):
        f, w = getattr(L, name), getattr(L, name + "_workspace")
        f.restype, f.argtypes = C.c_int, [C.POINTER(plan), _p, C.c_size_t, _p, _p]
        w.restype, w.argtypes = C.c_size_t, [C.POINTER(plan)]
    L.kvq_copy_pages.restype = C.c_int
    L.kvq_copy_pages.argtypes = [C.POINTER(PageCopy), _p, _p]
    L.kvq_q4_decode_workspace.restype = C.c_size_t
    L.kvq_q4_decode_workspace.argtypes = [C.POINTER(Q4Problem)]
    L.kvq_q4_decode.restype = C.c_int
    L.kvq_q4_decode.argtypes = [C.POINTER(Q4Problem), _p, _p, _p, C.c_size_t, _p, _p]


def _check(status: int):
    if status != 0:
        raise KvqError(status, lib().kvq_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)     # the handle without a Stream object
    if raw is not None:
        return raw(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


# ---------------------------------------------------------------------------------------

def kvq_version() -> int:
    return lib().kvq_version()


def kvq_set_fault(spec: str | None) -> None:
    _check(lib().kvq_set_fault(None if spec is None else spec.encode()))


def kvq_tq4_codebook():
    import numpy as np
    cb = np.empty(16, np.float32)
    thr = np.empty(15, np.float32)
    _check(lib().kvq_tq4_codebook(cb.ctypes.data, thr.ctypes.data))
    return cb, thr


def kvq_tq_codebook(bits: int):
    import numpy as np
    L = 1 << bits
    cb = np.empty(L, np.float32)
    thr = np.empty(L - 1, np.float32)
    _check(lib().kvq_tq_codebook(bits, cb.ctypes.data, thr.ctypes.data))
    return cb, thr


def kvq_encode_fp8(x, codes, scales, stream=None) -> None:
    """x fp32 [rows][>=dim] -> codes u8 [rows][>=dim], scales fp32 [rows]; dim = codes
    columns used = x.shape[1] unless x is a strided view."""
    rows, dim = x.shape
    _check(lib().kvq_encode_fp8(_ptr(x), rows, dim, x.stride(0), _ptr(codes), codes.stride(0),
                                _ptr(scales), _stream(stream)))


def kvq_encode_tq4(x, sign_bits, packed, radius, stream=None) -> None:
    rows, dim = x.shape
    _check(lib().kvq_encode_tq4(_ptr(x), rows, dim, x.stride(0), _ptr(sign_bits), _ptr(packed),
                                packed.stride(0), _ptr(radius), _stream(stream)))


def kvq_encode_tq(x, sign_bits, bits, packed, radius, stream=None) -> None:
    """Rotated-tier encode at 3, 4 or 6 bits: packed u8 [rows][>= dim*bits/8]."""
    rows, dim = x.shape
    _check(lib().kvq_encode_tq(_ptr(x), rows, dim, x.stride(0), int(bits), _ptr(sign_bits),
                               _ptr(packed), packed.stride(0), _ptr(radius), _stream(stream)))


def kvq_encode_mla(c_lat, k_rope, fmt, sign_bits, lat, lat_scale, rope, rope_scale, stream=None) -> None:
    """Append-time encode of MLA rows: latent c_lat fp32 [rows][512] into the tier `fmt`
    (lat u8 [rows][>= 512 * bits / 8], lat_scale fp32 [rows]) and rope key k_rope fp32
    [rows][64] into fp8 (rope u8 [rows][>= 64], rope_scale fp32 [rows]), in one call."""
    rows = c_lat.shape[0]
    _check(lib().kvq_encode_mla(_ptr(c_lat), c_lat.stride(0), _ptr(k_rope), k_rope.stride(0), rows,
                                int(fmt), _ptr(sign_bits), _ptr(lat), lat.stride(0), _ptr(lat_scale),
                                _ptr(rope), rope.stride(0), _ptr(rope_scale), _stream(stream)))


def kvq_append_q4(k, v, pos0, page_table, page_size, n_cells, k_pool, v_pool,
                  dev_status=None, stream=None) -> None:
    n_seq, n_tok, n_heads, hd = k.shape
    _check(lib().kvq_append_q4(_ptr(k), _ptr(v), n_seq, _ptr(pos0), n_tok, n_heads, hd,
                               _ptr(page_table), page_table.shape[1], page_size, n_cells,
                               _ptr(k_pool), _ptr(v_pool), _ptr(dev_status), _stream(stream)))


def kvq_project_append_q4(h, w_k, w_v, pos0, page_table, page_size, n_cells, k_pool, v_pool,
                          dev_status=None, stream=None) -> None:
    """h fp32 [n_seq][n_tok][d_model]; w_k, w_v [d_model][n_heads * 256] float32 or
    bfloat16 tensors; the projected rows are appended as kvq_append_q4 appends k, v."""
    n_seq, n_tok, d_model = h.shape
    w_type = WEIGHT_BF16 if str(w_k.dtype).endswith("bfloat16") else WEIGHT_F32
    n_heads = w_k.shape[1] // 256
    if tuple(w_k.shape) != (d_model, n_heads * 256) or tuple(w_v.shape) != tuple(w_k.shape) \
            or w_v.dtype != w_k.dtype:
        raise ValueError("w_k, w_v must both be [d_model][n_heads * 256] of one dtype")
    _check(lib().kvq_project_append_q4(_ptr(h), n_seq, _ptr(pos0), n_tok, d_model, _ptr(w_k),
                                       _ptr(w_v), w_type, n_heads, 256, _ptr(page_table),
                                       page_table.shape[1], page_size, n_cells, _ptr(k_pool),
                                       _ptr(v_pool), _ptr(dev_status), _stream(stream)))


def kvq_gather_q4(pool, pos0, n_tok, page_table, page_size, n_cells, out, dev_status=None,
                  stream=None) -> None:
    """q4_0 mode of kvq_gather: out u16/fp16 [n_seq][n_tok][n_heads][256]."""
    d = GatherDesc()
    d.format = FMT_Q4_0
    d.q4_pool, d.n_seq, d.n_tok = _ptr(pool), pos0.shape[0], n_tok
    d.n_heads, d.head_dim = out.shape[2], out.shape[3]
    d.pos0, d.n_cells, d.q4_out = _ptr(pos0), n_cells, _ptr(out)
    d.page_table, d.max_pages, d.page_size = _ptr(page_table), page_table.shape[-1], page_size
    d.dev_status = _ptr(dev_status)
    _check(lib().kvq_gather(C.byref(d), _stream(stream)))


def kvq_gather_rows(fmt, src: dict, src_rows, idx, dst: dict, page_table=None, page_size=0,
                    dev_status=None, stream=None) -> None:
    """fp8 / TQ4 mode of kvq_gather: copy rows idx of `src` planes into `dst` planes."""
    d = GatherDesc()
    d.format = fmt
    d.mla_src = MlaCache(_ptr(src["lat"]), _ptr(src["lat_scale"]), _ptr(src["rope"]),
                         _ptr(src["rope_scale"]), src["lat"].shape[0])
    d.mla_src_rows = src_rows
    d.idx, d.n_idx = _ptr(idx), idx.numel()
    if page_table is not None:
        d.page_table, d.max_pages, d.page_size = _ptr(page_table), page_table.shape[-1], page_size
    d.dst_lat, d.dst_lat_scale = _ptr(dst["lat"]), _ptr(dst["lat_scale"])
    d.dst_rope, d.dst_rope_scale = _ptr(dst["rope"]), _ptr(dst["rope_scale"])
    d.dev_status = _ptr(dev_status)
    _check(lib().kvq_gather(C.byref(d), _stream(stream)))


def _cache(planes):
    if planes is None:
        return MlaCache()
    return MlaCache(_ptr(planes["lat"]), _ptr(planes["lat_scale"]), _ptr(planes["rope"]),
                    _ptr(planes["rope_scale"]), planes["lat"].shape[0])


def make_problem(*, seq_len, q_lat, q_rope, sm_scale, max_seq_len, fmt=FMT_FP8, seq_fmt=None,
                 causal=False, block_table=None, page_size=0, seq_stride_rows=0, fp8=None,
                 tq4=None, signs=None, idx=None, split_rows=0, impl=0,
                 overlap_prior=0) -> MlaProblem:
    """Fill a kvq_mla_problem from torch tensors.  The returned object holds a reference
    to every tensor whose device pointer it carries, so the memory stays allocated (and
    is not handed to a later allocation) for as long as the problem is alive."""
    n_seq, n_q, H, DL = q_lat.shape
    p = MlaProblem()
    p.n_seq, p.n_q, p.n_heads, p.d_lat, p.d_rope = n_seq, n_q, H, DL, q_rope.shape[-1]
    p.causal, p.max_seq_len = int(bool(causal)), int(max_seq_len)
    p.seq_len, p.seq_fmt, p.fmt = _ptr(seq_len), _ptr(seq_fmt), fmt
    if block_table is not None:
        p.block_table, p.max_pages, p.page_size = _ptr(block_table), block_table.shape[-1], page_size
    p.seq_stride_rows = seq_stride_rows
    p.fp8, p.tq4, p.tq4_signs = _cache(fp8), _cache(tq4), _ptr(signs)
    p.q_lat, p.q_rope = _ptr(q_lat), _ptr(q_rope)
    if idx is not None:
        p.idx, p.top_k = _ptr(idx), idx.shape[-1]
    p.sm_scale, p.split_rows, p.impl = float(sm_scale), int(split_rows), int(impl)
    p.overlap_prior = int(overlap_prior)
    p._keep = [seq_len, seq_fmt, block_table, fp8, tq4, signs, q_lat, q_rope, idx]
    return p


def kvq_mla_decode_workspace(p: MlaProblem) -> int:
    return lib().kvq_mla_decode_workspace(C.byref(p))


def kvq_mla_decode_kernel(p: MlaProblem) -> int:
    """The kernel kvq_mla_decode runs for p: IMPL_SIMT, IMPL_TC, IMPL_MMA, IMPL_TC16, IMPL_TCF8
    or IMPL_BY_FMT (a batch of per-sequence formats split by tier)."""
    r = lib().kvq_mla_decode_kernel(C.byref(p))
    if r < 0:
        _check(-r)
    return r


def kvq_mla_decode(p: MlaProblem, out, lse=None, workspace=None, dev_status=None,
                   stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().kvq_mla_decode(C.byref(p), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
                                _ptr(dev_status), _stream(stream)))


def kvq_mla_decode_noalloc(p: MlaProblem, out, lse=None, dev_status=None, stream=None) -> None:
    """kvq_mla_decode with the library's fixed scratch array instead of a workspace, for
    callers that cannot allocate device memory (see include/kvq.h)."""
    _check(lib().kvq_mla_decode_noalloc(C.byref(p), _ptr(out), _ptr(lse), _ptr(dev_status),
                                        _stream(stream)))


def make_q4_problem(*, seq_len, page_table, page_size, k_pool, v_pool, q, sm_scale,
                    max_seq_len, gate=None, split_rows=0) -> Q4Problem:
    """Fill a kvq_q4_problem from torch tensors: pools [n_cells, n_kv, 144] uint8, q (and
    gate) [n_seq, n_qh, 256] fp32, page_table [n_seq, max_pages] int32.  The returned
    object keeps a reference to every tensor whose pointer it carries."""
    n_seq, n_qh, hd = q.shape
    p = Q4Problem()
    p.n_seq, p.n_qh, p.n_kv, p.head_dim = n_seq, n_qh, k_pool.shape[1], hd
    p.seq_len, p.max_seq_len = _ptr(seq_len), int(max_seq_len)
    p.page_table, p.max_pages, p.page_size = _ptr(page_table), page_table.shape[-1], int(page_size)
    p.n_cells = k_pool.shape[0]
    p.k_pool, p.v_pool, p.q, p.gate = _ptr(k_pool), _ptr(v_pool), _ptr(q), _ptr(gate)
    p.sm_scale, p.split_rows = float(sm_scale), int(split_rows)
    p._keep = [seq_len, page_table, k_pool, v_pool, q, gate]
    return p


def kvq_q4_decode_workspace(p: Q4Problem) -> int:
    return lib().kvq_q4_decode_workspace(C.byref(p))


def kvq_q4_decode(p: Q4Problem, out, lse=None, workspace=None, dev_status=None,
                  stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().kvq_q4_decode(C.byref(p), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
                               _ptr(dev_status), _stream(stream)))


# --- drafted tokens over a paged MLA cache ------------------------------------------------

def _want(name, t, dtype, *shape):
    """A contiguous tensor of `dtype` (a name) and `shape` (None: any size), or None."""
    if t is None:
        return
    import torch
    got = t.shape
    if t.dtype is not getattr(torch, dtype) or not t.is_contiguous() or \
            (got != shape and (len(got) != len(shape) or any(n is not None and n != m for n, m in zip(shape, got)))):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)}, is {t.dtype} {list(got)}")


def _want_signs(name, t, fmt):
    """The 512 rotation signs of a rotated tier: 16 words, one bit a dimension (None: left to the library)."""
    if t is None or fmt == FMT_FP8:
        return
    import torch
    if t.dtype not in (torch.int32, torch.uint32) or t.numel() != 16 or not t.is_contiguous():
        raise ValueError(f"{name} must be 16 contiguous 32-bit integers, is {t.dtype} {list(t.shape)}")


def _one_device(*tensors):
    """The index of the device that holds every tensor (-1: the host)."""
    d = {t.get_device() for t in tensors if t is not None}
    if len(d) != 1:
        raise ValueError(f"tensors on different devices: {sorted(d)}")
    return d.pop()


def _status_on(d, t):
    """The address of the dev_status word `t` (or None) of a call whose tensors are on device `d`."""
    if t is None:
        return None
    import torch
    if t.dtype not in (torch.int32, torch.uint32) or t.numel() < 1:
        raise ValueError(f"dev_status must be a 32-bit integer tensor, is {t.dtype} {list(t.shape)}")
    if t.get_device() != d:
        raise ValueError(f"tensors on different devices: dev_status on {t.device}")
    return t.data_ptr()


def _stream_on(d, stream):
    """The stream of a call whose tensors are on device `d`, which must be the current device: the kernels
    run there."""
    if d < 0:
        raise ValueError("the tensors are on the host")
    import torch
    now = torch.cuda.current_device()
    if d != now:
        raise ValueError(f"tensors on cuda:{d}, but the current device is cuda:{now}")
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if stream is None and raw is not None:
        return raw(d)
    return _stream(stream)


def make_page_plan(*, keep_len, n_new, block_table, n_held, free_list, n_free, page_size, seq_len,
                   tok_start, slot_map, tok_pos=None) -> PagePlan:
    """Fill a kvq_page_plan from int32 tensors: block_table [n_seq, max_pages], free_list
    [n_pages], n_free [1], tok_start [n_seq + 1], slot_map (and tok_pos) [max_tokens], the
    others [n_seq].  The returned object keeps a reference to every tensor it carries."""
    n = keep_len.shape[0]
    for name, t, shape in (("keep_len", keep_len, (n,)), ("n_new", n_new, (n,)),
                           ("block_table", block_table, (n, None)), ("n_held", n_held, (n,)),
                           ("free_list", free_list, (None,)), ("n_free", n_free, (1,)),
                           ("seq_len", seq_len, (n,)), ("tok_start", tok_start, (n + 1,)),
                           ("slot_map", slot_map, (None,)), ("tok_pos", tok_pos, slot_map.shape)):
        _want(name, t, "int32", *shape)
    p = PagePlan()
    p.n_seq, p.max_pages, p.page_size = n, block_table.shape[1], int(page_size)
    p.n_pages, p.max_tokens = free_list.shape[0], slot_map.shape[0]
    p.keep_len, p.n_new, p.block_table, p.n_held = _ptr(keep_len), _ptr(n_new), _ptr(block_table), _ptr(n_held)
    p.free_list, p.n_free, p.seq_len = _ptr(free_list), _ptr(n_free), _ptr(seq_len)
    p.tok_start, p.slot_map, p.tok_pos = _ptr(tok_start), _ptr(slot_map), _ptr(tok_pos)
    p._keep = [keep_len, n_new, block_table, n_held, free_list, n_free, seq_len, tok_start, slot_map, tok_pos]
    p._device = _one_device(*p._keep)
    return p


def kvq_resize_pages(p: PagePlan, dev_status=None, stream=None) -> None:
    status = _status_on(p._device, dev_status)
    _check(lib().kvq_resize_pages(C.byref(p), status, _stream_on(p._device, stream)))


_LAT_BYTES = {FMT_FP8: 512, FMT_TQ4: 256, FMT_TQ6: 384, FMT_TQ3: 192}


def _planes_of(planes):
    return planes["lat"], planes["lat_scale"], planes["rope"], planes["rope_scale"]


def _mla_planes(planes, fmt):
    import torch
    lat, ls, rope, rs = _planes_of(planes)
    n = lat.shape[0]
    one, u8, f32 = (n,), torch.uint8, torch.float32
    if not (lat.dtype is u8 and rope.dtype is u8 and ls.dtype is f32 and rs.dtype is f32 and
            lat.shape == (n, _LAT_BYTES.get(fmt)) and rope.shape == (n, 64) and ls.shape == one and rs.shape == one and
            lat.is_contiguous() and rope.is_contiguous() and ls.is_contiguous() and rs.is_contiguous()):
        _want("lat", lat, "uint8", n, _LAT_BYTES.get(fmt))            # (names the one at fault)
        _want("lat_scale", ls, "float32", n)
        _want("rope", rope, "uint8", n, 64)
        _want("rope_scale", rs, "float32", n)
    return MlaCache(lat.data_ptr(), ls.data_ptr(), rope.data_ptr(), rs.data_ptr(), n)


def kvq_append_mla(c_lat, k_rope, slot_map, fmt, sign_bits, planes: dict, dev_status=None,
                   stream=None) -> None:
    """Encode rows c_lat [rows, 512] and k_rope [rows, 64] (both float32 or both bfloat16, rows
    possibly strided) into the cache planes of tier `fmt` at pool rows slot_map int32 [rows]
    (negative: skipped)."""
    import torch
    rows, width = c_lat.shape
    kind = WEIGHT_F32 if c_lat.dtype is torch.float32 else WEIGHT_BF16 if c_lat.dtype is torch.bfloat16 else None
    ldx, one = c_lat.stride()
    ldr, one_r = k_rope.stride()
    if kind is None or k_rope.dtype is not c_lat.dtype or width != 512 or k_rope.shape != (rows, 64) or \
            (rows and (one != 1 or one_r != 1)):
        raise ValueError("c_lat, k_rope must be [rows, 512] and [rows, 64], both float32 or both bfloat16")
    if rows == 1:                                         # (a single row's stride is arbitrary)
        ldx, ldr = 512, 64
    _want("slot_map", slot_map, "int32", rows)
    _want_signs("sign_bits", sign_bits, fmt)
    c = _mla_planes(planes, fmt)
    d = _one_device(c_lat, k_rope, slot_map, sign_bits, *_planes_of(planes))
    status, stream = _status_on(d, dev_status), _stream_on(d, stream)
    _check(lib().kvq_append_mla(c_lat.data_ptr(), ldx, k_rope.data_ptr(), ldr, kind, rows, slot_map.data_ptr(),
                                int(fmt), _ptr(sign_bits), C.byref(c), status, stream))


def _row_stride(name, q, width):
    """Elements between the rows of q [n_seq, n_q, heads, width], which must be evenly spaced."""
    n, nq, h, w = q.shape
    ld = q.stride(2) if h > 1 else q.stride(1) if nq > 1 else q.stride(0) if n > 1 else w
    even = (w == width and q.stride(3) == 1 and (h == 1 or q.stride(2) == ld)
            and (nq == 1 or q.stride(1) == ld * h) and (n == 1 or q.stride(0) == ld * h * nq))
    if not str(q.dtype).endswith("bfloat16") or not even:
        raise ValueError(f"{name} must be bfloat16 [n_seq, n_q, heads, {width}] with evenly spaced rows")
    return ld


def make_tree_problem(*, seq_len, q_lat, q_rope, sm_scale, max_seq_len, fmt, cache, signs=None, n_node=None,
                      mask=None, block_table=None, page_size=0, seq_stride_rows=0, impl=0) -> TreeProblem:
    """Fill a kvq_mla_tree_problem from torch tensors: q_lat [n_seq, n_q, H, 512] and q_rope
    [n_seq, n_q, H, 64] bfloat16, mask int64 [n_seq, n_q] (bit k of an entry: sees node k), cache the
    planes of tier `fmt`.  The returned object keeps a reference to every tensor it carries."""
    n_seq, n_q, H, DL = q_lat.shape
    if tuple(q_rope.shape[:3]) != (n_seq, n_q, H):
        raise ValueError("q_rope must have the rows of q_lat")
    _want("seq_len", seq_len, "int32", n_seq)
    _want("n_node", n_node, "int32", n_seq)
    _want("mask", mask, "int64", n_seq, n_q)
    _want("block_table", block_table, "int32", n_seq, None)
    _want_signs("signs", signs, fmt)
    p = TreeProblem()
    p.n_seq, p.n_q, p.n_heads, p.d_lat, p.d_rope = n_seq, n_q, H, DL, q_rope.shape[-1]
    p.fmt, p.max_seq_len = int(fmt), int(max_seq_len)
    p.seq_len, p.n_node, p.mask = _ptr(seq_len), _ptr(n_node), _ptr(mask)
    if block_table is not None:
        p.block_table, p.max_pages, p.page_size = _ptr(block_table), block_table.shape[1], int(page_size)
    p.seq_stride_rows = int(seq_stride_rows)
    p.cache, p.signs = _mla_planes(cache, fmt), _ptr(signs)
    p.q_lat, p.q_rope = _ptr(q_lat), _ptr(q_rope)
    p.ldq_lat, p.ldq_rope = _row_stride("q_lat", q_lat, 512), _row_stride("q_rope", q_rope, 64)
    p.sm_scale, p.impl = float(sm_scale), int(impl)
    p._keep = [seq_len, n_node, mask, block_table, signs, q_lat, q_rope, *_planes_of(cache)]
    p._device = _one_device(*p._keep)
    return p


def kvq_mla_tree_decode_workspace(p: TreeProblem) -> int:
    return lib().kvq_mla_tree_decode_workspace(C.byref(p))


def kvq_mla_tree_decode_kernel(p: TreeProblem) -> int:
    """The form kvq_mla_tree_decode runs for p: TREE_PACKED or TREE_PER_QUERY."""
    r = lib().kvq_mla_tree_decode_kernel(C.byref(p))
    if r < 0:
        _check(-r)
    return r


def kvq_mla_tree_decode(p: TreeProblem, out, lse=None, workspace=None, dev_status=None, stream=None) -> None:
    _want("out", out, "bfloat16", p.n_seq, p.n_q, p.n_heads, 512)
    _want("lse", lse, "float32", p.n_seq, p.n_q, p.n_heads)
    d = _one_device(out, lse, workspace, p._keep[0])
    status, stream = _status_on(d, dev_status), _stream_on(d, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().kvq_mla_tree_decode(C.byref(p), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes, status, stream))


def make_accept(*, seq_len, path, n_acc, new_len, fmt, cache, n_node=None, block_table=None, page_size=0,
                seq_stride_rows=0) -> AcceptDesc:
    """Fill a kvq_mla_accept_desc from int32 tensors: path [n_seq, n_q], the others [n_seq].  The
    returned object keeps a reference to every tensor it carries."""
    n_seq, n_q = path.shape
    for name, t, shape in (("seq_len", seq_len, (n_seq,)), ("path", path, (n_seq, n_q)),
                           ("n_acc", n_acc, (n_seq,)), ("new_len", new_len, (n_seq,)),
                           ("n_node", n_node, (n_seq,)), ("block_table", block_table, (n_seq, None))):
        _want(name, t, "int32", *shape)
    d = AcceptDesc()
    d.n_seq, d.n_q, d.fmt = n_seq, n_q, int(fmt)
    d.seq_len, d.n_node, d.path = _ptr(seq_len), _ptr(n_node), _ptr(path)
    d.n_acc, d.new_len = _ptr(n_acc), _ptr(new_len)
    if block_table is not None:
        d.block_table, d.max_pages, d.page_size = _ptr(block_table), block_table.shape[1], int(page_size)
    d.seq_stride_rows, d.cache = int(seq_stride_rows), _mla_planes(cache, fmt)
    d._keep = [seq_len, n_node, path, n_acc, new_len, block_table, *_planes_of(cache)]
    d._device = _one_device(*d._keep)
    return d


def kvq_accept_mla(d: AcceptDesc, dev_status=None, stream=None) -> None:
    status = _status_on(d._device, dev_status)
    _check(lib().kvq_accept_mla(C.byref(d), status, _stream_on(d._device, stream)))


# --- beam search and samples over a paged fp8 K/V cache --------------------------------------

def _kv8_cache(planes):
    """The planes k, v uint8 [n_kv, rows, head_dim] and k_scale, v_scale float32 [n_kv, rows]."""
    import torch
    k, ks, v, vs = planes["k"], planes["k_scale"], planes["v"], planes["v_scale"]
    kv, n, d = shape = k.shape
    two, u8, f32 = (kv, n), torch.uint8, torch.float32
    if not (k.dtype is u8 and v.dtype is u8 and ks.dtype is f32 and vs.dtype is f32 and v.shape == shape and
            ks.shape == two and vs.shape == two and k.is_contiguous() and v.is_contiguous() and
            ks.is_contiguous() and vs.is_contiguous()):
        _want("k", k, "uint8", kv, n, d)                       # (names the one at fault)
        _want("v", v, "uint8", kv, n, d)
        _want("k_scale", ks, "float32", kv, n)
        _want("v_scale", vs, "float32", kv, n)
    return Kv8Cache(k.data_ptr(), ks.data_ptr(), v.data_ptr(), vs.data_ptr(), n, kv, d)


def _kv8_planes(planes):
    return planes["k"], planes["k_scale"], planes["v"], planes["v_scale"]


def kvq_append_kv8(k, v, slot_map, planes: dict, dev_status=None, stream=None) -> None:
    """Encode rows k, v [rows, n_kv, head_dim] (both float32 or both bfloat16; rows and heads possibly
    strided, as slices of a fused projection are) into the fp8 K/V planes at pool rows slot_map int32
    [rows] (negative: skipped)."""
    import torch
    c = _kv8_cache(planes)
    rows, kv, d = shape = k.shape
    dtype = k.dtype
    kind = WEIGHT_BF16 if dtype is torch.bfloat16 else WEIGHT_F32 if dtype is torch.float32 else None
    kr, kh, k1 = k.stride()
    vr, vh, v1 = v.stride()
    if kind is None or v.dtype is not dtype or v.shape != shape or kv != c.n_kv or d != c.head_dim or \
            (rows and (k1 != 1 or v1 != 1)):
        raise ValueError(f"k, v must be [rows, {c.n_kv}, {c.head_dim}], both float32 or both bfloat16")
    if rows <= 1:                                          # (the stride of a single row or head is arbitrary)
        kr = vr = kv * d
    if kv == 1:
        kh = vh = d
    _want("slot_map", slot_map, "int32", rows)
    dv = _one_device(k, v, slot_map, *_kv8_planes(planes))
    status, stream = _status_on(dv, dev_status), _stream_on(dv, stream)
    _check(lib().kvq_append_kv8(k.data_ptr(), kr, kh, v.data_ptr(), vr, vh, kind, rows, slot_map.data_ptr(), C.byref(c),
                                status, stream))


def make_kv8_problem(*, seq_len, q, sm_scale, max_seq_len, cache, block_table=None, page_size=0, seq_stride_rows=0,
                     window=0) -> Kv8Problem:
    """Fill a kvq_kv8_problem from torch tensors: q [n_seq, n_qh, head_dim] bfloat16 (sequences possibly
    strided), cache the planes k, k_scale, v, v_scale.  The returned object keeps a reference to
    every tensor it carries."""
    import torch
    c = _kv8_cache(cache)
    n_seq, n_qh, d = q.shape
    if q.dtype is not torch.bfloat16 or d != c.head_dim or q.stride(2) != 1 or (n_qh > 1 and q.stride(1) != d):
        raise ValueError(f"q must be bfloat16 [n_seq, n_qh, {c.head_dim}] with contiguous heads")
    _want("seq_len", seq_len, "int32", n_seq)
    _want("block_table", block_table, "int32", n_seq, None)
    p = Kv8Problem()
    p.n_seq, p.n_qh, p.max_seq_len, p.window = n_seq, n_qh, int(max_seq_len), int(window)
    p.seq_len = _ptr(seq_len)
    if block_table is not None:
        p.block_table, p.max_pages, p.page_size = _ptr(block_table), block_table.shape[1], int(page_size)
    p.seq_stride_rows, p.cache = int(seq_stride_rows), c
    p.q, p.ldq, p.sm_scale = _ptr(q), q.stride(0) if n_seq > 1 else n_qh * d, float(sm_scale)
    p._keep = [seq_len, block_table, q, *_kv8_planes(cache)]
    p._device = _one_device(*p._keep)
    return p


def kvq_kv8_decode_workspace(p: Kv8Problem) -> int:
    return lib().kvq_kv8_decode_workspace(C.byref(p))


def _scratch(d, t):
    """The address and the bytes of a call's workspace `t` (or None) on device `d`."""
    if t is None:
        return None, 0
    if t.get_device() != d:
        raise ValueError(f"tensors on different devices: workspace on {t.device}")
    if not t.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def kvq_kv8_decode(p: Kv8Problem, out, lse=None, workspace=None, dev_status=None, stream=None) -> None:
    """out bfloat16 [n_seq, n_qh, head_dim], lse float32 [n_seq, n_qh] or None."""
    _want("out", out, "bfloat16", p.n_seq, p.n_qh, p.cache.head_dim)
    _want("lse", lse, "float32", p.n_seq, p.n_qh)
    d = _one_device(out, lse, p._keep[0])
    ws, ws_bytes = _scratch(d, workspace)
    status, stream = _status_on(d, dev_status), _stream_on(d, stream)
    _check(lib().kvq_kv8_decode(C.byref(p), _ptr(out), _ptr(lse), ws, ws_bytes, status, stream))


def make_beam_problem(*, logits, score, out_score, out_token, out_parent, finished=None, out_finished=None, eos=-1,
                      pad=0) -> BeamProblem:
    """Fill a kvq_beam_problem from torch tensors: logits [n_req, n_beam, vocab] float32 or bfloat16 (rows
    evenly spaced), score float32 and finished int32 [n_req, n_beam], out_score float32 and out_token,
    out_parent, out_finished int32 [n_req, n_out].  The returned object keeps a reference to every tensor it
    carries."""
    import torch
    R, B, V = logits.shape
    kind = WEIGHT_F32 if logits.dtype is torch.float32 else WEIGHT_BF16 if logits.dtype is torch.bfloat16 else None
    ld = logits.stride(1) if B > 1 else logits.stride(0) if R > 1 else V
    if kind is None or (V > 1 and logits.stride(2) != 1) or (R > 1 and logits.stride(0) != ld * B):
        raise ValueError("logits must be float32 or bfloat16 [n_req, n_beam, vocab] with evenly spaced rows")
    n_out = out_score.shape[-1]
    for name, t, dt, w in (("score", score, "float32", B), ("finished", finished, "int32", B),
                           ("out_score", out_score, "float32", n_out), ("out_token", out_token, "int32", n_out),
                           ("out_parent", out_parent, "int32", n_out), ("out_finished", out_finished, "int32", n_out)):
        _want(name, t, dt, R, w)
    p = BeamProblem()
    p.n_req, p.n_beam, p.vocab, p.n_out, p.x_type, p.eos, p.pad = R, B, V, n_out, kind, int(eos), int(pad)
    p.logits, p.ld, p.score, p.finished = _ptr(logits), ld, _ptr(score), _ptr(finished)
    p.out_score, p.out_token, p.out_parent = _ptr(out_score), _ptr(out_token), _ptr(out_parent)
    p.out_finished = _ptr(out_finished)
    p._keep = [logits, score, finished, out_score, out_token, out_parent, out_finished]
    p._device = _one_device(*p._keep)
    return p


def kvq_beam_select_workspace(p: BeamProblem) -> int:
    return lib().kvq_beam_select_workspace(C.byref(p))


def kvq_beam_select(p: BeamProblem, workspace=None, dev_status=None, stream=None) -> None:
    ws, ws_bytes = _scratch(p._device, workspace)
    status, stream = _status_on(p._device, dev_status), _stream_on(p._device, stream)
    _check(lib().kvq_beam_select(C.byref(p), ws, ws_bytes, status, stream))


def make_fork_plan(*, parent, block_table, n_held, free_list, n_free, seq_len, page_size, copy_src, copy_dst, copy_rows,
                   n_copy, keep_len=None) -> ForkPlan:
    """Fill a kvq_fork_plan from int32 tensors: block_table [n_seq, max_pages], free_list [n_pages], n_free
    and n_copy [1], the others [n_seq].  The returned object keeps a reference to every tensor it carries."""
    n = parent.shape[0]
    for name, t, shape in (("parent", parent, (n,)), ("keep_len", keep_len, (n,)), ("block_table", block_table, (n, None)),
                           ("n_held", n_held, (n,)), ("free_list", free_list, (None,)), ("n_free", n_free, (1,)),
                           ("seq_len", seq_len, (n,)), ("copy_src", copy_src, (n,)), ("copy_dst", copy_dst, (n,)),
                           ("copy_rows", copy_rows, (n,)), ("n_copy", n_copy, (1,))):
        _want(name, t, "int32", *shape)
    p = ForkPlan()
    p.n_seq, p.max_pages, p.page_size, p.n_pages = n, block_table.shape[1], int(page_size), free_list.shape[0]
    p.parent, p.keep_len, p.block_table, p.n_held = _ptr(parent), _ptr(keep_len), _ptr(block_table), _ptr(n_held)
    p.free_list, p.n_free, p.seq_len = _ptr(free_list), _ptr(n_free), _ptr(seq_len)
    p.copy_src, p.copy_dst, p.copy_rows, p.n_copy = _ptr(copy_src), _ptr(copy_dst), _ptr(copy_rows), _ptr(n_copy)
    p._keep = [parent, keep_len, block_table, n_held, free_list, n_free, seq_len, copy_src, copy_dst, copy_rows, n_copy]
    p._device = _one_device(*p._keep)
    return p


def kvq_fork_pages_workspace(p: ForkPlan) -> int:
    return lib().kvq_fork_pages_workspace(C.byref(p))


def kvq_fork_pages(p: ForkPlan, workspace=None, dev_status=None, stream=None) -> None:
    ws, ws_bytes = _scratch(p._device, workspace)
    status, stream = _status_on(p._device, dev_status), _stream_on(p._device, stream)
    _check(lib().kvq_fork_pages(C.byref(p), ws, ws_bytes, status, stream))


def make_compact_plan(*, block_table, n_held, new_table, free_list, n_free, n_used, page_size, copy_src, copy_dst,
                      copy_rows, n_copy) -> CompactPlan:
    """Fill a kvq_compact_plan from int32 tensors: block_table and new_table [n_seq, max_pages] (possibly the
    same), n_held [n_seq], free_list [n_pages], copy_* [n_pages / 2 or more], the others [1].  The returned
    object keeps a reference to every tensor it carries."""
    n, mp = block_table.shape
    m = copy_src.shape[0]
    for name, t, shape in (("block_table", block_table, (n, mp)), ("n_held", n_held, (n,)), ("new_table", new_table, (n, mp)),
                           ("free_list", free_list, (None,)), ("n_free", n_free, (1,)), ("n_used", n_used, (1,)),
                           ("copy_src", copy_src, (m,)), ("copy_dst", copy_dst, (m,)), ("copy_rows", copy_rows, (m,)),
                           ("n_copy", n_copy, (1,))):
        _want(name, t, "int32", *shape)
    p = CompactPlan()
    p.n_seq, p.max_pages, p.page_size, p.n_pages, p.max_copy = n, mp, int(page_size), free_list.shape[0], m
    p.block_table, p.n_held, p.new_table = _ptr(block_table), _ptr(n_held), _ptr(new_table)
    p.free_list, p.n_free, p.n_used = _ptr(free_list), _ptr(n_free), _ptr(n_used)
    p.copy_src, p.copy_dst, p.copy_rows, p.n_copy = _ptr(copy_src), _ptr(copy_dst), _ptr(copy_rows), _ptr(n_copy)
    p._keep = [block_table, n_held, new_table, free_list, n_free, n_used, copy_src, copy_dst, copy_rows, n_copy]
    p._device = _one_device(*p._keep)
    return p


def kvq_compact_pages_workspace(p: CompactPlan) -> int:
    return lib().kvq_compact_pages_workspace(C.byref(p))


def kvq_compact_pages(p: CompactPlan, workspace=None, dev_status=None, stream=None) -> None:
    ws, ws_bytes = _scratch(p._device, workspace)
    status, stream = _status_on(p._device, dev_status), _stream_on(p._device, stream)
    _check(lib().kvq_compact_pages(C.byref(p), ws, ws_bytes, status, stream))


def _pool_planes(cache):
    """(tensor, axis of the pool's rows) of every plane of a cache."""
    if not isinstance(cache, dict):
        return [(cache, 0)]                                    # a q4_0 pool [n_cells, heads, 144], or any rows
    if "lat" in cache:
        return [(t, 0) for t in _planes_of(cache)]
    return [(t, 1) for t in _kv8_planes(cache)]


def make_page_copy(*, caches, page_size, copy_src, copy_dst, copy_rows, n_copy) -> PageCopy:
    """Fill a kvq_page_copy: `caches` lists what the copies are made in (64 planes at most): dictionaries of
    MLA planes or of fp8 K/V planes, or pools as tensors with their rows along the first axis; copy_* int32
    [max_copy] and n_copy int32 [1] as kvq_fork_pages or kvq_compact_pages wrote them.  The
    returned object keeps a reference to every tensor it carries."""
    m = copy_src.shape[0]
    for name, t, shape in (("copy_src", copy_src, (m,)), ("copy_dst", copy_dst, (m,)), ("copy_rows", copy_rows, (m,)),
                           ("n_copy", n_copy, (1,))):
        _want(name, t, "int32", *shape)
    planes = [x for c in caches for x in _pool_planes(c)]
    d = PageCopy()
    d._planes = (Plane * max(1, len(planes)))()
    for at, (t, axis) in zip(d._planes, planes):
        if not t.is_contiguous():
            raise ValueError(f"a plane is not contiguous: {list(t.shape)}")
        rows, size = t.shape[axis], t.element_size()
        for n in t.shape[axis + 1:]:
            size *= n
        at.base, at.row_bytes, at.n_rows = _ptr(t), size, rows
        at.n_outer, at.outer_stride = t.shape[0] if axis else 1, rows * size
    d.planes, d.n_planes, d.page_size, d.max_copy = d._planes, len(planes), int(page_size), m
    d.copy_src, d.copy_dst, d.copy_rows, d.n_copy = _ptr(copy_src), _ptr(copy_dst), _ptr(copy_rows), _ptr(n_copy)
    d._keep = [copy_src, copy_dst, copy_rows, n_copy, *(t for t, _ in planes)]
    d._device = _one_device(*d._keep)
    return d


def kvq_copy_pages(d: PageCopy, dev_status=None, stream=None) -> None:
    status = _status_on(d._device, dev_status)
    _check(lib().kvq_copy_pages(C.byref(d), status, _stream_on(d._device, stream)))


# --- cache files ------------------------------------------------------------------------

def kvq_cache_probe(path) -> CacheInfo:
    info = CacheInfo()
    _check(lib().kvq_cache_probe(os.fsencode(path), C.byref(info)))
    return info


def kvq_cache_save(path, fmt, planes: dict, rows, signs=None, stream=None) -> None:
    """planes: dict of device tensors lat, lat_scale, rope, rope_scale (a quantized tier)."""
    c = _cache(planes)
    _check(lib().kvq_cache_save(os.fsencode(path), int(fmt), C.byref(c), _ptr(signs), int(rows),
                                _stream(stream)))


def kvq_cache_save_f32(path, lat, rope, stream=None) -> None:
    _check(lib().kvq_cache_save_f32(os.fsencode(path), _ptr(lat), _ptr(rope), lat.shape[0],
                                    _stream(stream)))


def kvq_cache_append(path, fmt, planes: dict, row0, rows, stream=None) -> None:
    c = _cache(planes)
    _check(lib().kvq_cache_append(os.fsencode(path), int(fmt), C.byref(c), int(row0), int(rows),
                                  _stream(stream)))


def kvq_cache_load_workspace() -> int:
    return lib().kvq_cache_load_workspace()


def kvq_cache_load(path, fmt, planes: dict, signs=None, workspace=None, stream=None) -> int:
    """Load `path` under `fmt` into the device planes (their row count is the capacity);
    returns the rows loaded."""
    c = _cache(planes)
    n = _i64(0)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().kvq_cache_load(os.fsencode(path), int(fmt), _ptr(signs), C.byref(c), c.n_rows,
                                C.byref(n), _ptr(workspace), ws_bytes, _stream(stream)))
    return n.value
