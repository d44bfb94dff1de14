"""Python binding of libupipe: head-chunked, trunked causal (GQA) attention for one GB300.

Argument marshalling only: every step of the attention path runs in the library's CUDA
kernels, reached through the C ABI declared in ``include/upipe.h``. The functions named
``upipe_*`` mirror that ABI one to one (tensors may be passed where the ABI takes pointers);
``attention_forward`` / ``attention_backward`` allocate outputs and the workspace with torch
and call them. There is no fallback: if ``libupipe.so`` is missing, importing the binding
fails with an error that says how to build it.
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as _np  # noqa: F401  (kept for users that pass numpy-backed pinned buffers)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libupipe.so")

UPIPE_OK = 0
UPIPE_ERR_INVALID_ARG = 1
UPIPE_ERR_UNSUPPORTED = 2
UPIPE_ERR_WORKSPACE_TOO_SMALL = 3
UPIPE_ERR_CUDA = 4
UPIPE_ERR_TIMEOUT = 5
UPIPE_ERR_PAGE = 6

UPIPE_PASS_FWD, UPIPE_PASS_BWD, UPIPE_PASS_BOTH, UPIPE_PASS_FUSED = 0, 1, 2, 3
UPIPE_HOST_KV, UPIPE_HOST_ACT = 1, 2
UPIPE_ROPE_PLAIN, UPIPE_ROPE_LINEAR, UPIPE_ROPE_NTK, UPIPE_ROPE_BY_PARTS = 0, 1, 2, 3

KERNEL_CLASSES = ["layout", "attn_fwd", "bwd_pre", "attn_bwd", "dq_convert", "other",
                  "loss_gemm", "loss_merge", "kv_h2d", "dkdv_d2h", "kv_wait", "rope",
                  "kv_append", "attn_paged", "paged_merge", "attn_prefix", "norm_rope", "embed",
                  "logp"]

# Every symbol include/upipe.h declares, with (restype, argtypes).
_vp, _i, _i64, _sz, _u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_uint64


class KernelStat(ctypes.Structure):
    _fields_ = [("total_ms", ctypes.c_double), ("launches", ctypes.c_uint64)]


class Heads(ctypes.Structure):
    """upipe_heads: a strided [B, S, heads, D] bf16 tensor."""
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_int64),
                ("stride_s", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("heads", ctypes.c_int32)]


class Pages(ctypes.Structure):
    """upipe_pages: the k and v caches and their strides."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("stride_page", ctypes.c_int64), ("stride_slot", ctypes.c_int64),
                ("stride_head", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("D", ctypes.c_int32)]


class Norm(ctypes.Structure):
    """upipe_norm: the weights of q's and k's norms."""
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("offset", ctypes.c_double), ("eps", ctypes.c_double), ("wide", ctypes.c_int32)]


_pn = ctypes.POINTER(Norm)
_ph, _pp, _d = ctypes.POINTER(Heads), ctypes.POINTER(Pages), ctypes.c_double

SIGNATURES = {
    "upipe_workspace_bytes": (_sz, [_i, _i64, _i, _i, _i, _i, _i, _i64, _i, _i]),
    "upipe_attn_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i64, _i, _i, _i, _i, _i, _i64, _vp,
                            _sz, _vp]),
    "upipe_attn_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i64, _i, _i, _i,
                            _i, _i, _i64, _vp, _sz, _vp]),
    "upipe_attn_fwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i64, _i, _i, _i, _i, _i, _i64,
                                    _i, _vp]),
    "upipe_seq_to_head_major": (_i, [_vp, _vp, _i, _i64, _i, _i, _i, _i, _vp]),
    "upipe_head_to_seq_major": (_i, [_vp, _vp, _i, _i64, _i, _i, _i, _i, _vp]),
    "upipe_sync_status": (_i, [_vp]),
    "upipe_status_string": (ctypes.c_char_p, [_i]),
    "upipe_last_error_message": (ctypes.c_char_p, []),
    "upipe_shutdown": (None, []),
    "upipe_launch_count": (_u64, []),
    "upipe_debug_fail_copy_after": (_i, [_i]),
    "upipe_profile_enable": (_i, [_i]),
    "upipe_profile_read": (_i, [ctypes.POINTER(KernelStat), _i]),
    "upipe_selftest_umma": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp]),
    "upipe_selftest_wait_timeout": (_i, [_i, _vp]),
    "upipe_ce_workspace_bytes": (_sz, [_i64, _i, _i64, _i64, _i, _i]),
    "upipe_ce_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i64, _i, _i64, _i64, _vp, _sz, _vp]),
    "upipe_ce_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i, _i64, _i64, _vp, _sz,
                          _vp]),
    "upipe_ce_fwd_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i, _i64, _i64, _vp,
                              _sz, _vp]),
    "upipe_mlp_workspace_bytes": (_sz, [_i64, _i, _i, _i64, _i, _i]),
    "upipe_mlp_fwd": (_i, [_vp, _vp, _vp, _vp, _i64, _i, _i, _i64, _vp, _sz, _vp]),
    "upipe_mlp_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i, _i, _i64, _vp, _sz,
                           _vp]),
    "upipe_logp_workspace_bytes": (_sz, [_i64, _i, _i64, _i, _i64, _i]),
    "upipe_logp_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i, _i64, _i, _i64, _vp,
                            _sz, _vp]),
    "upipe_embed_fwd": (_i, [_vp, _vp, _vp, _i64, _i, _i64, _d, _vp]),
    "upipe_embed_workspace_bytes": (_sz, [_i64, _i, _i64]),
    "upipe_embed_bwd": (_i, [_vp, _vp, _vp, _i64, _i, _i64, _d, _i, _vp, _sz, _vp]),
    "upipe_rope_frequencies": (_i, [ctypes.POINTER(_d), ctypes.POINTER(_d), _i, _d, _i, _d, _d,
                                    _d, _d]),
    "upipe_rope_phases": (_i, [ctypes.POINTER(_d), ctypes.POINTER(_u64), _i]),
    "upipe_rope_fwd": (_i, [_ph, _ph, _ph, _ph, _vp, _i64, _vp, _d, _i, _i64, _i, _i, _i, _vp]),
    "upipe_rope_bwd": (_i, [_ph, _ph, _ph, _ph, _vp, _i64, _vp, _d, _i, _i64, _i, _i, _i, _vp]),
    "upipe_kv_append": (_i, [_ph, _ph, _ph, _ph, _pp, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp,
                             _d, _i, _i64, _i, _i, _vp]),
    "upipe_kv_append_norm": (_i, [_ph, _ph, _ph, _ph, _pn, _pp, _vp, _i64, _i64, _vp, _vp, _vp,
                                  _i64, _vp, _d, _i, _i64, _i, _i, _vp]),
    "upipe_norm_rope_fwd": (_i, [_ph, _ph, _ph, _ph, _pn, _vp, _i64, _vp, _d, _i, _i64, _i, _i, _i,
                                 _vp]),
    "upipe_norm_rope_workspace_bytes": (_sz, [_i, _i64, _i, _i, _i]),
    "upipe_norm_rope_bwd": (_i, [_ph, _ph, _ph, _ph, _ph, _ph, _vp, _vp, _pn, _vp, _i64, _vp, _d,
                                 _i, _i64, _i, _i, _i, _vp, _sz, _vp]),
    "upipe_attn_paged_workspace_bytes": (_sz, [_i, _i64, _i, _i, _i, _i64, _i64, _i64]),
    "upipe_attn_paged_fwd": (_i, [_ph, _ph, _vp, _pp, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _i,
                                  _i64, _i64, _i64, _vp, _sz, _vp]),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; "
            f"g.build()\"` (or `python context_parallelism_gb300/build.py`)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


class UpipeError(RuntimeError):
    def __init__(self, status, where):
        msg = _lib.upipe_last_error_message().decode()
        name = _lib.upipe_status_string(status).decode()
        super().__init__(f"{where}: {name}: {msg}")
        self.status = status


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    raise TypeError(f"cannot pass {type(x)} as a pointer")


def _stream(stream, *tensors):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    for t in tensors:
        if hasattr(t, "is_cuda") and t.is_cuda:
            return _current_stream(t)
    return None


_torch = None
_raw_stream = _raw_alloc = _raw_delete = None


def _lazy_torch():
    """torch, imported once: the calls for single tokens are bound by the host's time."""
    global _torch, _raw_stream, _raw_alloc, _raw_delete
    if _torch is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
        _raw_delete = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)
        _torch = torch
    return _torch


def _current_stream(t):
    """Handle of the current stream on a CUDA tensor's device."""
    torch = _torch or _lazy_torch()
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _check(status, where):
    if status != UPIPE_OK:
        raise UpipeError(status, where)


# ---- one-to-one ABI wrappers ------------------------------------------------------------

def upipe_workspace_bytes(B, S, Hq, Hkv, D, causal, head_chunk, seq_trunk, pass_=UPIPE_PASS_BOTH,
                          host_mask=0):
    """host_mask: UPIPE_HOST_KV | UPIPE_HOST_ACT bits (True/1 keeps meaning host k/v)."""
    return int(_lib.upipe_workspace_bytes(B, S, Hq, Hkv, D, int(causal), head_chunk, seq_trunk,
                                          pass_, int(host_mask)))


def upipe_attn_fwd(q, k, v, o, lse, B, S, Hq, Hkv, D, causal, head_chunk, seq_trunk, workspace,
                   workspace_bytes=None, stream=None):
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = _lib.upipe_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, S, Hq, Hkv, D,
                             int(causal), head_chunk, seq_trunk, _ptr(workspace), wb,
                             _stream(stream, q, o, workspace))
    _check(st, "upipe_attn_fwd")


def upipe_attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, S, Hq, Hkv, D, causal, head_chunk,
                   seq_trunk, workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = _lib.upipe_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                             _ptr(dk), _ptr(dv), B, S, Hq, Hkv, D, int(causal), head_chunk,
                             seq_trunk, _ptr(workspace), wb, _stream(stream, q, dq, lse, workspace))
    _check(st, "upipe_attn_bwd")


def upipe_attn_fwd_noalloc(q, k, v, o, lse, B, S, Hq, Hkv, D, causal, head_chunk, seq_trunk,
                           check_status=0, stream=None):
    """The forward with its scratch in the library's static device array (no allocation)."""
    st = _lib.upipe_attn_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, S, Hq, Hkv,
                                     D, int(causal), head_chunk, seq_trunk, int(check_status),
                                     _stream(stream, q, o))
    _check(st, "upipe_attn_fwd_noalloc")


def upipe_seq_to_head_major(src, dst, B, S, H, D, h_begin, h_count, stream=None):
    _check(_lib.upipe_seq_to_head_major(_ptr(src), _ptr(dst), B, S, H, D, h_begin, h_count,
                                        _stream(stream, src)), "upipe_seq_to_head_major")


def upipe_head_to_seq_major(src, dst, B, S, H, D, h_begin, h_count, stream=None):
    _check(_lib.upipe_head_to_seq_major(_ptr(src), _ptr(dst), B, S, H, D, h_begin, h_count,
                                        _stream(stream, src)), "upipe_head_to_seq_major")


def upipe_sync_status(stream=None):
    """Synchronise the stream and raise UpipeError if a kernel's bounded wait expired."""
    import torch
    s = stream if stream is not None else (torch.cuda.current_stream().cuda_stream
                                           if torch.cuda.is_available() else None)
    if s is not None and not isinstance(s, int):
        s = s.cuda_stream
    _check(_lib.upipe_sync_status(s), "upipe_sync_status")


def upipe_status_string(status):
    return _lib.upipe_status_string(status).decode()


def upipe_last_error_message():
    return _lib.upipe_last_error_message().decode()


def upipe_shutdown():
    _lib.upipe_shutdown()


def upipe_launch_count():
    return int(_lib.upipe_launch_count())


def upipe_debug_fail_copy_after(n):
    """Test hook: the n-th staging copy from now on fails (0 disarms)."""
    _check(_lib.upipe_debug_fail_copy_after(int(n)), "upipe_debug_fail_copy_after")


def upipe_profile_enable(on=True):
    _check(_lib.upipe_profile_enable(int(on)), "upipe_profile_enable")


def upipe_profile_read():
    """Returns {class name: (total_ms, launches)} for the launches recorded since last read."""
    arr = (KernelStat * len(KERNEL_CLASSES))()
    _check(_lib.upipe_profile_read(arr, len(KERNEL_CLASSES)), "upipe_profile_read")
    return {n: (arr[i].total_ms, int(arr[i].launches)) for i, n in enumerate(KERNEL_CLASSES)}


def upipe_selftest_umma(a, b, c, N, K, a_mn_major, b_mn_major, a_manual=0, lbo=16384, sbo=1024,
                        stream=None):
    _check(_lib.upipe_selftest_umma(_ptr(a), _ptr(b), _ptr(c), N, K, int(a_mn_major),
                                    int(b_mn_major), int(a_manual), lbo, sbo,
                                    _stream(stream, a)), "upipe_selftest_umma")


def upipe_selftest_wait_timeout(limit_us, stream=None):
    _check(_lib.upipe_selftest_wait_timeout(limit_us, _stream(stream)),
           "upipe_selftest_wait_timeout")


def upipe_ce_workspace_bytes(S, Dm, V, seq_tile, pass_=UPIPE_PASS_BOTH, host_mask=0):
    return int(_lib.upipe_ce_workspace_bytes(S, Dm, V, seq_tile, pass_, int(host_mask)))


def upipe_ce_fwd(h, w, target, loss, lse, S, Dm, V, seq_tile, workspace, workspace_bytes=None,
                 stream=None):
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = _lib.upipe_ce_fwd(_ptr(h), _ptr(w), _ptr(target), _ptr(loss), _ptr(lse), S, Dm, V,
                           seq_tile, _ptr(workspace), wb, _stream(stream, h, loss, workspace))
    _check(st, "upipe_ce_fwd")


def upipe_ce_bwd(h, w, target, lse, dloss, dh, dw, S, Dm, V, seq_tile, workspace,
                 workspace_bytes=None, stream=None):
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = _lib.upipe_ce_bwd(_ptr(h), _ptr(w), _ptr(target), _ptr(lse), _ptr(dloss), _ptr(dh),
                           _ptr(dw), S, Dm, V, seq_tile, _ptr(workspace), wb,
                           _stream(stream, h, dh, workspace))
    _check(st, "upipe_ce_bwd")


def upipe_ce_fwd_bwd(h, w, target, dloss, loss, lse, dh, dw, S, Dm, V, seq_tile, workspace,
                     workspace_bytes=None, stream=None):
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = _lib.upipe_ce_fwd_bwd(_ptr(h), _ptr(w), _ptr(target), _ptr(dloss), _ptr(loss),
                               _ptr(lse), _ptr(dh), _ptr(dw), S, Dm, V, seq_tile,
                               _ptr(workspace), wb, _stream(stream, h, loss, workspace))
    _check(st, "upipe_ce_fwd_bwd")


def upipe_mlp_workspace_bytes(S, Dm, F, seq_tile, pass_=UPIPE_PASS_BOTH, host_mask=0):
    return int(_lib.upipe_mlp_workspace_bytes(S, Dm, F, seq_tile, pass_, int(host_mask)))


def upipe_mlp_fwd(x, w_gu, w_d, y, S, Dm, F, seq_tile, workspace, workspace_bytes=None,
                  stream=None):
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = _lib.upipe_mlp_fwd(_ptr(x), _ptr(w_gu), _ptr(w_d), _ptr(y), S, Dm, F, seq_tile,
                            _ptr(workspace), wb, _stream(stream, x, y, workspace))
    _check(st, "upipe_mlp_fwd")


def upipe_mlp_bwd(x, w_gu, w_d, dy, dx, dw_gu, dw_d, S, Dm, F, seq_tile, workspace,
                  workspace_bytes=None, stream=None):
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = _lib.upipe_mlp_bwd(_ptr(x), _ptr(w_gu), _ptr(w_d), _ptr(dy), _ptr(dx), _ptr(dw_gu),
                            _ptr(dw_d), S, Dm, F, seq_tile, _ptr(workspace), wb,
                            _stream(stream, x, dx, workspace))
    _check(st, "upipe_mlp_bwd")


@functools.lru_cache(maxsize=4096)
def upipe_logp_workspace_bytes(S, Dm, V, top, seq_tile, host_mask=0):
    return int(_lib.upipe_logp_workspace_bytes(S, Dm, V, top, seq_tile, int(host_mask)))


def upipe_logp_fwd(h, w, target, logp, entropy, lse, top_logp, top_index, S, Dm, V, top, seq_tile,
                   workspace, workspace_bytes=None, stream=None):
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(_lib.upipe_logp_fwd(_ptr(h), _ptr(w), _ptr(target), _ptr(logp), _ptr(entropy), _ptr(lse),
                               _ptr(top_logp), _ptr(top_index), S, Dm, V, top, seq_tile,
                               _ptr(workspace), wb, _stream(stream, h, w, workspace)),
           "upipe_logp_fwd")


def upipe_embed_fwd(token, w, h, S, Dm, V, scale=1.0, stream=None):
    _check(_lib.upipe_embed_fwd(_ptr(token), _ptr(w), _ptr(h), S, Dm, V, scale,
                                _stream(stream, h, w)), "upipe_embed_fwd")


@functools.lru_cache(maxsize=4096)
def upipe_embed_workspace_bytes(S, Dm, V):
    return int(_lib.upipe_embed_workspace_bytes(S, Dm, V))


def upipe_embed_bwd(token, dh, dw, S, Dm, V, scale, add, workspace, workspace_bytes=None,
                    stream=None):
    wb = workspace_bytes
    if wb is None:
        wb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.upipe_embed_bwd(_ptr(token), _ptr(dh), _ptr(dw), S, Dm, V, scale, int(add),
                                _ptr(workspace), wb, _stream(stream, dw, dh)), "upipe_embed_bwd")


def upipe_rope_frequencies(rot_dim, theta=10000.0, scaling=UPIPE_ROPE_PLAIN, factor=1.0,
                           trained_len=0.0, turns_fast=32.0, turns_slow=1.0):
    """Returns (list of rot_dim / 2 frequencies in radians a position, mscale)."""
    f = (_d * max(1, rot_dim // 2))()
    m = _d()
    _check(_lib.upipe_rope_frequencies(f, ctypes.byref(m), rot_dim, theta, scaling, factor,
                                       trained_len, turns_fast, turns_slow),
           "upipe_rope_frequencies")
    return list(f), m.value


def upipe_rope_phases(inv_freq):
    """Frequencies (radians a position) as a list of unsigned 64-bit fractions of a turn."""
    n = len(inv_freq)
    out = (_u64 * max(1, n))()
    _check(_lib.upipe_rope_phases((_d * max(1, n))(*inv_freq), out, n), "upipe_rope_phases")
    return list(out)[:n]


def upipe_rope_fwd(q, k, q_out, k_out, pos, pos0, phase, mscale, B, S, D, rot_dim, interleaved,
                   stream=None):
    """q, k, q_out, k_out: Heads or None (absent)."""
    _check(_lib.upipe_rope_fwd(q, k, q_out, k_out, _ptr(pos), pos0, _ptr(phase), mscale, B, S, D,
                               rot_dim, int(interleaved), _stream(stream, phase)),
           "upipe_rope_fwd")


def upipe_rope_bwd(dq_out, dk_out, dq, dk, pos, pos0, phase, mscale, B, S, D, rot_dim,
                   interleaved, stream=None):
    _check(_lib.upipe_rope_bwd(dq_out, dk_out, dq, dk, _ptr(pos), pos0, _ptr(phase), mscale, B,
                               S, D, rot_dim, int(interleaved), _stream(stream, phase)),
           "upipe_rope_bwd")


def upipe_kv_append(q, q_out, k, v, cache, page_table, table_stride, max_pages, seq_len, cu_rows,
                    pos, pos0, phase, mscale, B, S, rot_dim, interleaved, stream=None):
    """q, q_out, k, v: Heads or None; cache: Pages."""
    _check(_lib.upipe_kv_append(q, q_out, k, v, cache, _ptr(page_table), table_stride, max_pages,
                                _ptr(seq_len), _ptr(cu_rows), _ptr(pos), pos0, _ptr(phase),
                                mscale, B, S, rot_dim, int(interleaved),
                                _stream(stream, page_table)), "upipe_kv_append")


def upipe_kv_append_norm(q, q_out, k, v, norm, cache, page_table, table_stride, max_pages, seq_len,
                         cu_rows, pos, pos0, phase, mscale, B, S, rot_dim, interleaved,
                         stream=None):
    """q, q_out, k, v: Heads or None; norm: Norm; cache: Pages."""
    _check(_lib.upipe_kv_append_norm(q, q_out, k, v, norm, cache, _ptr(page_table), table_stride,
                                     max_pages, _ptr(seq_len), _ptr(cu_rows), _ptr(pos), pos0,
                                     _ptr(phase), mscale, B, S, rot_dim, int(interleaved),
                                     _stream(stream, page_table)), "upipe_kv_append_norm")


def upipe_norm_rope_fwd(q, k, q_out, k_out, norm, pos, pos0, phase, mscale, B, S, D, rot_dim,
                        interleaved, stream=None):
    """q, k, q_out, k_out: Heads or None (absent); norm: Norm. Without phase and pos, whose device
    has a current stream, stream None is the default stream."""
    _check(_lib.upipe_norm_rope_fwd(q, k, q_out, k_out, norm, _ptr(pos), pos0, _ptr(phase), mscale,
                                    B, S, D, rot_dim, int(interleaved),
                                    _stream(stream, phase, pos)), "upipe_norm_rope_fwd")


@functools.lru_cache(maxsize=4096)
def upipe_norm_rope_workspace_bytes(B, S, Hq, Hkv, D):
    return int(_lib.upipe_norm_rope_workspace_bytes(B, S, Hq, Hkv, D))


def upipe_norm_rope_bwd(dq_out, dk_out, q, k, dq, dk, dq_weight, dk_weight, norm, pos, pos0, phase,
                        mscale, B, S, D, rot_dim, interleaved, workspace, workspace_bytes=None,
                        stream=None):
    """dq_out, dk_out, q, k, dq, dk: Heads or None (absent); norm: Norm."""
    wb = workspace_bytes
    if wb is None:
        wb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.upipe_norm_rope_bwd(dq_out, dk_out, q, k, dq, dk, _ptr(dq_weight), _ptr(dk_weight),
                                    norm, _ptr(pos), pos0, _ptr(phase), mscale, B, S, D, rot_dim,
                                    int(interleaved), _ptr(workspace), wb,
                                    _stream(stream, dq_weight, dk_weight, workspace)),
           "upipe_norm_rope_bwd")


@functools.lru_cache(maxsize=4096)
def upipe_attn_paged_workspace_bytes(B, rows, Hq, Hkv, D, prefix_len, max_q, max_len):
    return int(_lib.upipe_attn_paged_workspace_bytes(B, rows, Hq, Hkv, D, prefix_len, max_q,
                                                     max_len))


def upipe_attn_paged_fwd(q, o, lse, cache, page_table, table_stride, max_pages, seq_len, cu_rows,
                         prefix_table, prefix_len, B, S, max_q, max_len, workspace,
                         workspace_bytes=None, stream=None):
    """q, o: Heads; cache: Pages."""
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(_lib.upipe_attn_paged_fwd(q, o, _ptr(lse), cache, _ptr(page_table), table_stride,
                                     max_pages, _ptr(seq_len), _ptr(cu_rows), _ptr(prefix_table),
                                     prefix_len, B, S, max_q, max_len, _ptr(workspace), wb,
                                     _stream(stream, page_table)), "upipe_attn_paged_fwd")


# ---- convenience: allocate outputs / workspace with torch, then call the ABI -------------

def _dims(q, k):
    B, S, Hq, D = q.shape
    return B, S, Hq, k.shape[2], D


def _device_of(*tensors):
    import torch
    for t in tensors:
        if t is not None and t.is_cuda:
            return t.device
    return torch.device("cuda", torch.cuda.current_device())


def attention_forward(q, k, v, causal=True, head_chunk=None, seq_trunk=None, workspace=None,
                      stream=None, with_lse=True, o_on_host=False):
    """o, lse = attention over token-major bf16 q [B,S,Hq,D], k/v [B,S,Hkv,D].
    q, k/v may be pinned host tensors (staged head group by head group, trunk by trunk);
    o_on_host returns o as a pinned host tensor, copied out group by group. with_lse=False is
    the prefill (inference) form: lse is neither allocated nor written and None is returned."""
    import torch
    B, S, Hq, Hkv, D = _dims(q, k)
    hc = head_chunk or Hq
    T = seq_trunk or S
    dev = _device_of(q, k)
    kv_host = not k.is_cuda
    mask = (UPIPE_HOST_KV if kv_host else 0) | (UPIPE_HOST_ACT if (not q.is_cuda or o_on_host)
                                                else 0)
    if o_on_host:
        o = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    else:
        o = torch.empty(q.shape, dtype=q.dtype, device=dev)
    lse = torch.empty((B, Hq, S), dtype=torch.float32, device=dev) if with_lse else None
    need = upipe_workspace_bytes(B, S, Hq, Hkv, D, causal, hc, T, UPIPE_PASS_FWD, mask)
    if need == 0:
        upipe_attn_fwd(q, k, v, o, lse, B, S, Hq, Hkv, D, causal, hc, T, 0, 0, stream)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    upipe_attn_fwd(q, k, v, o, lse, B, S, Hq, Hkv, D, causal, hc, T, workspace, None, stream)
    return o, lse


def attention_backward(q, k, v, o, lse, dout, causal=True, head_chunk=None, seq_trunk=None,
                       workspace=None, stream=None, dkdv_on_host=False, dq_on_host=False):
    """dq, dk, dv for the forward above. q, o, dout may be pinned host tensors (staged head
    group by head group); dq_on_host returns dq as a pinned host tensor, copied out group by
    group. dk/dv are device tensors, or pinned host tensors when dkdv_on_host (which needs host
    k/v): then each trunk's dK/dV is copied out as it finishes."""
    import torch
    B, S, Hq, Hkv, D = _dims(q, k)
    hc = head_chunk or Hq
    T = seq_trunk or S
    dev = _device_of(q, k, lse)
    kv_host = not k.is_cuda
    act_host = dq_on_host or not (q.is_cuda and o.is_cuda and dout.is_cuda)
    mask = (UPIPE_HOST_KV if kv_host else 0) | (UPIPE_HOST_ACT if act_host else 0)
    if dq_on_host:
        dq = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    else:
        dq = torch.empty(q.shape, dtype=q.dtype, device=dev)
    if dkdv_on_host:
        dk = torch.empty((B, S, Hkv, D), dtype=q.dtype, pin_memory=True)
        dv = torch.empty((B, S, Hkv, D), dtype=q.dtype, pin_memory=True)
    else:
        dk = torch.empty((B, S, Hkv, D), dtype=q.dtype, device=dev)
        dv = torch.empty((B, S, Hkv, D), dtype=q.dtype, device=dev)
    need = upipe_workspace_bytes(B, S, Hq, Hkv, D, causal, hc, T, UPIPE_PASS_BWD, mask)
    if need == 0:
        upipe_attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, S, Hq, Hkv, D, causal, hc, T, 0, 0,
                       stream)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    upipe_attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, S, Hq, Hkv, D, causal, hc, T, workspace,
                   None, stream)
    return dq, dk, dv


def _tiled_device(*tensors):
    import torch
    for t in tensors:
        if t is not None and t.is_cuda:
            return t.device
    return torch.device("cuda", torch.cuda.current_device())


def _empty_like_on(shape, dtype, dev, on_host):
    import torch
    if on_host:
        return torch.empty(shape, dtype=dtype, pin_memory=True)
    return torch.empty(shape, dtype=dtype, device=dev)


def ce_loss_forward(h, w, target, seq_tile=8192, workspace=None, stream=None):
    """loss, lse (float32 [S]) of the readout h [S, Dm] @ w[V, Dm]^T followed by token-level
    cross-entropy against target [S] (int64, negative = ignored), computed seq_tile tokens at
    a time without storing logits. h may be a pinned host tensor (staged tile by tile)."""
    import torch
    S, Dm = h.shape
    V = w.shape[0]
    dev = _tiled_device(w, target)
    loss = torch.empty(S, dtype=torch.float32, device=dev)
    lse = torch.empty(S, dtype=torch.float32, device=dev)
    mask = 0 if h.is_cuda else UPIPE_HOST_ACT
    need = upipe_ce_workspace_bytes(S, Dm, V, seq_tile, UPIPE_PASS_FWD, mask)
    if need == 0:
        upipe_ce_fwd(h, w, target, loss, lse, S, Dm, V, seq_tile, 0, 0, stream)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    upipe_ce_fwd(h, w, target, loss, lse, S, Dm, V, seq_tile, workspace, None, stream)
    return loss, lse


def ce_loss_backward(h, w, target, lse, dloss, seq_tile=8192, workspace=None, stream=None,
                     dh_on_host=False):
    """dh (bf16 [S, Dm]) and dw (float32 [V, Dm]) of sum_i dloss[i] * loss[i] for the forward
    above; lse is the forward's. h may be a pinned host tensor; dh_on_host returns dh as one."""
    import torch
    S, Dm = h.shape
    V = w.shape[0]
    dev = _tiled_device(w, target)
    dh = _empty_like_on((S, Dm), h.dtype, dev, dh_on_host)
    dw = torch.empty((V, Dm), dtype=torch.float32, device=dev)
    mask = UPIPE_HOST_ACT if (dh_on_host or not h.is_cuda) else 0
    need = upipe_ce_workspace_bytes(S, Dm, V, seq_tile, UPIPE_PASS_BWD, mask)
    if need == 0:
        upipe_ce_bwd(h, w, target, lse, dloss, dh, dw, S, Dm, V, seq_tile, 0, 0, stream)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    upipe_ce_bwd(h, w, target, lse, dloss, dh, dw, S, Dm, V, seq_tile, workspace, None, stream)
    return dh, dw


def ce_loss_fused(h, w, target, dloss, seq_tile=8192, workspace=None, stream=None,
                  dh_on_host=False):
    """loss, lse, dh, dw in one call when the upstream gradient dloss is known up front (the
    loss is the last operation). Bitwise the results of ce_loss_forward + ce_loss_backward,
    without the backward's logits recompute; needs seq_tile * V * 6 more bytes of workspace."""
    import torch
    S, Dm = h.shape
    V = w.shape[0]
    dev = _tiled_device(w, target)
    loss = torch.empty(S, dtype=torch.float32, device=dev)
    lse = torch.empty(S, dtype=torch.float32, device=dev)
    dh = _empty_like_on((S, Dm), h.dtype, dev, dh_on_host)
    dw = torch.empty((V, Dm), dtype=torch.float32, device=dev)
    mask = UPIPE_HOST_ACT if (dh_on_host or not h.is_cuda) else 0
    need = upipe_ce_workspace_bytes(S, Dm, V, seq_tile, UPIPE_PASS_FUSED, mask)
    if need == 0:
        upipe_ce_fwd_bwd(h, w, target, dloss, loss, lse, dh, dw, S, Dm, V, seq_tile, 0, 0, stream)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    upipe_ce_fwd_bwd(h, w, target, dloss, loss, lse, dh, dw, S, Dm, V, seq_tile, workspace, None,
                     stream)
    return loss, lse, dh, dw


def mlp_forward(x, w_gu, w_d, seq_tile=8192, workspace=None, stream=None, y_on_host=False):
    """y = (silu(x Wg^T) * x Wu^T) Wd^T for x [S, Dm], w_gu = [Wg; Wu] [2F, Dm], w_d [Dm, F]
    (bf16), seq_tile tokens at a time. x may be a pinned host tensor; y_on_host returns y as
    one."""
    import torch
    S, Dm = x.shape
    F = w_d.shape[1]
    dev = _tiled_device(w_gu)
    y = _empty_like_on((S, Dm), x.dtype, dev, y_on_host)
    mask = UPIPE_HOST_ACT if (y_on_host or not x.is_cuda) else 0
    need = upipe_mlp_workspace_bytes(S, Dm, F, seq_tile, UPIPE_PASS_FWD, mask)
    if need == 0:
        upipe_mlp_fwd(x, w_gu, w_d, y, S, Dm, F, seq_tile, 0, 0, stream)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    upipe_mlp_fwd(x, w_gu, w_d, y, S, Dm, F, seq_tile, workspace, None, stream)
    return y


def mlp_backward(x, w_gu, w_d, dy, seq_tile=8192, workspace=None, stream=None,
                 dx_on_host=False):
    """dx (bf16 [S, Dm]), dw_gu (float32 [2F, Dm]) and dw_d (float32 [Dm, F]) for the forward
    above and the upstream gradient dy [S, Dm]. x and dy may be pinned host tensors;
    dx_on_host returns dx as one."""
    import torch
    S, Dm = x.shape
    F = w_d.shape[1]
    dev = _tiled_device(w_gu)
    dx = _empty_like_on((S, Dm), x.dtype, dev, dx_on_host)
    dw_gu = torch.empty((2 * F, Dm), dtype=torch.float32, device=dev)
    dw_d = torch.empty((Dm, F), dtype=torch.float32, device=dev)
    mask = UPIPE_HOST_ACT if (dx_on_host or not x.is_cuda or not dy.is_cuda) else 0
    need = upipe_mlp_workspace_bytes(S, Dm, F, seq_tile, UPIPE_PASS_BWD, mask)
    if need == 0:
        upipe_mlp_bwd(x, w_gu, w_d, dy, dx, dw_gu, dw_d, S, Dm, F, seq_tile, 0, 0, stream)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    upipe_mlp_bwd(x, w_gu, w_d, dy, dx, dw_gu, dw_d, S, Dm, F, seq_tile, workspace, None,
                  stream)
    return dx, dw_gu, dw_d


# ---- token log probabilities ----------------------------------------------------------------

def token_logprobs(h, w, target=None, top=0, seq_tile=4096, workspace=None, stream=None):
    """logp, entropy, lse (float32 [S]), top_logp (float32 [S, top]), top_index (int64 [S, top]) of the
    readout h [S, Dm] @ w[V, Dm]^T (bf16): the log probability of target [S] (int64, negative: 0;
    None: logp is None), the entropy, the log of the sum of the exponentials, and the `top` most
    likely tokens with theirs (None, None for top = 0), seq_tile tokens at a time. h may be a pinned
    host tensor (staged tile by tile). The gradient of sum g * logp: ce_loss_backward with
    dloss = -g and this lse. top_index goes by the exact logits; top_logp is what logp gives these tokens,
    so that nearly equal neighbours may be a rounding out of order. With top the workspace has room for a
    tile's logits, 512 bytes for each token and group of up to 128 columns: seq_tile * V * 4 bytes where the
    groups are full, more where they are not."""
    torch = _torch or _lazy_torch()
    f32, i64 = torch.float32, torch.int64
    if len(_matrix(h, "h", torch.bfloat16)) != 2 or len(_matrix(w, "w", torch.bfloat16)) != 2 or \
            h.shape[1] != w.shape[1]:
        raise ValueError(f"h and w must be [S, Dm] and [V, Dm], not {tuple(h.shape)} and "
                         f"{tuple(w.shape)}")
    S, Dm = h.shape
    V = w.shape[0]
    logp = None
    if target is not None:
        _dense(target, i64, (S,), "target")
        logp = _empty(stream, w, (S,), f32)
    entropy, lse = _empty(stream, w, (S,), f32), _empty(stream, w, (S,), f32)
    top_logp = top_index = None
    if top:
        top_logp = _empty(stream, w, (S, top), f32)
        top_index = _empty(stream, w, (S, top), i64)
    if workspace is None:
        need = upipe_logp_workspace_bytes(S, Dm, V, top, seq_tile, 0 if h.is_cuda else UPIPE_HOST_ACT)
        workspace = _empty(stream, w, (need,), torch.uint8)
    st = _lib.upipe_logp_fwd(h.data_ptr(), w.data_ptr(), _ptr(target), _ptr(logp),
                             entropy.data_ptr(), lse.data_ptr(), _ptr(top_logp), _ptr(top_index), S,
                             Dm, V, top, seq_tile, workspace.data_ptr(),
                             workspace.numel() * workspace.element_size(), _stream(stream, w))
    if st:
        raise UpipeError(st, "upipe_logp_fwd")
    return logp, entropy, lse, top_logp, top_index


# ---- token embedding ------------------------------------------------------------------------

def _matrix(t, name, dtype, dims=2):
    """Checks a dense tensor whose last dimension is a row of features; returns its sizes."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.dim() < dims or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {dims} dimensions or more, not "
                         f"{tuple(t.shape)}")
    return t.shape


def embed_forward(tokens, w, scale=1.0, stream=None):
    """h = scale * w[tokens], bf16 [*tokens.shape, Dm]: tokens int64, w bf16 [V, Dm]. A negative
    token (padding) gives zeros, one beyond the table NaN."""
    torch = _torch or _lazy_torch()
    shape = _matrix(tokens, "tokens", torch.int64, 0)
    if len(_matrix(w, "w", torch.bfloat16)) != 2:
        raise ValueError(f"w must be [V, Dm], not {tuple(w.shape)}")
    V, Dm = w.shape
    h = _empty(stream, w, (*shape, Dm), w.dtype)
    st = _lib.upipe_embed_fwd(tokens.data_ptr(), w.data_ptr(), h.data_ptr(), tokens.numel(), Dm, V,
                              scale, _stream(stream, w))
    if st:
        raise UpipeError(st, "upipe_embed_fwd")
    return h


def embed_backward(tokens, dh, V, scale=1.0, dw=None, workspace=None, stream=None):
    """The gradient of w (float32 [V, Dm]) from dh (bf16 [*tokens.shape, Dm]). dw: added to instead
    of a new one (tied weights: the readout's), returned."""
    torch = _torch or _lazy_torch()
    shape = _matrix(dh, "dh", torch.bfloat16, 1)
    if _matrix(tokens, "tokens", torch.int64, 0) != shape[:-1]:
        raise ValueError(f"dh must be {tuple(tokens.shape)} + [Dm], not {tuple(shape)}")
    S, Dm, add = tokens.numel(), shape[-1], dw is not None
    if not add:
        dw = _empty(stream, dh, (V, Dm), torch.float32)
    elif _matrix(dw, "dw", torch.float32) != (V, Dm):
        raise ValueError(f"dw must be [{V}, {Dm}], not {tuple(dw.shape)}")
    if workspace is None:
        workspace = _empty(stream, dh, (upipe_embed_workspace_bytes(S, Dm, V),), torch.uint8)
    st = _lib.upipe_embed_bwd(tokens.data_ptr(), dh.data_ptr(), dw.data_ptr(), S, Dm, V, scale,
                              1 if add else 0, workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), _stream(stream, dh))
    if st:
        raise UpipeError(st, "upipe_embed_bwd")
    return dw


# ---- rotary positions, paged cache ----------------------------------------------------------

def _heads(t, name, dims):
    """upipe_heads of a bf16 [B, S, heads, D] (dims 4) or packed [S, heads, D] (dims 3) tensor."""
    torch = _torch or _lazy_torch()
    st = t.stride()
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, not {t.dtype}")
    if len(st) != dims or st[-1] != 1:
        raise ValueError(f"{name} must have {dims} dimensions with contiguous features, not "
                         f"{tuple(t.shape)} with strides {st}")
    return Heads(t.data_ptr(), st[0] if dims == 4 else 0, st[-3], st[-2], t.shape[-2])


def _pages(k_pages, v_pages):
    torch = _torch or _lazy_torch()
    if k_pages.dtype is not torch.bfloat16 or v_pages.dtype is not torch.bfloat16:
        raise TypeError("the caches must be bfloat16")
    st, shape = k_pages.stride(), k_pages.shape
    if len(st) != 4 or st[3] != 1 or v_pages.shape != shape or v_pages.stride() != st:
        raise ValueError("k_pages and v_pages must be [n_pages, page_size, heads, D] of one shape "
                         "and one set of strides, with contiguous features")
    return Pages(k_pages.data_ptr(), v_pages.data_ptr(), shape[0], st[0], st[1], st[2], shape[1],
                 shape[2], shape[3])


def _dense(t, dtype, shape, name):
    """Checks a dense tensor that the kernels index; a missing one passes."""
    if t is not None and (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                         f"not {t.dtype} {tuple(t.shape)}")


def _empty(stream, like, shape, dtype, zero=False):
    """An uninitialised (or zeroed) tensor beside `like`, allocated for the stream that the call
    runs on, so that its memory is not handed to other work before that stream is done with it.
    shape None: like's own, and its layout."""
    torch = _torch or _lazy_torch()
    if stream is None:
        if shape is None:
            return torch.empty_like(like)
        if zero:
            return torch.zeros(shape, dtype=dtype, device=like.device)
        return torch.empty(shape, dtype=dtype, device=like.device)
    if isinstance(stream, int):  # handle 0 as an ExternalStream would be a stream of torch's pool
        stream = (torch.cuda.ExternalStream(stream, device=like.device) if stream
                  else torch.cuda.default_stream(like.device))
    with torch.cuda.stream(stream):
        return _empty(None, like, shape, dtype, zero)


def rope_phases(rot_dim, theta=10000.0, scaling=UPIPE_ROPE_PLAIN, factor=1.0, trained_len=0.0,
                turns_fast=32.0, turns_slow=1.0, inv_freq=None, device="cuda"):
    """phases (int64 [rot_dim / 2] on the device), mscale: what the rotary calls take. Made once
    and kept. inv_freq: own frequencies (radians a position, rot_dim / 2 values) instead of
    theta's."""
    import torch
    if inv_freq is None:
        inv_freq, mscale = upipe_rope_frequencies(rot_dim, theta, scaling, factor, trained_len,
                                                  turns_fast, turns_slow)
    else:
        inv_freq, mscale = [float(f) for f in inv_freq], 1.0
        if len(inv_freq) != rot_dim // 2:
            raise ValueError(f"inv_freq has {len(inv_freq)} values, not {rot_dim // 2}")
    words = [w - (1 << 64) if w >> 63 else w for w in upipe_rope_phases(inv_freq)]
    return torch.tensor(words, dtype=torch.int64, device=device), mscale


def _phases(phases):
    torch = _torch or _lazy_torch()
    if phases.dtype is not torch.int64 or phases.dim() != 1 or not phases.is_contiguous():
        raise ValueError("phases must be a contiguous int64 vector (see rope_phases)")
    return 2 * phases.shape[0]


def _rope(fn, where, q, k, phases, mscale, interleaved, positions, start, inplace, stream):
    torch = _torch or _lazy_torch()
    ref = q if q is not None else k
    if ref is None or ref.dim() != 4:
        raise ValueError("q and k must be [B, S, heads, D] (one may be None)")
    B, S, _, D = shape = ref.shape
    if k is not None and k is not ref:
        ks = k.shape
        if len(ks) != 4 or ks[0] != B or ks[1] != S or ks[3] != D:
            raise ValueError("q and k must agree in B, S and D")
    pos = None
    if positions is not None:
        _dense(positions, torch.int64, shape[:2], "positions")
        pos = positions.data_ptr()
    rot = _phases(phases)
    q_in = q_out = k_in = k_out = None
    if q is not None:
        q_in = q_out = _heads(q, "q", 4)
        if not inplace:
            q = torch.empty_like(q) if stream is None else _empty(stream, q, None, q.dtype)
            q_out = _heads(q, "q", 4)
    if k is not None:
        k_in = k_out = _heads(k, "k", 4)
        if not inplace:
            k = torch.empty_like(k) if stream is None else _empty(stream, k, None, k.dtype)
            k_out = _heads(k, "k", 4)
    st = fn(q_in, k_in, q_out, k_out, pos, start, phases.data_ptr(), mscale, B, S, D, rot,
            1 if interleaved else 0, _stream(stream, ref))
    if st:
        raise UpipeError(st, where)
    return q, k


def rope_forward(q, k, phases, mscale=1.0, interleaved=False, positions=None, start=0,
                 inplace=False, stream=None):
    """q, k (bf16 [B, S, heads, D], any strides with contiguous D; one may be None) with their
    first 2 * len(phases) features rotated by their positions: positions (int64 [B, S]) or
    start + s. phases, mscale: rope_phases. inplace writes the inputs. Returns (q, k)."""
    return _rope(_lib.upipe_rope_fwd, "upipe_rope_fwd", q, k, phases, mscale, interleaved,
                 positions, start, inplace, stream)


def rope_backward(dq, dk, phases, mscale=1.0, interleaved=False, positions=None, start=0,
                  inplace=False, stream=None):
    """The gradients with respect to rope_forward's inputs, from those of its outputs."""
    return _rope(_lib.upipe_rope_bwd, "upipe_rope_bwd", dq, dk, phases, mscale, interleaved,
                 positions, start, inplace, stream)


def _norm(q_weight, k_weight, D, offset, eps):
    """upipe_norm of two [D] weights of one type (bf16 or float32; None: ones)."""
    torch = _torch or _lazy_torch()
    wide, ptr = None, [None, None]
    for i, w in enumerate((q_weight, k_weight)):
        if w is None:
            continue
        if w.dtype is not torch.bfloat16 and w.dtype is not torch.float32:
            raise TypeError(f"a norm's weights must be bfloat16 or float32, not {w.dtype}")
        if w.shape != (D,) or not w.is_contiguous():
            raise ValueError(f"a norm's weights must be contiguous [{D}], not {tuple(w.shape)}")
        if wide is not None and wide != (w.dtype is torch.float32):
            raise TypeError("q_weight and k_weight must be of one type")
        wide = w.dtype is torch.float32
        ptr[i] = w.data_ptr()
    return Norm(ptr[0], ptr[1], offset, eps, 1 if wide else 0)


def _like(x, ref, name):
    """x must be of ref's shape, in [B, S, heads, D]."""
    if x.shape != ref.shape:
        raise ValueError(f"{name} must be {tuple(ref.shape)}, not {tuple(x.shape)}")
    return x


def _rotation(phases, positions, lead):
    """rot_dim, and the pointers of the phases and of the positions (None: start + place)."""
    pos = None
    if positions is not None:
        _dense(positions, (_torch or _lazy_torch()).int64, lead, "positions")
        pos = positions.data_ptr()
    if phases is None:
        return 0, None, pos
    return _phases(phases), phases.data_ptr(), pos


def _q_or_k(q, k):
    """B, S, D of the tensors that are there."""
    ref = q if q is not None else k
    if ref is None or ref.dim() != 4:
        raise ValueError("q and k must be [B, S, heads, D] (one may be None)")
    B, S, _, D = ref.shape
    if k is not None and k is not ref:
        ks = k.shape
        if len(ks) != 4 or ks[0] != B or ks[1] != S or ks[3] != D:
            raise ValueError("q and k must agree in B, S and D")
    return ref, B, S, D


def norm_rope_forward(q, k, q_weight, k_weight, phases=None, mscale=1.0, eps=1e-6, offset=0.0,
                      interleaved=False, positions=None, start=0, inplace=False, stream=None):
    """q, k (bf16 [B, S, heads, D], any strides with contiguous D; one may be None), each head
    normed by its root mean square, times its weights (bf16 or float32 [D]; None: ones; offset is
    added to them), and rotated as by rope_forward (phases None: not rotated). Returns (q, k)."""
    ref, B, S, D = _q_or_k(q, k)
    rot, ph, pos = _rotation(phases, positions, ref.shape[:2])
    norm = _norm(q_weight if q is not None else None, k_weight if k is not None else None, D,
                 offset, eps)
    q_in = q_out = k_in = k_out = None
    if q is not None:
        q_in = q_out = _heads(q, "q", 4)
        if not inplace:
            q = _empty(stream, q, None, q.dtype)
            q_out = _heads(q, "q", 4)
    if k is not None:
        k_in = k_out = _heads(k, "k", 4)
        if not inplace:
            k = _empty(stream, k, None, k.dtype)
            k_out = _heads(k, "k", 4)
    st = _lib.upipe_norm_rope_fwd(q_in, k_in, q_out, k_out, norm, pos, start, ph, mscale, B, S, D,
                                  rot, 1 if interleaved else 0, _stream(stream, ref))
    if st:
        raise UpipeError(st, "upipe_norm_rope_fwd")
    return q, k


def norm_rope_backward(dq, dk, q, k, q_weight, k_weight, phases=None, mscale=1.0, eps=1e-6,
                       offset=0.0, interleaved=False, positions=None, start=0, inplace=False,
                       workspace=None, stream=None):
    """The gradients with respect to norm_rope_forward's inputs q, k and weights, from those of its
    outputs (dq, dk; inplace writes them). Returns (dq, dk, dq_weight, dk_weight), the last two
    float32 [D] (None for weights that are None)."""
    torch = _torch or _lazy_torch()
    ref, B, S, D = _q_or_k(dq, dk)
    rot, ph, pos = _rotation(phases, positions, ref.shape[:2])
    if dq is None:
        q_weight = None
    if dk is None:
        k_weight = None
    norm = _norm(q_weight, k_weight, D, offset, eps)
    dq_in = dq_out = q_in = dk_in = dk_out = k_in = None
    if dq is not None:
        q_in, dq_in = _heads(_like(q, dq, "q"), "q", 4), _heads(dq, "dq", 4)
        dq_out = dq_in
        if not inplace:
            dq = _empty(stream, dq, None, dq.dtype)
            dq_out = _heads(dq, "dq", 4)
    if dk is not None:
        k_in, dk_in = _heads(_like(k, dk, "k"), "k", 4), _heads(dk, "dk", 4)
        dk_out = dk_in
        if not inplace:
            dk = _empty(stream, dk, None, dk.dtype)
            dk_out = _heads(dk, "dk", 4)
    dqw = _empty(stream, ref, (D,), torch.float32) if q_weight is not None else None
    dkw = _empty(stream, ref, (D,), torch.float32) if k_weight is not None else None
    ws, wb = None, 0
    if dqw is not None or dkw is not None:
        if workspace is None:
            wb = upipe_norm_rope_workspace_bytes(B, S, dq_in.heads if dq_in else 0,
                                                 dk_in.heads if dk_in else 0, D)
            workspace = _empty(stream, ref, (max(wb, 256),), torch.uint8)
        ws, wb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = _lib.upipe_norm_rope_bwd(dq_in, dk_in, q_in, k_in, dq_out, dk_out, _ptr(dqw), _ptr(dkw),
                                  norm, pos, start, ph, mscale, B, S, D, rot,
                                  1 if interleaved else 0, ws, wb, _stream(stream, ref))
    if st:
        raise UpipeError(st, "upipe_norm_rope_bwd")
    return dq, dk, dqw, dkw


def _batch(q, cu_seqlens, seq_len):
    """B, S, dimensions and leading shape of a padded [B, S, heads, D] or packed [S, heads, D]
    batch, and the pointers of its two integer vectors."""
    int32 = (_torch or _lazy_torch()).int32
    lens = seq_len.shape
    if seq_len.dtype is not int32 or len(lens) != 1 or not seq_len.is_contiguous():
        raise ValueError("seq_len must be a contiguous int32 vector")
    B, shape = lens[0], q.shape
    if cu_seqlens is None:
        if len(shape) != 4 or shape[0] != B:
            raise ValueError(f"a padded batch is [{B}, S, heads, D], not {tuple(shape)}")
        return B, shape[1], 4, seq_len.data_ptr(), None
    if cu_seqlens.dtype is not int32 or cu_seqlens.shape != (B + 1,) or \
            not cu_seqlens.is_contiguous():
        raise ValueError(f"cu_seqlens must be a contiguous int32 vector of {B + 1}")
    if len(shape) != 3:
        raise ValueError(f"a packed batch is [rows, heads, D], not {tuple(shape)}")
    return B, shape[0], 3, seq_len.data_ptr(), cu_seqlens.data_ptr()


def _table(page_table, B):
    torch = _torch or _lazy_torch()
    shape = page_table.shape
    if page_table.dtype is torch.int32 and len(shape) == 2 and shape[0] == B:
        st = page_table.stride()
        if st[1] == 1 or shape[1] <= 1:
            return page_table.data_ptr(), st[0], shape[1]
    raise ValueError(f"page_table must be int32 [{B}, max_pages] with contiguous rows")


def kv_append(k, v, k_pages, v_pages, page_table, seq_len, q=None, q_out=None, phases=None,
              mscale=1.0, interleaved=False, positions=None, start=0, cu_seqlens=None,
              stream=None, q_weight=None, k_weight=None, eps=None, offset=0.0):
    """Writes the new tokens' k (rotated) and v into the paged cache; returns q rotated (None
    without q).

    k, v (and q): bf16 [B, S, heads, D], or packed [rows, heads, D] with cu_seqlens (int32
    [B + 1]); k_pages, v_pages: bf16 [n_pages, page_size, heads, D] (any strides with contiguous
    D); page_table: int32 [B, max_pages]; seq_len: int32 [B], each sequence's tokens in its own
    pages with the new ones. Positions: positions (int64, one a row), or start + a token's index
    in its sequence. phases None: nothing is rotated. q_out: where q goes (q itself: in place).
    eps: each head of q and k is normed before, with q_weight, k_weight and offset, as by
    norm_rope_forward."""
    if eps is None and (q_weight is not None or k_weight is not None or offset):
        raise ValueError("a norm's weights or offset without its eps")
    B, S, dims, lens, cu = _batch(k, cu_seqlens, seq_len)
    shape = k.shape
    lead, D = shape[:-2], k_pages.shape[-1]
    if shape[-1] != D or v.shape != shape:
        raise ValueError(f"k and v must have one shape with {D} features, not {tuple(shape)} "
                         f"and {tuple(v.shape)}")
    table, ts, mp = _table(page_table, B)
    pos = None
    if positions is not None:
        _dense(positions, (_torch or _lazy_torch()).int64, lead, "positions")
        pos = positions.data_ptr()
    rot = ph = None
    if phases is not None:
        rot, ph = _phases(phases), phases.data_ptr()
    qv = qo = None
    if q is not None:
        if q_out is None:  # rows of no sequence are not written
            q_out = _empty(stream, q, q.shape, q.dtype, zero=cu is not None)
        if q.shape[:-2] != lead or q.shape[-1] != D or q_out.shape != q.shape:
            raise ValueError(f"q and q_out must be {tuple(lead)} + [heads, {D}], not "
                             f"{tuple(q.shape)} and {tuple(q_out.shape)}")
        qv, qo = _heads(q, "q", dims), _heads(q_out, "q_out", dims)
    if eps is None:
        st = _lib.upipe_kv_append(qv, qo, _heads(k, "k", dims), _heads(v, "v", dims),
                                  _pages(k_pages, v_pages), table, ts, mp, lens, cu, pos, start,
                                  ph, mscale, B, S, rot or 0, 1 if interleaved else 0,
                                  _stream(stream, k))
    else:
        norm = _norm(q_weight if q is not None else None, k_weight, D, offset, eps)
        st = _lib.upipe_kv_append_norm(qv, qo, _heads(k, "k", dims), _heads(v, "v", dims), norm,
                                       _pages(k_pages, v_pages), table, ts, mp, lens, cu, pos,
                                       start, ph, mscale, B, S, rot or 0, 1 if interleaved else 0,
                                       _stream(stream, k))
    if st:
        raise UpipeError(st, "upipe_kv_append" if eps is None else "upipe_kv_append_norm")
    return q_out if q is not None else None


def paged_attention(q, k_pages, v_pages, page_table, seq_len, prefix_table=None, prefix_len=0,
                    cu_seqlens=None, max_q=None, max_len=None, out=None, with_lse=False,
                    lse=None, workspace=None, stream=None):
    """o, lse of new tokens over a shared prefix and their sequences' own pages.

    q: bf16 [B, S, Hq, D], or packed [rows, Hq, D] with cu_seqlens (int32 [B + 1]). k_pages,
    v_pages, page_table, seq_len as for kv_append, called before for the same tokens. The first
    prefix_len tokens of the pages prefix_table (int32) are seen by every row and read once for
    all; then row i of a sequence with n new tokens sees its own keys 0 .. seq_len - n + i.
    max_q, max_len: the largest numbers of new and own tokens, hints for tiles and blocks only
    (default: the most that the tensors allow). lse: float32 [B, Hq, S] (packed: [Hq, rows]),
    returned when given or with_lse, else None."""
    torch = _torch or _lazy_torch()
    B, S, dims, lens, cu = _batch(q, cu_seqlens, seq_len)
    cache = _pages(k_pages, v_pages)
    shape = q.shape
    Hq, D = shape[-2], shape[-1]
    if D != cache.D:
        raise ValueError(f"q has D={D}, the cache {cache.D}")
    table, ts, mp = _table(page_table, B)
    ptable = None
    if prefix_len:
        if prefix_table is None:
            raise ValueError("prefix_len without prefix_table")
        _dense(prefix_table, torch.int32, (prefix_table.numel(),), "prefix_table")
        if prefix_table.shape[0] * cache.page_size < prefix_len:
            raise ValueError(f"prefix_table has {prefix_table.numel()} pages of "
                             f"{cache.page_size} for {prefix_len} tokens")
        ptable = prefix_table.data_ptr()
    if cu is not None:
        rows, mq = S, S if max_q is None else max_q
    else:
        rows, mq = B * S, S
    ml = max_len if max_len is not None else max(1, mp * cache.page_size)
    # rows of no sequence are not written: zeros in what is made here
    if out is None:
        out = _empty(stream, q, shape, q.dtype, zero=cu is not None)
    elif out.shape != shape:
        raise ValueError(f"out must be {tuple(shape)}, not {tuple(out.shape)}")
    lse_ptr = None
    if lse is not None or with_lse:
        ls = (Hq, S) if cu is not None else (B, Hq, S)
        if lse is None:
            lse = _empty(stream, q, ls, torch.float32, zero=cu is not None)
        else:
            _dense(lse, torch.float32, ls, "lse")
        lse_ptr = lse.data_ptr()
    qh, oh, sp = _heads(q, "q", dims), _heads(out, "out", dims), _stream(stream, q)
    wb, ws, own = 0, None, False
    if workspace is not None:
        wb, ws = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    elif rows:
        wb = max(256, upipe_attn_paged_workspace_bytes(B, rows, Hq, cache.heads, D, prefix_len, mq,
                                                       ml))
        # torch's allocator without a tensor around the block (8 us less of a call's 21 on the
        # host), for the stream that the call runs on
        own = _raw_delete is not None and q.is_cuda and q.get_device() == torch.cuda.current_device()
        if own:
            ws = _raw_alloc(wb, sp)
        else:
            workspace = _empty(stream, q, (wb,), torch.uint8)
            ws = workspace.data_ptr()
    try:
        st = _lib.upipe_attn_paged_fwd(qh, oh, lse_ptr, cache, table, ts, mp, lens, cu, ptable,
                                       prefix_len, B, S, mq, ml, ws, wb, sp)
    finally:
        if own:
            _raw_delete(ws)
    if st:
        raise UpipeError(st, "upipe_attn_paged_fwd")
    return out, lse
