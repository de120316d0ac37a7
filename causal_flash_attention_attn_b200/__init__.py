"""B200 (sm_100a) fused causal attention: Python binding of libforge_attn.so.

The functions named ``forge_attn_*`` mirror the C ABI in include/forge_attn.h one
to one (argument marshalling only: every pointer argument accepts a torch
tensor or an integer device address). ``attention_fwd`` / ``attention_bwd`` /
``attention_decode`` allocate outputs and workspace with torch and call them;
``attention`` wraps the first two in a torch.autograd.Function.

PyTorch is used for device memory and streams only; all arithmetic runs in the
library's CUDA kernels. There is no fallback: if the shared library is missing
or fails to load, every call raises.

Packed sequences of different lengths: ``attention_varlen_fwd`` / ``_bwd`` and
``attention_varlen`` (autograd). A paged KV cache: ``attention_decode_paged``,
``paged_append``, ``paged_copy``, and ``PagedCache``, which keeps a pool's books
(pages of each sequence, forks, compaction) and calls them.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import operator
import os

__all__ = [
    "FORGE_OK", "FORGE_ERR_INVALID_ARG", "FORGE_ERR_UNSUPPORTED", "FORGE_ERR_WORKSPACE",
    "FORGE_ERR_CUDA", "FORGE_ERR_TIMEOUT", "FORGE_DTYPE_F32", "FORGE_DTYPE_BF16", "FORGE_VARLEN_CLEAR_TAIL",
    "FORGE_VARLEN_SINK_FIXED", "ForgeError",
    "library", "library_path", "forge_attn_fwd", "forge_attn_bwd", "forge_attn_bwd_workspace_size",
    "forge_attn_bwd_noalloc", "forge_attn_fwd_ext", "forge_attn_bwd_ext", "forge_attn_decode",
    "forge_attn_decode_workspace_size", "attention_decode", "forge_attn_fwd_dkv", "forge_attn_bwd_dkv",
    "forge_attn_bwd_workspace_size_dkv",
    "forge_attn_bwd_preprocess", "forge_attn_bwd_main", "forge_attn_bwd_finalize", "forge_attn_check",
    "forge_attn_status_string", "forge_attn_selftest_timeout", "forge_attn_selftest_exp2", "forge_attn_last_cuda_error", "forge_attn_timeout_info", "forge_attn_version",
    "attention_fwd", "attention_bwd", "attention", "dtype_code",
    "forge_attn_varlen_fwd", "forge_attn_varlen_fwd_workspace_size", "forge_attn_varlen_bwd",
    "forge_attn_varlen_bwd_workspace_size", "forge_attn_decode_paged", "forge_attn_decode_paged_workspace_size",
    "forge_attn_paged_append", "forge_attn_paged_copy",
    "attention_varlen_fwd", "attention_varlen_bwd", "attention_varlen", "attention_decode_paged", "paged_append",
    "paged_copy", "PagedCache",
]

FORGE_OK = 0
FORGE_ERR_INVALID_ARG = 1
FORGE_ERR_UNSUPPORTED = 2
FORGE_ERR_WORKSPACE = 3
FORGE_ERR_CUDA = 4
FORGE_ERR_TIMEOUT = 5
FORGE_DTYPE_F32 = 0
FORGE_DTYPE_BF16 = 1
FORGE_VARLEN_CLEAR_TAIL = 1
FORGE_VARLEN_SINK_FIXED = 0x100

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libforge_attn.so")
_lib = None


class ForgeError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = forge_attn_status_string(status)
        if status == FORGE_ERR_CUDA:
            msg += f" ({forge_attn_last_cuda_error()})"
        if status == FORGE_ERR_TIMEOUT:
            try:
                msg += f" (wait info {forge_attn_timeout_info()[1]})"
            except Exception:
                pass
        super().__init__(f"{what}: {msg}" if what else msg)


def library():
    """Load (once) and return the ctypes handle of libforge_attn.so."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError(f"{library_path} is missing: run `python -m causal_flash_attention_attn_b200.build`")
    L = ctypes.CDLL(library_path)
    vp, i, f, st, u = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_uint
    L.forge_attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, f, i, vp]
    L.forge_attn_fwd.restype = i
    L.forge_attn_bwd_workspace_size.argtypes = [i, i, i, i, i, i]
    L.forge_attn_bwd_workspace_size.restype = st
    L.forge_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, f, i, vp, st, vp]
    L.forge_attn_bwd.restype = i
    L.forge_attn_fwd_ext.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, f, vp, vp, i, vp]
    L.forge_attn_fwd_ext.restype = i
    L.forge_attn_bwd_ext.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, f, vp, vp, i, vp, st, vp]
    L.forge_attn_bwd_ext.restype = i
    L.forge_attn_fwd_dkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, f, i, vp]
    L.forge_attn_fwd_dkv.restype = i
    L.forge_attn_bwd_workspace_size_dkv.argtypes = [i, i, i, i, i, i, i]
    L.forge_attn_bwd_workspace_size_dkv.restype = st
    L.forge_attn_bwd_dkv.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, f, i, vp, st, vp]
    L.forge_attn_bwd_dkv.restype = i
    L.forge_attn_decode_workspace_size.argtypes = [i, i, i, i, i]
    L.forge_attn_decode_workspace_size.restype = st
    L.forge_attn_decode.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, f, vp, i, vp, st, vp]
    L.forge_attn_decode.restype = i
    L.forge_attn_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, f, i, vp]
    L.forge_attn_bwd_noalloc.restype = i
    L.forge_attn_bwd_preprocess.argtypes = [vp, vp, i, i, i, i, i, i, vp, st, vp]
    L.forge_attn_bwd_preprocess.restype = i
    L.forge_attn_bwd_main.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, f, i, vp, st, vp]
    L.forge_attn_bwd_main.restype = i
    L.forge_attn_bwd_finalize.argtypes = [vp, i, i, i, i, i, i, vp, st, vp]
    L.forge_attn_bwd_finalize.restype = i
    L.forge_attn_varlen_fwd_workspace_size.argtypes = [i, i, i, i, i, i]
    L.forge_attn_varlen_fwd_workspace_size.restype = st
    L.forge_attn_varlen_fwd.argtypes = ([vp] * 7 + [i] * 5 + [st] * 3 + [f, i, f, vp, i, i, vp, st, vp])
    L.forge_attn_varlen_fwd.restype = i
    L.forge_attn_varlen_bwd_workspace_size.argtypes = [i, i, i, i, i, i]
    L.forge_attn_varlen_bwd_workspace_size.restype = st
    L.forge_attn_varlen_bwd.argtypes = ([vp] * 11 + [i] * 5 + [st] * 3 + [f, i, f, vp, vp, i, i, vp, st, vp])
    L.forge_attn_varlen_bwd.restype = i
    L.forge_attn_decode_paged_workspace_size.argtypes = [i, i, i, i, i]
    L.forge_attn_decode_paged_workspace_size.restype = st
    L.forge_attn_decode_paged.argtypes = [vp] * 7 + [i] * 7 + [st, f, i, f, vp, i, vp, st, vp]
    L.forge_attn_decode_paged.restype = i
    L.forge_attn_paged_append.argtypes = [vp] * 7 + [i] * 7 + [st, st, st, i, vp]
    L.forge_attn_paged_append.restype = i
    L.forge_attn_paged_copy.argtypes = [vp] * 4 + [i, i, st, i, i, i, i, st, i, vp]
    L.forge_attn_paged_copy.restype = i
    L.forge_attn_check.argtypes = [vp]
    L.forge_attn_check.restype = i
    L.forge_attn_status_string.argtypes = [i]
    L.forge_attn_status_string.restype = ctypes.c_char_p
    L.forge_attn_selftest_timeout.argtypes = [u, vp]
    L.forge_attn_selftest_timeout.restype = i
    L.forge_attn_selftest_exp2.argtypes = [vp, vp, vp, i, vp]
    L.forge_attn_selftest_exp2.restype = i
    L.forge_attn_timeout_info.argtypes = [vp]
    L.forge_attn_timeout_info.restype = i
    L.forge_attn_last_cuda_error.argtypes = []
    L.forge_attn_last_cuda_error.restype = ctypes.c_char_p
    L.forge_attn_version.argtypes = []
    L.forge_attn_version.restype = ctypes.c_char_p
    _lib = L
    return L


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def dtype_code(dtype) -> int:
    import torch
    if dtype == torch.float32:
        return FORGE_DTYPE_F32
    if dtype == torch.bfloat16:
        return FORGE_DTYPE_BF16
    raise ValueError(f"unsupported dtype {dtype}")


# ------------------------------------------------------------------ raw C ABI
def forge_attn_fwd(q, k, v, o, lse, B, Hq, Hkv, T, D, scale, window, softcap, dtype, stream=None) -> int:
    return library().forge_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, T, D,
                                    float(scale), int(window), float(softcap), int(dtype), _stream(stream))


def forge_attn_bwd_workspace_size(B, Hq, Hkv, T, D, dtype) -> int:
    return int(library().forge_attn_bwd_workspace_size(B, Hq, Hkv, T, D, int(dtype)))


def forge_attn_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, Hq, Hkv, T, D, scale, window, softcap, dtype,
                   workspace, workspace_bytes, stream=None) -> int:
    return library().forge_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                                    _ptr(dk), _ptr(dv), B, Hq, Hkv, T, D, float(scale), int(window),
                                    float(softcap), int(dtype), _ptr(workspace), int(workspace_bytes),
                                    _stream(stream))


def forge_attn_fwd_ext(q, k, v, o, lse, B, Hq, Hkv, T, D, scale, window, softcap, sink, max_logit, dtype,
                       stream=None) -> int:
    return library().forge_attn_fwd_ext(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, T, D,
                                        float(scale), int(window), float(softcap), _ptr(sink), _ptr(max_logit),
                                        int(dtype), _stream(stream))


def forge_attn_bwd_ext(q, k, v, o, lse, dO, dq, dk, dv, B, Hq, Hkv, T, D, scale, window, softcap, sink, dsink,
                       dtype, workspace, workspace_bytes, stream=None) -> int:
    return library().forge_attn_bwd_ext(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                                        _ptr(dk), _ptr(dv), B, Hq, Hkv, T, D, float(scale), int(window),
                                        float(softcap), _ptr(sink), _ptr(dsink), int(dtype), _ptr(workspace),
                                        int(workspace_bytes), _stream(stream))


def forge_attn_fwd_dkv(q, k, v, o, lse, B, Hq, Hkv, T, Dk, Dv, scale, window, softcap, dtype, stream=None) -> int:
    return library().forge_attn_fwd_dkv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, T, Dk, Dv,
                                        float(scale), int(window), float(softcap), int(dtype), _stream(stream))


def forge_attn_bwd_workspace_size_dkv(B, Hq, Hkv, T, Dk, Dv, dtype) -> int:
    return int(library().forge_attn_bwd_workspace_size_dkv(B, Hq, Hkv, T, Dk, Dv, int(dtype)))


def forge_attn_bwd_dkv(q, k, v, o, lse, dO, dq, dk, dv, B, Hq, Hkv, T, Dk, Dv, scale, window, softcap, dtype,
                       workspace, workspace_bytes, stream=None) -> int:
    return library().forge_attn_bwd_dkv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                                        _ptr(dk), _ptr(dv), B, Hq, Hkv, T, Dk, Dv, float(scale), int(window),
                                        float(softcap), int(dtype), _ptr(workspace), int(workspace_bytes),
                                        _stream(stream))


def forge_attn_decode_workspace_size(B, Hq, Hkv, T, D) -> int:
    return int(library().forge_attn_decode_workspace_size(B, Hq, Hkv, T, D))


def forge_attn_decode(q, k_cache, v_cache, o, lse, seq_lens, B, Hq, Hkv, T, Tmax, D, scale, window, softcap, sink,
                      dtype, workspace, workspace_bytes, stream=None) -> int:
    return library().forge_attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse), _ptr(seq_lens),
                                       B, Hq, Hkv, T, Tmax, D, float(scale), int(window), float(softcap),
                                       _ptr(sink), int(dtype), _ptr(workspace), int(workspace_bytes),
                                       _stream(stream))


def forge_attn_bwd_noalloc(q, k, v, o, lse, dO, dq, dk, dv, B, Hq, Hkv, T, D, scale, window, softcap, dtype,
                           stream=None) -> int:
    """forge_attn_bwd with the library's fixed 32 MiB internal scratch instead of a workspace."""
    return library().forge_attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                                            _ptr(dk), _ptr(dv), B, Hq, Hkv, T, D, float(scale), int(window),
                                            float(softcap), int(dtype), _stream(stream))


def forge_attn_bwd_preprocess(o, dO, B, Hq, Hkv, T, D, dtype, workspace, workspace_bytes, stream=None) -> int:
    return library().forge_attn_bwd_preprocess(_ptr(o), _ptr(dO), B, Hq, Hkv, T, D, int(dtype),
                                               _ptr(workspace), int(workspace_bytes), _stream(stream))


def forge_attn_bwd_main(q, k, v, lse, dO, dq, dk, dv, B, Hq, Hkv, T, D, scale, window, softcap, dtype,
                        workspace, workspace_bytes, stream=None) -> int:
    return library().forge_attn_bwd_main(_ptr(q), _ptr(k), _ptr(v), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk),
                                         _ptr(dv), B, Hq, Hkv, T, D, float(scale), int(window), float(softcap),
                                         int(dtype), _ptr(workspace), int(workspace_bytes), _stream(stream))


def forge_attn_bwd_finalize(dq, B, Hq, Hkv, T, D, dtype, workspace, workspace_bytes, stream=None) -> int:
    return library().forge_attn_bwd_finalize(_ptr(dq), B, Hq, Hkv, T, D, int(dtype), _ptr(workspace),
                                             int(workspace_bytes), _stream(stream))


def forge_attn_varlen_fwd_workspace_size(num_seqs, rows, Hq, Hkv, D, dtype) -> int:
    return int(library().forge_attn_varlen_fwd_workspace_size(num_seqs, rows, Hq, Hkv, D, int(dtype)))


def forge_attn_varlen_fwd(q, k, v, o, o_res, lse, cu_seqlens, num_seqs, rows, Hq, Hkv, D, q_stride, k_stride, v_stride,
                          scale, window, softcap, sink, clear_tail, dtype, workspace, workspace_bytes,
                          stream=None) -> int:
    """clear_tail: the C function's flags (FORGE_VARLEN_CLEAR_TAIL, FORGE_VARLEN_SINK_FIXED)."""
    return library().forge_attn_varlen_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(o_res), _ptr(lse),
                                           _ptr(cu_seqlens), num_seqs, rows, Hq, Hkv, D, int(q_stride), int(k_stride), int(v_stride), float(scale),
                                           int(window), float(softcap), _ptr(sink), int(clear_tail), int(dtype),
                                           _ptr(workspace), int(workspace_bytes), _stream(stream))


def forge_attn_varlen_bwd_workspace_size(num_seqs, rows, Hq, Hkv, D, dtype) -> int:
    return int(library().forge_attn_varlen_bwd_workspace_size(num_seqs, rows, Hq, Hkv, D, int(dtype)))


def forge_attn_varlen_bwd(q, k, v, o, o_res, lse, dO, dq, dk, dv, cu_seqlens, num_seqs, rows, Hq, Hkv, D, q_stride, k_stride,
                          v_stride, scale, window, softcap, sink, dsink, clear_tail, dtype, workspace, workspace_bytes,
                          stream=None) -> int:
    """clear_tail: the C function's flags (FORGE_VARLEN_CLEAR_TAIL)."""
    return library().forge_attn_varlen_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(o_res), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk),
                                           _ptr(dv), _ptr(cu_seqlens), num_seqs, rows, Hq, Hkv, D, int(q_stride),
                                           int(k_stride), int(v_stride), float(scale), int(window), float(softcap),
                                           _ptr(sink), _ptr(dsink), int(clear_tail), int(dtype), _ptr(workspace),
                                           int(workspace_bytes), _stream(stream))


def forge_attn_decode_paged_workspace_size(B, Hq, Hkv, D, dtype) -> int:
    return int(library().forge_attn_decode_paged_workspace_size(B, Hq, Hkv, D, int(dtype)))


def forge_attn_decode_paged(q, k_pages, v_pages, o, lse, page_table, seq_lens, B, Hq, Hkv, D, num_pages, page_size,
                            table_width, page_stride, scale, window, softcap, sink, dtype, workspace, workspace_bytes,
                            stream=None) -> int:
    return library().forge_attn_decode_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(o), _ptr(lse),
                                             _ptr(page_table), _ptr(seq_lens), B, Hq, Hkv, D, num_pages, page_size,
                                             table_width, int(page_stride), float(scale), int(window), float(softcap),
                                             _ptr(sink), int(dtype), _ptr(workspace), int(workspace_bytes),
                                             _stream(stream))


def forge_attn_paged_append(k, v, k_pages, v_pages, page_table, starts, cu_seqlens, num_seqs, rows, Hkv, D, num_pages,
                            page_size, table_width, k_stride, v_stride, page_stride, dtype, stream=None) -> int:
    return library().forge_attn_paged_append(_ptr(k), _ptr(v), _ptr(k_pages), _ptr(v_pages), _ptr(page_table),
                                             _ptr(starts), _ptr(cu_seqlens), num_seqs, rows, Hkv, D, num_pages,
                                             page_size, table_width, int(k_stride), int(v_stride), int(page_stride),
                                             int(dtype), _stream(stream))


def forge_attn_paged_copy(k_pages, v_pages, src, dst, n, num_layers, layer_stride, num_pages, Hkv, page_size, D,
                          page_stride, dtype, stream=None) -> int:
    """src and dst: host memory (an int32 CPU tensor, or the address of n ints)."""
    return library().forge_attn_paged_copy(_ptr(k_pages), _ptr(v_pages), _ptr(src), _ptr(dst), n, num_layers,
                                           int(layer_stride), num_pages, Hkv, page_size, D, int(page_stride),
                                           int(dtype), _stream(stream))


def forge_attn_check(stream=None) -> int:
    return library().forge_attn_check(_stream(stream))


def forge_attn_status_string(s: int) -> str:
    return library().forge_attn_status_string(int(s)).decode()


def forge_attn_selftest_timeout(limit_us: int, stream=None) -> int:
    return library().forge_attn_selftest_timeout(int(limit_us), _stream(stream))


def forge_attn_selftest_exp2(x, y, y_ref, n, stream=None) -> int:
    return library().forge_attn_selftest_exp2(_ptr(x), _ptr(y), _ptr(y_ref), int(n), _stream(stream))


def forge_attn_timeout_info():
    """(status, [barrier+1, block, thread, (threads << 20) | blocks]) of the first wait that ran out."""
    arr = (ctypes.c_uint * 4)()
    s = library().forge_attn_timeout_info(arr)
    return s, list(arr)


def forge_attn_last_cuda_error() -> str:
    return library().forge_attn_last_cuda_error().decode()


def forge_attn_version() -> str:
    return library().forge_attn_version().decode()


# ---------------------------------------------------------- torch conveniences
# The library reads raw pointers with the documented dense layouts, so these
# helpers reject what it would misread: host tensors, strided views, mixed
# dtypes or devices, and shapes that disagree.
def _check(what, dtype, device, shapes, **tensors):
    import torch
    given = {name: t for name, t in tensors.items() if t is not None}
    for name, t in given.items():
        want = dtype.get(name)
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: {name} must be a torch tensor")
        if not t.is_contiguous():
            raise ValueError(f"{what}: {name} must be contiguous")
        if want is not None and t.dtype != want:
            raise ValueError(f"{what}: {name} has dtype {t.dtype}, expected {want}")
        if name in shapes and tuple(t.shape) != tuple(shapes[name]):
            raise ValueError(f"{what}: {name} has shape {tuple(t.shape)}, expected {tuple(shapes[name])}")
    for name, t in given.items():
        if not t.is_cuda:
            raise ValueError(f"{what}: {name} must be a CUDA tensor")
        if t.device != device:
            raise ValueError(f"{what}: {name} is on {t.device}, expected {device}")


def _dims(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"q and k must be [B, H, T, D], got {tuple(q.shape)} and {tuple(k.shape)}")
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    return B, Hq, Hkv, T, D


def _check_bhtd(what, q, k, v, extras=False, **rest):
    """Checks q, k, v and the rest; v (and o, dO) may have a head dim Dv of its own,
    but then without the sink / max-logit extras. Returns (B, Hq, Hkv, T, D, Dv)."""
    import torch
    B, Hq, Hkv, T, D = _dims(q, k)
    if v.dim() != 4:
        raise ValueError(f"{what}: v must be [B, Hkv, T, Dv], got {tuple(v.shape)}")
    Dv = v.shape[3]
    if Dv != D and extras:
        raise ValueError(f"{what}: sinks and the max logit are not offered with d_k != d_v")
    qs, ks, vs, rows = (B, Hq, T, Dv), (B, Hkv, T, D), (B, Hkv, T, Dv), (B, Hq, T)
    shapes = dict(k=ks, v=vs, o=qs, dO=qs, lse=rows, sink=(Hq,))
    f = torch.float32
    dt = dict(k=q.dtype, v=q.dtype, o=q.dtype, dO=q.dtype, lse=f, sink=f)
    _check(what, dt, q.device, shapes, q=q, k=k, v=v, **rest)
    return B, Hq, Hkv, T, D, Dv


def attention_fwd(q, k, v, scale=None, window=0, softcap=0.0, stream=None, *, sink=None, return_max_logit=False):
    """Forward on device tensors q [B,Hq,T,D], k [B,Hkv,T,D], v [B,Hkv,T,Dv] (bf16
    or f32). Returns (o, lse), or (o, lse, max_logit [B,Hq]) with
    return_max_logit. sink: optional f32 [Hq] sink logits. Dv != D runs the
    d_k != d_v entry point (no sink, no max logit there)."""
    import torch
    B, Hq, Hkv, T, D, Dv = _check_bhtd("attention_fwd", q, k, v, extras=sink is not None or return_max_logit,
                                       sink=sink)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    dt = dtype_code(q.dtype)
    o = torch.empty((B, Hq, T, Dv), dtype=q.dtype, device=q.device)
    lse = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device)
    ml = None
    if Dv != D:
        s, what = forge_attn_fwd_dkv(q, k, v, o, lse, B, Hq, Hkv, T, D, Dv, scale, window, softcap, dt,
                                     stream), "forge_attn_fwd_dkv"
    elif sink is not None or return_max_logit:
        ml = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if return_max_logit else None
        s, what = forge_attn_fwd_ext(q, k, v, o, lse, B, Hq, Hkv, T, D, scale, window, softcap, sink, ml, dt,
                                     stream), "forge_attn_fwd_ext"
    else:
        s, what = forge_attn_fwd(q, k, v, o, lse, B, Hq, Hkv, T, D, scale, window, softcap, dt,
                                 stream), "forge_attn_fwd"
    if s != FORGE_OK:
        raise ForgeError(s, what)
    return (o, lse, ml) if return_max_logit else (o, lse)


def attention_decode(q, k_cache, v_cache, T=None, scale=None, window=0, softcap=0.0, seq_lens=None, sink=None,
                     stream=None):
    """Decode on device tensors: q [B,Hq,D], caches [B,Hkv,Tmax,D]; T defaults to
    Tmax (or the largest of seq_lens, an int32 device tensor [B]). Returns (o, lse)."""
    import torch
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError(f"attention_decode: q must be [B, Hq, D] and the caches [B, Hkv, Tmax, D], got "
                         f"{tuple(q.shape)} and {tuple(k_cache.shape)}")
    B, Hq, D = q.shape
    Hkv, Tmax = k_cache.shape[1], k_cache.shape[2]
    _check("attention_decode", dict(k_cache=q.dtype, v_cache=q.dtype, sink=torch.float32, seq_lens=torch.int32),
           q.device, dict(k_cache=(B, Hkv, Tmax, D), v_cache=(B, Hkv, Tmax, D), sink=(Hq,), seq_lens=(B,)),
           q=q, k_cache=k_cache, v_cache=v_cache, sink=sink, seq_lens=seq_lens)
    if T is None:
        T = int(seq_lens.max().item()) if seq_lens is not None else Tmax
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    ws = torch.empty(forge_attn_decode_workspace_size(B, Hq, Hkv, T, D), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    s = forge_attn_decode(q, k_cache, v_cache, o, lse, seq_lens, B, Hq, Hkv, T, Tmax, D, scale, window, softcap, sink,
                          dtype_code(q.dtype), ws, ws.numel(), stream)
    if s != FORGE_OK:
        raise ForgeError(s, "forge_attn_decode")
    return o, lse


def attention_bwd(q, k, v, o, lse, dO, scale=None, window=0, softcap=0.0, workspace=None, stream=None, *,
                  sink=None):
    """Backward on device tensors (o and lse from the matching forward). Returns
    (dq, dk, dv), or (dq, dk, dv, dsink [Hq]) when the forward had a sink. Dv != D
    runs the d_k != d_v entry point."""
    import torch
    B, Hq, Hkv, T, D, Dv = _check_bhtd("attention_bwd", q, k, v, extras=sink is not None, o=o, lse=lse, dO=dO,
                                       workspace=workspace, sink=sink)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    dt = dtype_code(q.dtype)
    if Dv != D:
        nbytes = forge_attn_bwd_workspace_size_dkv(B, Hq, Hkv, T, D, Dv, dt)
        if nbytes == 0:
            raise ForgeError(FORGE_ERR_UNSUPPORTED, "forge_attn_bwd_dkv")
    else:
        nbytes = forge_attn_bwd_workspace_size(B, Hq, Hkv, T, D, dt)
    if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    wbytes = workspace.numel() * workspace.element_size()
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    dsink = None
    if Dv != D:
        s, what = forge_attn_bwd_dkv(q, k, v, o, lse, dO, dq, dk, dv, B, Hq, Hkv, T, D, Dv, scale, window, softcap,
                                     dt, workspace, wbytes, stream), "forge_attn_bwd_dkv"
    elif sink is not None:
        dsink = torch.empty((Hq,), dtype=torch.float32, device=q.device)
        s, what = forge_attn_bwd_ext(q, k, v, o, lse, dO, dq, dk, dv, B, Hq, Hkv, T, D, scale, window, softcap,
                                     sink, dsink, dt, workspace, wbytes, stream), "forge_attn_bwd_ext"
    else:
        s, what = forge_attn_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, Hq, Hkv, T, D, scale, window, softcap, dt,
                                 workspace, wbytes, stream), "forge_attn_bwd"
    if s != FORGE_OK:
        raise ForgeError(s, what)
    return (dq, dk, dv, dsink) if sink is not None else (dq, dk, dv)


# ------------------------------------------------------------------ autograd
_attention_fn = None


def _attention_function():
    """The torch.autograd.Function over attention_fwd / attention_bwd (built on
    first use, so that importing this module does not import torch)."""
    global _attention_fn
    if _attention_fn is None:
        import torch

        class ForgeAttention(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, v, sink, scale, window, softcap):
                o, lse = attention_fwd(q, k, v, scale, window, softcap, sink=sink)
                ctx.save_for_backward(q, k, v, o, lse, sink)
                ctx.args = (scale, window, softcap)
                return o

            @staticmethod
            def backward(ctx, dO):
                q, k, v, o, lse, sink = ctx.saved_tensors
                g = attention_bwd(q, k, v, o, lse, dO.contiguous(), *ctx.args, sink=sink)
                return g[0], g[1], g[2], (g[3] if sink is not None else None), None, None, None

        _attention_fn = ForgeAttention
    return _attention_fn


def attention(q, k, v, scale=None, window=0, softcap=0.0, sink=None):
    """Causal attention with autograd: o = attention(q, k, v), gradients for q, k,
    v (and sink) through the library's backward. Shapes, dtypes and options as
    attention_fwd; scale defaults to 1/sqrt(head dim of q)."""
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else float(scale)
    return _attention_function().apply(q, k, v, sink, scale, int(window), float(softcap))


# ------------------------------------------------------------ packed sequences
_NOTHING = contextlib.nullcontext()


def _scope(device, stream):
    """Makes `device`, and the stream if one is given, current: outputs and workspaces allocated inside
    belong to the stream that the kernels run on."""
    import torch
    if stream is not None:
        return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream)
    return _NOTHING if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _here(device):
    """Handle of the current stream of `device`."""
    import torch
    try:  # without a Stream object: 0.2 instead of 3 us of a short call's host time
        return torch._C._cuda_getCurrentRawStream(device.index)
    except AttributeError:
        return torch.cuda.current_stream(device).cuda_stream


# The helpers below are called once per layer and token, so that their host time counts. Each takes
# arguments that are as they should be through one test (_is, _is_packed, _is_pool) and leaves the
# explanation of what is not to the _check functions, which test the same things one by one.
# They call the library without the raw binding in between for the same reason, and ask for the
# workspace of the same sizes on a device (its SM count counts) once.
@functools.lru_cache(maxsize=1024)
def _bytes(name, index, *sizes):
    return int(getattr(library(), name)(*sizes))


def _at(t):
    return None if t is None else t.data_ptr()


def _is(t, dtype, shape, index):
    return t is None or t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()


def _is_packed(q, k, v, cu_seqlens, sink):
    """(rows, Hq, Hkv, D, row strides) of packed arguments, or None: ask _check_packed."""
    import torch
    try:
        sq, sk, sv, dtype, index = q.stride(), k.stride(), v.stride(), q.dtype, q.get_device()
        rows, Hq, D = q.shape
        Hkv = k.shape[1]
        if (index >= 0 and rows > 1 and k.shape == v.shape == (rows, Hkv, D) and dtype is k.dtype is v.dtype and
                k.get_device() == v.get_device() == index and sq[1:] == sk[1:] == sv[1:] == (D, 1) and
                sq[0] >= Hq * D and sk[0] >= Hkv * D and sv[0] >= Hkv * D and not (sq[0] | sk[0] | sv[0]) % 8 and
                cu_seqlens.dim() == 1 and cu_seqlens.numel() > 1 and
                _is(cu_seqlens, torch.int32, cu_seqlens.shape, index) and _is(sink, torch.float32, (Hq,), index)):
            return rows, Hq, Hkv, D, (sq[0], sk[0], sv[0])
    except (AttributeError, TypeError, ValueError, IndexError):
        pass
    return None


def _is_pool(k_pages, v_pages, dtype, index, layers=False):
    """As _check_pool, or None: ask it."""
    try:
        st, shape = k_pages.stride(), k_pages.shape
        nl, ls = 1, 0
        if layers and len(shape) == 5:
            nl, ls, st, shape = shape[0], st[0], st[1:], shape[1:]
        P, Hkv, ps, D = shape
        if (index >= 0 and P > 1 and st[1:] == (ps * D, D, 1) and k_pages.shape == v_pages.shape and
                k_pages.stride() == v_pages.stride() and k_pages.dtype is dtype is v_pages.dtype and
                k_pages.get_device() == v_pages.get_device() == index):
            return nl, ls, P, Hkv, ps, D, st[0]
    except (AttributeError, TypeError, ValueError, IndexError):
        pass
    return None


def _check_dense(what, device, **specs):
    """Each name: (tensor or None, dtype, shape). Contiguous, on `device`."""
    _check(what, {n: d for n, (t, d, s) in specs.items()}, device, {n: s for n, (t, d, s) in specs.items()},
           **{n: t for n, (t, d, s) in specs.items()})


def _check_rows(what, dtype, device, **tensors):
    """Packed [rows, H, D] tensors whose heads are dense but whose rows may lie apart (parts of one
    projection's output). Returns their row strides in elements."""
    import torch
    strides = []
    for name, t in tensors.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: {name} must be a torch tensor")
        if t.dim() != 3:
            raise ValueError(f"{what}: {name} must be [rows, H, D], got {tuple(t.shape)}")
        if t.dtype != dtype:
            raise ValueError(f"{what}: {name} has dtype {t.dtype}, expected {dtype}")
        rows, H, D = t.shape
        if (D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D):
            raise ValueError(f"{what}: {name}'s heads must be contiguous (strides {t.stride()})")
        stride = t.stride(0) if rows > 1 else H * D
        if stride < H * D or stride * t.element_size() % 16:
            raise ValueError(f"{what}: {name}'s rows must be at least {H * D} elements and a multiple of 16 bytes "
                             f"apart (stride {stride})")
        strides.append(stride)
    for name, t in tensors.items():
        if not t.is_cuda:
            raise ValueError(f"{what}: {name} must be a CUDA tensor")
        if t.device != device:
            raise ValueError(f"{what}: {name} is on {t.device}, expected {device}")
    return strides


def _check_packed(what, q, k, v, cu_seqlens, sink):
    import torch
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dim() != 3:
            raise ValueError(f"{what}: {name} must be [rows, H, D], got {tuple(t.shape)}")
    rows, Hq, D = q.shape
    Hkv = k.shape[1]
    for name, t in (("k", k), ("v", v)):
        if tuple(t.shape) != (rows, Hkv, D):
            raise ValueError(f"{what}: {name} has shape {tuple(t.shape)}, expected {(rows, Hkv, D)}")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError(f"{what}: cu_seqlens must be [num_seqs + 1] with num_seqs >= 1, got {tuple(cu_seqlens.shape)}")
    strides = _check_rows(what, q.dtype, q.device, q=q, k=k, v=v)
    _check_dense(what, q.device, cu_seqlens=(cu_seqlens, torch.int32, cu_seqlens.shape),
                 sink=(sink, torch.float32, (Hq,)))
    return rows, Hq, Hkv, D, strides


def attention_varlen_fwd(q, k, v, cu_seqlens, scale=None, window=0, softcap=0.0, stream=None, *, sink=None,
                         return_residual=False, sink_fixed=False):
    """Causal attention over packed sequences: q [rows,Hq,D], k, v [rows,Hkv,D] (bf16 or f32; their rows
    may lie apart), cu_seqlens int32 [num_seqs + 1] on the device, from 0. Returns (o [rows,Hq,D], lse
    [Hq,rows]), or (o, lse, o_res) with return_residual: o's rounding residual for the backward (None in
    f32), and with a sink P in two terms for dsink, unless sink_fixed says that no gradient of the sink
    will be asked for. Rows behind the last sequence get zeros, lse -inf there. Nothing synchronises; bad
    cu_seqlens are reported by forge_attn_check."""
    import torch
    what = "attention_varlen_fwd"
    rows, Hq, Hkv, D, (qs, ks, vs) = (_is_packed(q, k, v, cu_seqlens, sink) or
                                      _check_packed(what, q, k, v, cu_seqlens, sink))
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    window, softcap, dt, n = int(window), float(softcap), dtype_code(q.dtype), cu_seqlens.numel() - 1
    with _scope(q.device, stream):
        o = q.new_empty((rows, Hq, D))
        o_res = torch.empty_like(o) if return_residual and dt == FORGE_DTYPE_BF16 else None
        lse = q.new_empty((Hq, rows), dtype=torch.float32)
        L = library()
        nbytes = _bytes("forge_attn_varlen_fwd_workspace_size", q.get_device(), n, rows, Hq, Hkv, D, dt)
        ws = q.new_empty(nbytes, dtype=torch.uint8)
        flags = FORGE_VARLEN_CLEAR_TAIL | (FORGE_VARLEN_SINK_FIXED if sink_fixed else 0)
        s = L.forge_attn_varlen_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _at(o_res), lse.data_ptr(),
                                    cu_seqlens.data_ptr(), n, rows, Hq, Hkv, D, qs, ks, vs, scale, window, softcap,
                                    _at(sink), flags, dt, ws.data_ptr(), nbytes, _here(q.device))
    if s != FORGE_OK:
        raise ForgeError(s, "forge_attn_varlen_fwd")
    return (o, lse, o_res) if return_residual else (o, lse)


def attention_varlen_bwd(q, k, v, o, lse, dO, cu_seqlens, scale=None, window=0, softcap=0.0, stream=None, *,
                         sink=None, o_res=None):
    """Backward of attention_varlen_fwd (its o and lse, and o_res if it returned one; dO contiguous).
    Returns (dq, dk, dv), or (dq, dk, dv, dsink [Hq]) with a sink (which only dsink needs); zeros in the rows
    behind the last sequence."""
    import torch
    what = "attention_varlen_bwd"
    rows, Hq, Hkv, D, (qs, ks, vs) = (_is_packed(q, k, v, cu_seqlens, sink) or
                                      _check_packed(what, q, k, v, cu_seqlens, sink))
    shape, dev = (rows, Hq, D), q.get_device()
    if not (_is(o, q.dtype, shape, dev) and _is(o_res, q.dtype, shape, dev) and _is(dO, q.dtype, shape, dev) and
            _is(lse, torch.float32, (Hq, rows), dev)):
        _check_dense(what, q.device, o=(o, q.dtype, shape), lse=(lse, torch.float32, (Hq, rows)),
                     o_res=(o_res, q.dtype, shape), dO=(dO, q.dtype, shape))
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    with _scope(q.device, stream):
        g = _varlen_bwd(q, k, v, o, o_res, lse, dO, cu_seqlens, sink, scale, int(window), float(softcap), rows, Hq, Hkv,
                        D, qs, ks, vs)
    return g if sink is not None else g[:3]


def _varlen_bwd(q, k, v, o, o_res, lse, dO, cu_seqlens, sink, scale, window, softcap, rows, Hq, Hkv, D, qs, ks, vs):
    """The call of attention_varlen_bwd on checked arguments, on the current device and stream."""
    import torch
    L, n, dt = library(), cu_seqlens.shape[0] - 1, dtype_code(q.dtype)
    dq = torch.empty_like(o)
    dk = q.new_empty((rows, Hkv, D))
    dv = torch.empty_like(dk)
    dsink = torch.empty_like(sink) if sink is not None else None
    nbytes = _bytes("forge_attn_varlen_bwd_workspace_size", q.get_device(), n, rows, Hq, Hkv, D, dt)
    ws = q.new_empty(nbytes, dtype=torch.uint8)
    s = L.forge_attn_varlen_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _at(o_res), lse.data_ptr(),
                                dO.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), cu_seqlens.data_ptr(), n,
                                rows, Hq, Hkv, D, qs, ks, vs, scale, window, softcap, _at(sink), _at(dsink), 1, dt,
                                ws.data_ptr(), nbytes, _here(q.device))
    if s != FORGE_OK:
        raise ForgeError(s, "forge_attn_varlen_bwd")
    return dq, dk, dv, dsink


_attention_varlen_fn = None


def _attention_varlen_function():
    global _attention_varlen_fn
    if _attention_varlen_fn is None:
        import torch

        class ForgeAttentionVarlen(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, v, cu_seqlens, sink, scale, window, softcap, residual):
                # a sink that requires no gradient: no second term of P, no dsink
                trained = sink if ctx.needs_input_grad[4] else None
                o, lse, *rest = attention_varlen_fwd(q, k, v, cu_seqlens, scale, window, softcap, sink=sink,
                                                     return_residual=residual, sink_fixed=trained is None)
                o_res = rest[0] if residual else None
                ctx.save_for_backward(q, k, v, o, o_res, lse, cu_seqlens, trained)
                rows, Hq, D = q.shape
                ctx.args = (scale, window, softcap, rows, Hq, k.shape[1], D,
                            *((x.stride(0) if rows > 1 else x.shape[1] * D) for x in (q, k, v)))
                return o

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dO):
                # the forward has checked everything but dO, which autograd gives o's type
                # and shape, with the device and the stream of the forward current
                q, k, v, o, o_res, lse, cu_seqlens, sink = ctx.saved_tensors
                dO = dO.contiguous()
                if dO.data_ptr() % 16:  # a part of another tensor's gradient may start anywhere
                    dO = dO.clone()
                dq, dk, dv, dsink = _varlen_bwd(q, k, v, o, o_res, lse, dO, cu_seqlens, sink, *ctx.args)
                return dq, dk, dv, None, dsink, None, None, None, None

        _attention_varlen_fn = ForgeAttentionVarlen
    return _attention_varlen_fn


def attention_varlen(q, k, v, cu_seqlens, scale=None, window=0, softcap=0.0, sink=None, residual=True):
    """attention_varlen_fwd with autograd: o, and gradients for q, k, v (and sink, if it requires one)
    through the library's backward (once: there are no second derivatives). In bf16 a second tensor
    of o's size, its rounding residual, is kept for the backward; residual=False does without (less
    memory and traffic, as `attention`), and then dq, dk and dsink carry o's rounding, which shows
    where rows attend to few keys. The lengths must not change between the forward and its backward.
    Capture a forward together with its backward, on one stream, while no graph of an earlier call on
    the same leaves is alive."""
    import torch
    # (a Function's forward cannot tell: inside it grad mode is off, and needs_input_grad says only
    # which inputs require one)
    if not (torch.is_grad_enabled() and any(x is not None and x.requires_grad for x in (q, k, v, sink))):
        return attention_varlen_fwd(q, k, v, cu_seqlens, scale, window, softcap, sink=sink)[0]
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else float(scale)
    return _attention_varlen_function().apply(q, k, v, cu_seqlens, sink, scale, int(window), float(softcap),
                                              bool(residual))


# ---------------------------------------------------------------- paged cache
def _check_pool(what, dtype, device, k_pages, v_pages, layers=False):
    """[num_pages, Hkv, page_size, D] pools (layers: or [layers, num_pages, ...]) whose pages are dense.
    Returns (num_layers, layer stride, num_pages, Hkv, page_size, D, page stride), strides in elements."""
    import torch
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: {name} must be a torch tensor")
        if t.dim() != 4 and not (layers and t.dim() == 5):
            raise ValueError(f"{what}: {name} must be [num_pages, Hkv, page_size, D]"
                             f"{' or [layers, num_pages, Hkv, page_size, D]' if layers else ''}, got {tuple(t.shape)}")
        if t.dtype != dtype:
            raise ValueError(f"{what}: {name} has dtype {t.dtype}, expected {dtype}")
        if t.shape != k_pages.shape or t.stride() != k_pages.stride():
            raise ValueError(f"{what}: {name} has shape {tuple(t.shape)} and strides {t.stride()}, expected those of "
                             f"k_pages, {tuple(k_pages.shape)} and {k_pages.stride()}")
        Hkv, ps, D = t.shape[-3:]
        if (D > 1 and t.stride(-1) != 1) or (ps > 1 and t.stride(-2) != D) or (Hkv > 1 and t.stride(-3) != ps * D):
            raise ValueError(f"{what}: {name}'s pages must be contiguous (strides {t.stride()})")
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if not t.is_cuda:
            raise ValueError(f"{what}: {name} must be a CUDA tensor")
        if t.device != device:
            raise ValueError(f"{what}: {name} is on {t.device}, expected {device}")
    P, Hkv, ps, D = k_pages.shape[-4:]
    page_stride = k_pages.stride(-4) if P > 1 else Hkv * ps * D
    nl, ls = (k_pages.shape[0], k_pages.stride(0)) if k_pages.dim() == 5 else (1, 0)
    return nl, ls, P, Hkv, ps, D, page_stride


def attention_decode_paged(q, k_pages, v_pages, page_table, seq_lens, scale=None, window=0, softcap=0.0, sink=None,
                           stream=None):
    """One new query per sequence against a paged cache: q [B,Hq,D], pools [num_pages,Hkv,page_size,D] (bf16
    or f32; page_size a multiple of 16), page_table int32 [B,width], seq_lens int32 [B] (0 = padded
    entry: o = 0, lse = -inf or the sink). Returns (o [B,Hq,D], lse [B,Hq]). Nothing synchronises; bad
    lengths and pages are reported by forge_attn_check."""
    import torch
    what = "attention_decode_paged"
    if q.dim() != 3 or page_table.dim() != 2:
        raise ValueError(f"{what}: q must be [B, Hq, D] and page_table [B, width], got {tuple(q.shape)} and "
                         f"{tuple(page_table.shape)}")
    B, Hq, D = q.shape
    width, dev = page_table.shape[1], q.get_device()
    _, _, P, Hkv, ps, Dk, stride = (_is_pool(k_pages, v_pages, q.dtype, dev) or
                                    _check_pool(what, q.dtype, q.device, k_pages, v_pages))
    if Dk != D:
        raise ValueError(f"{what}: q has head dim {D}, the pools {Dk}")
    if not (_is(q, q.dtype, q.shape, dev) and _is(page_table, torch.int32, (B, width), dev) and
            _is(seq_lens, torch.int32, (B,), dev) and _is(sink, torch.float32, (Hq,), dev)):
        _check_dense(what, q.device, q=(q, q.dtype, q.shape), page_table=(page_table, torch.int32, (B, width)),
                     seq_lens=(seq_lens, torch.int32, (B,)), sink=(sink, torch.float32, (Hq,)))
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    window, softcap, dt = int(window), float(softcap), dtype_code(q.dtype)
    with _scope(q.device, stream):
        o = torch.empty_like(q)
        lse = q.new_empty((B, Hq), dtype=torch.float32)
        L = library()
        nbytes = _bytes("forge_attn_decode_paged_workspace_size", dev, B, Hq, Hkv, D, dt)
        ws = q.new_empty(nbytes, dtype=torch.uint8)
        s = L.forge_attn_decode_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), o.data_ptr(),
                                      lse.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), B, Hq, Hkv, D, P, ps,
                                      width, stride, scale, window, softcap, _at(sink), dt, ws.data_ptr(), nbytes,
                                      _here(q.device))
    if s != FORGE_OK:
        raise ForgeError(s, "forge_attn_decode_paged")
    return o, lse


def paged_append(k, v, k_pages, v_pages, page_table, starts, cu_seqlens=None, stream=None):
    """Write new tokens' keys and values into their sequences' pages: k, v [rows,Hkv,D] (their rows may lie
    apart), page_table int32 [num_seqs,width], starts int32 [num_seqs] (tokens each sequence holds
    already), cu_seqlens int32 [num_seqs + 1] as in attention_varlen_fwd, or None: one token per sequence.
    Rows behind the last sequence are skipped. Bad places are skipped and reported by forge_attn_check."""
    import torch
    what = "paged_append"
    if k.dim() != 3 or page_table.dim() != 2:
        raise ValueError(f"{what}: k must be [rows, Hkv, D] and page_table [num_seqs, width], got {tuple(k.shape)} and "
                         f"{tuple(page_table.shape)}")
    rows, Hkv, D = k.shape
    if v.shape != k.shape:
        raise ValueError(f"{what}: v has shape {tuple(v.shape)}, expected {tuple(k.shape)}")
    n, width = page_table.shape
    if cu_seqlens is None and n != rows:
        raise ValueError(f"{what}: {rows} rows for {n} sequences need cu_seqlens")
    dev, sk, sv = k.get_device(), k.stride(), v.stride()
    if (rows > 1 and sk[1:] == sv[1:] == (D, 1) and k.dtype is v.dtype and v.get_device() == dev >= 0 and
            sk[0] >= Hkv * D and sv[0] >= Hkv * D and not (sk[0] | sv[0]) % 8):
        ks, vs = sk[0], sv[0]
    else:
        ks, vs = _check_rows(what, k.dtype, k.device, k=k, v=v)
    if not (_is(page_table, torch.int32, (n, width), dev) and _is(starts, torch.int32, (n,), dev) and
            _is(cu_seqlens, torch.int32, (n + 1,), dev)):
        _check_dense(what, k.device, page_table=(page_table, torch.int32, (n, width)),
                     starts=(starts, torch.int32, (n,)), cu_seqlens=(cu_seqlens, torch.int32, (n + 1,)))
    _, _, P, Hp, ps, Dp, stride = (_is_pool(k_pages, v_pages, k.dtype, dev) or
                                   _check_pool(what, k.dtype, k.device, k_pages, v_pages))
    if (Hp, Dp) != (Hkv, D):
        raise ValueError(f"{what}: k has {Hkv} heads of {D}, the pools {Hp} of {Dp}")
    with _scope(k.device, stream):
        s = library().forge_attn_paged_append(k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                              page_table.data_ptr(), starts.data_ptr(), _at(cu_seqlens), n, rows, Hkv,
                                              D, P, ps, width, ks, vs, stride, dtype_code(k.dtype), _here(k.device))
    if s != FORGE_OK:
        raise ForgeError(s, "forge_attn_paged_append")


def _host_ints(what, name, x):
    import torch
    if isinstance(x, torch.Tensor):
        if x.is_cuda:
            raise ValueError(f"{what}: {name} must be on the host")
        if x.dim() == 1 and x.dtype is torch.int32 and x.is_contiguous():
            return x
        if x.dim() != 1 or x.dtype not in (torch.int32, torch.int64):
            raise ValueError(f"{what}: {name} must be a list of page numbers")
        if x.dtype == torch.int64 and x.numel() and (int(x.min()) < 0 or int(x.max()) >= 1 << 31):
            raise ValueError(f"{what}: {name} has a page number out of range")
        return x.to(torch.int32).contiguous()
    try:
        pages = [operator.index(i) for i in x]
    except TypeError:
        raise ValueError(f"{what}: {name} must be a list of page numbers") from None
    if pages and (min(pages) < -1 << 31 or max(pages) >= 1 << 31):
        raise ValueError(f"{what}: {name} has a page number out of range")
    return torch.tensor(pages, dtype=torch.int32)


def paged_copy(k_pages, v_pages, src, dst, stream=None):
    """Copy page src[i] onto page dst[i], i = 0, 1, .. in that order, in both pools: [num_pages,Hkv,page_size,D],
    or [layers,num_pages,..] for every layer at once. src, dst: page numbers on the host (lists or CPU
    tensors), read before the call returns."""
    what = "paged_copy"
    src, dst = _host_ints(what, "src", src), _host_ints(what, "dst", dst)
    if src.numel() != dst.numel():
        raise ValueError(f"{what}: {src.numel()} sources for {dst.numel()} destinations")
    nl, ls, P, Hkv, ps, D, stride = (_is_pool(k_pages, v_pages, k_pages.dtype, k_pages.get_device(), layers=True) or
                                     _check_pool(what, k_pages.dtype, k_pages.device, k_pages, v_pages, layers=True))
    with _scope(k_pages.device, stream):
        s = library().forge_attn_paged_copy(k_pages.data_ptr(), v_pages.data_ptr(), src.data_ptr(), dst.data_ptr(),
                                            src.numel(), nl, ls, P, Hkv, ps, D, stride, dtype_code(k_pages.dtype),
                                            _here(k_pages.device))
    if s != FORGE_OK:
        raise ForgeError(s, "forge_attn_paged_copy")


from .paged_cache import PagedCache  # noqa: E402  (imports no torch)
