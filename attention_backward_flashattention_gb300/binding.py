"""ctypes binding of the C ABI in ``include/attn.h`` (libattn_gb300.so).

The functions named like the C entry points (``attn_fwd``, ``attn_bwd``, ...)
only marshal arguments: tensors become device pointers, streams become
``cudaStream_t`` handles, and the integer status comes back unchanged.
``forward`` / ``backward`` are conveniences on top that allocate outputs and
the workspace with PyTorch (device memory only) and raise ``AttnError`` on a
non-zero status.  Every step of the computation runs in the library's CUDA
kernels: there is no CPU path, and a missing library raises at first use.
"""
from __future__ import annotations

import array
import ctypes
import math
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libattn_gb300.so")

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = -1
ATTN_ERR_UNSUPPORTED = -2
ATTN_ERR_WORKSPACE_TOO_SMALL = -3
ATTN_ERR_CUDA = -4
ATTN_ERR_TIMEOUT = -5
ATTN_ERR_INTERNAL = -6
ATTN_ERR_SCRATCH_TOO_SMALL = -7
ATTN_ERR_BAD_PAGE = -8
ATTN_ERR_WORKSPACE_NOT_READY = -9
LAYOUT_BTHD = 0
LAYOUT_PACKED_QKV = 1
MAX_VARLEN_SEQS = 1024
ROPE_HALVES, ROPE_PAIRS = 0, 1
CACHE_BF16, CACHE_E4M3 = 0, 1

EXPORTED = ("attn_fwd", "attn_bwd_workspace_size", "attn_bwd", "attn_bwd_status",
            "attn_fwd_status", "attn_strerror", "attn_varlen_order", "attn_debug_set_wait_bias",
            "attn_profile_main_kernel", "attn_profile_aux_kernels", "attn_bwd_noalloc",
            "attn_bwd_noalloc_status", "attn_step_host_scratch_size", "attn_step_host",
            "attn_step_host_status", "attn_fwd_window", "attn_bwd_window", "attn_fwd_ex",
            "attn_bwd_ex", "attn_debug_cache_stats", "attn_debug_set_bwd_variant",
            "attn_rope_rates", "attn_rope", "attn_cache_append", "attn_cache_status",
            "attn_decode", "attn_decode_workspace_size", "attn_decode_workspace_init",
            "attn_fwd_grouped", "attn_bwd_grouped", "attn_bwd_grouped_workspace_size",
            "attn_prefill",
            "attn_prefill_workspace_size", "attn_norm_rope", "attn_norm_rope_bwd",
            "attn_norm_rope_bwd_workspace_size", "attn_cache_append_norm")
BLOCK = 128  # rows per block of a block-sparse mask

_lock = threading.Lock()
_lib = None


class AttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {strerror(code)} ({code})")
        self.code = code


class _RotationStruct(ctypes.Structure):
    """attn_rotation of include/attn.h."""
    _fields_ = [("rates", ctypes.c_void_p), ("begin", ctypes.c_int), ("dim", ctypes.c_int),
                ("style", ctypes.c_int)]


class _NormStruct(ctypes.Structure):
    """attn_head_norm of include/attn.h."""
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


class _NormRowsStruct(ctypes.Structure):
    """attn_norm_rows of include/attn.h."""
    _fields_ = [(n, ctypes.c_longlong) for n in ("q", "k", "dq_out", "dk_out", "dq", "dk")]


class _RowsStruct(ctypes.Structure):
    """attn_rows of include/attn.h."""
    _fields_ = [(n, ctypes.c_longlong) for n in ("q", "k", "v", "o", "d_o", "dq", "dk", "dv")]


class _CacheStruct(ctypes.Structure):
    """attn_paged_cache of include/attn.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + \
               [(f"{s}_{n}_stride", ctypes.c_longlong) for s in "kv"
                for n in ("page", "token", "head")] + \
               [(n, ctypes.c_int) for n in ("type", "num_pages", "page_size", "heads", "dqk",
                                            "dv")]


def load():
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m attention_backward_flashattention_gb300.build`")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.attn_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, F, P, I, P]
        lib.attn_fwd.restype = I
        lib.attn_fwd_window.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, P, I, P]
        lib.attn_fwd_window.restype = I
        lib.attn_bwd_window.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F,
                                        P, I, I, P, SZ, P]
        lib.attn_bwd_window.restype = I
        lib.attn_fwd_ex.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, P, I, I, F, P, P,
                                    I, P]
        lib.attn_fwd_ex.restype = I
        lib.attn_bwd_ex.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, P, I, I,
                                    F, P, P, I, I, P, SZ, P]
        lib.attn_bwd_ex.restype = I
        lib.attn_bwd_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
        lib.attn_bwd_workspace_size.restype = SZ
        lib.attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, P, I, I, P,
                                 SZ, P]
        lib.attn_bwd.restype = I
        lib.attn_bwd_noalloc.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, P, I,
                                         I, P]
        lib.attn_bwd_noalloc.restype = I
        lib.attn_bwd_noalloc_status.argtypes = [P]
        lib.attn_bwd_noalloc_status.restype = I
        lib.attn_bwd_status.argtypes = [P, P]
        lib.attn_bwd_status.restype = I
        lib.attn_fwd_status.argtypes = [P]
        lib.attn_fwd_status.restype = I
        lib.attn_strerror.argtypes = [I]
        lib.attn_strerror.restype = ctypes.c_char_p
        lib.attn_varlen_order.argtypes = [P, I, P]
        lib.attn_varlen_order.restype = I
        lib.attn_profile_main_kernel.argtypes = [P, P]
        lib.attn_profile_main_kernel.restype = I
        lib.attn_profile_aux_kernels.argtypes = [P, P, P, P]
        lib.attn_profile_aux_kernels.restype = I
        lib.attn_debug_set_bwd_variant.argtypes = [I]
        lib.attn_debug_set_bwd_variant.restype = I
        lib.attn_debug_cache_stats.argtypes = [P]
        lib.attn_debug_cache_stats.restype = I
        lib.attn_debug_set_wait_bias.argtypes = [I]
        lib.attn_debug_set_wait_bias.restype = I
        lib.attn_step_host_scratch_size.argtypes = [I, I, I, I, I, I, I]
        lib.attn_step_host_scratch_size.restype = SZ
        lib.attn_step_host.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, I, P, SZ,
                                       P, P, P, P]
        lib.attn_step_host.restype = I
        lib.attn_step_host_status.argtypes = [P, I, I, I, I, I, I, I, P]
        lib.attn_step_host_status.restype = I
        L = ctypes.c_longlong
        lib.attn_rope_rates.argtypes = [P, I, P]
        lib.attn_rope_rates.restype = I
        lib.attn_rope.argtypes = [P, P, P, P, I, I, I, I, I, I, L, L, L, L, P, I, I, P, P, P]
        lib.attn_rope.restype = I
        lib.attn_cache_append.argtypes = [P, P, I, L, P, I, I, P, P, L, P, L, P, L, P, L, I, P, P]
        lib.attn_cache_append.restype = I
        lib.attn_cache_status.argtypes = [P]
        lib.attn_cache_status.restype = I
        lib.attn_decode_workspace_size.argtypes = []
        lib.attn_decode_workspace_size.restype = SZ
        lib.attn_decode_workspace_init.argtypes = [P, SZ, P]
        lib.attn_decode_workspace_init.restype = I
        lib.attn_decode.argtypes = [P, P, I, L, P, I, P, L, P, P, I, I, F, P, SZ, P]
        lib.attn_decode.restype = I
        lib.attn_fwd_grouped.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, P, I, I, I, F, P, P,
                                         P]
        lib.attn_fwd_grouped.restype = I
        lib.attn_bwd_grouped_workspace_size.argtypes = [I, I, I, I, I, I, I, I, I]
        lib.attn_bwd_grouped_workspace_size.restype = SZ
        lib.attn_bwd_grouped.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, I, I,
                                         I, F, P, P, I, P, SZ, P]
        lib.attn_bwd_grouped.restype = I
        lib.attn_prefill_workspace_size.argtypes = []
        lib.attn_prefill_workspace_size.restype = SZ
        lib.attn_prefill.argtypes = [P, P, I, L, P, I, I, P, P, L, P, P, I, I, F, P, SZ, P]
        lib.attn_prefill.restype = I
        lib.attn_norm_rope.argtypes = [P, P, P, P, I, I, I, I, I, I, L, L, L, L, P, P, I, P, P, P]
        lib.attn_norm_rope.restype = I
        lib.attn_norm_rope_bwd_workspace_size.argtypes = [I]
        lib.attn_norm_rope_bwd_workspace_size.restype = SZ
        lib.attn_norm_rope_bwd.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, P, P, P, I, P,
                                           P, P, SZ, P]
        lib.attn_norm_rope_bwd.restype = I
        lib.attn_cache_append_norm.argtypes = [P, P, I, L, P, I, I, P, P, L, P, L, P, L, P, L, I,
                                               P, P, P]
        lib.attn_cache_append_norm.restype = I
        _lib = lib
        return lib


def _ptr(x):
    if isinstance(x, torch.Tensor):
        return x.data_ptr()
    if x is None:
        return None
    return int(x)


# the current stream's handle without a Stream object (a tenth of the time, where it exists)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(s):
    if s is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, torch.cuda.Stream):
        return s.cuda_stream
    return int(s)


def _c_int(v):
    """v as the nearest int that C's has room for (ctypes would cut off the upper bits): a window
    longer than any sequence stays one, and a position out of range is refused by the library."""
    v = int(v)
    return v if -2 ** 31 <= v < 2 ** 31 else 2 ** 31 - 1 if v > 0 else -2 ** 31


class _HostInts:
    """Keeps a host int32 array alive for the duration of a call."""

    __slots__ = ("arr",)

    def __init__(self, values):
        if values is None:
            self.arr = None
            return
        if hasattr(values, "tolist"):
            values = values.tolist()
        try:
            self.arr = array.array("i", values)
        except TypeError:
            self.arr = array.array("i", [int(v) for v in values])

    @property
    def ptr(self):
        return None if self.arr is None else self.arr.buffer_info()[0]


# ----------------------------------------------------------------------------
# C entry points (same names, argument marshalling only)
# ----------------------------------------------------------------------------
def attn_fwd(q, k, v, o, lse, B, H, Tq, Tk, dqk, dv, causal, scale, cu_seqlens=None,
             layout=LAYOUT_BTHD, stream=None) -> int:
    cu = _HostInts(cu_seqlens)
    return load().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Tq, Tk, dqk, dv,
                           int(causal), float(scale), cu.ptr, layout, _stream(stream))


def attn_fwd_window(q, k, v, o, lse, B, H, Tq, Tk, dqk, dv, causal, window_left, window_right,
                    scale, cu_seqlens=None, layout=LAYOUT_BTHD, stream=None) -> int:
    cu = _HostInts(cu_seqlens)
    return load().attn_fwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Tq, Tk,
                                  dqk, dv, int(causal), _c_int(window_left), _c_int(window_right),
                                  float(scale), cu.ptr, layout, _stream(stream))


def attn_bwd_window(q, k, v, o, dO, lse, dq, dk, dv_out, B, H, Tq, Tk, dqk, dv, causal,
                    window_left, window_right, scale, cu_seqlens=None, layout=LAYOUT_BTHD,
                    deterministic=False, workspace=None, workspace_bytes=0, stream=None) -> int:
    cu = _HostInts(cu_seqlens)
    return load().attn_bwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse),
                                  _ptr(dq), _ptr(dk), _ptr(dv_out), B, H, Tq, Tk, dqk, dv,
                                  int(causal), _c_int(window_left), _c_int(window_right),
                                  float(scale), cu.ptr, layout, int(deterministic),
                                  _ptr(workspace), int(workspace_bytes), _stream(stream))


def attn_fwd_ex(q, k, v, o, lse, B, H, Tq, Tk, dqk, dv, causal, window_left, window_right,
                block_mask, mask_batches, mask_heads, scale, cu_seqlens_q=None,
                cu_seqlens_k=None, layout=LAYOUT_BTHD, stream=None) -> int:
    cq, ck = _HostInts(cu_seqlens_q), _HostInts(cu_seqlens_k)
    return load().attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Tq, Tk, dqk,
                              dv, int(causal), _c_int(window_left), _c_int(window_right),
                              _ptr(block_mask), int(mask_batches), int(mask_heads), float(scale),
                              cq.ptr, ck.ptr, layout, _stream(stream))


def attn_bwd_ex(q, k, v, o, dO, lse, dq, dk, dv_out, B, H, Tq, Tk, dqk, dv, causal, window_left,
                window_right, block_mask, mask_batches, mask_heads, scale, cu_seqlens_q=None,
                cu_seqlens_k=None, layout=LAYOUT_BTHD, deterministic=False, workspace=None,
                workspace_bytes=0, stream=None) -> int:
    cq, ck = _HostInts(cu_seqlens_q), _HostInts(cu_seqlens_k)
    return load().attn_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(dq),
                              _ptr(dk), _ptr(dv_out), B, H, Tq, Tk, dqk, dv, int(causal),
                              _c_int(window_left), _c_int(window_right), _ptr(block_mask),
                              int(mask_batches), int(mask_heads), float(scale), cq.ptr, ck.ptr,
                              layout, int(deterministic), _ptr(workspace), int(workspace_bytes),
                              _stream(stream))


def attn_fwd_grouped(q, k, v, o, lse, B, Hq, Hk, Tq, Tk, dqk, dv, rows, causal, window_left,
                     window_right, scale, cu_seqlens_q=None, cu_seqlens_k=None,
                     stream=None) -> int:
    cq, ck = _HostInts(cu_seqlens_q), _HostInts(cu_seqlens_k)
    return load().attn_fwd_grouped(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hk, Tq,
                                   Tk, dqk, dv, _struct(rows), int(causal), _c_int(window_left),
                                   _c_int(window_right), float(scale), cq.ptr, ck.ptr,
                                   _stream(stream))


def attn_bwd_grouped_workspace_size(B, Hq, Hk, Tq, Tk, dqk, dv, varlen=False,
                                    deterministic=False) -> int:
    return int(load().attn_bwd_grouped_workspace_size(B, Hq, Hk, Tq, Tk, dqk, dv, int(varlen),
                                                      int(deterministic)))


def attn_bwd_grouped(q, k, v, o, dO, lse, dq, dk, dv_out, B, Hq, Hk, Tq, Tk, dqk, dv, rows,
                     causal, window_left, window_right, scale, cu_seqlens_q=None,
                     cu_seqlens_k=None, deterministic=False, workspace=None, workspace_bytes=0,
                     stream=None) -> int:
    cq, ck = _HostInts(cu_seqlens_q), _HostInts(cu_seqlens_k)
    return load().attn_bwd_grouped(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse),
                                   _ptr(dq), _ptr(dk), _ptr(dv_out), B, Hq, Hk, Tq, Tk, dqk, dv,
                                   _struct(rows), int(causal), _c_int(window_left),
                                   _c_int(window_right), float(scale), cq.ptr, ck.ptr,
                                   int(deterministic), _ptr(workspace), int(workspace_bytes),
                                   _stream(stream))


def _mask_dims(block_mask):
    """(mask, mask_batches, mask_heads) of a [NQ][NK] or [Bm][Hm][NQ][NK] uint8
    device tensor (None: no block mask)."""
    if block_mask is None:
        return None, 1, 1
    if block_mask.dtype != torch.uint8 or not block_mask.is_contiguous():
        raise ValueError("block_mask must be a contiguous uint8 tensor")
    if block_mask.dim() == 2:
        return block_mask, 1, 1
    if block_mask.dim() != 4:
        raise ValueError("block_mask must be [NQ][NK] or [Bm][Hm][NQ][NK]")
    return block_mask, block_mask.shape[0], block_mask.shape[1]


def attn_bwd_workspace_size(B, H, Tq, Tk, dqk, dv, varlen=False, deterministic=False) -> int:
    return int(load().attn_bwd_workspace_size(B, H, Tq, Tk, dqk, dv, int(varlen),
                                              int(deterministic)))


def attn_bwd(q, k, v, o, dO, lse, dq, dk, dv_out, B, H, Tq, Tk, dqk, dv, causal, scale,
             cu_seqlens=None, layout=LAYOUT_BTHD, deterministic=False, workspace=None,
             workspace_bytes=0, stream=None) -> int:
    cu = _HostInts(cu_seqlens)
    return load().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(dq),
                           _ptr(dk), _ptr(dv_out), B, H, Tq, Tk, dqk, dv, int(causal),
                           float(scale), cu.ptr, layout, int(deterministic), _ptr(workspace),
                           int(workspace_bytes), _stream(stream))


def attn_bwd_noalloc(q, k, v, o, dO, lse, dq, dk, dv_out, B, H, Tq, Tk, dqk, dv, causal, scale,
                     cu_seqlens=None, layout=LAYOUT_BTHD, deterministic=False,
                     stream=None) -> int:
    """attn_bwd without a caller workspace (the library's 32 MiB device array)."""
    cu = _HostInts(cu_seqlens)
    return load().attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse),
                                   _ptr(dq), _ptr(dk), _ptr(dv_out), B, H, Tq, Tk, dqk, dv,
                                   int(causal), float(scale), cu.ptr, layout, int(deterministic),
                                   _stream(stream))


def attn_bwd_noalloc_status(stream=None) -> int:
    return load().attn_bwd_noalloc_status(_stream(stream))


def attn_bwd_status(workspace, stream=None) -> int:
    return load().attn_bwd_status(_ptr(workspace), _stream(stream))


def attn_fwd_status(stream=None) -> int:
    return load().attn_fwd_status(_stream(stream))


def attn_strerror(code: int) -> str:
    return load().attn_strerror(int(code)).decode()


def strerror(code: int) -> str:
    try:
        return attn_strerror(code)
    except RuntimeError:
        return f"code {code}"


def attn_profile_main_kernel(event_start=None, event_stop=None) -> int:
    """Record torch.cuda.Event (or raw cudaEvent_t) pairs around the backward main kernel."""
    conv = lambda e: None if e is None else (e.cuda_event if hasattr(e, "cuda_event") else int(e))
    return load().attn_profile_main_kernel(conv(event_start), conv(event_stop))


def attn_profile_aux_kernels(pre_start=None, pre_stop=None, convert_start=None,
                             convert_stop=None) -> int:
    """Record event pairs around the backward's preprocess and dQ conversion kernels."""
    conv = lambda e: None if e is None else (e.cuda_event if hasattr(e, "cuda_event") else int(e))
    return load().attn_profile_aux_kernels(conv(pre_start), conv(pre_stop), conv(convert_start),
                                           conv(convert_stop))


BWD_AUTO, BWD_ONE_CTA, BWD_CTA_PAIR = 0, 1, 2


def attn_debug_set_bwd_variant(variant: int) -> int:
    """Backward main kernel where both apply: 0 library's choice, 1 one CTA, 2 CTA pairs."""
    return load().attn_debug_set_bwd_variant(int(variant))


def attn_debug_cache_stats() -> dict:
    """Host-side cache counters (tensor maps encoded / reused, tables built / reused)."""
    out = (ctypes.c_longlong * 4)()
    rc = load().attn_debug_cache_stats(ctypes.cast(out, ctypes.c_void_p))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_debug_cache_stats")
    return {"map_encodes": out[0], "map_hits": out[1], "table_builds": out[2],
            "table_hits": out[3]}


def attn_debug_set_wait_bias(bias: int) -> int:
    return load().attn_debug_set_wait_bias(int(bias))


def attn_step_host_scratch_size(B, H, T, dqk, dv, heads_per_group=0, deterministic=False) -> int:
    return int(load().attn_step_host_scratch_size(B, H, T, dqk, dv, int(heads_per_group),
                                                  int(deterministic)))


def attn_step_host(q, k, v, dO, o, dq, dk, dv_out, B, H, T, dqk, dv, causal, scale,
                   deterministic=False, heads_per_group=0, scratch=None, scratch_bytes=0,
                   stream=None, stream2=None, h2d_stream=None, d2h_stream=None) -> int:
    """Host tensors in and out (pinned CPU tensors); copies overlapped with the kernels."""
    opt = lambda s: None if s is None else _stream(s)
    return load().attn_step_host(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(o), _ptr(dq),
                                 _ptr(dk), _ptr(dv_out), B, H, T, dqk, dv, int(causal),
                                 float(scale), int(deterministic), int(heads_per_group),
                                 _ptr(scratch), int(scratch_bytes), _stream(stream),
                                 opt(stream2), opt(h2d_stream), opt(d2h_stream))


def attn_step_host_status(scratch, B, H, T, dqk, dv, heads_per_group=0, deterministic=False,
                          stream=None) -> int:
    return load().attn_step_host_status(_ptr(scratch), B, H, T, dqk, dv, int(heads_per_group),
                                        int(deterministic), _stream(stream))


def attn_varlen_order(cu_seqlens) -> list:
    cu = _HostInts(cu_seqlens)
    n = len(cu.arr) - 1
    out = (ctypes.c_int * max(n, 1))()
    rc = load().attn_varlen_order(cu.ptr, n, ctypes.cast(out, ctypes.c_void_p))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_varlen_order")
    return list(out)[:n]


def attn_rope_rates(rates_rad) -> list:
    """Fixed-point form (turns per position, times 2^64) of rates in radians per position."""
    vals = [float(r) for r in rates_rad]
    src = (ctypes.c_double * max(len(vals), 1))(*vals)
    out = (ctypes.c_ulonglong * max(len(vals), 1))()
    rc = load().attn_rope_rates(ctypes.cast(src, ctypes.c_void_p), len(vals),
                                ctypes.cast(out, ctypes.c_void_p))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_rope_rates")
    return list(out)[:len(vals)]


def _struct(x):
    """Address of a ctypes structure (or of a Rotation's or PagedCache's), or None."""
    if x is None:
        return None
    if isinstance(x, ctypes.Structure):
        return ctypes.addressof(x)
    return x.address


def attn_rope(q, k, q_out, k_out, B, Hq, Hk, Tq, Tk, d, q_row, k_row, q_out_row, k_out_row,
              rotation, inverse=False, pos0=0, cu_seqlens_q=None, cu_seqlens_k=None,
              stream=None) -> int:
    cq, ck = _HostInts(cu_seqlens_q), _HostInts(cu_seqlens_k)
    return load().attn_rope(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), B, Hq, Hk, Tq, Tk, d,
                            q_row, k_row, q_out_row, k_out_row, _struct(rotation), int(inverse),
                            _c_int(pos0), cq.ptr, ck.ptr, _stream(stream))


def attn_cache_append(cache, block_table, max_pages, table_stride, lens, B, T, cu_seqlens, k,
                      k_row, v, v_row, q, q_row, q_out, q_out_row, Hq, rotation=None,
                      stream=None) -> int:
    cu = _HostInts(cu_seqlens)
    return load().attn_cache_append(_struct(cache), _ptr(block_table), max_pages, table_stride,
                                    _ptr(lens), B, T, cu.ptr, _ptr(k), k_row, _ptr(v), v_row,
                                    _ptr(q), q_row, _ptr(q_out), q_out_row, Hq,
                                    _struct(rotation), _stream(stream))


def attn_cache_append_norm(cache, block_table, max_pages, table_stride, lens, B, T, cu_seqlens, k,
                           k_row, v, v_row, q, q_row, q_out, q_out_row, Hq, norm=None,
                           rotation=None, stream=None) -> int:
    cu = _HostInts(cu_seqlens)
    return load().attn_cache_append_norm(_struct(cache), _ptr(block_table), max_pages,
                                         table_stride, _ptr(lens), B, T, cu.ptr, _ptr(k), k_row,
                                         _ptr(v), v_row, _ptr(q), q_row, _ptr(q_out), q_out_row,
                                         Hq, _struct(norm), _struct(rotation), _stream(stream))


def attn_norm_rope(q, k, q_out, k_out, B, Hq, Hk, Tq, Tk, d, q_row, k_row, q_out_row, k_out_row,
                   norm, rotation=None, pos0=0, cu_seqlens_q=None, cu_seqlens_k=None,
                   stream=None) -> int:
    cq, ck = _HostInts(cu_seqlens_q), _HostInts(cu_seqlens_k)
    return load().attn_norm_rope(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), B, Hq, Hk, Tq, Tk, d,
                                 q_row, k_row, q_out_row, k_out_row, _struct(norm),
                                 _struct(rotation), _c_int(pos0), cq.ptr, ck.ptr, _stream(stream))


def attn_norm_rope_bwd_workspace_size(d) -> int:
    return int(load().attn_norm_rope_bwd_workspace_size(int(d)))


def attn_norm_rope_bwd(q, k, dq_out, dk_out, dq, dk, dq_weight, dk_weight, B, Hq, Hk, Tq, Tk, d,
                       rows, norm, rotation=None, pos0=0, cu_seqlens_q=None, cu_seqlens_k=None,
                       workspace=None, workspace_bytes=0, stream=None) -> int:
    cq, ck = _HostInts(cu_seqlens_q), _HostInts(cu_seqlens_k)
    return load().attn_norm_rope_bwd(_ptr(q), _ptr(k), _ptr(dq_out), _ptr(dk_out), _ptr(dq),
                                     _ptr(dk), _ptr(dq_weight), _ptr(dk_weight), B, Hq, Hk, Tq, Tk,
                                     d, _struct(rows), _struct(norm), _struct(rotation),
                                     _c_int(pos0), cq.ptr, ck.ptr, _ptr(workspace),
                                     int(workspace_bytes), _stream(stream))


def attn_cache_status(stream=None) -> int:
    return load().attn_cache_status(_stream(stream))


def attn_decode_workspace_size() -> int:
    return int(load().attn_decode_workspace_size())


def attn_decode_workspace_init(workspace, workspace_bytes, stream=None) -> int:
    return load().attn_decode_workspace_init(_ptr(workspace), int(workspace_bytes),
                                             _stream(stream))


def attn_decode(cache, block_table, max_pages, table_stride, lens, B, q, q_row, o, lse, Hq,
                window_left, scale, workspace, workspace_bytes, stream=None) -> int:
    return load().attn_decode(_struct(cache), _ptr(block_table), max_pages, table_stride,
                              _ptr(lens), B, _ptr(q), q_row, _ptr(o), _ptr(lse), Hq,
                              _c_int(window_left), float(scale), _ptr(workspace),
                              int(workspace_bytes), _stream(stream))


def attn_prefill_workspace_size() -> int:
    return int(load().attn_prefill_workspace_size())


def attn_prefill(cache, block_table, max_pages, table_stride, lens, B, T, cu_seqlens, q, q_row, o,
                 lse, Hq, window_left, scale, workspace, workspace_bytes, stream=None) -> int:
    cu = _HostInts(cu_seqlens)
    return load().attn_prefill(_struct(cache), _ptr(block_table), max_pages, table_stride,
                               _ptr(lens), B, T, cu.ptr, _ptr(q), q_row, _ptr(o), _ptr(lse), Hq,
                               _c_int(window_left), float(scale), _ptr(workspace),
                               int(workspace_bytes), _stream(stream))


# ----------------------------------------------------------------------------
# Conveniences: shapes from tensors, outputs allocated with torch
# ----------------------------------------------------------------------------
def _dims(q, k, v, cu_seqlens, layout):
    # the library sees only pointers: a tensor whose rank does not match the
    # layout would be read with the wrong sizes
    rank = (3 if cu_seqlens is not None else 4) + (1 if layout == LAYOUT_PACKED_QKV else 0)
    if layout == LAYOUT_PACKED_QKV:
        rank -= 1  # q, k, v are slot views: (..., H, d) of a (..., 3, H, d) buffer
    if any(t.dim() != rank for t in (q, k, v)):
        raise ValueError(f"q, k, v must have {rank} dimensions for this layout "
                         f"({'variable length' if cu_seqlens is not None else 'fixed length'})")
    if layout == LAYOUT_PACKED_QKV:
        # q, k, v are slot views of one (..., 3, H, d) buffer
        H, dqk = q.shape[-2], q.shape[-1]
        dv = v.shape[-1]
    else:
        H, dqk, dv = q.shape[-2], q.shape[-1], v.shape[-1]
    if cu_seqlens is not None:
        B = len(cu_seqlens) - 1
        Tq, Tk = q.shape[0], k.shape[0]
    else:
        B, Tq, Tk = q.shape[0], q.shape[1], k.shape[1]
    return B, H, Tq, Tk, dqk, dv


def forward(q, k, v, causal=False, scale=None, cu_seqlens=None, layout=LAYOUT_BTHD,
            with_lse=True, stream=None, window=None, block_mask=None, cu_seqlens_k=None):
    """O (bf16, like q with v's head size) and LSE (fp32) or None.
    window: (left, right) local-attention bounds (-1: open side), or None.
    block_mask: device uint8 [NQ][NK] or [Bm][Hm][NQ][NK] (NQ, NK: blocks of
    BLOCK rows), non-zero = the block pair takes part, or None.
    cu_seqlens_k: key offsets of a variable-length batch when they differ
    from cu_seqlens (the query offsets), or None.
    k and v may have fewer heads than q (grouped heads: query head h uses key
    head h * Hk // Hq), and q, k, v rows that lie apart (slices of one
    projection); neither goes with a block mask."""
    B, H, Tq, Tk, dqk, dv = _dims(q, k, v, cu_seqlens, layout)
    scale = 1.0 / math.sqrt(dqk) if scale is None else scale
    if layout == LAYOUT_BTHD and _is_grouped(q, k, v):
        return _forward_grouped(q, k, v, causal, scale, cu_seqlens, with_lse, stream, window,
                                block_mask, cu_seqlens_k)
    o = torch.empty(q.shape[:-2] + (H, dv), dtype=torch.bfloat16, device=q.device)
    lse = None
    if with_lse:
        lse = torch.empty((H, Tq) if cu_seqlens is not None else (B, H, Tq),
                          dtype=torch.float32, device=q.device)
    wl, wr = (-1, -1) if window is None else window
    bm, mb, mh = _mask_dims(block_mask)
    rc = attn_fwd_ex(q, k, v, o, lse, B, H, Tq, Tk, dqk, dv, causal, wl, wr, bm, mb, mh, scale,
                     cu_seqlens, cu_seqlens_k, layout, stream)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd")
    return o, lse


def backward(q, k, v, o, dO, lse, causal=False, scale=None, cu_seqlens=None,
             layout=LAYOUT_BTHD, deterministic=False, workspace=None, stream=None, out=None,
             window=None, block_mask=None, cu_seqlens_k=None):
    """(dq, dk, dv) as bf16 tensors shaped like q, k, v (a packed buffer for layout 1).
    window, block_mask, cu_seqlens_k, grouped heads and rows that lie apart: as in
    forward(); dk and dv then have the key heads, summed over their query heads."""
    B, H, Tq, Tk, dqk, dv = _dims(q, k, v, cu_seqlens, layout)
    scale = 1.0 / math.sqrt(dqk) if scale is None else scale
    if layout == LAYOUT_BTHD and _is_grouped(q, k, v, o, dO, *(out if out is not None else ())):
        return _backward_grouped(q, k, v, o, dO, lse, causal, scale, cu_seqlens, deterministic,
                                 workspace, stream, out, window, block_mask, cu_seqlens_k)
    if out is not None:
        dq, dk, dvt = out
    elif layout == LAYOUT_PACKED_QKV:
        g = torch.empty(q.shape[:-2] + (3, H, dqk), dtype=torch.bfloat16, device=q.device)
        dq, dk, dvt = g.select(-3, 0), g.select(-3, 1), g.select(-3, 2)
    else:
        dq = torch.empty_like(q)
        dk = torch.empty_like(k)
        dvt = torch.empty_like(v)
    need = attn_bwd_workspace_size(B, H, Tq, Tk, dqk, dv, cu_seqlens is not None, deterministic)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    wl, wr = (-1, -1) if window is None else window
    bm, mb, mh = _mask_dims(block_mask)
    rc = attn_bwd_ex(q, k, v, o, dO, lse, dq, dk, dvt, B, H, Tq, Tk, dqk, dv, causal, wl, wr, bm,
                     mb, mh, scale, cu_seqlens, cu_seqlens_k, layout, deterministic, workspace,
                     workspace.numel() * workspace.element_size(), stream)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_bwd")
    return dq, dk, dvt


def step_host(q, k, v, dO, causal=False, scale=None, deterministic=False, heads_per_group=0,
              with_o=False, out=None, scratch=None, streams=None, device=None):
    """Forward + backward of host (B,T,H,d) bf16 tensors through attn_step_host.

    Returns (dq, dk, dv, o) as host tensors (o is None unless with_o).  Pass
    pinned tensors for overlapped copies; `out` reuses (dq, dk, dv, o) host
    buffers, `scratch` a device uint8 buffer, `streams` a (compute, compute2,
    h2d, d2h) tuple (compute2 may be None).  The call is asynchronous: synchronise the compute stream before
    reading the outputs (this helper does so unless `streams` is given)."""
    B, T, H, dqk = q.shape
    dv = v.shape[-1]
    scale = 1.0 / math.sqrt(dqk) if scale is None else scale
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    if out is None:
        mk = lambda t: torch.empty(t.shape, dtype=torch.bfloat16, pin_memory=True)
        out = (mk(q), mk(k), mk(v), mk(v) if with_o else None)
    need = attn_step_host_scratch_size(B, H, T, dqk, dv, heads_per_group, deterministic)
    if scratch is None or scratch.numel() * scratch.element_size() < need:
        scratch = torch.empty(need, dtype=torch.uint8, device=dev)
    own = streams is None
    if own:
        streams = (torch.cuda.current_stream(dev), torch.cuda.Stream(dev), torch.cuda.Stream(dev),
                   torch.cuda.Stream(dev))
    cs, cs2, hs, ds = streams
    dq, dk, dvt, o = out
    rc = attn_step_host(q, k, v, dO, o, dq, dk, dvt, B, H, T, dqk, dv, causal, scale,
                        deterministic, heads_per_group, scratch,
                        scratch.numel() * scratch.element_size(), cs, cs2, hs, ds)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_step_host")
    if own:
        cs.synchronize()
    return dq, dk, dvt, o


# ----------------------------------------------------------------------------
# Position rotation, paged cache, decode
# ----------------------------------------------------------------------------
class Rotation:
    """The position rotation of a head's columns begin .. begin + 2 * len(inv_freq) - 1.

    inv_freq: the angle (radians) that each pair of columns turns per position, a
    float64 tensor or sequence (any frequencies: base 10000, rescaled ones, ...).
    interleaved: pairs are adjacent columns; else they lie dim/2 apart."""

    def __init__(self, inv_freq, begin=0, interleaved=False, device=None):
        if device is None:
            device = inv_freq.device if getattr(inv_freq, "is_cuda", False) else "cuda"
        vals = inv_freq.double().tolist() if isinstance(inv_freq, torch.Tensor) else inv_freq
        words = attn_rope_rates(vals)
        signed = [w - (1 << 64) if w >> 63 else w for w in words]
        self.rates = torch.tensor(signed, dtype=torch.int64, device=device)
        self.begin, self.dim, self.interleaved = int(begin), 2 * len(words), bool(interleaved)
        self.struct = _RotationStruct(self.rates.data_ptr(), _c_int(self.begin), self.dim,
                                      ROPE_PAIRS if interleaved else ROPE_HALVES)
        self.address = ctypes.addressof(self.struct)


def _rows_apart(t):
    """Whether the rows of a cache tensor (pages, page_size, heads, d) have their own memory each,
    as those of any slice or permutation of a dense tensor have."""
    extent = t.shape[3]
    for stride, size in sorted(zip(t.stride()[:3], t.shape[:3])):
        if size > 1:
            if stride < extent:
                return False
            extent += stride * (size - 1)
    return True


class PagedCache:
    """A paged key / value cache over the caller's tensors.

    k_cache (pages, page_size, heads, dqk) and v_cache (pages, page_size, heads, dv),
    bf16 or float8_e4m3fn, with any strides whose columns are adjacent (a cache kept
    as (pages, heads, page_size, d) is passed transposed; one with broadcast dimensions can be
    read, but not appended to).  k_scale, v_scale: fp32
    per key head, the value of one stored unit of an e4m3 cache (None: 1)."""

    def __init__(self, k_cache, v_cache, k_scale=None, v_scale=None):
        if k_cache.dim() != 4 or v_cache.dim() != 4 or k_cache.shape[:3] != v_cache.shape[:3]:
            raise ValueError("k_cache and v_cache must be (pages, page_size, heads, d) with the "
                             "same pages, page_size and heads")
        kinds = {torch.bfloat16: CACHE_BF16, torch.float8_e4m3fn: CACHE_E4M3}
        if k_cache.dtype not in kinds or v_cache.dtype != k_cache.dtype:
            raise ValueError("the caches must both be bfloat16 or both float8_e4m3fn")
        pages, page_size, heads, dqk = k_cache.shape
        if max(k_cache.shape) > 2 ** 31 - 1:
            raise ValueError("a cache's sizes must be below 2^31")
        for t in (k_cache, v_cache):
            if t.stride(3) != 1:
                raise ValueError("the columns of a cache row must be adjacent")
            if t.device != k_cache.device:
                raise ValueError("the caches must be on one device")
        for t in (k_scale, v_scale):
            if t is not None and (t.dtype != torch.float32 or t.numel() != heads
                                  or not t.is_contiguous() or t.device != k_cache.device):
                raise ValueError("k_scale and v_scale must be contiguous fp32, one per key head, "
                                 "on the cache's device")
        self.k_cache, self.v_cache, self.k_scale, self.v_scale = k_cache, v_cache, k_scale, v_scale
        self.rows_apart = _rows_apart(k_cache) and _rows_apart(v_cache)
        self.page_size, self.heads, self.dqk, self.dv = page_size, heads, dqk, v_cache.shape[3]
        self.struct = _CacheStruct(
            k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_scale), _ptr(v_scale),
            *k_cache.stride()[:3], *v_cache.stride()[:3], kinds[k_cache.dtype], pages, page_size,
            heads, dqk, self.dv)
        self.address = ctypes.addressof(self.struct)


class _On:
    """Runs a call on a device and stream: outputs are allocated, and the kernel launched, on
    `stream` (None: the device's current stream)."""

    def __init__(self, index, stream):
        self.stack = []
        if index != torch.cuda.current_device():
            self.stack.append(torch.cuda.device(index))
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=index)
            self.stack.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.stack:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.stack):
            c.__exit__(*exc)


# Uninitialised memory on the current device without torch.empty's way through its dispatcher,
# which takes about 3 us after a launch (two outputs: 16 us a decode call, 11 this way).  Where
# that way is looked at (modes, the filling of new memory in deterministic mode) it is taken.
_empty_strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None),
                         "_empty_strided_cuda", None)
_dispatch_modes = getattr(torch._C, "_len_torch_dispatch_stack", None)
_function_modes = getattr(torch._C, "_len_torch_function_stack", None)
if _dispatch_modes is None or _function_modes is None:
    _empty_strided = None
_empty_is_known = False


def _know_empty(device):
    """The private function is used only where it does what this file takes it to do."""
    global _empty_strided, _empty_is_known
    try:
        got = _empty_strided((2, 3), (3, 1), torch.float32)
        want = torch.empty((2, 3), dtype=torch.float32, device=device)
        same = all(getattr(got, a) == getattr(want, a)
                   for a in ("shape", "dtype", "device", "requires_grad", "layout"))
        if not same or got.stride() != want.stride():
            _empty_strided = None
    except Exception:  # (whatever another version of it raises)
        _empty_strided = None
    _empty_is_known = True


def _empty(shape, dtype, device):
    """torch.empty(shape, dtype=dtype, device=device) for the current CUDA device."""
    shape = tuple(shape)
    if (_empty_strided is None or 0 in shape or _dispatch_modes() or _function_modes()
            or torch.are_deterministic_algorithms_enabled()):
        return torch.empty(shape, dtype=dtype, device=device)
    if not _empty_is_known:
        _know_empty(device)
        return _empty(shape, dtype, device)
    strides, n = (1,), 1
    for d in shape[:0:-1]:
        n *= d
        strides = (n,) + strides
    return _empty_strided(shape, strides, dtype)


# (the current device, once CUDA is up)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _here(index, stream):
    """Whether a call for tensors on device `index` and for `stream` runs where the caller is."""
    return stream is None and index == _get_device()


def _current(index):
    """Handle of the current stream of the current device, `index`."""
    return _stream(None) if _raw_stream is None else _raw_stream(index)


def _rows(t, shape, name):
    """Distance in elements between the token rows of a bf16 tensor t of this shape, (T, H, d) or
    (B, T, H, d), whose rows are evenly spaced, each of adjacent heads and with its own memory."""
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16")
    H, d = shape[-2], shape[-1]
    if t.is_contiguous():
        return H * d
    stride = t.stride()
    if (d > 1 and stride[-1] != 1) or (H > 1 and stride[-2] != d):
        raise ValueError(f"the heads of a row of {name} must be adjacent")
    T = shape[-3]
    row = stride[-3] if T > 1 else H * d
    if len(shape) == 4 and shape[0] > 1:
        if T > 1 and stride[0] != row * T:
            raise ValueError(f"the rows of {name} must be evenly spaced")
        if T == 1:
            row = stride[0]
    if row < H * d:  # (a broadcast dimension has a stride of 0)
        raise ValueError(f"the rows of {name} must have their own memory")
    return row


def _device_of(t, *others):
    """The CUDA device that all of these are on (None entries are passed over).  The kernels
    would read a host pointer as a device address."""
    index = t.get_device()
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    for o in others:
        if o is not None and o.get_device() != index:
            raise ValueError(f"tensors must be on one CUDA device (cuda:{index})")
    return index


# ----------------------------------------------------------------------------
# Grouped heads, rows apart
# ----------------------------------------------------------------------------
def _is_grouped(q, k, v, *others):
    """Whether a call goes to the entry points for grouped heads and rows that lie apart."""
    return (k.shape[-2] != q.shape[-2] or v.shape[-2] != q.shape[-2]
            or not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
                    and all(t.is_contiguous() for t in others)))


def _grouped_dims(q, k, v, cu_seqlens, cu_seqlens_k, window, block_mask):
    """(B, Hq, Hk, Tq, Tk, dqk, dv), (window_left, window_right) of a checked call."""
    if block_mask is not None:
        raise ValueError("a block mask needs as many key heads as query heads, and dense tensors")
    B, Hq, Tq, Tk, dqk, dv = _dims(q, k, v, cu_seqlens, LAYOUT_BTHD)
    Hk = k.shape[-2]
    if k.shape[:-1] != v.shape[:-1] or k.shape[-1] != dqk:
        raise ValueError("k and v must agree in rows and heads, and k with q in head size")
    if Hk == 0 or Hq % Hk:
        raise ValueError("the query heads must be a multiple of the key heads")
    if cu_seqlens is None and k.shape[0] != B:
        raise ValueError("q, k and v must agree in batch")
    if cu_seqlens is not None and cu_seqlens_k is not None and len(cu_seqlens_k) != B + 1:
        raise ValueError("cu_seqlens and cu_seqlens_k must have the same length")
    if cu_seqlens is None and cu_seqlens_k is not None:
        raise ValueError("cu_seqlens_k needs cu_seqlens")
    return (B, Hq, Hk, Tq, Tk, dqk, dv), ((-1, -1) if window is None else window)


def _forward_grouped(q, k, v, causal, scale, cu_seqlens, with_lse, stream, window, block_mask,
                     cu_seqlens_k):
    dims, (wl, wr) = _grouped_dims(q, k, v, cu_seqlens, cu_seqlens_k, window, block_mask)
    B, Hq, Hk, Tq, Tk, dqk, dv = dims
    rows = _RowsStruct(_rows(q, q.shape, "q"), _rows(k, k.shape, "k"), _rows(v, v.shape, "v"))
    index = _device_of(q, k, v)
    if not _here(index, stream):
        with _On(index, stream):
            return _forward_grouped(q, k, v, causal, scale, cu_seqlens, with_lse, None, window,
                                    block_mask, cu_seqlens_k)
    device = q.device
    o = _empty(q.shape[:-1] + (dv,), torch.bfloat16, device)
    lse = None
    if with_lse:
        lse = _empty((Hq, Tq) if cu_seqlens is not None else (B, Hq, Tq), torch.float32, device)
    if q.numel() == 0:  # (tensors without elements have no address)
        return o, lse
    rc = attn_fwd_grouped(q, k, v, o, lse, *dims, rows, causal, wl, wr, scale, cu_seqlens,
                          cu_seqlens_k, _current(index))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_grouped")
    return o, lse


def _backward_grouped(q, k, v, o, dO, lse, causal, scale, cu_seqlens, deterministic, workspace,
                      stream, out, window, block_mask, cu_seqlens_k):
    dims, (wl, wr) = _grouped_dims(q, k, v, cu_seqlens, cu_seqlens_k, window, block_mask)
    B, Hq, Hk, Tq, Tk, dqk, dv = dims
    shape = q.shape[:-1] + (dv,)
    if o.shape != shape or dO.shape != shape:
        raise ValueError("o and dO must have q's rows and heads, and v's head size")
    if (lse.dtype is not torch.float32 or not lse.is_contiguous()
            or lse.shape != ((Hq, Tq) if cu_seqlens is not None else (B, Hq, Tq))):
        raise ValueError("lse must be the forward's contiguous fp32 statistic")
    grads = out if out is not None else (None, None, None)
    for g, t, name in zip(grads, (q, k, v), "qkv"):
        if out is not None and g.shape != t.shape:
            raise ValueError(f"out must hold a tensor like {name}")
    if workspace is not None and not workspace.is_contiguous():  # (nbytes counts its memory)
        raise ValueError("workspace must be contiguous")
    rows = _RowsStruct(_rows(q, q.shape, "q"), _rows(k, k.shape, "k"), _rows(v, v.shape, "v"),
                       _rows(o, shape, "o"), _rows(dO, shape, "dO"),
                       *(0 if g is None else _rows(g, g.shape, "out") for g in grads))
    index = _device_of(q, k, v, o, dO, lse, workspace, *grads)
    if not _here(index, stream):
        with _On(index, stream):
            return _backward_grouped(q, k, v, o, dO, lse, causal, scale, cu_seqlens,
                                     deterministic, workspace, None, out, window, block_mask,
                                     cu_seqlens_k)
    device = q.device
    if out is None:
        grads = [_empty(t.shape, torch.bfloat16, device) for t in (q, k, v)]
    dq, dk, dvt = grads
    if q.numel() == 0:  # (tensors without elements have no address; no query sees a key)
        return dq, dk.zero_(), dvt.zero_()
    need = attn_bwd_grouped_workspace_size(*dims, cu_seqlens is not None, deterministic)
    if workspace is None or workspace.nbytes < need:
        workspace = _empty((max(need, 1),), torch.uint8, device)
    rc = attn_bwd_grouped(q, k, v, o, dO, lse, dq, dk, dvt, *dims, rows, causal, wl, wr, scale,
                          cu_seqlens, cu_seqlens_k, deterministic, workspace, workspace.nbytes,
                          _current(index))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_bwd_grouped")
    return dq, dk, dvt


def rope(q, k, rotation, inverse=False, pos0=0, cu_seqlens=None, cu_seqlens_k=None, out=None,
         stream=None):
    """(q, k) rotated by their positions, as bf16 tensors (either may be None).

    q (B,Tq,Hq,d), k (B,Tk,Hk,d), or (sum T, H, d) with host offsets; slots of a packed
    buffer work as they are.  Positions: key j of a sequence at pos0 + j, and the queries
    are its last ones, as in forward().  inverse=True turns the other way, which is the
    gradient: gradients of the rotated tensors in, of the unrotated ones out.  out: (q_out,
    k_out), which may be the inputs themselves."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q and k are both None")
    shape = x.shape
    varlen = cu_seqlens is not None
    if len(shape) != (3 if varlen else 4):
        raise ValueError(f"q and k must have {3 if varlen else 4} dimensions")
    other = k.shape if q is not None and k is not None else shape
    if len(other) != len(shape) or other[-1] != shape[-1] or (not varlen and other[0] != shape[0]):
        raise ValueError("q and k must agree in batch and head size")
    if varlen:
        B, Tq, Tk = len(cu_seqlens) - 1, shape[0], other[0]
        if cu_seqlens_k is not None and len(cu_seqlens_k) != B + 1:
            raise ValueError("cu_seqlens and cu_seqlens_k must have the same length")
        if k is None and B >= 0 and cu_seqlens_k is not None:  # the keys that the queries end
            Tk = int(cu_seqlens_k[-1])
        if q is None and cu_seqlens_k is not None:
            cu_seqlens = cu_seqlens_k
    else:
        B, Tq, Tk = shape[0], shape[1], other[1]
    q_row = 0 if q is None else _rows(q, shape, "q")
    k_row = 0 if k is None else _rows(k, other, "k")
    q_out, k_out = out if out is not None else (None, None)
    q_out_row = k_out_row = 0  # dense
    if out is not None:
        for name, t, o in (("q", q, q_out), ("k", k, k_out)):
            if (t is None) != (o is None) or (o is not None and o.shape != t.shape):
                raise ValueError(f"out must hold a tensor like {name}")
        q_out_row = 0 if q is None else _rows(q_out, shape, "out[0]")
        k_out_row = 0 if k is None else _rows(k_out, other, "out[1]")
    index = _device_of(x, k, q_out, k_out, rotation.rates)
    if not _here(index, stream):
        with _On(index, stream):
            return rope(q, k, rotation, inverse, pos0, cu_seqlens, cu_seqlens_k, out)
    if out is None:
        device = x.device
        q_out = None if q is None else _empty(shape, torch.bfloat16, device)
        k_out = None if k is None else _empty(other, torch.bfloat16, device)
    if x.numel() == 0:
        if q is not None and k is not None and k.numel() > 0:  # no queries: the keys alone
            cu = cu_seqlens if cu_seqlens_k is None else cu_seqlens_k
            rope(None, k, rotation, inverse, pos0, cu, None, (None, k_out))
        return q_out, k_out
    if k is not None and k.numel() == 0:  # no keys: the queries alone, in front of the first
        k = None
    cu, cuk = _HostInts(cu_seqlens), _HostInts(cu_seqlens_k)
    rc = load().attn_rope(_ptr(q), _ptr(k), _ptr(q_out), None if k is None else _ptr(k_out),
                          B, 0 if q is None else shape[-2], 0 if k is None else other[-2], Tq, Tk,
                          shape[-1], q_row, k_row, q_out_row, k_out_row, rotation.address,
                          int(inverse), _c_int(pos0), cu.ptr, cuk.ptr, _current(index))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_rope")
    return q_out, k_out


def _check_tables(cache, block_table, lens):
    """(sequences, table width, table stride)."""
    if block_table.dtype is not torch.int32 or len(block_table.shape) != 2:
        raise ValueError("block_table must be int32 (sequences, pages) with adjacent entries")
    B, width = block_table.shape
    stride = width
    if not block_table.is_contiguous():
        if B > 1:
            stride = block_table.stride(0)
        if (width > 1 and block_table.stride(1) != 1) or stride < width:
            raise ValueError("block_table must be int32 (sequences, pages) with adjacent entries, "
                             "each row with its own memory")
    if lens.dtype is not torch.int32 or lens.shape != (B,) or not lens.is_contiguous():
        raise ValueError("lens must be contiguous int32, one per row of block_table")
    return B, width, stride


class HeadNorm:
    """The norm of each query and key head: x / sqrt(mean(x^2) + eps) times a weight per column
    (q_weight, k_weight: contiguous fp32, one value per column of a head; None: ones)."""

    def __init__(self, q_weight=None, k_weight=None, eps=1e-6):
        for w in (q_weight, k_weight):
            if w is not None:
                self._check_kind(w)
        self.q_weight, self.k_weight, self.eps = q_weight, k_weight, float(eps)
        self.struct = _NormStruct(_ptr(q_weight), _ptr(k_weight), self.eps)
        self.address = ctypes.addressof(self.struct)

    @staticmethod
    def _check_kind(w):
        if w.dtype is not torch.float32 or w.dim() != 1 or not w.is_contiguous():
            raise ValueError("q_weight and k_weight must be contiguous fp32, one per column")

    def check(self, d):
        """For heads of d columns.  The weights are looked at anew, as a parameter's memory may move,
        and its type may change with it (a module turned to bf16)."""
        for name in ("q_weight", "k_weight"):
            w = getattr(self, name)
            if w is not None:
                self._check_kind(w)
                if w.shape[0] != d:
                    raise ValueError("the norm's weights must have one value per column of a head")
                setattr(self.struct, name, w.data_ptr())


def _norm_dims(q, k, cu_seqlens, cu_seqlens_k):
    """(B, Hq, Hk, Tq, Tk, d) and the offsets of queries and keys, of which one may be None."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q and k are both None")
    varlen = cu_seqlens is not None
    rank = 3 if varlen else 4
    if any(t is not None and t.dim() != rank for t in (q, k)):
        raise ValueError(f"q and k must have {rank} dimensions")
    if q is not None and k is not None and (q.shape[-1] != k.shape[-1] or
                                            (not varlen and q.shape[0] != k.shape[0])):
        raise ValueError("q and k must agree in batch and head size")
    if cu_seqlens_k is not None:
        if not varlen:
            raise ValueError("cu_seqlens_k needs cu_seqlens")
        if len(cu_seqlens_k) != len(cu_seqlens):
            raise ValueError("cu_seqlens and cu_seqlens_k must have the same length")
    if varlen:
        B = len(cu_seqlens) - 1
        if q is None and cu_seqlens_k is not None:
            cu_seqlens = cu_seqlens_k
        Tq = q.shape[0] if q is not None else k.shape[0]
        if k is not None:
            Tk = k.shape[0]
        else:  # the keys that the queries end
            Tk = int(cu_seqlens_k[-1]) if cu_seqlens_k is not None else Tq
    else:
        B = x.shape[0]
        Tq, Tk = (t.shape[1] if t is not None else x.shape[1] for t in (q, k))
    heads = lambda t: 0 if t is None else t.shape[-2]
    return (B, heads(q), heads(k), Tq, Tk, x.shape[-1]), cu_seqlens, cu_seqlens_k


def _like(name, t, o):
    if (t is None) != (o is None) or (o is not None and o.shape != t.shape):
        raise ValueError(f"there must be a tensor like {name}")


def _or_rows(t, name):
    return 0 if t is None else _rows(t, t.shape, name)


def norm_rope(q, k, norm, rotation=None, pos0=0, cu_seqlens=None, cu_seqlens_k=None, out=None,
              stream=None):
    """(q, k) with each head normed by a HeadNorm and then rotated to its position, as bf16
    tensors (either may be None; rotation None: normed alone).

    Tensors, positions, offsets and out: as in rope()."""
    dims, cu, cuk = _norm_dims(q, k, cu_seqlens, cu_seqlens_k)
    norm.check(dims[-1])
    q_out, k_out = out if out is not None else (None, None)
    if out is not None:
        _like("q", q, q_out)
        _like("k", k, k_out)
    rows = [_or_rows(t, n) for t, n in ((q, "q"), (k, "k"), (q_out, "out[0]"), (k_out, "out[1]"))]
    x = q if q is not None else k
    index = _device_of(x, k, q_out, k_out, norm.q_weight, norm.k_weight,
                       None if rotation is None else rotation.rates)
    if not _here(index, stream):
        with _On(index, stream):
            return norm_rope(q, k, norm, rotation, pos0, cu_seqlens, cu_seqlens_k, out)
    if out is None:
        q_out, k_out = (None if t is None else _empty(t.shape, torch.bfloat16, t.device)
                        for t in (q, k))
    # (tensors without elements have no address)
    full = lambda t: None if t is None or t.numel() == 0 else t
    if full(q) is None and full(k) is None:
        return q_out, k_out
    if full(q) is None and q is not None and cuk is not None:
        cu = cuk
    B, Hq, Hk, Tq, Tk, d = dims
    if full(q) is None:
        Tq = Tk if cu_seqlens is not None else 0
    rc = attn_norm_rope(full(q), full(k), full(q_out), full(k_out), B, Hq, Hk, Tq, Tk, d, *rows,
                        norm, rotation, pos0, cu, cuk, _current(index))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_norm_rope")
    return q_out, k_out


def norm_rope_backward(q, k, dq_out, dk_out, norm, rotation=None, pos0=0, cu_seqlens=None,
                       cu_seqlens_k=None, workspace=None, out=None, stream=None):
    """(dq, dk, dq_weight, dk_weight): the gradients of norm_rope(q, k, norm, ...) from those of
    its outputs, dq_out and dk_out.  dq, dk: bf16 like q, k; those of the weights: fp32, one per
    column (None where norm has no weight, or q or k is None).  out: (dq, dk) to write to, which
    may be dq_out, dk_out or q, k themselves."""
    dims, cu, cuk = _norm_dims(q, k, cu_seqlens, cu_seqlens_k)
    d = dims[-1]
    norm.check(d)
    _like("q", q, dq_out)
    _like("k", k, dk_out)
    dq, dk = out if out is not None else (None, None)
    if out is not None:
        _like("q", q, dq)
        _like("k", k, dk)
    if workspace is not None and not workspace.is_contiguous():  # (nbytes counts its memory)
        raise ValueError("workspace must be contiguous")
    rows = _NormRowsStruct(*(_or_rows(t, n) for t, n in (
        (q, "q"), (k, "k"), (dq_out, "dq_out"), (dk_out, "dk_out"), (dq, "out[0]"),
        (dk, "out[1]"))))
    x = q if q is not None else k
    index = _device_of(x, k, dq_out, dk_out, dq, dk, workspace, norm.q_weight, norm.k_weight,
                       None if rotation is None else rotation.rates)
    if not _here(index, stream):
        with _On(index, stream):
            return norm_rope_backward(q, k, dq_out, dk_out, norm, rotation, pos0, cu_seqlens,
                                      cu_seqlens_k, workspace, out)
    device = x.device
    if out is None:
        dq, dk = (None if t is None else _empty(t.shape, torch.bfloat16, device) for t in (q, k))
    full = lambda t: None if t is None or t.numel() == 0 else t
    dqw, dkw = (None if t is None or w is None else
                _empty((d,), torch.float32, device) if full(t) is not None else
                torch.zeros(d, device=device)
                for t, w in ((q, norm.q_weight), (k, norm.k_weight)))
    if full(q) is None and full(k) is None:
        return dq, dk, dqw, dkw
    if full(q) is None and q is not None and cuk is not None:
        cu = cuk
    B, Hq, Hk, Tq, Tk, _ = dims
    if full(q) is None:
        Tq = Tk if cu_seqlens is not None else 0
    if workspace is None:
        workspace = _empty((max(1, attn_norm_rope_bwd_workspace_size(d)),), torch.uint8, device)
    of = lambda t, o: None if full(t) is None else o
    rc = attn_norm_rope_bwd(full(q), full(k), of(q, dq_out), of(k, dk_out), of(q, dq), of(k, dk),
                            of(q, dqw), of(k, dkw), B, Hq, Hk, Tq, Tk, d, rows, norm, rotation,
                            pos0, cu, cuk, workspace, workspace.nbytes, _current(index))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_norm_rope_bwd")
    return dq, dk, dqw, dkw


def cache_append(cache, k, v, block_table, lens, q=None, rotation=None, cu_seqlens=None,
                 q_out=None, stream=None, norm=None):
    """Appends new tokens' keys (T,heads,dqk) and values (T,heads,dv) to a PagedCache.

    lens: device int32, each sequence's length with the new tokens counted; block_table:
    device int32 (sequences, pages).  Without cu_seqlens (host offsets of the new rows) every
    sequence brings T / sequences tokens.  k is normed by a HeadNorm if one is given, then
    rotated to its position if a rotation is given, and so is q (T,Hq,dqk), which is returned
    (in q_out, which may be q)."""
    B, width, stride = _check_tables(cache, block_table, lens)
    k_shape, v_shape, heads = k.shape, v.shape, cache.heads
    T = k_shape[0]
    if not cache.rows_apart:
        raise ValueError("the rows of k_cache and v_cache must have their own memory each to be "
                         "appended to")
    if k_shape != (T, heads, cache.dqk) or v_shape != (T, heads, cache.dv):
        raise ValueError("k and v must be (T, heads, d) with the cache's heads and the same T")
    if cu_seqlens is not None and len(cu_seqlens) != B + 1:
        raise ValueError("cu_seqlens must have one entry more than there are sequences")
    k_row, v_row = _rows(k, k_shape, "k"), _rows(v, v_shape, "v")
    q_row = out_row = Hq = 0
    if q is not None:
        q_shape = q.shape
        if len(q_shape) != 3 or q_shape[0] != T or q_shape[2] != cache.dqk:
            raise ValueError("q must be (T, heads, dqk)")
        Hq, q_row = q_shape[1], _rows(q, q_shape, "q")
    if q_out is not None:
        if q is None or q_out.shape != q_shape:
            raise ValueError("q_out must have q's shape")
        out_row = _rows(q_out, q_shape, "q_out")
    index = _device_of(cache.k_cache, k, v, q, q_out, block_table, lens,
                       None if rotation is None else rotation.rates)
    if norm is not None:
        norm.check(cache.dqk)
        _device_of(cache.k_cache, norm.q_weight, norm.k_weight)
    if not _here(index, stream):
        with _On(index, stream):
            return cache_append(cache, k, v, block_table, lens, q, rotation, cu_seqlens, q_out,
                                norm=norm)
    if q is not None and q_out is None:
        q_out = _empty(q_shape, torch.bfloat16, q.device)
    if T == 0:  # (tensors without elements have no address)
        return q_out
    cu = _HostInts(cu_seqlens)
    rc = load().attn_cache_append_norm(cache.address, block_table.data_ptr(), width, stride,
                                       lens.data_ptr(), B, T, cu.ptr, k.data_ptr(), k_row,
                                       v.data_ptr(), v_row, _ptr(q), q_row, _ptr(q_out), out_row,
                                       Hq, None if norm is None else norm.address,
                                       None if rotation is None else rotation.address,
                                       _current(index))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_cache_append")
    return q_out


def decode_workspace(device=None, stream=None):
    """A workspace for decode(), initialised on `stream`; calls that share one must be
    ordered on the GPU."""
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError("a decode workspace must be on a CUDA device")
    index = torch.cuda.current_device() if device.index is None else device.index
    with _On(index, stream):
        ws = torch.empty(attn_decode_workspace_size(), dtype=torch.uint8, device=device)
        rc = attn_decode_workspace_init(ws, ws.numel())
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_decode_workspace_init")
    return ws


def decode(cache, q, block_table, lens, scale=None, window_left=-1, with_lse=True,
           workspace=None, out=None, stream=None):
    """Attention of one new token per sequence over a PagedCache: o (B,Hq,dv) bf16 and the
    log-sum-exp (B,Hq) fp32 (None unless with_lse).

    q (B,Hq,dqk) bf16, Hq a multiple of the cache's heads; lens counts the new token, whose
    key is in the cache already.  window_left >= 0: only the last window_left + 1 keys.
    workspace: from decode_workspace() (None: one is made and initialised for this call).
    out: (o, lse) to write to (lse may be None)."""
    B, width, stride = _check_tables(cache, block_table, lens)
    shape = q.shape
    if len(shape) != 3 or shape[0] != B or shape[2] != cache.dqk:
        raise ValueError("q must be (sequences, heads, dqk)")
    Hq, q_row = shape[1], _rows(q, shape, "q")
    o, lse = out if out is not None else (None, None)
    if out is not None and (o.dtype is not torch.bfloat16 or o.shape != (B, Hq, cache.dv)
                            or not o.is_contiguous()):
        raise ValueError("out[0] must be contiguous bfloat16 (sequences, heads, dv)")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (B, Hq)
                            or not lse.is_contiguous()):
        raise ValueError("out[1] must be contiguous float32 (sequences, heads)")
    if workspace is not None and not workspace.is_contiguous():  # (nbytes counts its memory)
        raise ValueError("workspace must be contiguous")
    index = _device_of(cache.k_cache, q, block_table, lens, workspace, o, lse)
    if scale is None:
        scale = 1.0 / math.sqrt(cache.dqk)
    if not _here(index, stream):
        with _On(index, stream):
            return decode(cache, q, block_table, lens, scale, window_left, with_lse, workspace,
                          out)
    if out is None:
        device = q.device
        o = _empty((B, Hq, cache.dv), torch.bfloat16, device)
        lse = _empty((B, Hq), torch.float32, device) if with_lse else None
    if B == 0:  # (tensors without elements have no address)
        return o, lse
    if workspace is None:
        workspace = decode_workspace(index)
    rc = load().attn_decode(cache.address, block_table.data_ptr(), width, stride, lens.data_ptr(),
                            B, q.data_ptr(), q_row, o.data_ptr(),
                            None if lse is None else lse.data_ptr(), Hq, _c_int(window_left),
                            float(scale), workspace.data_ptr(), workspace.nbytes, _current(index))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_decode")
    return o, lse


def prefill_workspace(device=None):
    """A workspace for prefill(); calls that share one must be ordered on the GPU."""
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError("a prefill workspace must be on a CUDA device")
    return torch.empty(attn_prefill_workspace_size(), dtype=torch.uint8, device=device)


def prefill(cache, q, block_table, lens, scale=None, window_left=-1, with_lse=True,
            cu_seqlens=None, workspace=None, out=None, stream=None):
    """Attention of a chunk of new tokens per sequence over a PagedCache that holds them already:
    o (T,Hq,dv) bf16 and the log-sum-exp (T,Hq) fp32 (None unless with_lse).

    q (T,Hq,dqk) bf16, Hq a multiple of the cache's heads; lens: device int32, each sequence's
    length with the new tokens counted.  Without cu_seqlens (host offsets of the new rows) every
    sequence brings T / sequences tokens.  A token sees the keys up to its own, with
    window_left >= 0 only the last window_left + 1 of them.  workspace: from
    prefill_workspace() (None: one is made for this call).  out: (o, lse) to write to (lse may
    be None)."""
    B, width, stride = _check_tables(cache, block_table, lens)
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.dqk:
        raise ValueError("q must be (T, heads, dqk)")
    T, Hq, q_row = shape[0], shape[1], _rows(q, shape, "q")
    if cu_seqlens is not None and len(cu_seqlens) != B + 1:
        raise ValueError("cu_seqlens must have one entry more than there are sequences")
    o, lse = out if out is not None else (None, None)
    if out is not None and (o.dtype is not torch.bfloat16 or o.shape != (T, Hq, cache.dv)
                            or not o.is_contiguous()):
        raise ValueError("out[0] must be contiguous bfloat16 (T, heads, dv)")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (T, Hq)
                            or not lse.is_contiguous()):
        raise ValueError("out[1] must be contiguous float32 (T, heads)")
    if workspace is not None and not workspace.is_contiguous():  # (nbytes counts its memory)
        raise ValueError("workspace must be contiguous")
    index = _device_of(cache.k_cache, q, block_table, lens, workspace, o, lse)
    if scale is None:
        scale = 1.0 / math.sqrt(cache.dqk)
    if not _here(index, stream):
        with _On(index, stream):
            return prefill(cache, q, block_table, lens, scale, window_left, with_lse, cu_seqlens,
                           workspace, out)
    if out is None:
        device = q.device
        o = _empty((T, Hq, cache.dv), torch.bfloat16, device)
        lse = _empty((T, Hq), torch.float32, device) if with_lse else None
    if T == 0 or B == 0:  # (tensors without elements have no address)
        return o, lse
    if workspace is None:
        workspace = _empty((attn_prefill_workspace_size(),), torch.uint8, q.device)
    cu = _HostInts(cu_seqlens)
    rc = load().attn_prefill(cache.address, block_table.data_ptr(), width, stride,
                             lens.data_ptr(), B, T, cu.ptr, q.data_ptr(), q_row, o.data_ptr(),
                             None if lse is None else lse.data_ptr(), Hq, _c_int(window_left),
                             float(scale), workspace.data_ptr(), workspace.nbytes,
                             _current(index))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_prefill")
    return o, lse
