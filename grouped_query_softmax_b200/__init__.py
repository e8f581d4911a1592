"""Causal grouped-query softmax attention on B200 (sm_100a): Python binding of libgqa.

Every step of the computation runs in the CUDA kernels of ``libgqa.so``; this
module only marshals arguments across the C ABI declared in ``include/gqa.h``.
The functions named ``gqa_*`` mirror the C entry points one to one (device
pointers as integers, sizes, strides, a stream handle). ``attn_fwd`` and
``attn_decode`` are conveniences for torch tensors: they check dtype, device and
layout, allocate the outputs (and the decode workspace) with torch, and call the
same entry points. PyTorch supplies device memory and streams only.

Around the attention calls, for torch tensors in the same way: ``paged_plan`` (block
tables and cache rows of a step, on the device), ``qk_norm_rope`` with its backward and
its cache-writing form, and a paged cache held in 4 bits (``kv4_append``,
``kv4_gather``, ``attn_decode_kv4``). Their checks and allocations are in C++
(``_torch_calls.so``, built with the library where torch with CUDA is installed), since these
calls take microseconds on the device. All operands must be on the current device; a ``stream``
other than the current one has to be ordered after it by the caller.

There is no CPU fallback: importing this package fails loudly if the CUDA
library has not been built.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

__all__ = [
    "GqaError", "gqa_attn_fwd", "gqa_attn_fwd_ex", "gqa_attn_fwd_split", "gqa_attn_fwd_split_workspace_bytes",
    "gqa_attn_decode", "gqa_attn_decode_workspace_bytes",
    "gqa_attn_decode_num_splits", "gqa_attn_decode_static", "gqa_attn_decode_ex",
    "gqa_attn_decode_ex_workspace_bytes", "gqa_attn_decode_ex_num_splits", "gqa_status_string", "gqa_get_device_error",
    "gqa_selftest_bounded_wait", "attn_fwd", "attn_decode", "library_path",
    "GqaLayout", "gqa_attn_fwd_varlen", "gqa_attn_fwd_varlen_workspace_bytes", "gqa_attn_decode_varlen",
    "gqa_attn_decode_varlen_workspace_bytes", "gqa_attn_decode_varlen_num_splits",
    "gqa_attn_bwd", "gqa_attn_bwd_workspace_bytes", "attn_bwd", "gqa_attn_fwd_varlen_paged",
    "attn_fwd_varlen", "attn_decode_varlen",
    "GqaRope", "GqaKv4Layout", "gqa_paged_plan", "gqa_qk_norm_rope", "gqa_qk_norm_rope_bwd",
    "gqa_qk_norm_rope_bwd_workspace_bytes", "gqa_qk_norm_rope_append", "gqa_kv4_append", "gqa_kv4_gather",
    "gqa_attn_decode_kv4", "gqa_attn_decode_kv4_workspace_bytes", "PagedPlan", "paged_plan", "qk_norm_rope",
    "qk_norm_rope_bwd", "qk_norm_rope_append", "kv4_pool", "kv4_append", "kv4_gather", "attn_decode_kv4",
    "GQA_OK", "GQA_ERR_INVALID_ARGUMENT", "GQA_ERR_UNSUPPORTED", "GQA_ERR_WORKSPACE",
    "GQA_ERR_CUDA", "GQA_ERR_TIMEOUT",
]

GQA_OK = 0
GQA_ERR_INVALID_ARGUMENT = 1
GQA_ERR_UNSUPPORTED = 2
GQA_ERR_WORKSPACE = 3
GQA_ERR_CUDA = 4
GQA_ERR_TIMEOUT = 5

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libgqa.so")

if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is missing: build the CUDA library first "
        "(python -c 'import __graft_entry__ as g; g.build()'). There is no CPU fallback.")

_lib = ctypes.CDLL(_LIB_PATH)

_vp, _i32, _ll, _f32, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t

_lib.gqa_attn_fwd.restype = _i32
_lib.gqa_attn_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                              _ll, _ll, _ll, _ll, _f32, _vp]
_lib.gqa_attn_fwd_ex.restype = _i32
_lib.gqa_attn_fwd_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                 _ll, _ll, _ll, _ll, _f32, _i32, _vp]
_lib.gqa_attn_fwd_split_workspace_bytes.restype = _sz
_lib.gqa_attn_fwd_split_workspace_bytes.argtypes = [_i32] * 7
_lib.gqa_attn_fwd_split.restype = _i32
_lib.gqa_attn_fwd_split.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                    _ll, _ll, _ll, _ll, _f32, _i32, _vp, _sz, _vp]
_lib.gqa_attn_fwd_host_workspace_bytes.restype = _sz
_lib.gqa_attn_fwd_host_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
_lib.gqa_attn_fwd_host.restype = _i32
_lib.gqa_attn_fwd_host.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32,
                                   _vp, _sz, _vp]
_lib.gqa_attn_decode_workspace_bytes.restype = _sz
_lib.gqa_attn_decode_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
_lib.gqa_attn_decode_num_splits.restype = _i32
_lib.gqa_attn_decode_num_splits.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
_lib.gqa_attn_decode.restype = _i32
_lib.gqa_attn_decode.argtypes = [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                 _ll, _ll, _ll, _ll, _f32, _i32, _vp, _sz, _vp]
_lib.gqa_attn_decode_ex_workspace_bytes.restype = _sz
_lib.gqa_attn_decode_ex_workspace_bytes.argtypes = [_i32] * 8
_lib.gqa_attn_decode_ex_num_splits.restype = _i32
_lib.gqa_attn_decode_ex_num_splits.argtypes = [_i32] * 8
_lib.gqa_attn_decode_ex.restype = _i32
_lib.gqa_attn_decode_ex.argtypes = [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                    _ll, _ll, _ll, _ll, _f32, _i32, _i32, _vp, _sz, _vp]
_lib.gqa_attn_decode_static.restype = _i32
_lib.gqa_attn_decode_static.argtypes = [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                        _ll, _ll, _ll, _ll, _f32, _i32, _vp]


class GqaLayout(ctypes.Structure):
    """C ``gqa_layout``: element strides (batch, head, row) of a bf16 operand; d is contiguous."""
    _fields_ = [("sb", _ll), ("sh", _ll), ("st", _ll)]


_lay = ctypes.POINTER(GqaLayout)
_lib.gqa_attn_fwd_varlen_workspace_bytes.restype = _sz
_lib.gqa_attn_fwd_varlen_workspace_bytes.argtypes = [_i32] * 4
_lib.gqa_attn_fwd_varlen.restype = _i32
_lib.gqa_attn_fwd_varlen.argtypes = ([_vp] * 9 + [_i32] * 7 + [_lay] * 4 + [_f32, _i32, _vp, _sz, _vp])
_lib.gqa_attn_fwd_varlen_paged.restype = _i32
_lib.gqa_attn_fwd_varlen_paged.argtypes = ([_vp] * 9 + [_i32] * 9 + [_lay] * 4 + [_f32, _i32, _vp, _sz, _vp])
_lib.gqa_attn_decode_varlen_workspace_bytes.restype = _sz
_lib.gqa_attn_decode_varlen_workspace_bytes.argtypes = [_i32] * 8
_lib.gqa_attn_decode_varlen_num_splits.restype = _i32
_lib.gqa_attn_decode_varlen_num_splits.argtypes = [_i32] * 8
_lib.gqa_attn_decode_varlen.restype = _i32
_lib.gqa_attn_decode_varlen.argtypes = ([_vp] * 6 + [_i32] * 9 + [_lay] * 2 + [_f32, _i32, _i32, _vp, _sz, _vp])
_lib.gqa_attn_bwd_workspace_bytes.restype = _sz
_lib.gqa_attn_bwd_workspace_bytes.argtypes = [_i32] * 6
_lib.gqa_attn_bwd.restype = _i32
_lib.gqa_attn_bwd.argtypes = [_vp] * 9 + [_i32] * 6 + [_ll] * 4 + [_f32, _i32, _vp, _sz, _vp]


class GqaRope(ctypes.Structure):
    """C ``gqa_rope``: norm weights, angle tables and positions (device addresses; 0 = none)."""
    _fields_ = [("q_weight", _vp), ("k_weight", _vp), ("cos", _vp), ("sin", _vp), ("positions", _vp),
                ("positions_sb", _ll), ("n_positions", _i32), ("rot", _i32), ("interleaved", _i32),
                ("weight_fp32", _i32), ("eps", _f32)]


class GqaKv4Layout(ctypes.Structure):
    """C ``gqa_kv4_layout``: byte strides (page, head) of a 4-bit pool."""
    _fields_ = [("sb", _ll), ("sh", _ll)]


_rope, _lay4 = ctypes.POINTER(GqaRope), ctypes.POINTER(GqaKv4Layout)
_lib.gqa_paged_plan.restype = _i32
_lib.gqa_paged_plan.argtypes = [_vp] * 11 + [_i32] * 6 + [_vp]
_lib.gqa_qk_norm_rope.restype = _i32
_lib.gqa_qk_norm_rope.argtypes = [_vp] * 4 + [_i32] * 5 + [_lay] * 4 + [_rope, _vp]
_lib.gqa_qk_norm_rope_append.restype = _i32
_lib.gqa_qk_norm_rope_append.argtypes = [_vp] * 7 + [_i32] * 6 + [_lay] * 6 + [_rope, _vp]
_lib.gqa_qk_norm_rope_bwd_workspace_bytes.restype = _sz
_lib.gqa_qk_norm_rope_bwd_workspace_bytes.argtypes = [_i32] * 5
_lib.gqa_qk_norm_rope_bwd.restype = _i32
_lib.gqa_qk_norm_rope_bwd.argtypes = [_vp] * 8 + [_i32] * 5 + [_lay] * 6 + [_rope, _vp, _sz, _vp]
_lib.gqa_kv4_append.restype = _i32
_lib.gqa_kv4_append.argtypes = [_vp] * 5 + [_i32] * 5 + [_lay] * 2 + [_lay4] * 2 + [_vp]
_lib.gqa_kv4_gather.restype = _i32
_lib.gqa_kv4_gather.argtypes = [_vp] * 5 + [_i32] * 5 + [_lay4] * 2 + [_lay] * 2 + [_vp]
_lib.gqa_attn_decode_kv4_workspace_bytes.restype = _sz
_lib.gqa_attn_decode_kv4_workspace_bytes.argtypes = [_i32] * 7
_lib.gqa_attn_decode_kv4.restype = _i32
_lib.gqa_attn_decode_kv4.argtypes = [_vp] * 6 + [_i32] * 9 + [_lay4] * 2 + [_f32, _i32, _vp, _sz, _vp]
_lib.gqa_status_string.restype = ctypes.c_char_p
_lib.gqa_status_string.argtypes = [_i32]
_lib.gqa_get_device_error.restype = _i32
_lib.gqa_get_device_error.argtypes = [_vp]
_lib.gqa_selftest_bounded_wait.restype = _i32
_lib.gqa_selftest_bounded_wait.argtypes = [ctypes.c_ulonglong, _vp]


def library_path() -> str:
    return _LIB_PATH


class GqaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {gqa_status_string(status)}" if what else gqa_status_string(status))


# ---------------------------------------------------------------- raw C entry points
def gqa_attn_fwd(q, k, v, o, lse, B, Hq, Hkv, Tq, Tk, D, k_sb, k_sh, v_sb, v_sh,
                 softmax_scale=0.0, stream=None) -> int:
    """C ``gqa_attn_fwd``; pointers are integers (device addresses). Returns the status."""
    return _lib.gqa_attn_fwd(q, k, v, o, lse, B, Hq, Hkv, Tq, Tk, D, k_sb, k_sh, v_sb, v_sh,
                             float(softmax_scale), stream)


def gqa_attn_fwd_ex(q, k, v, o, lse, B, Hq, Hkv, Tq, Tk, D, k_sb, k_sh, v_sb, v_sh,
                    softmax_scale=0.0, window=0, stream=None) -> int:
    """C ``gqa_attn_fwd_ex``: ``gqa_attn_fwd`` with a sliding window (0 = causal only)."""
    return _lib.gqa_attn_fwd_ex(q, k, v, o, lse, B, Hq, Hkv, Tq, Tk, D, k_sb, k_sh, v_sb, v_sh,
                                float(softmax_scale), int(window), stream)


def gqa_attn_fwd_split_workspace_bytes(B, Hq, Hkv, Tq, Tk, D, window=0) -> int:
    """C ``gqa_attn_fwd_split_workspace_bytes`` (0: the launch does not split)."""
    return _lib.gqa_attn_fwd_split_workspace_bytes(B, Hq, Hkv, Tq, Tk, D, window)


def gqa_attn_fwd_split(q, k, v, o, lse, B, Hq, Hkv, Tq, Tk, D, k_sb, k_sh, v_sb, v_sh,
                       softmax_scale=0.0, window=0, workspace=None, workspace_bytes=0, stream=None) -> int:
    """C ``gqa_attn_fwd_split``: ``gqa_attn_fwd_ex`` that may split the keys of the last wave's
    units over several CTAs (partials merged by log-sum-exp in a workspace). Returns the status."""
    return _lib.gqa_attn_fwd_split(q, k, v, o, lse, B, Hq, Hkv, Tq, Tk, D, k_sb, k_sh, v_sb, v_sh,
                                   float(softmax_scale), window, workspace, workspace_bytes, stream)


def gqa_attn_fwd_host_workspace_bytes(B, Hq, Hkv, Tq, Tk, D) -> int:
    return int(_lib.gqa_attn_fwd_host_workspace_bytes(B, Hq, Hkv, Tq, Tk, D))


def gqa_attn_fwd_host(q, k, v, o, lse, B, Hq, Hkv, Tq, Tk, D, softmax_scale=0.0, window=0,
                      workspace=None, workspace_bytes=0, stream=None) -> int:
    """C ``gqa_attn_fwd_host``: q, k, v, o, lse are HOST addresses; workspace a device address."""
    return _lib.gqa_attn_fwd_host(q, k, v, o, lse, B, Hq, Hkv, Tq, Tk, D, float(softmax_scale), int(window),
                                  workspace, workspace_bytes, stream)


def gqa_attn_decode_workspace_bytes(B, Hq, Hkv, Tk, D, num_splits=0) -> int:
    return int(_lib.gqa_attn_decode_workspace_bytes(B, Hq, Hkv, Tk, D, num_splits))


def gqa_attn_decode_num_splits(B, Hq, Hkv, Tk, D, num_splits=0) -> int:
    return int(_lib.gqa_attn_decode_num_splits(B, Hq, Hkv, Tk, D, num_splits))


def gqa_attn_decode(q, k_cache, v_cache, o, B, Hq, Hkv, Tk, D, k_sb, k_sh, v_sb, v_sh,
                    softmax_scale=0.0, num_splits=0, workspace=None, workspace_bytes=0,
                    stream=None) -> int:
    """C ``gqa_attn_decode``; pointers are integers (device addresses). Returns the status."""
    return _lib.gqa_attn_decode(q, k_cache, v_cache, o, B, Hq, Hkv, Tk, D, k_sb, k_sh, v_sb, v_sh,
                                float(softmax_scale), num_splits, workspace, workspace_bytes, stream)


def gqa_attn_decode_ex_workspace_bytes(B, Hq, Hkv, Tq, Tk, D, window=0, num_splits=0) -> int:
    return int(_lib.gqa_attn_decode_ex_workspace_bytes(B, Hq, Hkv, Tq, Tk, D, window, num_splits))


def gqa_attn_decode_ex_num_splits(B, Hq, Hkv, Tq, Tk, D, window=0, num_splits=0) -> int:
    return int(_lib.gqa_attn_decode_ex_num_splits(B, Hq, Hkv, Tq, Tk, D, window, num_splits))


def gqa_attn_decode_ex(q, k_cache, v_cache, o, B, Hq, Hkv, Tq, Tk, D, k_sb, k_sh, v_sb, v_sh,
                       softmax_scale=0.0, window=0, num_splits=0, workspace=None, workspace_bytes=0,
                       stream=None) -> int:
    """C ``gqa_attn_decode_ex``: decode of 1 <= Tq <= 16 new queries per head, optional window."""
    return _lib.gqa_attn_decode_ex(q, k_cache, v_cache, o, B, Hq, Hkv, Tq, Tk, D, k_sb, k_sh, v_sb,
                                   v_sh, float(softmax_scale), int(window), int(num_splits), workspace,
                                   workspace_bytes, stream)


def gqa_attn_decode_static(q, k_cache, v_cache, o, B, Hq, Hkv, Tk, D, k_sb, k_sh, v_sb, v_sh,
                           softmax_scale=0.0, num_splits=0, stream=None) -> int:
    """C ``gqa_attn_decode_static``: decode with the library's fixed 16 MiB device scratch
    instead of a caller workspace, for callers that cannot allocate device memory."""
    return _lib.gqa_attn_decode_static(q, k_cache, v_cache, o, B, Hq, Hkv, Tk, D, k_sb, k_sh, v_sb,
                                       v_sh, float(softmax_scale), num_splits, stream)


def _layout(x):
    if isinstance(x, GqaLayout):
        return x
    sb, sh, st = x
    return GqaLayout(int(sb), int(sh), int(st))


def gqa_attn_fwd_varlen_workspace_bytes(S, Hq, Hkv, max_seqlen_q) -> int:
    return int(_lib.gqa_attn_fwd_varlen_workspace_bytes(S, Hq, Hkv, max_seqlen_q))


def gqa_attn_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, seqlens_q, seqlens_k, S, Hq, Hkv,
                        D, rows_q, rows_k, max_seqlen_q, q_layout, k_layout, v_layout, o_layout,
                        softmax_scale=0.0, window=0, workspace=None, workspace_bytes=0,
                        stream=None) -> int:
    """C ``gqa_attn_fwd_varlen``; layouts are GqaLayout or (sb, sh, st) tuples in elements."""
    lq, lk, lv, lo = (_layout(x) for x in (q_layout, k_layout, v_layout, o_layout))
    return _lib.gqa_attn_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, seqlens_q, seqlens_k,
                                    S, Hq, Hkv, D, rows_q, rows_k, max_seqlen_q, ctypes.byref(lq),
                                    ctypes.byref(lk), ctypes.byref(lv), ctypes.byref(lo),
                                    float(softmax_scale), int(window), workspace, workspace_bytes, stream)


def gqa_attn_fwd_varlen_paged(q, k_pool, v_pool, o, lse, cu_seqlens_q, seqlens_q, seqlens_k, block_table,
                              page_size, num_pages, max_pages, S, Hq, Hkv, D, rows_q, max_seqlen_q, q_layout,
                              k_layout, v_layout, o_layout, softmax_scale=0.0, window=0, workspace=None,
                              workspace_bytes=0, stream=None) -> int:
    """C ``gqa_attn_fwd_varlen_paged``: variable-length forward over a paged key/value cache."""
    lq, lk, lv, lo = (_layout(x) for x in (q_layout, k_layout, v_layout, o_layout))
    return _lib.gqa_attn_fwd_varlen_paged(q, k_pool, v_pool, o, lse, cu_seqlens_q, seqlens_q, seqlens_k,
                                          block_table, page_size, num_pages, max_pages, S, Hq, Hkv, D, rows_q,
                                          max_seqlen_q, ctypes.byref(lq), ctypes.byref(lk), ctypes.byref(lv),
                                          ctypes.byref(lo), float(softmax_scale), int(window), workspace,
                                          workspace_bytes, stream)


def gqa_attn_decode_varlen_workspace_bytes(B, Hq, Hkv, Tq, max_seqlen_k, D, window=0, num_splits=0) -> int:
    return int(_lib.gqa_attn_decode_varlen_workspace_bytes(B, Hq, Hkv, Tq, max_seqlen_k, D, window, num_splits))


def gqa_attn_decode_varlen_num_splits(B, Hq, Hkv, Tq, max_seqlen_k, D, window=0, num_splits=0) -> int:
    return int(_lib.gqa_attn_decode_varlen_num_splits(B, Hq, Hkv, Tq, max_seqlen_k, D, window, num_splits))


def gqa_attn_decode_varlen(q, k_cache, v_cache, o, seqlens_k, block_table, page_size, num_pages,
                           max_pages, B, Hq, Hkv, Tq, max_seqlen_k, D, k_layout, v_layout,
                           softmax_scale=0.0, window=0, num_splits=0, workspace=None, workspace_bytes=0,
                           stream=None) -> int:
    """C ``gqa_attn_decode_varlen``: decode over per-sequence cache lengths, contiguous or paged."""
    lk, lv = _layout(k_layout), _layout(v_layout)
    return _lib.gqa_attn_decode_varlen(q, k_cache, v_cache, o, seqlens_k, block_table, page_size,
                                       num_pages, max_pages, B, Hq, Hkv, Tq, max_seqlen_k, D,
                                       ctypes.byref(lk), ctypes.byref(lv), float(softmax_scale),
                                       int(window), int(num_splits), workspace, workspace_bytes, stream)


def gqa_attn_bwd_workspace_bytes(B, Hq, Hkv, Tq, Tk, D) -> int:
    return int(_lib.gqa_attn_bwd_workspace_bytes(B, Hq, Hkv, Tq, Tk, D))


def gqa_attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, Tq, Tk, D, k_sb, k_sh, v_sb, v_sh,
                 softmax_scale=0.0, window=0, workspace=None, workspace_bytes=0, stream=None) -> int:
    """C ``gqa_attn_bwd``: dq, dk, dv of the causal GQA forward for the output gradient dout."""
    return _lib.gqa_attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, Tq, Tk, D, k_sb, k_sh, v_sb, v_sh,
                             float(softmax_scale), int(window), workspace, workspace_bytes, stream)


def gqa_paged_plan(seqlens, keep, new_tokens, block_table, free_list, free_count, seqlens_out, cu_seqlens, positions,
                   slots, free_count_out, S, max_pages, page_size, num_pages, free_capacity, max_tokens,
                   stream=None) -> int:
    """C ``gqa_paged_plan``; pointers are integers (device addresses). Returns the status."""
    return _lib.gqa_paged_plan(seqlens, keep, new_tokens, block_table, free_list, free_count, seqlens_out, cu_seqlens,
                               positions, slots, free_count_out, S, max_pages, page_size, num_pages, free_capacity,
                               max_tokens, stream)


def gqa_qk_norm_rope(q, k, q_out, k_out, B, T, Hq, Hkv, D, q_layout, k_layout, q_out_layout, k_out_layout, rope,
                     stream=None) -> int:
    """C ``gqa_qk_norm_rope``; ``rope`` is a GqaRope, layouts GqaLayout or (sb, sh, st) tuples."""
    return _lib.gqa_qk_norm_rope(q, k, q_out, k_out, B, T, Hq, Hkv, D, _layout(q_layout), _layout(k_layout),
                                 _layout(q_out_layout), _layout(k_out_layout), rope, stream)


def gqa_qk_norm_rope_append(q, k, v, q_out, k_pool, v_pool, slots, N, Hq, Hkv, D, page_size, num_pages, q_layout,
                            k_layout, v_layout, q_out_layout, k_pool_layout, v_pool_layout, rope, stream=None) -> int:
    """C ``gqa_qk_norm_rope_append``: the norm and rotation, with k and v written into their pages."""
    return _lib.gqa_qk_norm_rope_append(q, k, v, q_out, k_pool, v_pool, slots, N, Hq, Hkv, D, page_size, num_pages,
                                        _layout(q_layout), _layout(k_layout), _layout(v_layout),
                                        _layout(q_out_layout), _layout(k_pool_layout), _layout(v_pool_layout), rope,
                                        stream)


def gqa_qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hkv, D) -> int:
    return int(_lib.gqa_qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hkv, D))


def gqa_qk_norm_rope_bwd(dq_out, dk_out, q, k, dq, dk, dq_weight, dk_weight, B, T, Hq, Hkv, D, dq_out_layout,
                         dk_out_layout, q_layout, k_layout, dq_layout, dk_layout, rope, workspace=None,
                         workspace_bytes=0, stream=None) -> int:
    """C ``gqa_qk_norm_rope_bwd``: gradients of q, k and the norm weights."""
    return _lib.gqa_qk_norm_rope_bwd(dq_out, dk_out, q, k, dq, dk, dq_weight, dk_weight, B, T, Hq, Hkv, D,
                                     _layout(dq_out_layout), _layout(dk_out_layout), _layout(q_layout),
                                     _layout(k_layout), _layout(dq_layout), _layout(dk_layout), rope, workspace,
                                     workspace_bytes, stream)


def _layout4(x):
    return x if isinstance(x, GqaKv4Layout) else GqaKv4Layout(*x)


def gqa_kv4_append(k, v, k_pool, v_pool, slots, N, Hkv, D, page_size, num_pages, k_layout, v_layout, k_pool_layout,
                   v_pool_layout, stream=None) -> int:
    """C ``gqa_kv4_append``; pool layouts are GqaKv4Layout or (sb, sh) tuples in bytes."""
    return _lib.gqa_kv4_append(k, v, k_pool, v_pool, slots, N, Hkv, D, page_size, num_pages, _layout(k_layout),
                               _layout(v_layout), _layout4(k_pool_layout), _layout4(v_pool_layout), stream)


def gqa_kv4_gather(k_pool, v_pool, k, v, slots, N, Hkv, D, page_size, num_pages, k_pool_layout, v_pool_layout,
                   k_layout, v_layout, stream=None) -> int:
    """C ``gqa_kv4_gather``: rows of the 4-bit cache back as bf16."""
    return _lib.gqa_kv4_gather(k_pool, v_pool, k, v, slots, N, Hkv, D, page_size, num_pages, _layout4(k_pool_layout),
                               _layout4(v_pool_layout), _layout(k_layout), _layout(v_layout), stream)


def gqa_attn_decode_kv4_workspace_bytes(B, Hq, Hkv, Tq, max_seqlen_k, D, window=0) -> int:
    return int(_lib.gqa_attn_decode_kv4_workspace_bytes(B, Hq, Hkv, Tq, max_seqlen_k, D, window))


def gqa_attn_decode_kv4(q, k_pool, v_pool, o, seqlens_k, block_table, page_size, num_pages, max_pages, B, Hq, Hkv, Tq,
                        max_seqlen_k, D, k_layout, v_layout, softmax_scale=0.0, window=0, workspace=None,
                        workspace_bytes=0, stream=None) -> int:
    """C ``gqa_attn_decode_kv4``: decode over a paged cache held in 4 bits."""
    return _lib.gqa_attn_decode_kv4(q, k_pool, v_pool, o, seqlens_k, block_table, page_size, num_pages, max_pages, B,
                                    Hq, Hkv, Tq, max_seqlen_k, D, _layout4(k_layout), _layout4(v_layout),
                                    softmax_scale, window, workspace, workspace_bytes, stream)


def gqa_status_string(status: int) -> str:
    return _lib.gqa_status_string(int(status)).decode()


def gqa_get_device_error(stream=None) -> int:
    return _lib.gqa_get_device_error(stream)


def gqa_selftest_bounded_wait(timeout_ns: int, stream=None) -> int:
    return _lib.gqa_selftest_bounded_wait(int(timeout_ns), stream)


# ---------------------------------------------------------------- torch conveniences
def _torch():
    import torch
    return torch


def _stream_handle(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check_bf16_cuda(t, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a bf16 CUDA tensor")


def _plane_strides(t, name):
    """(batch, head) element strides of a [B, H, T, D] tensor with packed rows."""
    if t.dim() != 4 or t.stride(3) != 1 or (t.size(2) > 1 and t.stride(2) != t.size(3)):
        raise ValueError(f"{name} must be [B, H, T, D] with rows packed (stride(3)=1, stride(2)=D)")
    return t.stride(0), t.stride(1)


def attn_fwd(q, k, v, *, Tk=None, scale=None, window=0, return_lse=False, out=None, stream=None, split=True,
             workspace=None):
    """o = causal GQA attention of q [B,Hq,Tq,D] over k, v [B,Hkv,T_cap,D] (first Tk rows).

    Query row i sits at position Tk - Tq + i; ``window`` > 0 limits it to its
    ``window`` most recent positions. Returns o (bf16, [B,Hq,Tq,D]) and, if
    ``return_lse``, the fp32 natural-log log-sum-exp [B,Hq,Tq].

    With ``split`` (the default) the call goes through gqa_attn_fwd_split, which may
    split the keys of the last wave's units over several CTAs (the results then agree with
    ``split=False``, gqa_attn_fwd_ex, within rounding rather than bit for bit);
    ``workspace`` is then a uint8 CUDA tensor of at least
    gqa_attn_fwd_split_workspace_bytes(...) bytes, allocated here when omitted.
    """
    torch = _torch()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_bf16_cuda(t, n)
    if not q.is_contiguous():
        raise ValueError("q must be contiguous [B, Hq, Tq, D]")
    B, Hq, Tq, D = q.shape
    Hkv = k.shape[1]
    Tk = k.shape[2] if Tk is None else int(Tk)
    if k.shape[0] != B or v.shape[:2] != k.shape[:2] or k.shape[3] != D or v.shape[3] != D:
        raise ValueError("q, k, v shapes disagree")
    if Tk > k.shape[2] or Tk > v.shape[2]:
        raise ValueError("Tk exceeds the cache capacity")
    k_sb, k_sh = _plane_strides(k, "k")
    v_sb, v_sh = _plane_strides(v, "v")
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=q.device) if return_lse else None
    lse_ptr = lse.data_ptr() if lse is not None else None
    if not split:
        st = gqa_attn_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_ptr, B, Hq, Hkv, Tq, Tk,
                             D, k_sb, k_sh, v_sb, v_sh, float(scale or 0.0), int(window), _stream_handle(stream))
        if st != GQA_OK:
            raise GqaError(st, "gqa_attn_fwd_ex")
        return (out, lse) if return_lse else out
    need = gqa_attn_fwd_split_workspace_bytes(B, Hq, Hkv, Tq, Tk, D, int(window))
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if (need and workspace is not None) else None
    ws_bytes = workspace.numel() * workspace.element_size() if (need and workspace is not None) else 0
    st = gqa_attn_fwd_split(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_ptr, B, Hq, Hkv, Tq, Tk, D,
                            k_sb, k_sh, v_sb, v_sh, float(scale or 0.0), int(window), ws_ptr, ws_bytes,
                            _stream_handle(stream))
    if st != GQA_OK:
        raise GqaError(st, "gqa_attn_fwd_split")
    return (out, lse) if return_lse else out


def attn_fwd_host(q, k, v, *, scale=None, window=0, return_lse=False, out=None, workspace=None, device=None,
                  stream=None, synchronize=True):
    """attn_fwd for operands in host memory: q [B,Hq,Tq,D] and k, v [B,Hkv,Tk,D], contiguous
    bf16 CPU tensors (pinned, for the copies to overlap the kernels). The library streams
    query-row chunks through a device workspace (gqa_attn_fwd_host) and writes o (and the
    fp32 LSE) into CPU tensors. With ``synchronize=False`` the call returns once the work is
    enqueued on ``stream``, and the outputs are valid once the stream reaches that point."""
    torch = _torch()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.is_cuda or not t.is_contiguous():
            raise TypeError(f"{n} must be a contiguous bf16 CPU tensor")
    B, Hq, Tq, D = q.shape
    Hkv, Tk = k.shape[1], k.shape[2]
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != D:
        raise ValueError("q, k, v shapes disagree")
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, pin_memory=q.is_pinned())
    elif out.shape != q.shape or out.dtype != torch.bfloat16 or out.is_cuda or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 CPU tensor shaped like q")
    lse = torch.empty((B, Hq, Tq), dtype=torch.float32, pin_memory=q.is_pinned()) if return_lse else None
    need = gqa_attn_fwd_host_workspace_bytes(B, Hq, Hkv, Tq, Tk, D)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8,
                                device=device if device is not None else torch.cuda.current_device())
    st = gqa_attn_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                           lse.data_ptr() if lse is not None else None, B, Hq, Hkv, Tq, Tk, D,
                           float(scale or 0.0), int(window), workspace.data_ptr(),
                           workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if st != GQA_OK:
        raise GqaError(st, "gqa_attn_fwd_host")
    if synchronize:
        if stream is None:
            torch.cuda.current_stream().synchronize()
        elif hasattr(stream, "synchronize"):
            stream.synchronize()
        else:
            torch.cuda.synchronize()
    return (out, lse) if return_lse else out


def attn_decode(q, k_cache, v_cache, *, Tk=None, scale=None, window=0, num_splits=0, out=None,
                workspace=None, stream=None):
    """One decode step: q [B,Hq,Tq,D] (Tq <= 16; or [B,Hq,D] for Tq = 1) over the first Tk
    cached keys; query row i sits at position Tk - Tq + i."""
    torch = _torch()
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _check_bf16_cuda(t, n)
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    B, Hq, D = q.shape[0], q.shape[1], q.shape[-1]
    Tq = q.shape[2] if q.dim() == 4 else 1
    if q.numel() != B * Hq * Tq * D:
        raise ValueError("q must be [B, Hq, Tq, D] or [B, Hq, D]")
    Hkv = k_cache.shape[1]
    Tk = k_cache.shape[2] if Tk is None else int(Tk)
    k_sb, k_sh = _plane_strides(k_cache, "k_cache")
    v_sb, v_sh = _plane_strides(v_cache, "v_cache")
    if out is None:
        out = torch.empty_like(q)
    need = gqa_attn_decode_ex_workspace_bytes(B, Hq, Hkv, Tq, Tk, D, window, num_splits)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = gqa_attn_decode_ex(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
                            B, Hq, Hkv, Tq, Tk, D, k_sb, k_sh, v_sb, v_sh, float(scale or 0.0),
                            int(window), int(num_splits), ws_ptr, ws_bytes, _stream_handle(stream))
    if st != GQA_OK:
        raise GqaError(st, "gqa_attn_decode_ex")
    return out


def _side_layout(t, name):
    """(packed?, rows, H, layout) of a varlen operand: packed [rows, H, D] or padded [S, H, rows, D]."""
    if t.stride(-1) != 1:
        raise ValueError(f"{name}: the last (D) axis must be contiguous")
    if t.dim() == 3:
        return True, t.shape[0], t.shape[1], (0, t.stride(1), t.stride(0))
    if t.dim() == 4:
        return False, t.shape[2], t.shape[1], (t.stride(0), t.stride(1), t.stride(2))
    raise ValueError(f"{name} must be packed [rows, H, D] or padded [S, H, rows, D]")


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _int32_cuda(t, name):
    torch = _torch()
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 CUDA tensor")
    return t


def attn_fwd_varlen(q, k, v, *, cu_seqlens_q=None, cu_seqlens_k=None, seqlens_q=None, seqlens_k=None,
                    max_seqlen_q=None, scale=None, window=0, return_lse=False, out=None, workspace=None,
                    block_table=None, pool_layout="NHD", stream=None):
    """S independent causal GQA problems of different lengths in one call.

    Each side is packed, a 3-D [rows, H, D] tensor (any row/head strides, so token-major
    [total, H, D] and a transposed head-major buffer both work) with int32 boundaries
    ``cu_seqlens_*`` [S + 1], or padded, a 4-D [S, H, rows, D] tensor with optional
    lengths ``seqlens_*`` [S]. Sequence s's L_q query rows sit at positions L_k - L_q ..
    L_k - 1 of its own keys. Returns o shaped like q (rows of no sequence untouched)
    and, with ``return_lse``, the fp32 LSE [Hq, rows_q] (packed) or [S, Hq, rows_q].

    With ``block_table`` (int32 [S, max_pages]) the keys are paged: k and v are pools
    [pages, page, Hkv, D] ("NHD") or [pages, Hkv, page, D] ("HND") and ``seqlens_k`` gives
    each sequence's key count.
    """
    if block_table is not None:
        return _attn_fwd_varlen_paged(q, k, v, cu_seqlens_q, seqlens_q, seqlens_k, block_table, max_seqlen_q,
                                      scale, window, return_lse, out, workspace, pool_layout, stream)
    torch = _torch()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_bf16_cuda(t, n)
    cu_q, cu_k = _int32_cuda(cu_seqlens_q, "cu_seqlens_q"), _int32_cuda(cu_seqlens_k, "cu_seqlens_k")
    len_q, len_k = _int32_cuda(seqlens_q, "seqlens_q"), _int32_cuda(seqlens_k, "seqlens_k")
    packed_q, rows_q, Hq, lay_q = _side_layout(q, "q")
    packed_k, rows_k, Hkv, lay_k = _side_layout(k, "k")
    _, _, _, lay_v = _side_layout(v, "v")
    if packed_q != (cu_q is not None) or packed_k != (cu_k is not None):
        raise ValueError("a packed (3-D) side needs cu_seqlens; a padded (4-D) side must not have it")
    if v.shape != k.shape or q.shape[-1] != k.shape[-1]:
        raise ValueError("q, k, v shapes disagree")
    D = q.shape[-1]
    S = cu_q.numel() - 1 if packed_q else q.shape[0]
    S_k = cu_k.numel() - 1 if packed_k else k.shape[0]
    if S != S_k or S <= 0:
        raise ValueError("queries and keys describe different numbers of sequences")
    if max_seqlen_q is None:  # convenience: one device-to-host read
        if packed_q:
            max_seqlen_q = int((cu_q[1:] - cu_q[:-1]).max().item())
        else:
            max_seqlen_q = int(len_q.max().item()) if len_q is not None else rows_q
    max_seqlen_q = max(1, int(max_seqlen_q))
    if out is None:
        out = torch.empty_like(q)
    _, _, _, lay_o = _side_layout(out, "out")
    lse = None
    if return_lse:
        lse = torch.empty(((Hq, rows_q) if packed_q else (S, Hq, rows_q)), dtype=torch.float32,
                          device=q.device)
    need = gqa_attn_fwd_varlen_workspace_bytes(S, Hq, Hkv, max_seqlen_q)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    st = gqa_attn_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _ptr(lse),
                             _ptr(cu_q), _ptr(cu_k), _ptr(len_q), _ptr(len_k), S, Hq, Hkv, D, rows_q,
                             rows_k, max_seqlen_q, lay_q, lay_k, lay_v, lay_o, float(scale or 0.0),
                             int(window), workspace.data_ptr(), workspace.numel(), _stream_handle(stream))
    if st != GQA_OK:
        raise GqaError(st, "gqa_attn_fwd_varlen")
    return (out, lse) if return_lse else out


def attn_decode_varlen(q, k_cache, v_cache, seqlens_k, *, block_table=None, max_seqlen_k=None,
                       pool_layout="NHD", scale=None, window=0, num_splits=0, out=None, workspace=None,
                       stream=None):
    """Decode of q [B, Hq, Tq, D] (Tq <= 16; or [B, Hq, D]) over per-sequence cache lengths.

    Contiguous cache (``block_table`` None): k_cache/v_cache [B, Hkv, T_cap, D] with any
    batch/head/row strides. Paged cache: a pool [pages, page, Hkv, D] ("NHD") or
    [pages, Hkv, page, D] ("HND") and an int32 block table [B, max_pages]. Sequence b's
    queries are the last Tq of its seqlens_k[b] positions.
    """
    torch = _torch()
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _check_bf16_cuda(t, n)
    seqlens_k = _int32_cuda(seqlens_k, "seqlens_k")
    table = _int32_cuda(block_table, "block_table")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    B, Hq, D = q.shape[0], q.shape[1], q.shape[-1]
    Tq = q.shape[2] if q.dim() == 4 else 1
    if seqlens_k is None or seqlens_k.numel() != B:
        raise ValueError("seqlens_k must hold one length per sequence")
    if k_cache.shape != v_cache.shape or k_cache.dim() != 4 or k_cache.stride(3) != 1:
        raise ValueError("k_cache and v_cache must be 4-D with a contiguous D axis and equal shapes")

    def lay(t):
        if table is None:
            return (t.stride(0), t.stride(1), t.stride(2))
        if pool_layout == "NHD":
            return (t.stride(0), t.stride(2), t.stride(1))
        if pool_layout == "HND":
            return (t.stride(0), t.stride(1), t.stride(2))
        raise ValueError("pool_layout must be 'NHD' or 'HND'")

    if table is None:
        Hkv = k_cache.shape[1]
        page_size = num_pages = max_pages = 0
        cap = k_cache.shape[2]
        max_seqlen_k = cap if max_seqlen_k is None else int(max_seqlen_k)
        if max_seqlen_k > cap:
            raise ValueError("max_seqlen_k exceeds the cache rows")
    else:
        Hkv = k_cache.shape[2] if pool_layout == "NHD" else k_cache.shape[1]
        page_size = k_cache.shape[1] if pool_layout == "NHD" else k_cache.shape[2]
        num_pages = k_cache.shape[0]
        if table.dim() != 2 or table.shape[0] != B:
            raise ValueError("block_table must be [B, max_pages]")
        max_pages = table.shape[1]
        max_seqlen_k = max_pages * page_size if max_seqlen_k is None else int(max_seqlen_k)
    if out is None:
        out = torch.empty_like(q)
    need = gqa_attn_decode_varlen_workspace_bytes(B, Hq, Hkv, Tq, max_seqlen_k, D, window, num_splits)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = gqa_attn_decode_varlen(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
                                seqlens_k.data_ptr(), _ptr(table), page_size, num_pages, max_pages, B, Hq,
                                Hkv, Tq, max_seqlen_k, D, lay(k_cache), lay(v_cache), float(scale or 0.0),
                                int(window), int(num_splits), _ptr(workspace),
                                workspace.numel() if workspace is not None else 0, _stream_handle(stream))
    if st != GQA_OK:
        raise GqaError(st, "gqa_attn_decode_varlen")
    return out


def attn_bwd(q, k, v, o, dout, lse, *, Tk=None, scale=None, window=0, dq=None, dk=None, dv=None,
             workspace=None, stream=None):
    """Gradients (dq, dk, dv) of ``attn_fwd(q, k, v)`` for the output gradient ``dout``.

    o and lse are the forward's output and its log-sum-exp (``attn_fwd(..., return_lse=True)``);
    q, o, dout [B,Hq,Tq,D] contiguous; k, v [B,Hkv,T_cap,D] (first Tk rows). dk and dv are
    [B,Hkv,Tk,D]; a KV head's gradient sums over the query heads that read it.
    """
    torch = _torch()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _check_bf16_cuda(t, n)
    for t, n in ((q, "q"), (o, "o"), (dout, "dout")):
        if not t.is_contiguous() or t.shape != q.shape:
            raise ValueError(f"{n} must be contiguous and shaped like q")
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous():
        raise TypeError("lse must be a contiguous fp32 CUDA tensor")
    B, Hq, Tq, D = q.shape
    Hkv = k.shape[1]
    Tk = k.shape[2] if Tk is None else int(Tk)
    k_sb, k_sh = _plane_strides(k, "k")
    v_sb, v_sh = _plane_strides(v, "v")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty((B, Hkv, Tk, D), dtype=q.dtype, device=q.device) if dk is None else dk
    dv = torch.empty((B, Hkv, Tk, D), dtype=q.dtype, device=q.device) if dv is None else dv
    need = gqa_attn_bwd_workspace_bytes(B, Hq, Hkv, Tq, Tk, D)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    st = gqa_attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(),
                      dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, Tq, Tk, D, k_sb, k_sh, v_sb, v_sh,
                      float(scale or 0.0), int(window), workspace.data_ptr(), workspace.numel(),
                      _stream_handle(stream))
    if st != GQA_OK:
        raise GqaError(st, "gqa_attn_bwd")
    return dq, dk, dv


def _attn_fwd_varlen_paged(q, k_pool, v_pool, cu_seqlens_q, seqlens_q, seqlens_k, block_table, max_seqlen_q,
                           scale, window, return_lse, out, workspace, pool_layout, stream):
    torch = _torch()
    for t, n in ((q, "q"), (k_pool, "k_pool"), (v_pool, "v_pool")):
        _check_bf16_cuda(t, n)
    cu_q = _int32_cuda(cu_seqlens_q, "cu_seqlens_q")
    len_q, len_k = _int32_cuda(seqlens_q, "seqlens_q"), _int32_cuda(seqlens_k, "seqlens_k")
    table = _int32_cuda(block_table, "block_table")
    if len_k is None:
        raise ValueError("a paged cache needs seqlens_k")
    packed_q, rows_q, Hq, lay_q = _side_layout(q, "q")
    if packed_q != (cu_q is not None):
        raise ValueError("packed (3-D) queries need cu_seqlens_q; padded (4-D) queries must not have it")
    if k_pool.shape != v_pool.shape or k_pool.dim() != 4 or k_pool.stride(3) != 1:
        raise ValueError("k_pool and v_pool must be 4-D with a contiguous D axis and equal shapes")
    if pool_layout == "NHD":
        num_pages, page, Hkv, D = k_pool.shape
        lay = lambda t: (t.stride(0), t.stride(2), t.stride(1))
    elif pool_layout == "HND":
        num_pages, Hkv, page, D = k_pool.shape
        lay = lambda t: (t.stride(0), t.stride(1), t.stride(2))
    else:
        raise ValueError("pool_layout must be 'NHD' or 'HND'")
    S = cu_q.numel() - 1 if packed_q else q.shape[0]
    if table.dim() != 2 or table.shape[0] != S or len_k.numel() != S:
        raise ValueError("block_table must be [S, max_pages] and seqlens_k [S]")
    if max_seqlen_q is None:
        if packed_q:
            max_seqlen_q = int((cu_q[1:] - cu_q[:-1]).max().item())
        else:
            max_seqlen_q = int(len_q.max().item()) if len_q is not None else rows_q
    max_seqlen_q = max(1, int(max_seqlen_q))
    if out is None:
        out = torch.empty_like(q)
    _, _, _, lay_o = _side_layout(out, "out")
    lse = None
    if return_lse:
        lse = torch.empty(((Hq, rows_q) if packed_q else (S, Hq, rows_q)), dtype=torch.float32, device=q.device)
    need = gqa_attn_fwd_varlen_workspace_bytes(S, Hq, Hkv, max_seqlen_q)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    st = gqa_attn_fwd_varlen_paged(q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), out.data_ptr(), _ptr(lse),
                                   _ptr(cu_q), _ptr(len_q), len_k.data_ptr(), table.data_ptr(), page, num_pages,
                                   table.shape[1], S, Hq, Hkv, D, rows_q, max_seqlen_q, lay_q, lay(k_pool),
                                   lay(v_pool), lay_o, float(scale or 0.0), int(window), workspace.data_ptr(),
                                   workspace.numel(), _stream_handle(stream))
    if st != GQA_OK:
        raise GqaError(st, "gqa_attn_fwd_varlen_paged")
    return (out, lse) if return_lse else out


# ---------------------------------------------------------------- around the attention calls
_calls = None  # _torch_calls: checks, allocation and the C calls of the functions below


def _load_calls():
    """Load _torch_calls.so and give it the C entry points' addresses."""
    global _calls
    _torch()  # before the module, which needs its libraries
    path = os.path.join(_HERE, "_torch_calls.so")
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build the library with torch installed "
                          "(python -c 'import __graft_entry__ as g; g.build()'). There is no fallback.")
    from . import _torch_calls as calls
    calls.set_functions(*[ctypes.cast(getattr(_lib, n), _vp).value for n in (
        "gqa_paged_plan", "gqa_qk_norm_rope", "gqa_qk_norm_rope_append", "gqa_qk_norm_rope_bwd",
        "gqa_qk_norm_rope_bwd_workspace_bytes", "gqa_kv4_append", "gqa_kv4_gather", "gqa_attn_decode_kv4",
        "gqa_attn_decode_kv4_workspace_bytes")])
    _calls = calls
    return calls


def _handle(stream):
    return None if stream is None else _stream_handle(stream)


def _keep_until(stream, *tensors):
    """Tensors allocated for a call on another stream than the current one stay allocated until
    that stream has passed the call."""
    torch = _torch()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)))
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


class PagedPlan(NamedTuple):
    """What ``paged_plan`` returns: int32 CUDA tensors."""
    seqlens_k: object   # [S] rows each request holds afterwards
    cu_seqlens: object  # [S + 1] first token of each request
    positions: object   # [max_tokens]
    slots: object       # [max_tokens] cache rows, -1: none
    free_count: object  # [1]


def paged_plan(seqlens, new_tokens, block_table, free_list, free_count, *, page_size, num_pages, max_tokens, keep=None,
               out=None, stream=None):
    """The plan of one step over a paged cache, made on the device from request lengths.

    Request s holds ``seqlens[s]`` rows, keeps the first ``keep[s]`` (default: all; 0 for a
    finished request) and adds ``new_tokens[s]``. Pages given back are pushed on the stack
    ``free_list[:free_count]`` in (request, page) order, then the wanted ones are popped;
    ``block_table`` [S, max_pages] and ``free_list`` are updated in place. Returns a PagedPlan:
    new lengths (``seqlens_k`` of the attention calls), token boundaries (``cu_seqlens_q``),
    ``positions`` and ``slots`` of ``max_tokens`` tokens (padding: 0 and -1), and the new free
    count. ``out`` is a PagedPlan to write into; its ``seqlens_k`` and ``free_count`` may be
    ``seqlens`` and ``free_count`` themselves. Lengths that do not fit, or too few pages, leave
    everything as it is and are reported by ``gqa_get_device_error``.
    """
    r = (_calls or _load_calls()).paged_plan(seqlens, new_tokens, block_table, free_list, free_count, keep, out, page_size,
                                             num_pages, max_tokens, _handle(stream))
    if type(r) is int:
        raise GqaError(r, "gqa_paged_plan")
    if out is not None:
        return out
    if stream is not None:
        _keep_until(stream, *r)
    return PagedPlan(*r)


def qk_norm_rope(q, k, *, q_weight=None, k_weight=None, eps=1e-6, cos=None, sin=None, positions=None,
                 interleaved=False, q_out=None, k_out=None, stream=None):
    """RMS norm of each query and key head, then the position rotation, in one pass.

    q [B, Hq, T, D] and k [B, Hkv, T, D], bf16, any batch/head/row strides (so the projection's
    [B, T, heads, D] output is read where it lies). ``q_weight``/``k_weight`` [D] (bf16 or fp32;
    None: that side is not normalised); ``cos``/``sin`` fp32 [positions, rot / 2] (None: no
    rotation; rot = D rotates whole rows); ``positions`` int32 [T] or [B, T] (default 0 .. T - 1);
    pairs are (i, i + rot/2), or (2i, 2i + 1) when ``interleaved``. Returns contiguous (q, k) of
    the same shapes, or writes ``q_out``/``k_out`` (which may be q and k themselves).
    """
    r = (_calls or _load_calls()).qk_norm_rope(q, k, q_weight, k_weight, eps, cos, sin, positions, interleaved, q_out, k_out,
                                               _handle(stream))
    if type(r) is int:
        raise GqaError(r, "gqa_qk_norm_rope")
    if stream is not None:
        _keep_until(stream, *(t for t, given in zip(r, (q_out, k_out)) if given is None))
    return r


def qk_norm_rope_bwd(dq_out, dk_out, q, k, *, q_weight=None, k_weight=None, eps=1e-6, cos=None, sin=None,
                     positions=None, interleaved=False, dq=None, dk=None, workspace=None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of ``qk_norm_rope(q, k, ...)`` for the gradients of
    its outputs (for instance ``attn_bwd``'s dq and dk). The weights' gradients are fp32 [D], None
    for a side without a weight. dq and dk may be dq_out and dk_out themselves."""
    r = (_calls or _load_calls()).qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, eps, cos, sin, positions,
                                                   interleaved, dq, dk, workspace, _handle(stream))
    if type(r) is int:
        raise GqaError(r, "gqa_qk_norm_rope_bwd")
    if stream is not None:  # a workspace made for the call lies in front of the weights' gradients
        _keep_until(stream, *(t for t, given in zip(r, (dq, dk, None, None)) if given is None))
    return r


def qk_norm_rope_append(q, k, v, k_pool, v_pool, slots, *, q_weight=None, k_weight=None, eps=1e-6, cos=None, sin=None,
                        positions=None, interleaved=False, pool_layout="NHD", q_out=None, stream=None):
    """``qk_norm_rope`` for N packed tokens that writes the keys and values into their cache pages.

    q [N, Hq, D], k and v [N, Hkv, D], any token/head strides; ``slots`` int32 [N] (``paged_plan``'s;
    distinct, negative: no row is written); ``positions`` int32 [N]. k_pool and v_pool are the bf16
    pools of ``attn_decode_varlen``, [pages, page, Hkv, D] ("NHD") or [pages, Hkv, page, D] ("HND").
    Returns the queries [N, Hq, D].
    """
    if pool_layout not in ("NHD", "HND"):
        raise ValueError("pool_layout must be 'NHD' or 'HND'")
    r = (_calls or _load_calls()).qk_norm_rope_append(q, k, v, k_pool, v_pool, slots, q_weight, k_weight, eps, cos, sin,
                                                      positions, interleaved, pool_layout == "NHD", q_out, _handle(stream))
    if type(r) is int:
        raise GqaError(r, "gqa_qk_norm_rope_append")
    if stream is not None and q_out is None:
        _keep_until(stream, r)
    return r


def kv4_pool(num_pages, num_heads, page_size, D, device=None):
    """A pool of zero rows for a paged cache held in 4 bits: uint8 [pages, Hkv, page, D / 2 + 4]."""
    torch = _torch()
    return torch.zeros((num_pages, num_heads, page_size, D // 2 + 4), dtype=torch.uint8,
                       device=torch.cuda.current_device() if device is None else device)


def kv4_append(k, v, k_pool, v_pool, slots, *, stream=None):
    """Write k and v, bf16 [N, Hkv, D] (any token/head strides), as 4-bit rows to the rows
    ``slots`` (int32 [N], distinct; negative: none) of the pools [pages, Hkv, page, D / 2 + 4]."""
    st = (_calls or _load_calls()).kv4_append(k, v, k_pool, v_pool, slots, _handle(stream))
    if st != GQA_OK:
        raise GqaError(st, "gqa_kv4_append")


def kv4_gather(k_pool, v_pool, slots, *, k=None, v=None, stream=None):
    """Rows ``slots`` (int32 [N]) of the 4-bit pools as bf16 (k, v) [N, Hkv, D]; a slot outside
    the pool gives zeros."""
    r = (_calls or _load_calls()).kv4_gather(k_pool, v_pool, slots, k, v, _handle(stream))
    if type(r) is int:
        raise GqaError(r, "gqa_kv4_gather")
    if stream is not None:
        _keep_until(stream, *(t for t, given in zip(r, (k, v)) if given is None))
    return r


def attn_decode_kv4(q, k_pool, v_pool, seqlens_k, block_table, *, max_seqlen_k=None, scale=None, window=0, out=None,
                    workspace=None, stream=None):
    """``attn_decode_varlen`` over a paged cache held in 4 bits (``kv4_append``'s pools).

    q [B, Hq, Tq, D] (Tq <= 16; or [B, Hq, D]); sequence b's queries are the last Tq of its
    ``seqlens_k[b]`` positions, a query at a negative position gets zeros; ``block_table`` int32
    [B, max_pages]. ``workspace``: a uint8 CUDA tensor of gqa_attn_decode_kv4_workspace_bytes(...)
    bytes, allocated here when omitted.
    """
    r = (_calls or _load_calls()).attn_decode_kv4(q, k_pool, v_pool, seqlens_k, block_table, max_seqlen_k, scale or 0.0, window,
                                                  out, workspace, _handle(stream))
    if type(r) is int:
        raise GqaError(r, "gqa_attn_decode_kv4")
    if stream is not None:
        _keep_until(stream, None if out is not None else r[0], None if workspace is not None else r[1])
    return r[0]
