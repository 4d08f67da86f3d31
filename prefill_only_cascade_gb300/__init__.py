"""Python binding of libquail: the GB300 (sm_103a) prefill-only cascade attention and
restricted head of Quail's AI.IF / AI_JOIN step.

This module only marshals arguments (tensor pointers, sizes, the current CUDA stream) to
the C ABI declared in include/quail.h; every step of the computation runs in the
library's CUDA kernels. PyTorch supplies device memory and streams. There is no CPU or
PyTorch fallback: importing fails loudly when libquail.so has not been built.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libquail.so")

QUAIL_OK = 0
QUAIL_ERR_INVALID_ARG = 1
QUAIL_ERR_UNSUPPORTED = 2
QUAIL_ERR_CUDA = 3
QUAIL_ERR_TIMEOUT = 4
QUAIL_ERR_DEVICE_BOUNDS = 5
QUAIL_BF16 = 0
QUAIL_FP8_E4M3 = 1
QUAIL_FP4_E2M1 = 2

# Every symbol include/quail.h declares.
EXPORTED_SYMBOLS = (
    "quail_cascade_attn", "quail_cascade_workspace_size", "quail_restricted_head",
    "quail_quantize_kv_fp8", "quail_status_string", "quail_get_device_error",
    "quail_set_wait_timeout_ns", "quail_debug_inject", "quail_set_cta_pairs", "quail_version",
    "quail_cascade_attn_noalloc", "quail_causal_prefill_attn",
    "quail_causal_prefill_workspace_size", "quail_kv_plan", "quail_shard_anchors",
    "quail_join_select", "quail_join_select_workspace_size", "quail_shard_batch",
    "quail_cascade_attn_two_pass", "quail_cascade_two_pass_workspace_size",
    "quail_quantize_kv_fp8_with_scales", "quail_paged_kv_append", "quail_paged_decode_attn",
    "quail_paged_decode_workspace_size", "quail_attn_scores", "quail_paged_kv_evict",
    "quail_paged_evict_workspace_size", "quail_paged_kv_read", "quail_paged_page_bytes",
)


class QuailError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class ShardSizes(ctypes.Structure):
    _fields_ = [("num_anchors", ctypes.c_int32), ("num_suffixes", ctypes.c_int32),
                ("anchor_tokens", ctypes.c_int64), ("suffix_tokens", ctypes.c_int64)]


class KvPlanStats(ctypes.Structure):
    _fields_ = [("hits", ctypes.c_int64), ("misses", ctypes.c_int64),
                ("compulsory_tokens", ctypes.c_int64), ("regret_tokens", ctypes.c_int64),
                ("peak_resident_tokens", ctypes.c_int64)]


KV_LRU, KV_FURTHEST_NEXT_USE = 0, 1


class CascadeDesc(ctypes.Structure):
    _fields_ = [
        ("num_anchors", ctypes.c_int32),
        ("num_suffixes", ctypes.c_int32),
        ("total_anchor_tokens", ctypes.c_int64),
        ("total_suffix_tokens", ctypes.c_int64),
        ("max_anchor_len", ctypes.c_int32),
        ("max_suffix_len", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float),
        ("kv_anchor_dtype", ctypes.c_int32),
    ]


class PagedDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_seqs", "max_seq_len", "num_pages", "page_size", "max_pages_per_seq", "num_q_heads",
        "num_kv_heads", "head_dim")] + [("softmax_scale", ctypes.c_float),
                                        ("kv_dtype", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python prefill_only_cascade_gb300/build.py` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32p, f32p = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
    lib.quail_cascade_attn.argtypes = [ctypes.POINTER(CascadeDesc), vp, vp, vp, vp, vp, i32p,
                                       i32p, i32p, f32p, f32p, vp, f32p, vp, ctypes.c_size_t, vp]
    lib.quail_cascade_attn.restype = ctypes.c_int
    lib.quail_cascade_attn_noalloc.argtypes = [ctypes.POINTER(CascadeDesc), vp, vp, vp, vp, vp,
                                               i32p, i32p, i32p, f32p, f32p, vp, f32p, vp]
    lib.quail_cascade_attn_noalloc.restype = ctypes.c_int
    lib.quail_cascade_workspace_size.argtypes = [ctypes.POINTER(CascadeDesc)]
    lib.quail_cascade_workspace_size.restype = ctypes.c_size_t
    lib.quail_cascade_attn_two_pass.argtypes = [ctypes.POINTER(CascadeDesc), vp, vp, vp, vp,
                                                vp, i32p, i32p, i32p, f32p, f32p,
                                                ctypes.c_int32, vp, f32p, vp, ctypes.c_size_t,
                                                vp]
    lib.quail_cascade_attn_two_pass.restype = ctypes.c_int
    lib.quail_cascade_two_pass_workspace_size.argtypes = [ctypes.POINTER(CascadeDesc)]
    lib.quail_cascade_two_pass_workspace_size.restype = ctypes.c_size_t
    lib.quail_restricted_head.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_float, vp,
                                          ctypes.c_int64, ctypes.c_int64, i32p, vp, vp, f32p,
                                          i32p, vp]
    lib.quail_restricted_head.restype = ctypes.c_int
    lib.quail_quantize_kv_fp8.argtypes = [ctypes.c_int32, i32p, ctypes.c_int64, ctypes.c_int32,
                                          ctypes.c_int32, vp, vp, f32p, vp]
    lib.quail_quantize_kv_fp8.restype = ctypes.c_int
    lib.quail_quantize_kv_fp8_with_scales.argtypes = [ctypes.c_int32, i32p, ctypes.c_int64,
                                                      ctypes.c_int32, ctypes.c_int32, vp, f32p,
                                                      vp, f32p, vp]
    lib.quail_quantize_kv_fp8_with_scales.restype = ctypes.c_int
    lib.quail_status_string.argtypes = [ctypes.c_int]
    lib.quail_status_string.restype = ctypes.c_char_p
    lib.quail_get_device_error.argtypes = [vp]
    lib.quail_get_device_error.restype = ctypes.c_int
    lib.quail_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
    lib.quail_set_wait_timeout_ns.restype = None
    lib.quail_debug_inject.argtypes = [ctypes.c_int32]
    lib.quail_debug_inject.restype = None
    lib.quail_set_cta_pairs.argtypes = [ctypes.c_int32]
    lib.quail_set_cta_pairs.restype = ctypes.c_int
    lib.quail_version.argtypes = []
    lib.quail_version.restype = ctypes.c_char_p
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    lib.quail_causal_prefill_attn.argtypes = [i32, i64, i32, i32, i32, i32, ctypes.c_float, vp,
                                              vp, vp, i32p, vp, f32p, f32p, f32p, vp,
                                              ctypes.c_size_t, vp]
    lib.quail_causal_prefill_attn.restype = ctypes.c_int
    lib.quail_causal_prefill_workspace_size.argtypes = [i32, i64, i32, i32, i32, i32]
    lib.quail_causal_prefill_workspace_size.restype = ctypes.c_size_t
    lib.quail_kv_plan.argtypes = [i32, vp, i64, vp, i64, i32, vp, ctypes.POINTER(KvPlanStats)]
    lib.quail_kv_plan.restype = ctypes.c_int
    lib.quail_shard_anchors.argtypes = [i32, vp, vp, vp, i32, vp, vp]
    lib.quail_shard_anchors.restype = ctypes.c_int
    lib.quail_shard_batch.argtypes = [i32, vp, vp, vp, vp, i32, ctypes.POINTER(ShardSizes),
                                      vp, vp, vp, vp, vp, vp]
    lib.quail_shard_batch.restype = ctypes.c_int
    lib.quail_join_select_workspace_size.argtypes = [i32]
    lib.quail_join_select_workspace_size.restype = ctypes.c_size_t
    lib.quail_join_select.argtypes = [i32, i32, vp, vp, i32, vp, vp, vp, vp, vp,
                                      ctypes.c_size_t, vp]
    lib.quail_join_select.restype = ctypes.c_int
    sz = ctypes.c_size_t
    paged = ctypes.POINTER(PagedDesc)
    lib.quail_paged_kv_append.argtypes = [paged, i64, vp, vp, i64, i64, i32p, i32p, i32p, f32p,
                                          f32p, vp, vp, vp]
    lib.quail_paged_kv_append.restype = ctypes.c_int
    lib.quail_paged_kv_read.argtypes = [paged, i64, i32p, i32p, i32p, f32p, f32p, vp, vp, vp, vp,
                                        i64, i64, vp]
    lib.quail_paged_kv_read.restype = ctypes.c_int
    lib.quail_paged_page_bytes.argtypes = [paged]
    lib.quail_paged_page_bytes.restype = sz
    lib.quail_paged_decode_attn.argtypes = [paged, vp, i64, vp, vp, i32p, i32p, f32p, f32p, vp,
                                            f32p, f32p, f32p, i64, vp, sz, vp]
    lib.quail_paged_decode_attn.restype = ctypes.c_int
    lib.quail_paged_decode_workspace_size.argtypes = [paged, i32]
    lib.quail_paged_decode_workspace_size.restype = sz
    lib.quail_attn_scores.argtypes = [i32, i64, i64, i32, i32, i32, i32, i32, ctypes.c_float, i32,
                                      i32, vp, i64, vp, i64, f32p, i32p, i32p, f32p, f32p, i64, vp]
    lib.quail_attn_scores.restype = ctypes.c_int
    lib.quail_paged_kv_evict.argtypes = [paged, i32, i32, vp, vp, i32p, i32p, f32p, i64, i32p,
                                         i32, i32, vp, vp, i32p, i32p, f32p, i64, vp, sz, vp]
    lib.quail_paged_kv_evict.restype = ctypes.c_int
    lib.quail_paged_evict_workspace_size.argtypes = [paged, i32]
    lib.quail_paged_evict_workspace_size.restype = sz
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.quail_status_string(int(status)).decode()


def version() -> str:
    return lib.quail_version().decode()


def _check(status: int, what: str):
    if status != QUAIL_OK:
        raise QuailError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_desc(num_anchors, num_suffixes, total_anchor_tokens, total_suffix_tokens,
              max_anchor_len, max_suffix_len, num_q_heads, num_kv_heads, head_dim,
              softmax_scale=0.0, kv_fp8=False) -> CascadeDesc:
    return CascadeDesc(int(num_anchors), int(num_suffixes), int(total_anchor_tokens),
                       int(total_suffix_tokens), int(max_anchor_len), int(max_suffix_len),
                       int(num_q_heads), int(num_kv_heads), int(head_dim), float(softmax_scale),
                       QUAIL_FP8_E4M3 if kv_fp8 else QUAIL_BF16)


def cascade_workspace_size(desc: CascadeDesc) -> int:
    return int(lib.quail_cascade_workspace_size(ctypes.byref(desc)))


def cascade_attn(desc: CascadeDesc, q_suf, k_anc, v_anc, k_suf, v_suf, anchor_offsets,
                 anchor_suffix_ptr, suffix_offsets, out, lse=None, workspace=None,
                 k_scale=None, v_scale=None, stream=None):
    """quail_cascade_attn on torch CUDA tensors (see include/quail.h for layouts)."""
    if workspace is None:
        raise ValueError("workspace is required (size: cascade_workspace_size(desc))")
    st = lib.quail_cascade_attn(
        ctypes.byref(desc), _ptr(q_suf), _ptr(k_anc), _ptr(v_anc), _ptr(k_suf), _ptr(v_suf),
        _ptr(anchor_offsets), _ptr(anchor_suffix_ptr), _ptr(suffix_offsets), _ptr(k_scale),
        _ptr(v_scale), _ptr(out), _ptr(lse), _ptr(workspace),
        ctypes.c_size_t(workspace.numel() * workspace.element_size()), _stream(stream))
    _check(st, "quail_cascade_attn")


def cascade_two_pass_workspace_size(desc: CascadeDesc) -> int:
    return int(lib.quail_cascade_two_pass_workspace_size(ctypes.byref(desc)))


def cascade_attn_two_pass(desc: CascadeDesc, q_suf, k_anc, v_anc, k_suf, v_suf,
                          anchor_offsets, anchor_suffix_ptr, suffix_offsets, out, lse=None,
                          workspace=None, k_scale=None, v_scale=None, merge_in_suffix_pass=True,
                          stream=None):
    """quail_cascade_attn_two_pass: anchor pass, suffix pass and LSE merge run apart
    (workspace size: cascade_two_pass_workspace_size(desc))."""
    if workspace is None:
        raise ValueError("workspace is required (size: cascade_two_pass_workspace_size(desc))")
    st = lib.quail_cascade_attn_two_pass(
        ctypes.byref(desc), _ptr(q_suf), _ptr(k_anc), _ptr(v_anc), _ptr(k_suf), _ptr(v_suf),
        _ptr(anchor_offsets), _ptr(anchor_suffix_ptr), _ptr(suffix_offsets), _ptr(k_scale),
        _ptr(v_scale), 1 if merge_in_suffix_pass else 0, _ptr(out), _ptr(lse), _ptr(workspace),
        ctypes.c_size_t(workspace.numel() * workspace.element_size()), _stream(stream))
    _check(st, "quail_cascade_attn_two_pass")


def cascade_attn_noalloc(desc: CascadeDesc, q_suf, k_anc, v_anc, k_suf, v_suf, anchor_offsets,
                         anchor_suffix_ptr, suffix_offsets, out, lse=None, k_scale=None,
                         v_scale=None, stream=None):
    """quail_cascade_attn_noalloc: the same computation with the library's fixed device
    scratch array instead of a caller workspace (for callers that may not allocate).
    Calls must not overlap on the GPU; the first call on a device must precede any
    stream capture."""
    st = lib.quail_cascade_attn_noalloc(
        ctypes.byref(desc), _ptr(q_suf), _ptr(k_anc), _ptr(v_anc), _ptr(k_suf), _ptr(v_suf),
        _ptr(anchor_offsets), _ptr(anchor_suffix_ptr), _ptr(suffix_offsets), _ptr(k_scale),
        _ptr(v_scale), _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "quail_cascade_attn_noalloc")


def causal_prefill_workspace_size(num_seqs, total_tokens, max_seq_len, num_q_heads,
                                  num_kv_heads, head_dim):
    return int(lib.quail_causal_prefill_workspace_size(num_seqs, total_tokens, max_seq_len,
                                                       num_q_heads, num_kv_heads, head_dim))


def causal_prefill_attn(q, k, v, seq_offsets, out, max_seq_len, lse=None, workspace=None,
                        softmax_scale=0.0, k_amax=None, v_amax=None, stream=None):
    """quail_causal_prefill_attn: causal self-attention over packed sequences
    (q [T, Hq, d], k/v [T, Hkv, d] bf16, seq_offsets [S+1] int32 on the device); with
    k_amax / v_amax ([S, Hkv] fp32) also the max |k| and |v| per (sequence, KV head)."""
    if workspace is None:
        raise ValueError("workspace is required (size: causal_prefill_workspace_size(...))")
    st = lib.quail_causal_prefill_attn(
        int(seq_offsets.numel() - 1), int(q.shape[0]), int(max_seq_len), int(q.shape[1]),
        int(k.shape[1]), int(q.shape[2]), float(softmax_scale), _ptr(q), _ptr(k), _ptr(v),
        _ptr(seq_offsets), _ptr(out), _ptr(lse), _ptr(k_amax), _ptr(v_amax), _ptr(workspace),
        ctypes.c_size_t(workspace.numel() * workspace.element_size()), _stream(stream))
    _check(st, "quail_causal_prefill_attn")


def kv_plan(access_anchor, anchor_tokens, capacity_tokens, policy=KV_FURTHEST_NEXT_USE):
    """quail_kv_plan on host arrays: returns (hit flags uint8 [accesses], stats dict)."""
    import numpy as np
    acc = np.ascontiguousarray(access_anchor, dtype=np.int32)
    size = np.ascontiguousarray(anchor_tokens, dtype=np.int64)
    hit = np.zeros(acc.size, dtype=np.uint8)
    st = KvPlanStats()
    code = lib.quail_kv_plan(int(size.size), size.ctypes.data, int(acc.size), acc.ctypes.data,
                             int(capacity_tokens), int(policy), hit.ctypes.data,
                             ctypes.byref(st))
    _check(code, "quail_kv_plan")
    return hit, {f: getattr(st, f) for f, _ in KvPlanStats._fields_}


def shard_anchors(anchor_offsets, anchor_suffix_ptr, suffix_offsets, num_ranks):
    """quail_shard_anchors on host arrays: returns (rank of each anchor int32 [A], visible
    (query, key) pairs per rank int64 [num_ranks])."""
    import numpy as np
    ao = np.ascontiguousarray(anchor_offsets, dtype=np.int32)
    asp = np.ascontiguousarray(anchor_suffix_ptr, dtype=np.int32)
    so = np.ascontiguousarray(suffix_offsets, dtype=np.int32)
    rank_of = np.zeros(max(ao.size - 1, 0), dtype=np.int32)
    pairs = np.zeros(int(num_ranks), dtype=np.int64)
    code = lib.quail_shard_anchors(int(ao.size - 1), ao.ctypes.data, asp.ctypes.data,
                                   so.ctypes.data, int(num_ranks), rank_of.ctypes.data,
                                   pairs.ctypes.data)
    _check(code, "quail_shard_anchors")
    return rank_of, pairs


def shard_batch(anchor_offsets, anchor_suffix_ptr, suffix_offsets, rank_of_anchor, rank):
    """quail_shard_batch on host arrays: one rank's sub-batch (its anchors in their original
    order with their suffixes). Returns int32 offset arrays rebased to the sub-batch
    (anchor_offsets, anchor_suffix_ptr, suffix_offsets, as quail_cascade_attn takes them),
    the kept anchors' ids and int64 row indices into the full batch: anchor_rows (rows of
    k_anc / v_anc) and suffix_rows (rows of q_suf / k_suf / v_suf and of out / lse)."""
    import numpy as np
    ao = np.ascontiguousarray(anchor_offsets, dtype=np.int32)
    asp = np.ascontiguousarray(anchor_suffix_ptr, dtype=np.int32)
    so = np.ascontiguousarray(suffix_offsets, dtype=np.int32)
    ro = np.ascontiguousarray(rank_of_anchor, dtype=np.int32)
    A = int(ao.size - 1)
    sz = ShardSizes()
    args = (A, ao.ctypes.data, asp.ctypes.data, so.ctypes.data, ro.ctypes.data, int(rank))
    _check(lib.quail_shard_batch(*args, ctypes.byref(sz), None, None, None, None, None, None),
           "quail_shard_batch")
    out = {"anchor_offsets": np.zeros(sz.num_anchors + 1, np.int32),
           "anchor_suffix_ptr": np.zeros(sz.num_anchors + 1, np.int32),
           "suffix_offsets": np.zeros(sz.num_suffixes + 1, np.int32),
           "anchors": np.zeros(sz.num_anchors, np.int32),
           "anchor_rows": np.zeros(sz.anchor_tokens, np.int64),
           "suffix_rows": np.zeros(sz.suffix_tokens, np.int64)}
    _check(lib.quail_shard_batch(*args, ctypes.byref(sz), *(out[k].ctypes.data for k in (
        "anchor_offsets", "anchor_suffix_ptr", "suffix_offsets", "anchors", "anchor_rows",
        "suffix_rows"))), "quail_shard_batch")
    return out


def restricted_head(h, gamma, w8, logits, argmax, eps=1e-6, row_index=None, n_rows=None,
                    stream=None):
    """quail_restricted_head: RMSNorm + 8-column head + argmax over rows of h (or over
    h[row_index]; indices outside h's rows are reported on the device, not read)."""
    if n_rows is None:
        n_rows = row_index.numel() if row_index is not None else h.shape[0]
    st = lib.quail_restricted_head(int(n_rows), int(h.shape[-1]), float(eps), _ptr(h),
                                   int(h.shape[0]), int(h.stride(0)), _ptr(row_index),
                                   _ptr(gamma), _ptr(w8), _ptr(logits), _ptr(argmax),
                                   _stream(stream))
    _check(st, "quail_restricted_head")


def join_select_workspace_size(num_suffixes) -> int:
    return int(lib.quail_join_select_workspace_size(int(num_suffixes)))


def join_select(argmax, true_index, selected, num_selected, workspace, verdict=None,
                anchor_suffix_ptr=None, anchor_count=None, stream=None):
    """quail_join_select on torch CUDA tensors: verdicts of the head's argmax, the passing
    suffix ids in increasing order, their number, and (optionally) a count per anchor."""
    num_anchors = 0 if anchor_suffix_ptr is None else int(anchor_suffix_ptr.numel() - 1)
    st = lib.quail_join_select(num_anchors, int(argmax.numel()), _ptr(anchor_suffix_ptr),
                               _ptr(argmax), int(true_index), _ptr(verdict), _ptr(selected),
                               _ptr(num_selected), _ptr(anchor_count), _ptr(workspace),
                               int(workspace.numel() * workspace.element_size()),
                               _stream(stream))
    _check(st, "quail_join_select")


def quantize_kv_fp8(kv_bf16, anchor_offsets, codes, scale, stream=None):
    """quail_quantize_kv_fp8: per-(anchor, KV head) E4M3 codes and fp32 scales."""
    T, hkv, d = kv_bf16.shape
    st = lib.quail_quantize_kv_fp8(int(anchor_offsets.numel() - 1), _ptr(anchor_offsets), int(T),
                                   int(hkv), int(d), _ptr(kv_bf16), _ptr(codes), _ptr(scale),
                                   _stream(stream))
    _check(st, "quail_quantize_kv_fp8")


def quantize_kv_fp8_with_scales(kv_bf16, anchor_offsets, amax, codes, scale, stream=None):
    """quail_quantize_kv_fp8_with_scales: the same codes and scales given the max |x| of
    every (anchor, KV head) (e.g. the causal prefill's k_amax / v_amax)."""
    T, hkv, d = kv_bf16.shape
    st = lib.quail_quantize_kv_fp8_with_scales(
        int(anchor_offsets.numel() - 1), _ptr(anchor_offsets), int(T), int(hkv), int(d),
        _ptr(kv_bf16), _ptr(amax), _ptr(codes), _ptr(scale), _stream(stream))
    _check(st, "quail_quantize_kv_fp8_with_scales")


def _int32(what, x):
    """x as an int that the C ABI's int32 holds (ctypes would drop the bits above)."""
    x = int(x)
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{what}: {x} does not fit 32 bits")
    return x


def make_paged_desc(num_seqs, max_seq_len, num_pages, page_size, max_pages_per_seq, num_q_heads,
                    num_kv_heads, head_dim, softmax_scale=0.0, kv_fp8=False,
                    kv_fp4=False) -> PagedDesc:
    """quail_paged_desc with bf16 pages, e4m3 codes (kv_fp8) or fp4 (kv_fp4)."""
    if kv_fp8 and kv_fp4:
        raise ValueError("kv_fp8 and kv_fp4: pages have one form")
    return PagedDesc(_int32("num_seqs", num_seqs), _int32("max_seq_len", max_seq_len),
                     _int32("num_pages", num_pages), _int32("page_size", page_size),
                     _int32("max_pages_per_seq", max_pages_per_seq),
                     _int32("num_q_heads", num_q_heads), _int32("num_kv_heads", num_kv_heads),
                     _int32("head_dim", head_dim), float(softmax_scale),
                     QUAIL_FP4_E2M1 if kv_fp4 else QUAIL_FP8_E4M3 if kv_fp8 else QUAIL_BF16)


def paged_pool_shape(desc: PagedDesc, pages=None):
    """Shape of a K or V pool of `pages` pages (the descriptor's): [pages, page_size, Hkv, d], or
    with fp4 pages [pages, Hkv, bytes of a page's head] of uint8 (its codes, then its block
    scales; see include/quail.h)."""
    if pages is None:
        pages = desc.num_pages
    if desc.kv_dtype == QUAIL_FP4_E2M1:
        return (pages, desc.num_kv_heads, desc.page_size * desc.head_dim * 9 // 16)
    return (pages, desc.page_size, desc.num_kv_heads, desc.head_dim)


def paged_page_bytes(desc: PagedDesc) -> int:
    return int(lib.quail_paged_page_bytes(ctypes.byref(desc)))


# The paged calls run once per generated token. Plain arguments on the current device and stream go
# through one native pass (csrc/paged_calls.cpp, built beside the library where PyTorch's and Python's
# headers are: 4-5 us a call on the host instead of 9-10); it answers None to anything else, and without
# it, or with a stream given, the checks below do the same. They too are written to be cheap: one test
# per tensor, the reason worked out only when it fails, the stream's handle without a
# Stream object, the device switched only when it is not the current one.
# (PyTorch's own short cuts where it has them: 0.08 us instead of 1.1 for the stream, 0.12
# instead of 0.25 for the device.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
try:
    from . import _paged_calls as _calls
    _calls.bind(PagedDesc, *(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.quail_paged_kv_append, lib.quail_paged_kv_read, lib.quail_paged_decode_attn,
        lib.quail_paged_kv_evict)))
except ImportError:
    _calls = None
_POOL_DTYPES = {QUAIL_BF16: (_BF16,), QUAIL_FP8_E4M3: (torch.float8_e4m3fn, torch.uint8),
                QUAIL_FP4_E2M1: (torch.uint8,)}


def _explain(what, t, dtypes, shape, index):
    """Why `t` is not a tensor of the given type and shape (None: any size) on CUDA device
    `index`, contiguous in its last axes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if index < 0 or t.get_device() != index:
        raise ValueError(f"{what}: on {t.device}, expected CUDA tensors of one device")
    raise ValueError(f"{what}: strides {t.stride()} are not those of contiguous rows")


def _axes(what, t, axes):
    """Why `t` is not a tensor with so many axes, if it is not."""
    if not isinstance(t, torch.Tensor) or t.dim() != axes:
        _explain(what, t, (getattr(t, "dtype", None),), (None,) * axes, 0)


# What is no tensor has no `dtype` or `get_device`: found out by the AttributeError, since asking
# for the type first costs 0.04 us a tensor.
def _need(what, t, dtype, shape, index):
    """A contiguous tensor of exactly this type, shape and device; its address."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == index
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _explain(what, t, (dtype,), shape, index)


def _need_rows(what, t, shape, index):
    """bf16 rows [n, heads, d] any distance apart: their address and that distance."""
    try:
        st = t.stride()
        if (t.dtype is _BF16 and t.shape == shape and index >= 0 and t.get_device() == index
                and len(st) == 3
                and (st[2] == 1 or not shape[0])
                and (st[1] == shape[2] or shape[1] <= 1 or not shape[0])):
            return t.data_ptr(), st[0] if shape[0] > 1 else shape[1] * shape[2]
    except AttributeError:
        pass
    _explain(what, t, (_BF16,), shape, index)


def _need_pool(k_name, k, v_name, v, desc, pages, index):
    """K and V of a pool of `pages` pages; their addresses."""
    form = desc.kv_dtype
    shape = paged_pool_shape(desc, pages)
    dtypes = _POOL_DTYPES.get(form, ())
    try:
        dtype = k.dtype
        if (dtype in dtypes and k.shape == shape
                and k.get_device() == index and k.is_contiguous() and v.dtype is dtype
                and v.shape == shape and v.get_device() == index and v.is_contiguous()):
            return k.data_ptr(), v.data_ptr()
    except AttributeError:
        pass
    for name, t in ((k_name, k), (v_name, v)):
        if (not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.shape != shape
                or t.get_device() != index or not t.is_contiguous()):
            _explain(name, t, dtypes, shape, index)
    raise ValueError(f"{k_name} and {v_name}: dtypes {k.dtype} and {v.dtype} differ")


def _need_scales(desc, k_scale, v_scale, index):
    if k_scale is None and v_scale is None and not desc.kv_dtype:
        return None, None
    if k_scale is None or v_scale is None:
        raise ValueError("e4m3 and fp4 pages need k_scale and v_scale, bf16 pages neither")
    shape = (desc.num_seqs, desc.num_kv_heads)
    return (_need("k_scale", k_scale, _F32, shape, index),
            _need("v_scale", v_scale, _F32, shape, index))


def _need_score(what, t, rows, heads, least, index):
    """[rows, heads, n] fp32 with n >= least: its address and n."""
    try:
        shape = t.shape
        good = (t.dtype is _F32 and len(shape) == 3 and shape[0] == rows and shape[1] == heads
                and t.get_device() == index and t.is_contiguous())
    except AttributeError:
        good = False
    if not good:
        _explain(what, t, (_F32,), (rows, heads, None), index)
    if shape[2] < least:
        raise ValueError(f"{what}: {shape[2]} entries a row, at least {least} are needed")
    return t.data_ptr(), shape[2]


def _need_workspace(t, index):
    try:
        if (t.dtype is torch.uint8 and t.dim() == 1 and t.get_device() == index
                and t.is_contiguous()):
            return t.data_ptr(), t.numel()
    except AttributeError:
        pass
    _explain("workspace", t, (torch.uint8,), (None,), index)


def _on_device(fn, what, index, stream, *args):
    """fn(*args, stream) with the tensors' device current and a stream of that device."""
    if index < 0:
        raise ValueError(f"{what}: expected CUDA tensors")
    if stream is None:
        handle = _raw_stream(index)
    elif stream.device_index != index:
        raise ValueError(f"{what}: stream of cuda:{stream.device_index}, tensors on cuda:{index}")
    else:
        handle = stream.cuda_stream
    if _current_device() == index:
        code = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            code = fn(*args, handle)
    if code != QUAIL_OK:
        raise QuailError(code, what)


def paged_kv_append(desc: PagedDesc, k_new, v_new, start_pos, block_table, k_pages, v_pages,
                    new_offsets=None, k_scale=None, v_scale=None, stream=None):
    """quail_paged_kv_append: rows k_new / v_new ([T, Hkv, d] bf16, any row stride) into the
    pages at start_pos[b] + i; new_offsets ([B+1] int32) delimits the sequences' rows (None:
    one token each). With e4m3 and fp4 pages the rows become codes under the given scales (fp4:
    amax / 2688, or 1 where amax is 0, uses the format whole)."""
    if _calls is not None and stream is None:
        code = _calls.append(desc, k_new, v_new, start_pos, block_table, k_pages, v_pages, new_offsets,
                             k_scale, v_scale)
        if code is not None:
            return _check(code, "quail_paged_kv_append")
    B, pages = desc.num_seqs, desc.num_pages
    try:
        dev, shape = k_new.get_device(), (k_new.shape[0], desc.num_kv_heads, desc.head_dim)
    except (AttributeError, IndexError):
        _axes("k_new", k_new, 3)
    k, k_stride = _need_rows("k_new", k_new, shape, dev)
    v, v_stride = _need_rows("v_new", v_new, shape, dev)
    off = None
    if new_offsets is not None:
        off = _need("new_offsets", new_offsets, _I32, (B + 1,), dev)
    ks, vs = _need_scales(desc, k_scale, v_scale, dev)
    _on_device(lib.quail_paged_kv_append, "quail_paged_kv_append", dev, stream,
               ctypes.byref(desc), shape[0], k, v, k_stride, v_stride, off,
               _need("start_pos", start_pos, _I32, (B,), dev),
               _need("block_table", block_table, _I32, (B, desc.max_pages_per_seq), dev), ks, vs,
               *_need_pool("k_pages", k_pages, "v_pages", v_pages, desc, pages, dev))


def paged_kv_read(desc: PagedDesc, k_pages, v_pages, start_pos, block_table, k_out, v_out,
                  offsets=None, k_scale=None, v_scale=None, stream=None):
    """quail_paged_kv_read: positions start_pos[b] + i of the sequences as bf16 rows into k_out /
    v_out ([T, Hkv, d] bf16, any row stride; None: not read); offsets ([B+1] int32) delimits the
    sequences' rows (None: one each)."""
    if _calls is not None and stream is None:
        code = _calls.read(desc, k_pages, v_pages, start_pos, block_table, k_out, v_out, offsets, k_scale,
                           v_scale)
        if code is not None:
            return _check(code, "quail_paged_kv_read")
    B, pages = desc.num_seqs, desc.num_pages
    some = k_out if k_out is not None else v_out
    if some is None:
        raise ValueError("k_out and v_out: at least one is needed")
    try:
        dev, shape = some.get_device(), (some.shape[0], desc.num_kv_heads, desc.head_dim)
    except (AttributeError, IndexError):
        _axes("k_out" if k_out is not None else "v_out", some, 3)
    k = v = kp = vp = None
    k_stride = v_stride = 0
    if k_out is not None:
        k, k_stride = _need_rows("k_out", k_out, shape, dev)
    if v_out is not None:
        v, v_stride = _need_rows("v_out", v_out, shape, dev)
    if k_out is not None and v_out is not None:
        kp, vp = _need_pool("k_pages", k_pages, "v_pages", v_pages, desc, pages, dev)
    elif k_out is not None:
        kp, _ = _need_pool("k_pages", k_pages, "k_pages", k_pages, desc, pages, dev)
    else:
        vp, _ = _need_pool("v_pages", v_pages, "v_pages", v_pages, desc, pages, dev)
    off = None
    if offsets is not None:
        off = _need("offsets", offsets, _I32, (B + 1,), dev)
    ks, vs = _need_scales(desc, k_scale, v_scale, dev)
    _on_device(lib.quail_paged_kv_read, "quail_paged_kv_read", dev, stream, ctypes.byref(desc),
               shape[0], off, _need("start_pos", start_pos, _I32, (B,), dev),
               _need("block_table", block_table, _I32, (B, desc.max_pages_per_seq), dev), ks, vs,
               kp, vp, k, v, k_stride, v_stride)


def paged_decode_workspace_size(desc: PagedDesc, with_scores=False) -> int:
    return int(lib.quail_paged_decode_workspace_size(ctypes.byref(desc), 1 if with_scores else 0))


def paged_decode_attn(desc: PagedDesc, q, k_pages, v_pages, block_table, seq_lens, out, workspace,
                      lse=None, k_scale=None, v_scale=None, score_in=None, score_out=None,
                      stream=None):
    """quail_paged_decode_attn: attention of one new token per sequence (q [B, Hq, d] bf16, any
    row stride) over its cached tokens; with score_out ([B, Hkv, n] fp32) also score_in plus
    the weight that each cached token receives (score_in may be score_out)."""
    if _calls is not None and stream is None:
        code = _calls.decode(desc, q, k_pages, v_pages, block_table, seq_lens, out, workspace, lse, k_scale,
                             v_scale, score_in, score_out)
        if code is not None:
            return _check(code, "quail_paged_decode_attn")
    if workspace is None:
        raise ValueError("workspace is required (size: paged_decode_workspace_size(...))")
    B, hq, pages = desc.num_seqs, desc.num_q_heads, desc.num_pages
    shape = (B, hq, desc.head_dim)
    try:
        dev = q.get_device()
    except AttributeError:
        _axes("q", q, 3)
    qp, q_stride = _need_rows("q", q, shape, dev)
    ws, ws_bytes = _need_workspace(workspace, dev)
    ks, vs = _need_scales(desc, k_scale, v_scale, dev)
    si = so = None
    width = 0
    if score_out is not None:
        so, width = _need_score("score_out", score_out, B, desc.num_kv_heads, desc.max_seq_len, dev)
        if score_in is not None:
            si = _need("score_in", score_in, _F32, score_out.shape, dev)
    elif score_in is not None:
        raise ValueError("score_in without score_out")
    _on_device(lib.quail_paged_decode_attn, "quail_paged_decode_attn", dev, stream,
               ctypes.byref(desc), qp, q_stride,
               *_need_pool("k_pages", k_pages, "v_pages", v_pages, desc, pages, dev),
               _need("block_table", block_table, _I32, (B, desc.max_pages_per_seq), dev),
               _need("seq_lens", seq_lens, _I32, (B,), dev), ks, vs,
               _need("out", out, _BF16, shape, dev),
               None if lse is None else _need("lse", lse, _F32, (B, hq), dev), si, so, width, ws,
               ws_bytes)


def attn_scores(q, k, lse, q_offsets, k_offsets, score_out, max_q_len, max_k_len, causal=True,
                window=0, score_in=None, softmax_scale=0.0, stream=None):
    """quail_attn_scores: the attention weight that each key receives from the queries of its
    sequence (q [Tq, Hq, d], k [Tk, Hkv, d] bf16 with any row stride, lse [Tq, Hq] from the
    attention call), added to score_in into score_out [num_seqs, Hkv, n] fp32."""
    try:
        dev = k.get_device()
        tq, hq, d = q.shape
        tk, hkv, _ = k.shape
        seqs = k_offsets.shape[0] - 1
    except (AttributeError, IndexError, ValueError):
        _axes("q", q, 3)
        _axes("k", k, 3)
        _axes("k_offsets", k_offsets, 1)
    qp, q_stride = _need_rows("q", q, (tq, hq, d), dev)
    kp, k_stride = _need_rows("k", k, (tk, hkv, d), dev)
    max_q_len, max_k_len, window = int(max_q_len), int(max_k_len), int(window)
    if (max_q_len | max_k_len | window) >> 31:
        for name, x in (("max_q_len", max_q_len), ("max_k_len", max_k_len), ("window", window)):
            _int32(name, x)
    ko = _need("k_offsets", k_offsets, _I32, (seqs + 1,), dev)
    so, width = _need_score("score_out", score_out, seqs, hkv, max_k_len, dev)
    _on_device(lib.quail_attn_scores, "quail_attn_scores", dev, stream, seqs, tq, tk, max_q_len,
               max_k_len, hq, hkv, d, softmax_scale, 1 if causal else 0, window, qp, q_stride,
               kp, k_stride, _need("lse", lse, _F32, (tq, hq), dev),
               _need("q_offsets", q_offsets, _I32, (seqs + 1,), dev),
               ko,
               None if score_in is None else _need("score_in", score_in, _F32, score_out.shape, dev),
               so, width)


def paged_evict_workspace_size(desc: PagedDesc, dst_num_pages) -> int:
    return int(lib.quail_paged_evict_workspace_size(ctypes.byref(desc),
                                                    _int32("dst_num_pages", dst_num_pages)))


def paged_kv_evict(desc: PagedDesc, budget, recent, k_pages, v_pages, block_table, seq_lens, score,
                   dst_table, k_dst, v_dst, kept, new_lens, workspace, score_out=None,
                   stream=None):
    """quail_paged_kv_evict: per (sequence, KV head) the last `recent` tokens and the best
    scored others, `budget` in all, copied in order into the pages that dst_table names (of
    the same pool or another); kept [B, Hkv, budget] and new_lens [B] int32 say which and how
    many, score_out [B, Hkv, n] takes their scores."""
    if _calls is not None and stream is None:
        code = _calls.evict(desc, budget, recent, k_pages, v_pages, block_table, seq_lens, score, dst_table,
                            k_dst, v_dst, kept, new_lens, workspace, score_out)
        if code is not None:
            return _check(code, "quail_paged_kv_evict")
    if workspace is None:
        raise ValueError("workspace is required (size: paged_evict_workspace_size(...))")
    budget, recent = int(budget), int(recent)
    if (budget | recent) >> 31:
        _int32("budget", budget), _int32("recent", recent)
    B, hkv, pages = desc.num_seqs, desc.num_kv_heads, desc.num_pages
    try:
        dev = k_pages.get_device()
        dst_shape, dst_pages = dst_table.shape, k_dst.shape[0]
    except (AttributeError, IndexError):
        _axes("k_pages", k_pages, 4)
        _axes("dst_table", dst_table, 2)
        _axes("k_dst", k_dst, 4)
    ws, ws_bytes = _need_workspace(workspace, dev)
    sp, width = _need_score("score", score, B, hkv, desc.max_seq_len, dev)
    so, out_width = None, 0
    if score_out is not None:
        so, out_width = _need_score("score_out", score_out, B, hkv, budget, dev)
    if len(dst_shape) != 2:
        _explain("dst_table", dst_table, (_I32,), (B, None), dev)
    _on_device(lib.quail_paged_kv_evict, "quail_paged_kv_evict", dev, stream, ctypes.byref(desc),
               budget, recent,
               *_need_pool("k_pages", k_pages, "v_pages", v_pages, desc, pages, dev),
               _need("block_table", block_table, _I32, (B, desc.max_pages_per_seq), dev),
               _need("seq_lens", seq_lens, _I32, (B,), dev), sp, width,
               _need("dst_table", dst_table, _I32, (B, dst_shape[1]), dev), dst_shape[1],
               dst_pages, *_need_pool("k_dst", k_dst, "v_dst", v_dst, desc, dst_pages, dev),
               _need("kept", kept, _I32, (B, hkv, budget), dev),
               _need("new_lens", new_lens, _I32, (B,), dev), so, out_width, ws, ws_bytes)


def get_device_error(stream=None) -> int:
    return int(lib.quail_get_device_error(_stream(stream)))


def set_wait_timeout_ns(ns: int):
    lib.quail_set_wait_timeout_ns(int(ns))


def debug_inject(skip_first_kv_load: bool):
    lib.quail_debug_inject(1 if skip_first_kv_load else 0)


CTA_PAIRS_OFF, CTA_PAIRS_AUTO, CTA_PAIRS_ALWAYS = 0, 1, 2


def set_cta_pairs(mode: int) -> int:
    """head_dim 128 kernel choice: CTA_PAIRS_OFF (single-SM kernel), CTA_PAIRS_AUTO (the
    default: SM pairs for every fused call, except with the fault-injection switch on) or
    CTA_PAIRS_ALWAYS. Returns the status."""
    return lib.quail_set_cta_pairs(int(mode))


def default_scale(head_dim: int) -> float:
    return 1.0 / math.sqrt(head_dim)
