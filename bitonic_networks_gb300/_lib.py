"""ctypes loader of libgsort.so: declares every entry point of include/gsort.h.

Loading the library needs no GPU (nothing runs at load time); calling a
compute entry point does.  There is no fallback: if the library is missing
and cannot be built, loading raises.
"""
from __future__ import annotations

import ctypes
import importlib
import os
import threading

from . import build as _build

_lock = threading.Lock()
_lib = None

c_u32p = ctypes.POINTER(ctypes.c_uint32)
c_i64p = ctypes.POINTER(ctypes.c_int64)


class Options(ctypes.Structure):
    """struct gsort_options."""
    _fields_ = [
        ("spin_limit", ctypes.c_uint32),
        ("stall_tile", ctypes.c_int64),
        ("events", ctypes.POINTER(ctypes.c_void_p)),
        ("num_events", ctypes.c_int),
        ("variant", ctypes.c_int),
    ]


class Adjustments(ctypes.Structure):
    """struct gsort_adjustments."""
    _fields_ = [
        ("d_history", ctypes.c_void_p),
        ("length", ctypes.c_int64),
        ("history_stride", ctypes.c_int64),
        ("history_bytes", ctypes.c_int),
        ("d_prompt", ctypes.c_void_p),
        ("d_repetition", ctypes.c_void_p),
        ("d_presence", ctypes.c_void_p),
        ("d_frequency", ctypes.c_void_p),
        ("d_bias_tokens", ctypes.c_void_p),
        ("d_bias", ctypes.c_void_p),
        ("biases", ctypes.c_int64),
        ("bias_stride", ctypes.c_int64),
        ("bias_bytes", ctypes.c_int),
        ("d_allowed", ctypes.c_void_p),
        ("allowed_stride", ctypes.c_int64),
    ]


# name -> (restype, argtypes); every symbol that include/gsort.h declares
SIGNATURES = {
    "gsort_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "gsort_version": (ctypes.c_int, []),
    "gsort_radix_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int]),
    "gsort_radix_keys": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.c_void_p]),
    "gsort_radix_pairs": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                         ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                         ctypes.c_size_t, ctypes.c_void_p]),
    "gsort_radix_pairs_ex": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                            ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                            ctypes.c_size_t, ctypes.c_void_p,
                                            ctypes.POINTER(Options)]),
    "gsort_radix_sort_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int, ctypes.c_int]),
    "gsort_radix_sort": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.c_void_p]),
    "gsort_radix_sort_ex": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                           ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                           ctypes.c_size_t, ctypes.c_void_p,
                                           ctypes.POINTER(Options)]),
    "gsort_radix_sort_launch_count": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                                     ctypes.c_int, ctypes.c_int]),
    "gsort_digit_histograms": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                              ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                              ctypes.c_void_p]),
    "gsort_compact_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64]),
    "gsort_compact_positive": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                              ctypes.c_void_p]),
    "gsort_compact_positive_ex": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p,
                                                 ctypes.c_int64, ctypes.c_void_p,
                                                 ctypes.c_void_p, ctypes.c_size_t,
                                                 ctypes.c_void_p, ctypes.POINTER(Options)]),
    "gsort_compact_positive_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p,
                                                      ctypes.c_int64, ctypes.c_void_p,
                                                      ctypes.c_void_p]),
    "gsort_segmented_bitonic": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                               ctypes.c_void_p]),
    "gsort_segmented_sort_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64,
                                                               ctypes.c_int]),
    "gsort_segmented_sort": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                            ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                            ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "gsort_segmented_sort_ex": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                               ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                               ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                               ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                               ctypes.POINTER(Options)]),
    "gsort_partition_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64]),
    "gsort_partition": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                       ctypes.c_uint32, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "gsort_split_sort_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int]),
    "gsort_split_sort": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "gsort_route_experts": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
        ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "gsort_route_experts_backward": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int64,
        ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_void_p,
        ctypes.c_void_p]),
    "gsort_group_capacity": (ctypes.c_int64, [ctypes.c_int64, ctypes.c_int, ctypes.c_int]),
    "gsort_group_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int]),
    "gsort_group_by_expert": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
        ctypes.c_void_p]),
    "gsort_dispatch_rows": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "gsort_combine_rows": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "gsort_combine_rows_backward": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "gsort_token_logprobs": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p]),
    "gsort_token_logprobs_backward": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
        ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_int64, ctypes.c_void_p]),
    "gsort_embed_tokens": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p]),
    "gsort_embed_tokens_backward_workspace_bytes": (ctypes.c_size_t, [
        ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    "gsort_embed_tokens_backward": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64,
        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "gsort_embed_tokens_backward_ex": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64,
        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.POINTER(Options)]),
    "gsort_adjust_logits": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
        ctypes.POINTER(Adjustments), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
    "gsort_adjust_logits_backward": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_int64, ctypes.POINTER(Adjustments), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
    "gsort_adjust_logits_ex": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
        ctypes.POINTER(Adjustments), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.POINTER(Options)]),
    "gsort_adjust_logits_backward_ex": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_int64, ctypes.POINTER(Adjustments), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
        ctypes.POINTER(Options)]),
    "gsort_gradient_norm_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64]),
    "gsort_gradient_norm": (ctypes.c_int, [
        ctypes.POINTER(ctypes.c_void_p), c_i64p, ctypes.POINTER(ctypes.c_int), ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "gsort_gradient_norm_ex": (ctypes.c_int, [
        ctypes.POINTER(ctypes.c_void_p), c_i64p, ctypes.POINTER(ctypes.c_int), ctypes.c_int64, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.POINTER(Options)]),
    "gsort_clip_gradients": (ctypes.c_int, [
        ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_void_p), c_i64p, ctypes.POINTER(ctypes.c_int),
        ctypes.c_int64, ctypes.c_float, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
        ctypes.c_void_p]),
    "gsort_clip_gradients_ex": (ctypes.c_int, [
        ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_void_p), c_i64p, ctypes.POINTER(ctypes.c_int),
        ctypes.c_int64, ctypes.c_float, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
        ctypes.c_void_p, ctypes.POINTER(Options)]),
    "gsort_check": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "gsort_radix_num_variants": (ctypes.c_int, []),
    "gsort_radix_variant_name": (ctypes.c_char_p, [ctypes.c_int]),
    "gsort_radix_launch_count": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                                ctypes.c_int]),
}


def library_path() -> str:
    return _build.LIB_PATH


def load(build_if_missing: bool = True):
    """Load libgsort.so (building it first if it is missing and nvcc exists)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if not os.path.exists(path):
            if not build_if_missing:
                raise OSError(f"{path} not found; run __graft_entry__.build()")
            _build.build_library()
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def load_ops(build_if_missing: bool = True):
    """The module _ops: the language-model operators on torch tensors (built
    first, with the library, if it is missing or for another torch)."""
    if not _build.ops_match():
        if not build_if_missing:
            raise OSError(f"{_build.OPS_PATH} not found, or for another torch; run __graft_entry__.build()")
        _build.build()
    import torch  # noqa: F401  (its libraries come first)
    load(build_if_missing)
    return importlib.import_module("._ops", __package__)
