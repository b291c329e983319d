"""ctypes loader for librssm.so (argument marshalling only)."""
from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "librssm.so")
_lock = threading.Lock()
_lib = None
_fast = None
_fast_kv = None


class RssmCacheStruct(ctypes.Structure):
    """Mirror of `rssm_cache` in include/rssm.h."""

    _fields_ = [
        ("num_slots", ctypes.c_int32), ("nheads", ctypes.c_int32), ("ngroups", ctypes.c_int32),
        ("dim", ctypes.c_int32), ("dstate", ctypes.c_int32), ("max_window", ctypes.c_int32),
        ("npredicted", ctypes.c_int32), ("state_dtype", ctypes.c_int32), ("rounding", ctypes.c_int32),
        ("state", ctypes.c_void_p), ("state_slot_stride", ctypes.c_int64),
        ("scale", ctypes.c_void_p), ("scale_slot_stride", ctypes.c_int64),
        ("x_cache", ctypes.c_void_p), ("x_slot_stride", ctypes.c_int64),
        ("B_cache", ctypes.c_void_p), ("B_slot_stride", ctypes.c_int64),
        ("dt_cache", ctypes.c_void_p), ("dt_slot_stride", ctypes.c_int64),
        ("ring_start", ctypes.c_void_p), ("flush_epoch", ctypes.c_void_p), ("error_word", ctypes.c_void_p),
        ("read_state", ctypes.c_void_p), ("read_slot_stride", ctypes.c_int64),
        ("read_scale", ctypes.c_void_p), ("read_scale_slot_stride", ctypes.c_int64),
        ("read_dtype", ctypes.c_int32),
        ("read_sf", ctypes.c_void_p), ("read_sf_slot_stride", ctypes.c_int64),
        ("read_gs", ctypes.c_void_p),
    ]


class RssmDeltaCacheStruct(ctypes.Structure):
    """Mirror of `rssm_delta_cache` in include/rssm.h."""

    _fields_ = [
        ("num_slots", ctypes.c_int32), ("nkheads", ctypes.c_int32), ("nvheads", ctypes.c_int32),
        ("dkey", ctypes.c_int32), ("dvalue", ctypes.c_int32), ("npredicted", ctypes.c_int32),
        ("state_dtype", ctypes.c_int32),
        ("state", ctypes.c_void_p), ("state_slot_stride", ctypes.c_int64),
        ("pend_k", ctypes.c_void_p), ("pend_k_slot_stride", ctypes.c_int64),
        ("pend_w", ctypes.c_void_p), ("pend_w_slot_stride", ctypes.c_int64),
        ("pend_c", ctypes.c_void_p), ("pend_c_slot_stride", ctypes.c_int64),
        ("pend", ctypes.c_void_p), ("error_word", ctypes.c_void_p),
        ("pend_cl", ctypes.c_void_p), ("pend_cl_slot_stride", ctypes.c_int64),
    ]


class RssmKvCacheStruct(ctypes.Structure):
    """Mirror of `rssm_kv_cache` in include/rssm.h."""

    _fields_ = [
        ("num_pages", ctypes.c_int32), ("nlayers", ctypes.c_int32), ("nheads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("format", ctypes.c_int32),
        ("k", ctypes.c_void_p), ("k_layer_stride", ctypes.c_int64), ("k_page_stride", ctypes.c_int64),
        ("v", ctypes.c_void_p), ("v_layer_stride", ctypes.c_int64), ("v_page_stride", ctypes.c_int64),
        ("k_scale", ctypes.c_void_p), ("k_scale_layer_stride", ctypes.c_int64), ("k_scale_page_stride", ctypes.c_int64),
        ("v_scale", ctypes.c_void_p), ("v_scale_layer_stride", ctypes.c_int64), ("v_scale_page_stride", ctypes.c_int64),
        ("error_word", ctypes.c_void_p),
    ]


class RssmLogitsArgs(ctypes.Structure):
    """Mirror of `rssm_logits_args` in include/rssm.h."""

    _fields_ = [
        ("logits", ctypes.c_void_p), ("logits_stride", ctypes.c_int64), ("logits_dtype", ctypes.c_int32),
        ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64), ("out_dtype", ctypes.c_int32),
        ("vocab", ctypes.c_int32), ("batch", ctypes.c_int32), ("T", ctypes.c_int32), ("probs", ctypes.c_int32),
        ("ntok", ctypes.c_int64), ("cu_seqlens", ctypes.c_void_p),
        ("temperature", ctypes.c_void_p), ("repetition", ctypes.c_void_p), ("presence", ctypes.c_void_p),
        ("frequency", ctypes.c_void_p),
        ("history", ctypes.c_void_p), ("history_stride", ctypes.c_int64), ("history_max", ctypes.c_int32),
        ("history_len", ctypes.c_void_p),
        ("prompt_len", ctypes.c_void_p), ("tokens", ctypes.c_void_p), ("parents", ctypes.c_void_p),
        ("bias_start", ctypes.c_void_p), ("bias_id", ctypes.c_void_p), ("bias_value", ctypes.c_void_p),
        ("biases", ctypes.c_int64), ("mask", ctypes.c_void_p), ("mask_stride", ctypes.c_int64),
        ("error_word", ctypes.c_void_p),
    ]


EXPORTS = ("rssm_scratch_bytes", "rssm_init_state", "rssm_flush", "rssm_step", "rssm_step_precompute",
           "rssm_step_readout", "rssm_step_gated", "rssm_step_readout_gated", "rssm_flush_step", "rssm_flush_step_classify", "rssm_flush_step_main", "rssm_accept", "rssm_accept_flush", "rssm_eval_spec_math", "rssm_selftest_wait_timeout",
           "rssm_status_string", "rssm_delta_scratch_bytes", "rssm_delta_step", "rssm_delta_prefill", "rssm_verify",
           "rssm_gated_norm", "rssm_residual_norm", "rssm_kv_append", "rssm_kv_read", "rssm_attention_scratch_bytes",
           "rssm_tree_attention", "rssm_tree_accept", "rssm_logits")


def load(path: str | None = None):
    """Load librssm.so; raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"librssm.so not found at {p}: build it with `python -c 'import __graft_entry__ as g; "
                               "g.build()'` (needs nvcc); there is no CPU fallback")
        lib = ctypes.CDLL(p)
        vp, i32, i64, u64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t
        cp = ctypes.POINTER(RssmCacheStruct)
        lib.rssm_scratch_bytes.restype = sz
        lib.rssm_scratch_bytes.argtypes = [cp, i32, i32]
        lib.rssm_init_state.restype = ctypes.c_int
        lib.rssm_init_state.argtypes = [cp, vp, vp, i32, u64, vp]
        lib.rssm_flush.restype = ctypes.c_int
        lib.rssm_flush.argtypes = [cp, vp, vp, vp, vp, i32, i32, i32, u64, vp, sz, vp]
        step_args = [cp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, vp, vp, sz, vp]
        for name in ("rssm_step", "rssm_step_precompute", "rssm_step_readout"):
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = step_args
        gated_args = step_args[:13] + [vp] + step_args[13:]  # z before out
        for name in ("rssm_step_gated", "rssm_step_readout_gated"):
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = gated_args
        for name in ("rssm_flush_step", "rssm_flush_step_classify", "rssm_flush_step_main"):
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = [cp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, u64, vp, vp, sz, vp]
        lib.rssm_accept.restype = ctypes.c_int
        lib.rssm_accept.argtypes = [cp, vp, vp, vp, vp, i32, i32, vp]
        lib.rssm_accept_flush.restype = ctypes.c_int
        lib.rssm_accept_flush.argtypes = [cp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, u64, vp, sz, vp]
        lib.rssm_eval_spec_math.restype = ctypes.c_int
        lib.rssm_eval_spec_math.argtypes = [vp, vp, vp, i64, vp]
        lib.rssm_selftest_wait_timeout.restype = ctypes.c_int
        lib.rssm_selftest_wait_timeout.argtypes = [vp, i32, vp]
        f32, dp = ctypes.c_float, ctypes.POINTER(RssmDeltaCacheStruct)
        lib.rssm_delta_scratch_bytes.restype = sz
        lib.rssm_delta_scratch_bytes.argtypes = [dp, i32, i64]
        tok_args = [dp, vp, i64, vp, i64, vp, i64, vp, vp, f32, i32, vp]  # cache, q, k, v, g, beta, scale, l2norm, slots
        lib.rssm_delta_step.restype = ctypes.c_int
        lib.rssm_delta_step.argtypes = tok_args + [vp, vp, i32, i32, i64, vp, vp, sz, vp]
        lib.rssm_delta_prefill.restype = ctypes.c_int
        lib.rssm_delta_prefill.argtypes = tok_args + [vp, vp, i32, i64, vp, vp, sz, vp]
        lib.rssm_verify.restype = ctypes.c_int
        lib.rssm_verify.argtypes = [vp, i64, vp, i64, i32, i32, vp, vp, vp, vp, i32, i32, i64, vp, vp, vp, vp]
        lib.rssm_gated_norm.restype = ctypes.c_int
        lib.rssm_gated_norm.argtypes = [vp, i64, vp, i64, i32, vp, i32, i64, i32, i32, f32, i32, vp, i64, vp]
        lib.rssm_residual_norm.restype = ctypes.c_int
        lib.rssm_residual_norm.argtypes = [vp, i64, vp, i64, i32, i32, vp, vp, f32, vp, i64, i32, f32, vp, i64, vp, i64,
                                           vp]
        kp = ctypes.POINTER(RssmKvCacheStruct)
        lib.rssm_kv_append.restype = ctypes.c_int
        lib.rssm_kv_append.argtypes = [kp, i32, vp, i64, vp, i64, vp, i64, i32, vp, vp, i32, i32, i64, vp]
        lib.rssm_kv_read.restype = ctypes.c_int
        lib.rssm_kv_read.argtypes = [kp, i32, vp, i64, i32, vp, vp, i32, i64, i32, vp, i64, vp, i64, vp]
        lib.rssm_attention_scratch_bytes.restype = sz
        lib.rssm_attention_scratch_bytes.argtypes = [kp, i32]
        lib.rssm_tree_attention.restype = ctypes.c_int
        lib.rssm_tree_attention.argtypes = [kp, i32, vp, i64, i32, f32, vp, i64, i32, vp, vp, vp, i32, i32, i64, vp, i64, vp, sz, vp]
        lib.rssm_tree_accept.restype = ctypes.c_int
        lib.rssm_tree_accept.argtypes = [kp, vp, i64, i32, vp, vp, vp, vp, vp, i32, i32, i64, vp, vp, vp, vp, vp]
        lib.rssm_logits.restype = ctypes.c_int
        lib.rssm_logits.argtypes = [ctypes.POINTER(RssmLogitsArgs), vp]
        lib.rssm_status_string.restype = ctypes.c_char_p
        lib.rssm_status_string.argtypes = [ctypes.c_int]
        _lib = lib
        return lib


def fast():
    """The C module that calls librssm with checked arguments (csrc/rssm_call.c); the library is loaded first, so that
    a missing build is reported as in load()."""
    global _fast
    if _fast is None:
        load()
        from . import _call

        _fast = _call
    return _fast


def fast_kv():
    """The same for the calls of attention layers and of the sampler (csrc/rssm_call_kv.c)."""
    global _fast_kv
    if _fast_kv is None:
        load()
        from . import _call_kv

        _fast_kv = _call_kv
    return _fast_kv
