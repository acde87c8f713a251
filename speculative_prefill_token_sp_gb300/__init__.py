"""SpecPrefill token-importance scoring and chunk selection on one GB300.

Python binding of libspecprefill.so (C ABI in include/specprefill.h).  The
functions named ``sp_*`` mirror the C entry points one to one and only marshal
arguments (torch tensors or raw integer addresses become pointers, streams
become cudaStream_t handles).  ``score``/``score_varlen``/``select``/
``select_varlen`` additionally allocate outputs and workspaces with torch and
raise ``SpError`` on a non-zero status.  Every step of the computation runs in
the library's CUDA kernels; if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

__all__ = [
    "SP_OK", "SP_EINVAL", "SP_ENOMEM", "SP_ECUDA", "SP_EDEVICE", "SP_ETIMEOUT", "SP_EUNSUPPORTED",
    "SP_BF16", "SP_F32", "SP_SELECT_TOPK", "SP_SELECT_MASS", "SpBoost", "SpError", "lib", "lib_path",
    "sp_score_workspace_size", "sp_score", "sp_score_lse_workspace_size", "sp_score_lse",
    "sp_score_prefill_workspace_size", "sp_score_prefill",
    "sp_score_varlen_workspace_size", "sp_score_varlen",
    "sp_score_lse_varlen_workspace_size", "sp_score_lse_varlen",
    "sp_select_workspace_size", "sp_select", "sp_select_varlen_workspace_size", "sp_select_varlen",
    "sp_select_noalloc", "sp_select_rules_workspace_size", "sp_select_rules", "SpKeepRules", "GUIDE_RULES",
    "sp_gather_kept", "sp_workspace_status", "sp_last_error", "sp_status_string", "sp_version",
    "sp_kernel_launches", "sp_test_set_exchange_wait_ns", "sp_test_score_plan",
    "score", "score_lse", "score_prefill", "score_varlen", "score_lse_varlen", "select", "select_rules", "select_varlen", "gather_kept", "V3_BOOST",
    "SP_CACHE_SAME", "SP_CACHE_E4M3", "SP_CACHE_INT8", "SpRows", "SpRotaryPlan", "SpCache", "SpBatch",
    "sp_rotary_plan_init", "sp_rotary", "sp_cache_workspace_size", "sp_cache_write", "sp_cache_read",
    "sp_attend_workspace_size", "sp_attend",
    "rotary_plan", "rotary", "Cache", "Batch", "cache_alloc", "cache_write", "cache_read", "attend_workspace_size",
    "attend",
    "sp_tree_workspace_size", "sp_tree_seen", "sp_attend_tree_workspace_size", "sp_attend_tree", "sp_tree_accept",
    "sp_attend_weights_workspace_size", "sp_attend_weights", "sp_cache_choose", "sp_cache_keep",
    "tree_seen", "attend_tree_workspace_size", "attend_tree", "tree_accept", "weights_alloc", "attend_weights_workspace_size",
    "attend_weights", "cache_choose", "cache_keep",
]

SP_OK, SP_EINVAL, SP_ENOMEM, SP_ECUDA, SP_EDEVICE, SP_ETIMEOUT, SP_EUNSUPPORTED = range(7)
SP_BF16, SP_F32 = 0, 1
SP_SELECT_TOPK, SP_SELECT_MASS = 0, 1
SP_CACHE_SAME, SP_CACHE_E4M3, SP_CACHE_INT8 = 0, 1, 2

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libspecprefill.so")


class SpBoost(ctypes.Structure):
    """sp_boost: v3 normalisation and structural boost."""
    _fields_ = [("first_n", ctypes.c_int32), ("first_mult", ctypes.c_double),
                ("last_n", ctypes.c_int32), ("last_mult", ctypes.c_double),
                ("normalize", ctypes.c_int32)]


# The llama.cpp guide's v3 defaults: first 64 tokens x1.5, last 128 x1.3, normalised.
V3_BOOST = (64, 1.5, 128, 1.3, 1)


class SpKeepRules(ctypes.Structure):
    """sp_keep_rules: the guide's v2 keep rules after the chunk selection."""
    _fields_ = [("min_tok", ctypes.c_int32), ("always_keep", ctypes.c_int32), ("max_keep", ctypes.c_int64)]


# The rules the llama.cpp guide runs with: min_tok 128, always-kept tokens, SP_MAX_KEEP 2000.
GUIDE_RULES = (128, 1, 2000)


class SpRows(ctypes.Structure):
    """sp_rows: a tensor [rows, heads, d] by its address and strides."""
    _fields_ = [("data", ctypes.c_void_p), ("stride_row", ctypes.c_int64), ("stride_head", ctypes.c_int64)]


class SpRotaryPlan(ctypes.Structure):
    """sp_rotary_plan: frequencies, filled by sp_rotary_plan_init."""
    _fields_ = [("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("turns", ctypes.c_uint64 * 128), ("axis", ctypes.c_uint8 * 128)]


class SpCache(ctypes.Structure):
    """sp_cache: one layer's paged keys and values."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("stride_page", ctypes.c_int64), ("stride_head", ctypes.c_int64),
                ("stride_slot", ctypes.c_int64), ("pages", ctypes.c_int64), ("page", ctypes.c_int32),
                ("H_kv", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("kind", ctypes.c_int32)]


class SpBatch(ctypes.Structure):
    """sp_batch: the new tokens of B sequences and where they stand."""
    _fields_ = [("B", ctypes.c_int32), ("max_new", ctypes.c_int32), ("T", ctypes.c_int64), ("cu_new", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("table", ctypes.c_void_p), ("table_width", ctypes.c_int32),
                ("table_stride", ctypes.c_int64)]


class SpError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_status_name(status)}: {message}")
        self.status = status


_lib = None
_c = ctypes
_vp, _sz, _i32, _i64, _dbl = _c.c_void_p, _c.c_size_t, _c.c_int, _c.c_int64, _c.c_double
_SIGS = {
    "sp_score_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i64, _i32, _i32]),
    "sp_score": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i64, _i32, _i32, _vp, _vp, _sz, _vp]),
    "sp_score_lse_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i64, _i32, _i32]),
    "sp_score_prefill_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i64, _i32, _i32]),
    "sp_score_prefill": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i64, _i32, _i32, _vp, _vp, _sz, _vp]),
    "sp_score_lse": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i64, _i32, _i32, _vp, _vp, _sz, _vp]),
    "sp_score_varlen_workspace_size": (_sz, [_i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32]),
    "sp_score_varlen": (_i32, [_vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp,
                               _sz, _vp]),
    "sp_score_lse_varlen_workspace_size": (_sz, [_i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32]),
    "sp_score_lse_varlen": (_i32, [_vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp,
                                   _sz, _vp]),
    "sp_select_workspace_size": (_sz, [_i64, _i32]),
    "sp_select": (_i32, [_vp, _i64, _i32, _i32, _i32, _dbl, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sp_select_varlen_workspace_size": (_sz, [_i32, _vp, _i32]),
    "sp_select_varlen": (_i32, [_vp, _i32, _vp, _i32, _i32, _i32, _dbl, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sp_select_noalloc": (_i32, [_vp, _i64, _i32, _i32, _i32, _dbl, _vp, _vp, _vp, _vp]),
    "sp_select_rules_workspace_size": (_sz, [_i64, _i32]),
    "sp_select_rules": (_i32, [_vp, _i64, _i32, _i32, _i32, _dbl, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sp_gather_kept": (_i32, [_vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "sp_rotary_plan_init": (_i32, [_vp, _i32, _vp, _vp, _i32, _i32]),
    "sp_rotary": (_i32, [_vp, _vp, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _vp]),
    "sp_cache_workspace_size": (_sz, []),
    "sp_cache_write": (_i32, [_vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sp_cache_read": (_i32, [_vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sp_attend_workspace_size": (_sz, [_vp, _vp, _i32]),
    "sp_attend": (_i32, [_vp, _vp, _vp, _i32, _dbl, _i64, _vp, _vp, _i64, _i64, _vp, _sz, _vp]),
    "sp_tree_workspace_size": (_sz, []),
    "sp_tree_seen": (_i32, [_vp, _vp, _vp, _i64, _i32, _vp, _vp, _sz, _vp]),
    "sp_attend_tree_workspace_size": (_sz, [_vp, _vp, _i32]),
    "sp_attend_tree": (_i32, [_vp, _vp, _vp, _i32, _dbl, _i64, _vp, _i64, _i32, _vp, _vp, _i64, _i64, _vp, _sz, _vp]),
    "sp_tree_accept": (_i32, [_vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _sz, _vp]),
    "sp_attend_weights_workspace_size": (_sz, [_vp, _vp, _i32]),
    "sp_attend_weights": (_i32, [_vp, _vp, _vp, _i32, _dbl, _i64, _vp, _i64, _i64, _dbl, _vp, _vp, _sz, _vp]),
    "sp_cache_choose": (_i32, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _sz, _vp]),
    "sp_cache_keep": (_i32, [_vp, _vp, _vp, _i32, _i64, _i64, _vp, _i64, _i32, _vp, _i32, _i64, _vp, _vp, _vp, _sz, _vp]),
    "sp_workspace_status": (_i32, [_vp, _vp]),
    "sp_last_error": (_c.c_char_p, []),
    "sp_status_string": (_c.c_char_p, [_i32]),
    "sp_version": (_i32, []),
    "sp_kernel_launches": (_c.c_uint64, []),
    "sp_test_set_exchange_wait_ns": (_c.c_uint64, [_c.c_uint64]),
    "sp_test_score_plan": (_i32, [_i32, _i32, _i32, _i32, _c.c_int64, _i32, _i32, _c.POINTER(_c.c_int)]),
}


def lib():
    """The loaded libspecprefill.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise ImportError(f"{lib_path} is missing: build it with "
                              "`python -m speculative_prefill_token_sp_gb300.build`")
        handle = ctypes.CDLL(lib_path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _status_name(s: int) -> str:
    names = ["SP_OK", "SP_EINVAL", "SP_ENOMEM", "SP_ECUDA", "SP_EDEVICE", "SP_ETIMEOUT", "SP_EUNSUPPORTED"]
    return names[s] if 0 <= s < len(names) else f"status {s}"


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if isinstance(x, ctypes.Array):
        return ctypes.addressof(x)
    raise TypeError(f"cannot pass {type(x).__name__} as a pointer")


def _stream(s) -> Optional[int]:
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _i64_array(values):
    arr = (ctypes.c_int64 * len(values))(*[int(v) for v in values])
    return arr


def _boost(b):
    if b is None:
        return None
    if isinstance(b, SpBoost):
        return ctypes.pointer(b)
    return ctypes.pointer(SpBoost(*b))


# ----------------------------------------------------------------------------
# One-to-one marshalling of the C entry points
# ----------------------------------------------------------------------------

def sp_score_workspace_size(L, H, H_kv, d, M, N, dtype) -> int:
    return lib().sp_score_workspace_size(L, H, H_kv, d, M, N, dtype)


def sp_score(Q_la, K_prompt, K_la, L, H, H_kv, d, M, N, dtype, importance, ws, ws_bytes, stream=None) -> int:
    return lib().sp_score(_ptr(Q_la), _ptr(K_prompt), _ptr(K_la), L, H, H_kv, d, M, N, dtype,
                          _ptr(importance), _ptr(ws), ws_bytes, _stream(stream))


def sp_score_prefill_workspace_size(L, H, H_kv, d, M, N, dtype) -> int:
    return lib().sp_score_prefill_workspace_size(L, H, H_kv, d, M, N, dtype)


def sp_score_prefill(Q_rows, K_prompt, K_la, L, H, H_kv, d, M, N, dtype, importance, ws, ws_bytes,
                     stream=None) -> int:
    return lib().sp_score_prefill(_ptr(Q_rows), _ptr(K_prompt), _ptr(K_la), L, H, H_kv, d, M, N, dtype,
                                  _ptr(importance), _ptr(ws), ws_bytes, _stream(stream))


def sp_score_lse_workspace_size(L, H, H_kv, d, M, N, dtype) -> int:
    return lib().sp_score_lse_workspace_size(L, H, H_kv, d, M, N, dtype)


def sp_score_lse(Q_la, K_prompt, lse, L, H, H_kv, d, M, N, dtype, importance, ws, ws_bytes, stream=None) -> int:
    return lib().sp_score_lse(_ptr(Q_la), _ptr(K_prompt), _ptr(lse), L, H, H_kv, d, M, N, dtype,
                              _ptr(importance), _ptr(ws), ws_bytes, _stream(stream))


def sp_score_varlen_workspace_size(B, cu_M_host, L, H, H_kv, d, N, dtype) -> int:
    cu = _i64_array(cu_M_host)
    return lib().sp_score_varlen_workspace_size(B, ctypes.addressof(cu), L, H, H_kv, d, N, dtype)


def sp_score_varlen(Q_la, K_prompt, K_la, B, cu_M_host, L, H, H_kv, d, N, dtype, importance, ws, ws_bytes,
                    stream=None) -> int:
    cu = _i64_array(cu_M_host)
    return lib().sp_score_varlen(_ptr(Q_la), _ptr(K_prompt), _ptr(K_la), B, ctypes.addressof(cu), L, H, H_kv,
                                 d, N, dtype, _ptr(importance), _ptr(ws), ws_bytes, _stream(stream))


def sp_score_lse_varlen_workspace_size(B, cu_M_host, L, H, H_kv, d, N, dtype) -> int:
    cu = _i64_array(cu_M_host)
    return lib().sp_score_lse_varlen_workspace_size(B, ctypes.addressof(cu), L, H, H_kv, d, N, dtype)


def sp_score_lse_varlen(Q_la, K_prompt, lse, B, cu_M_host, L, H, H_kv, d, N, dtype, importance, ws, ws_bytes,
                        stream=None) -> int:
    cu = _i64_array(cu_M_host)
    return lib().sp_score_lse_varlen(_ptr(Q_la), _ptr(K_prompt), _ptr(lse), B, ctypes.addressof(cu), L, H,
                                     H_kv, d, N, dtype, _ptr(importance), _ptr(ws), ws_bytes, _stream(stream))


def sp_select_workspace_size(M, chunk) -> int:
    return lib().sp_select_workspace_size(M, chunk)


def sp_select(importance, M, chunk, pool_k, mode, rate, boost, kept_pos, n_kept, ws, ws_bytes,
              stream=None) -> int:
    return lib().sp_select(_ptr(importance), M, chunk, pool_k, mode, rate, _boost(boost), _ptr(kept_pos),
                           _ptr(n_kept), _ptr(ws), ws_bytes, _stream(stream))


def _rules(rules):
    if rules is None:
        return None
    if isinstance(rules, SpKeepRules):
        return ctypes.pointer(rules)
    return ctypes.pointer(SpKeepRules(*rules))


def sp_select_rules_workspace_size(M, chunk) -> int:
    return lib().sp_select_rules_workspace_size(M, chunk)


def sp_select_rules(importance, M, chunk, pool_k, mode, rate, boost, rules, kept_pos, n_kept, ws, ws_bytes,
                    stream=None) -> int:
    return lib().sp_select_rules(_ptr(importance), M, chunk, pool_k, mode, rate, _boost(boost), _rules(rules),
                                 _ptr(kept_pos), _ptr(n_kept), _ptr(ws), ws_bytes, _stream(stream))


def sp_select_varlen_workspace_size(B, cu_M_host, chunk) -> int:
    cu = _i64_array(cu_M_host)
    return lib().sp_select_varlen_workspace_size(B, ctypes.addressof(cu), chunk)


def sp_select_varlen(importance, B, cu_M_host, chunk, pool_k, mode, rate, boost, kept_pos, n_kept, ws,
                     ws_bytes, stream=None) -> int:
    cu = _i64_array(cu_M_host)
    return lib().sp_select_varlen(_ptr(importance), B, ctypes.addressof(cu), chunk, pool_k, mode, rate,
                                  _boost(boost), _ptr(kept_pos), _ptr(n_kept), _ptr(ws), ws_bytes,
                                  _stream(stream))


def sp_select_noalloc(importance, M, chunk, pool_k, mode, rate, boost, kept_pos, n_kept, stream=None) -> int:
    """sp_select without a workspace (scratch in a fixed device array of the library)."""
    return lib().sp_select_noalloc(_ptr(importance), M, chunk, pool_k, mode, rate, _boost(boost), _ptr(kept_pos),
                                   _ptr(n_kept), _stream(stream))


def sp_gather_kept(token_ids, B, cu_M_host, kept_pos, n_kept, out_tokens, out_positions, cu_kept,
                   stream=None) -> int:
    cu = _i64_array(cu_M_host)
    return lib().sp_gather_kept(_ptr(token_ids), B, ctypes.addressof(cu), _ptr(kept_pos), _ptr(n_kept),
                                _ptr(out_tokens), _ptr(out_positions), _ptr(cu_kept), _stream(stream))


def _struct(x):
    return None if x is None else ctypes.addressof(x)


def sp_rotary_plan_init(plan, rot, inv_freq_host, axis_of_pair_host, axes, interleaved) -> int:
    freq = (ctypes.c_double * max(len(inv_freq_host), 1))(*inv_freq_host) if inv_freq_host is not None else None
    axis = (ctypes.c_uint8 * max(len(axis_of_pair_host), 1))(*axis_of_pair_host) if axis_of_pair_host is not None else None
    return lib().sp_rotary_plan_init(_struct(plan), rot, _ptr(freq), _ptr(axis), axes, interleaved)


def sp_rotary(plan, positions, pos_stride, T, d, dtype, inverse, q, q_out, H, k, k_out, H_kv, stream=None) -> int:
    return lib().sp_rotary(_struct(plan), _ptr(positions), pos_stride, T, d, dtype, inverse, _struct(q),
                           _struct(q_out), H, _struct(k), _struct(k_out), H_kv, _stream(stream))


def sp_cache_workspace_size() -> int:
    return lib().sp_cache_workspace_size()


def sp_cache_write(cache, batch, k_new, v_new, ws, ws_bytes, stream=None) -> int:
    return lib().sp_cache_write(_struct(cache), _struct(batch), _struct(k_new), _struct(v_new), _ptr(ws), ws_bytes,
                                _stream(stream))


def sp_cache_read(cache, batch, out_k, out_v, ws, ws_bytes, stream=None) -> int:
    return lib().sp_cache_read(_struct(cache), _struct(batch), _struct(out_k), _struct(out_v), _ptr(ws), ws_bytes,
                               _stream(stream))


def sp_attend_workspace_size(cache, batch, H) -> int:
    return lib().sp_attend_workspace_size(_struct(cache), _struct(batch), H)


def sp_attend(q, cache, batch, H, scale, window, out, lse, lse_stride_row, lse_stride_head, ws, ws_bytes,
              stream=None) -> int:
    return lib().sp_attend(_struct(q), _struct(cache), _struct(batch), H, scale, window, _struct(out), _ptr(lse),
                           lse_stride_row, lse_stride_head, _ptr(ws), ws_bytes, _stream(stream))


def sp_tree_workspace_size() -> int:
    return lib().sp_tree_workspace_size()


def sp_tree_seen(batch, parent, seen, seen_stride, seen_words, positions, ws, ws_bytes, stream=None) -> int:
    return lib().sp_tree_seen(_struct(batch), _ptr(parent), _ptr(seen), seen_stride, seen_words, _ptr(positions), _ptr(ws),
                              ws_bytes, _stream(stream))


def sp_attend_tree_workspace_size(cache, batch, H) -> int:
    return lib().sp_attend_tree_workspace_size(_struct(cache), _struct(batch), H)


def sp_attend_tree(q, cache, batch, H, scale, window, seen, seen_stride, seen_words, out, lse, lse_stride_row,
                   lse_stride_head, ws, ws_bytes, stream=None) -> int:
    return lib().sp_attend_tree(_struct(q), _struct(cache), _struct(batch), H, scale, window, _ptr(seen), seen_stride,
                                seen_words, _struct(out), _ptr(lse), lse_stride_row, lse_stride_head, _ptr(ws), ws_bytes,
                                _stream(stream))


def sp_tree_accept(batch, parent, draft, target, path, path_stride, n_path, next, ws, ws_bytes, stream=None) -> int:
    return lib().sp_tree_accept(_struct(batch), _ptr(parent), _ptr(draft), _ptr(target), _ptr(path), path_stride,
                                _ptr(n_path), _ptr(next), _ptr(ws), ws_bytes, _stream(stream))


def sp_attend_weights_workspace_size(cache, batch, H) -> int:
    return lib().sp_attend_weights_workspace_size(_struct(cache), _struct(batch), H)


def sp_attend_weights(q, cache, batch, H, scale, window, lse, lse_stride_row, lse_stride_head, decay, weights, ws, ws_bytes,
                      stream=None) -> int:
    return lib().sp_attend_weights(_struct(q), _struct(cache), _struct(batch), H, scale, window, _ptr(lse), lse_stride_row,
                                   lse_stride_head, decay, _ptr(weights), _ptr(ws), ws_bytes, _stream(stream))


def sp_cache_choose(cache, batch, weights, shared, budget, first, last, kept, kept_stride_seq, kept_stride_head, n_kept, ws,
                    ws_bytes, stream=None) -> int:
    return lib().sp_cache_choose(_struct(cache), _struct(batch), _ptr(weights), shared, budget, first, last, _ptr(kept),
                                 kept_stride_seq, kept_stride_head, _ptr(n_kept), _ptr(ws), ws_bytes, _stream(stream))


def sp_cache_keep(cache, batch, kept, heads, kept_stride_seq, kept_stride_head, n_kept, most, drafted, to, to_width,
                  to_stride, weights, kv_out, ws, ws_bytes, stream=None) -> int:
    return lib().sp_cache_keep(_struct(cache), _struct(batch), _ptr(kept), heads, kept_stride_seq, kept_stride_head,
                               _ptr(n_kept), most, drafted, _ptr(to), to_width, to_stride, _ptr(weights), _ptr(kv_out),
                               _ptr(ws), ws_bytes, _stream(stream))


def sp_workspace_status(ws, stream=None) -> int:
    return lib().sp_workspace_status(_ptr(ws), _stream(stream))


def sp_last_error() -> str:
    return lib().sp_last_error().decode()


def sp_status_string(s: int) -> str:
    return lib().sp_status_string(s).decode()


def sp_version() -> int:
    return lib().sp_version()


def sp_kernel_launches() -> int:
    return lib().sp_kernel_launches()


def sp_test_set_exchange_wait_ns(ns: int) -> int:
    """Test hook: limit (ns) of the scoring kernel's waits on other CTAs' exchange
    entries; 0 restores the default.  Returns the previous limit."""
    return lib().sp_test_set_exchange_wait_ns(int(ns))


def sp_test_score_plan(L: int, H: int, H_kv: int, d: int, M: int, N: int, sms: int = 152):
    """Test hook: the tensor-core scoring plan of one bf16 prompt as a dict
    (F, Pc, P, tiles, tiles_per_group, land, held, lag, smem_bytes), or None when
    that path does not take the shape.  Host only."""
    out = (_c.c_int * 9)()
    if not lib().sp_test_score_plan(L, H, H_kv, d, int(M), N, sms, out):
        return None
    keys = ("F", "Pc", "P", "tiles", "tiles_per_group", "land", "held", "lag", "smem_bytes")
    return dict(zip(keys, list(out)))


# ----------------------------------------------------------------------------
# Helpers that allocate with torch
# ----------------------------------------------------------------------------

def _check(status: int) -> None:
    if status != SP_OK:
        raise SpError(status, sp_last_error())


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return SP_BF16
    if t.dtype == torch.float32:
        return SP_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _workspace(nbytes: int, device, ws=None):
    import torch
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise SpError(SP_ENOMEM, f"workspace smaller than {nbytes} bytes")
        return ws
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _check_device(ws, stream, check):
    if check:
        _check(sp_workspace_status(ws, stream))


def score(Q_la, K_prompt, K_la, *, importance=None, ws=None, stream=None, check=False):
    """Importance [M] (fp32) of one prompt: Q_la [N,L,H,d], K_prompt [L,H_kv,M,d], K_la [L,H_kv,N,d].
    check=True synchronises and raises if a kernel recorded a run-time error."""
    import torch
    N, L, H, d = Q_la.shape
    _, H_kv, M, _ = K_prompt.shape
    dt = _dtype_code(K_prompt)
    if importance is None:
        importance = torch.empty(M, dtype=torch.float32, device=K_prompt.device)
    need = sp_score_workspace_size(L, H, H_kv, d, M, N, dt)
    ws = _workspace(need, K_prompt.device, ws)
    _check(sp_score(Q_la, K_prompt, K_la, L, H, H_kv, d, M, N, dt, importance, ws, ws.numel(), stream))
    _check_device(ws, stream, check)
    return importance


def score_prefill(Q_rows, K_prompt, K_la, *, importance=None, ws=None, stream=None, check=False):
    """Importance [M] (fp32) from the prefill's last query (Q_rows[0]) and N decode steps (Q_rows[1:]):
    Q_rows [N+1,L,H,d], K_prompt [L,H_kv,M,d], K_la [L,H_kv,N,d]."""
    import torch
    N1, L, H, d = Q_rows.shape
    _, H_kv, M, _ = K_prompt.shape
    dt = _dtype_code(K_prompt)
    if importance is None:
        importance = torch.empty(M, dtype=torch.float32, device=K_prompt.device)
    need = sp_score_prefill_workspace_size(L, H, H_kv, d, M, N1 - 1, dt)
    ws = _workspace(need, K_prompt.device, ws)
    _check(sp_score_prefill(Q_rows, K_prompt, K_la, L, H, H_kv, d, M, N1 - 1, dt, importance, ws, ws.numel(),
                            stream))
    _check_device(ws, stream, check)
    return importance


def score_lse(Q_la, K_prompt, lse, *, importance=None, ws=None, stream=None, check=False):
    """Importance [M] (fp32) of one prompt from given row normalisers: Q_la [N,L,H,d],
    K_prompt [L,H_kv,M,d], lse [L,H,N] fp32 (device)."""
    import torch
    N, L, H, d = Q_la.shape
    _, H_kv, M, _ = K_prompt.shape
    dt = _dtype_code(K_prompt)
    if importance is None:
        importance = torch.empty(M, dtype=torch.float32, device=K_prompt.device)
    need = sp_score_lse_workspace_size(L, H, H_kv, d, M, N, dt)
    ws = _workspace(need, K_prompt.device, ws)
    _check(sp_score_lse(Q_la, K_prompt, lse, L, H, H_kv, d, M, N, dt, importance, ws, ws.numel(), stream))
    _check_device(ws, stream, check)
    return importance


def score_varlen(Q_la, K_prompt, K_la, cu_M, *, importance=None, ws=None, stream=None, check=False):
    """Packed importance [T] of B prompts: Q_la [B,N,L,H,d], K_prompt [L,H_kv,T,d], K_la [B,L,H_kv,N,d]."""
    import torch
    B, N, L, H, d = Q_la.shape
    H_kv, T = K_prompt.shape[1], K_prompt.shape[2]
    cu = [int(x) for x in cu_M]
    dt = _dtype_code(K_prompt)
    if importance is None:
        importance = torch.empty(T, dtype=torch.float32, device=K_prompt.device)
    need = sp_score_varlen_workspace_size(B, cu, L, H, H_kv, d, N, dt)
    ws = _workspace(need, K_prompt.device, ws)
    _check(sp_score_varlen(Q_la, K_prompt, K_la, B, cu, L, H, H_kv, d, N, dt, importance, ws, ws.numel(),
                           stream))
    _check_device(ws, stream, check)
    return importance


def score_lse_varlen(Q_la, K_prompt, lse, cu_M, *, importance=None, ws=None, stream=None, check=False):
    """Packed importance [T] of B prompts from given row normalisers: Q_la [B,N,L,H,d],
    K_prompt [L,H_kv,T,d], lse [B,L,H,N] fp32 (device)."""
    import torch
    B, N, L, H, d = Q_la.shape
    H_kv, T = K_prompt.shape[1], K_prompt.shape[2]
    cu = [int(x) for x in cu_M]
    dt = _dtype_code(K_prompt)
    if importance is None:
        importance = torch.empty(T, dtype=torch.float32, device=K_prompt.device)
    need = sp_score_lse_varlen_workspace_size(B, cu, L, H, H_kv, d, N, dt)
    ws = _workspace(need, K_prompt.device, ws)
    _check(sp_score_lse_varlen(Q_la, K_prompt, lse, B, cu, L, H, H_kv, d, N, dt, importance, ws, ws.numel(),
                               stream))
    _check_device(ws, stream, check)
    return importance


def _mode(mode) -> int:
    if mode in (SP_SELECT_TOPK, "topk"):
        return SP_SELECT_TOPK
    if mode in (SP_SELECT_MASS, "mass"):
        return SP_SELECT_MASS
    raise ValueError(f"unknown mode {mode!r}")


def select(importance, chunk, pool_k, mode, rate, boost=None, *, kept_pos=None, n_kept=None, ws=None,
           stream=None, trim=True):
    """Kept position IDs of one prompt.  With trim=True (synchronises) returns
    kept_pos[:n]; otherwise (kept_pos buffer, n_kept device tensor)."""
    import torch
    M = importance.shape[0]
    dev = importance.device
    if kept_pos is None:
        kept_pos = torch.empty(max(M, 1), dtype=torch.int32, device=dev)
    if n_kept is None:
        n_kept = torch.empty(1, dtype=torch.int64, device=dev)
    ws = _workspace(sp_select_workspace_size(M, chunk), dev, ws)
    _check(sp_select(importance, M, chunk, pool_k, _mode(mode), float(rate), boost, kept_pos, n_kept, ws,
                     ws.numel(), stream))
    if trim:
        return kept_pos[: int(n_kept.item())]
    return kept_pos, n_kept


def select_rules(importance, chunk, pool_k, mode, rate, boost=None, rules=GUIDE_RULES, *, ws=None, stream=None):
    """Kept position IDs of one prompt after the selection and the keep rules (synchronises)."""
    import torch
    M = importance.shape[0]
    dev = importance.device
    kept_pos = torch.empty(max(M, 1), dtype=torch.int32, device=dev)
    n_kept = torch.empty(1, dtype=torch.int64, device=dev)
    ws = _workspace(sp_select_rules_workspace_size(M, chunk), dev, ws)
    _check(sp_select_rules(importance, M, chunk, pool_k, _mode(mode), float(rate), boost, rules, kept_pos, n_kept,
                           ws, ws.numel(), stream))
    return kept_pos[: int(n_kept.item())]


def select_varlen(importance, cu_M, chunk, pool_k, mode, rate, boost=None, *, kept_pos=None, n_kept=None,
                  ws=None, stream=None, trim=True):
    """Per-prompt kept position IDs of a packed batch.  trim=True returns a list of tensors."""
    import torch
    cu = [int(x) for x in cu_M]
    B = len(cu) - 1
    dev = importance.device
    if kept_pos is None:
        kept_pos = torch.empty(max(cu[-1], 1), dtype=torch.int32, device=dev)
    if n_kept is None:
        n_kept = torch.empty(B, dtype=torch.int64, device=dev)
    ws = _workspace(sp_select_varlen_workspace_size(B, cu, chunk), dev, ws)
    _check(sp_select_varlen(importance, B, cu, chunk, pool_k, _mode(mode), float(rate), boost, kept_pos,
                            n_kept, ws, ws.numel(), stream))
    if trim:
        n = n_kept.tolist()
        return [kept_pos[cu[b]: cu[b] + n[b]] for b in range(B)]
    return kept_pos, n_kept


def gather_kept(token_ids, cu_M, kept_pos, n_kept, *, stream=None):
    """Sparse-prefill batch of packed prompts: (tokens int32, positions int32, cu_kept int64 [B+1]),
    each prompt's kept tokens packed after the previous prompt's (device tensors, capacity T)."""
    import torch
    cu = [int(x) for x in cu_M]
    B, T = len(cu) - 1, cu[-1]
    dev = kept_pos.device
    tokens = torch.empty(max(T, 1), dtype=torch.int32, device=dev)
    positions = torch.empty(max(T, 1), dtype=torch.int32, device=dev)
    cu_kept = torch.empty(B + 1, dtype=torch.int64, device=dev)
    _check(sp_gather_kept(token_ids, B, cu, kept_pos, n_kept, tokens, positions, cu_kept, stream))
    return tokens, positions, cu_kept


# ----------------------------------------------------------------------------
# Positions, the paged cache, and attention over it
# ----------------------------------------------------------------------------

def rotary_plan(rot, *, base=10000.0, inv_freq=None, sections=None, axis_of_pair=None, interleaved=False):
    """Rotary frequencies for `rotary`: base ** (-2 i / rot), or the given inv_freq (rot / 2 values).
    sections: how many consecutive pairs each position axis has (time, height, width, say), or
    axis_of_pair: each pair's axis.  interleaved: pair i is entries 2i, 2i + 1, not i, i + rot / 2."""
    rot = int(rot)
    pairs = rot // 2
    freq = [float(base) ** (-i / pairs) for i in range(pairs)] if inv_freq is None else [float(f) for f in inv_freq]
    if sections is not None:
        if axis_of_pair is not None:
            raise ValueError("give sections or axis_of_pair, not both")
        axis_of_pair = [a for a, n in enumerate(sections) for _ in range(n)]
    axis = [0] * pairs if axis_of_pair is None else [int(a) for a in axis_of_pair]
    if len(freq) != pairs or len(axis) != pairs:
        raise ValueError(f"a plan of {rot} entries has {pairs} pairs: got {len(freq)} frequencies, {len(axis)} axes")
    if any(not 0 <= a < 8 for a in axis):
        raise ValueError("axes are numbered 0 to 7")
    plan = SpRotaryPlan()
    axes = max(len(sections) if sections is not None else 0, max(axis, default=0) + 1)
    _check(sp_rotary_plan_init(plan, rot, freq, axis, axes, int(bool(interleaved))))
    return plan


def _rows(t, heads_first=False):
    """sp_rows of a tensor [rows, heads, d] (heads_first: [heads, rows, d]) whose last axis is contiguous.  The stride
    of an axis with one entry may be anything in torch: d takes its place."""
    s0, s1, s2 = t.stride()
    if s2 != 1 and t.numel():
        raise ValueError("the last axis must be contiguous")
    if (s0 | s1) & 7:
        n0, n1, d = t.shape
        if n0 == 1:
            s0 = d
        if n1 == 1:
            s1 = d
    return SpRows(t.data_ptr(), s1, s0) if heads_first else SpRows(t.data_ptr(), s0, s1)


# The helpers below are called for every layer of every step, so their own time on the host counts: torch is looked
# up once, and a call for the current device and stream (nearly all of them) enters no context.
_torch = None


def _load_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _on(device, stream, call):
    """call(stream handle) with `device` and `stream` (None: its current one) current, so that what the call
    allocates belongs to the stream that uses it."""
    torch = _torch
    if device.type != "cuda":
        raise ValueError(f"the tensors must be on a GPU (got {device})")
    index = device.index
    if stream is None and index == torch._C._cuda_getDevice():
        return call(torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(device):
        if stream is None:
            return call(torch.cuda.current_stream().cuda_stream)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _same_device(device, *tensors):
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"tensors on different devices: {device} and {t.device}")


def _space(nbytes, device, ws):
    """(workspace, its bytes): the caller's, or a new one."""
    if ws is None:
        return _torch.empty(nbytes or 256, dtype=_torch.uint8, device=device), nbytes
    if ws.device != device:
        raise ValueError(f"the workspace is on {ws.device}, the tensors on {device}")
    return ws, ws.numel() * ws.element_size()


def rotary(q, k, positions, plan, *, inverse=False, q_out=None, k_out=None, stream=None):
    """Rotates q [T, H, d] and k [T, H_kv, d] (either may be None) at positions [T] or [axes, T] (int32) and returns
    (q_out, k_out).  q_out=q rotates in place.  inverse=True undoes the rotation (and is its gradient)."""
    torch = _torch or _load_torch()
    some = k if q is None else q
    if some is None:
        raise ValueError("neither q nor k")
    T, H, d = some.shape
    H_kv, dtype, device, code = 0, some.dtype, some.device, _dtype_code(some)
    if q is None:
        H, H_kv = 0, H
    elif k is not None:
        T2, H_kv, d2 = k.shape
        if T2 != T or d2 != d or k.dtype != dtype or k.device != device:
            raise ValueError("q and k must be [T, heads, d] of the same T, d, dtype and device")
    per_axis = positions.stride()
    axes = positions.shape[0] if len(per_axis) == 2 else 1
    if positions.dtype != torch.int32 or positions.shape[-1] != T or len(per_axis) > 2 or positions.device != device:
        raise ValueError("positions must be int32, [T] or [axes, T], on the device of q and k")
    if axes < plan.axes:
        raise ValueError(f"the plan has {plan.axes} axes: positions must be [{plan.axes}, T]")
    for t, o in ((q, q_out), (k, k_out)):
        if o is not None and (t is None or o.shape != t.shape or o.dtype != dtype or o.device != device):
            raise ValueError("q_out and k_out must have the shape, dtype and device of q and k")

    def call(handle):
        p, qo, ko = positions, q_out, k_out
        if per_axis[-1] != 1 and T > 1:
            p = p.contiguous()
        qr = kr = qor = kor = None
        if q is not None:
            if qo is None:
                qo = torch.empty((T, H, d), dtype=dtype, device=device)
            qr, qor = _rows(q), _rows(qo)
        if k is not None:
            if ko is None:
                ko = torch.empty((T, H_kv, d), dtype=dtype, device=device)
            kr, kor = _rows(k), _rows(ko)
        at = ctypes.addressof
        status = lib().sp_rotary(at(plan), p.data_ptr(), p.stride(0) if len(per_axis) == 2 else 0, T, d, code,
                                 1 if inverse else 0, qr and at(qr), qor and at(qor), H, kr and at(kr), kor and at(kor),
                                 H_kv, handle)
        if status:
            _check(status)
        return qo, ko

    return _on(device, stream, call)


class Cache:
    """One layer's paged keys and values: k and v [pages, H_kv, page, d] (any strides with the last axis contiguous;
    the same for both), of `dtype` (bf16 or f32) or, for an 8-bit cache, float8_e4m3fn or int8 with k_scale and
    v_scale fp32 [pages, H_kv, page].  cache_write makes the scales powers of two; those of a cache that was filled
    elsewhere may be any.  dtype: of the rows that are written and read (default: k's)."""

    def __init__(self, k, v, k_scale=None, v_scale=None, *, dtype=None):
        torch = _torch or _load_torch()
        kinds = {torch.float8_e4m3fn: SP_CACHE_E4M3, torch.int8: SP_CACHE_INT8}
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride():
            raise ValueError("k and v must be [pages, H_kv, page, d] of the same shape, dtype and strides")
        if k.stride(3) != 1:
            raise ValueError("the last axis of k and v must be contiguous")
        kind = kinds.get(k.dtype, SP_CACHE_SAME)
        dtype = dtype or (k.dtype if kind == SP_CACHE_SAME else torch.bfloat16)
        if kind == SP_CACHE_SAME:
            if dtype != k.dtype or k_scale is not None or v_scale is not None:
                raise ValueError(f"a cache of {k.dtype} holds rows of that dtype and has no scales")
        else:
            for s in (k_scale, v_scale):
                if s is None or s.dtype != torch.float32 or s.shape != k.shape[:3] or not s.is_contiguous():
                    raise ValueError("an 8-bit cache needs k_scale and v_scale, contiguous fp32 [pages, H_kv, page]")
        _same_device(k.device, v, k_scale, v_scale)
        code = {torch.bfloat16: SP_BF16, torch.float32: SP_F32}.get(dtype)
        if code is None:
            raise TypeError(f"unsupported dtype {dtype}")
        self.k, self.v, self.k_scale, self.v_scale, self.dtype, self.kind = k, v, k_scale, v_scale, dtype, kind
        self.device = k.device
        self.ws_bytes = sp_cache_workspace_size()
        self.pages, self.H_kv, self.page, self.d = k.shape
        sp_, sh, ss, _ = k.stride()
        self.c = SpCache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), sp_, sh, ss, self.pages, self.page,
                         self.H_kv, self.d, code, kind)
        self.at = ctypes.addressof(self.c)


def cache_alloc(pages, H_kv, page, d, *, dtype=None, kind="same", device="cuda"):
    """A Cache of uninitialised pages.  kind: "same" (rows held in dtype), "e4m3" or "int8"."""
    import torch
    dtype = dtype or torch.bfloat16
    kinds = {"same": dtype, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
    if kind not in kinds:
        raise ValueError(f"kind must be one of {sorted(kinds)} (got {kind!r})")
    held = kinds[kind]
    new = lambda: torch.empty(pages, H_kv, page, d, dtype=held, device=device)          # noqa: E731
    scale = lambda: None if kind == "same" else torch.empty(pages, H_kv, page, dtype=torch.float32, device=device)  # noqa: E731
    return Cache(new(), new(), scale(), scale(), dtype=dtype)


class Batch:
    """The new tokens of B sequences: cu_new int64 [B + 1] (offsets of their rows), kv_len int64 [B] (tokens in the
    cache, the new ones included) and table int32 [B, width] (page of each `page` tokens), on the device, read when
    the work runs.  rows: rows of the calls' tensors; max_new: at least the largest number of new tokens of a
    sequence (default: rows)."""

    def __init__(self, cu_new, kv_len, table, *, rows, max_new=None):
        torch = _torch or _load_torch()
        B = kv_len.shape[0]
        if cu_new.dtype != torch.int64 or kv_len.dtype != torch.int64 or table.dtype != torch.int32:
            raise TypeError("cu_new and kv_len must be int64, table int32")
        if cu_new.shape != (B + 1,) or kv_len.dim() != 1 or table.dim() != 2 or table.shape[0] != B:
            raise ValueError("cu_new must be [B + 1], kv_len [B] and table [B, width]")
        if not cu_new.is_contiguous() or not kv_len.is_contiguous() or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError("cu_new, kv_len and the rows of table must be contiguous")
        _same_device(cu_new.device, kv_len, table)
        self.cu_new, self.kv_len, self.table, self.rows = cu_new, kv_len, table, int(rows)
        self.device = cu_new.device
        self.max_new = self.rows if max_new is None else int(max_new)
        self.c = SpBatch(B, self.max_new, self.rows, _ptr(cu_new), _ptr(kv_len), _ptr(table), table.shape[1],
                         table.stride(0) if B > 1 else 0)
        self.at = ctypes.addressof(self.c)


def _check_rows_of(t, name, rows, heads, d, dtype, device):
    if t.shape != (rows, heads, d) or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be {dtype} [{rows}, {heads}, {d}] on {device}: "
                         f"got {t.dtype} {list(t.shape)} on {t.device}")


def cache_write(cache, batch, k_new, v_new, *, ws=None, stream=None, check=False):
    """Writes the batch's new tokens, k_new and v_new [rows, H_kv, d], into the cache."""
    device = cache.device
    _check_rows_of(k_new, "k_new", batch.rows, cache.H_kv, cache.d, cache.dtype, device)
    _check_rows_of(v_new, "v_new", batch.rows, cache.H_kv, cache.d, cache.dtype, device)
    _same_device(device, batch)

    def call(handle):
        w, size = _space(cache.ws_bytes, device, ws)
        kr, vr = _rows(k_new), _rows(v_new)
        status = lib().sp_cache_write(cache.at, batch.at, ctypes.addressof(kr), ctypes.addressof(vr), w.data_ptr(), size,
                                      handle)
        if status:
            _check(status)
        if check:
            _check(sp_workspace_status(w, handle))

    _on(device, stream, call)


def cache_read(cache, batch, *, out_k=None, out_v=None, ws=None, stream=None, check=False):
    """Reads the batch's tokens back: (out_k, out_v) [H_kv, rows, d], a layer of score's K_prompt each.  Given
    outputs are written in place (any strides with the last axis contiguous), and one that is not given while the
    other is stays out.  With neither given both are made, and rows that are not a token of the batch are not set."""
    device = cache.device
    for t, name in ((out_k, "out_k"), (out_v, "out_v")):
        if t is not None:
            _check_rows_of(t, name, cache.H_kv, batch.rows, cache.d, cache.dtype, device)
    _same_device(device, batch)

    def call(handle):
        k, v = out_k, out_v
        if k is None and v is None:
            k, v = (_torch.empty(cache.H_kv, batch.rows, cache.d, dtype=cache.dtype, device=device) for _ in range(2))
        w, size = _space(cache.ws_bytes, device, ws)
        kr, vr = None if k is None else _rows(k, True), None if v is None else _rows(v, True)
        status = lib().sp_cache_read(cache.at, batch.at, kr and ctypes.addressof(kr), vr and ctypes.addressof(vr),
                                     w.data_ptr(), size, handle)
        if status:
            _check(status)
        if check:
            _check(sp_workspace_status(w, handle))
        return k, v

    return _on(device, stream, call)


def attend_workspace_size(q, cache, batch):
    """Workspace bytes of attend for these arguments."""
    return _on(cache.device, None, lambda handle: sp_attend_workspace_size(cache.c, batch.c, q.shape[1]))


def attend(q, cache, batch, *, scale=None, window=0, out=None, lse=None, ws=None, stream=None, check=False):
    """Causal attention of the batch's new tokens, q [rows, H, d], over their sequences' cached tokens (their own
    among them): (out [rows, H, d], lse fp32 [H, rows]).  scale: default 1 / sqrt(d).  window > 0: each token sees
    itself and the window - 1 tokens before it.  lse may be any strided fp32 [H, rows], such as [l, :, j:j+1] of
    score_lse's [L, H, N].  out must not overlap q.  Rows that are not a token of the batch are not written."""
    return _attend(q, cache, batch, None, scale, window, out, lse, ws, stream, check)


def _attend(q, cache, batch, seen, scale, window, out, lse, ws, stream, check):
    device, rows = cache.device, batch.rows
    H = q.shape[1] if q.dim() == 3 else 0
    _check_rows_of(q, "q", rows, H, cache.d, cache.dtype, device)
    if out is not None:
        _check_rows_of(out, "out", rows, H, cache.d, cache.dtype, device)
    if lse is not None and (lse.shape != (H, rows) or lse.dtype != _torch.float32 or lse.device != device):
        raise ValueError(f"lse must be fp32 [{H}, {rows}] on {device}")
    _same_device(device, batch)

    def call(handle):
        o, z = out, lse
        if o is None:
            o = _torch.empty((rows, H, cache.d), dtype=cache.dtype, device=device)
        if z is None:
            z = _torch.empty(H, rows, dtype=_torch.float32, device=device)
        w, size = _space(sp_attend_workspace_size(cache.c, batch.c, H) if ws is None else 0, device, ws)
        zh, zr = z.stride()
        qr, outr = _rows(q), _rows(o)
        scale_ = cache.d ** -0.5 if scale is None else float(scale)
        if seen is None:
            status = lib().sp_attend(ctypes.addressof(qr), cache.at, batch.at, H, scale_, int(window),
                                     ctypes.addressof(outr), z.data_ptr(), zr, zh, w.data_ptr(), size, handle)
        else:
            status = lib().sp_attend_tree(ctypes.addressof(qr), cache.at, batch.at, H, scale_, int(window), seen.data_ptr(),
                                          _row_stride(seen), seen.shape[1], ctypes.addressof(outr), z.data_ptr(), zr, zh,
                                          w.data_ptr(), size, handle)
        if status:
            _check(status)
        if check:
            _check(sp_workspace_status(w, handle))
        return o, z

    return _on(device, stream, call)


# ----------------------------------------------------------------------------
# Trees of drafted tokens
# ----------------------------------------------------------------------------

def _check_ints(t, name, shape, device, dtype=None):
    """An integer tensor of this shape (None: any extent, of all axes but the first) whose last axis is contiguous."""
    dtype = dtype or _torch.int32
    have = t.shape
    if t.dtype is dtype and t.is_contiguous() and t.get_device() == device.index and \
            (have == shape or (shape[-1] is None and len(have) == len(shape) and have[0] == shape[0])):
        return                  # nearly every call's: the rest takes four times as long
    if t.dtype != dtype or t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        want = ", ".join("*" if n is None else str(n) for n in shape)
        raise ValueError(f"{name} must be {str(dtype)[6:]} [{want}]: got {t.dtype} {list(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")


def _row_stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[-1]


def tree_seen(batch, parent, *, seen=None, positions=None, ws=None, stream=None, check=False):
    """What the batch's new tokens see if they are drafted ones that form a tree: parent int32 [rows], the new token of the
    same sequence that each hangs on, counted from the sequence's first and before its child, or -1.  Returns (seen int32
    [rows, words], the bits that attend_tree takes, and positions int32 [rows], which rotary takes).  Rows that are not
    a token of the batch are not written.  At most 4096 new tokens a sequence."""
    device, rows = batch.device, batch.rows
    words = max(1, -(-batch.max_new // 32))
    _check_ints(parent, "parent", (rows,), device)
    if seen is not None:
        _check_ints(seen, "seen", (rows, None), device)
    if positions is not None:
        _check_ints(positions, "positions", (rows,), device)

    def call(handle):
        s, p = seen, positions
        if s is None:
            s = _torch.empty(rows, words, dtype=_torch.int32, device=device)
        if p is None:
            p = _torch.empty(rows, dtype=_torch.int32, device=device)
        w, size = _space(sp_tree_workspace_size() if ws is None else 0, device, ws)
        status = lib().sp_tree_seen(batch.at, parent.data_ptr(), s.data_ptr(), _row_stride(s), s.shape[1], p.data_ptr(),
                                    w.data_ptr(), size, handle)
        if status:
            _check(status)
        if check:
            _check(sp_workspace_status(w, handle))
        return s, p

    return _on(device, stream, call)


def attend_tree_workspace_size(q, cache, batch):
    """Workspace bytes of attend_tree for these arguments."""
    return _on(cache.device, None, lambda handle: sp_attend_tree_workspace_size(cache.c, batch.c, q.shape[1]))


def attend_tree(q, cache, batch, seen, *, scale=None, window=0, out=None, lse=None, ws=None, stream=None, check=False):
    """Attention of drafted tokens: as attend, but of the new tokens each row sees those whose bits are set in seen int32
    [rows, words], as tree_seen makes them (word u // 32, bit u % 32 for the sequence's new token u).  A window counts from
    a row's place, behind the cached tokens and the new ones that it sees, and hides cached tokens only."""
    _check_ints(seen, "seen", (batch.rows, None), cache.device)
    return _attend(q, cache, batch, seen, scale, window, out, lse, ws, stream, check)


def tree_accept(batch, parent, draft, target, *, path=None, n_path=None, next_token=None, ws=None, stream=None, check=False):
    """The drafted tokens that the target agrees with.  draft and target int32 [rows]: the token that each row is, and the
    target's choice after it.  A sequence's first new token is accepted, and after an accepted token its first child that is
    the target's choice.  Returns (path int32 [B, max_new], the accepted ones of each sequence counted from its first, then -1;
    n_path int64 [B]; next_token int32 [B], the target's choice after the last).  path and n_path go to cache_keep."""
    device, rows, B = batch.device, batch.rows, batch.c.B
    for t, name in ((parent, "parent"), (draft, "draft"), (target, "target")):
        _check_ints(t, name, (rows,), device)
    if path is not None:
        _check_ints(path, "path", (B, batch.max_new), device)
    if n_path is not None:
        _check_ints(n_path, "n_path", (B,), device, _torch.int64)
    if next_token is not None:
        _check_ints(next_token, "next_token", (B,), device)

    def call(handle):
        p, n, x = path, n_path, next_token
        if p is None:
            p = _torch.empty(B, batch.max_new, dtype=_torch.int32, device=device)
        if n is None:
            n = _torch.empty(B, dtype=_torch.int64, device=device)
        if x is None:
            x = _torch.empty(B, dtype=_torch.int32, device=device)
        w, size = _space(sp_tree_workspace_size() if ws is None else 0, device, ws)
        status = lib().sp_tree_accept(batch.at, parent.data_ptr(), draft.data_ptr(), target.data_ptr(), p.data_ptr(),
                                      _row_stride(p), n.data_ptr(), x.data_ptr(), w.data_ptr(), size, handle)
        if status:
            _check(status)
        if check:
            _check(sp_workspace_status(w, handle))
        return p, n, x

    return _on(device, stream, call)


# ----------------------------------------------------------------------------
# Cutting a cache
# ----------------------------------------------------------------------------

def weights_alloc(cache):
    """Weights of a cache's tokens, fp32 [pages, H_kv, page], for attend_weights (uninitialised: a new token's starts from 0)."""
    torch = _torch or _load_torch()
    return torch.empty(cache.pages, cache.H_kv, cache.page, dtype=torch.float32, device=cache.device)


def _check_weights(weights, cache):
    if weights.shape != (cache.pages, cache.H_kv, cache.page) or weights.dtype != _torch.float32 or \
            not weights.is_contiguous() or weights.device != cache.device:
        raise ValueError(f"weights must be contiguous fp32 [{cache.pages}, {cache.H_kv}, {cache.page}] on {cache.device}")


def attend_weights_workspace_size(q, cache, batch):
    """Workspace bytes of attend_weights for these arguments."""
    return _on(cache.device, None, lambda handle: sp_attend_weights_workspace_size(cache.c, batch.c, q.shape[1]))


def attend_weights(q, cache, batch, lse, weights, *, scale=None, window=0, decay=1.0, ws=None, stream=None, check=False):
    """Adds the attention weights that the batch's new tokens give their sequences' cached tokens to weights fp32 [pages, H_kv,
    page], summed over new tokens and the query heads of a KV head: weights = decay * weights + the sum.  q, scale and window
    as given to attend, lse fp32 [H, rows] as it returned it.  New tokens start from 0; with decay=0 all do (the weights that
    the last tokens of a prompt give it, say).  Returns weights."""
    device, rows = cache.device, batch.rows
    H = q.shape[1] if q.dim() == 3 else 0
    _check_rows_of(q, "q", rows, H, cache.d, cache.dtype, device)
    if lse.shape != (H, rows) or lse.dtype != _torch.float32 or lse.device != device:
        raise ValueError(f"lse must be fp32 [{H}, {rows}] on {device}")
    _check_weights(weights, cache)
    _same_device(device, batch)

    def call(handle):
        w, size = _space(sp_attend_weights_workspace_size(cache.c, batch.c, H) if ws is None else 0, device, ws)
        zh, zr = lse.stride()
        qr = _rows(q)
        status = lib().sp_attend_weights(ctypes.addressof(qr), cache.at, batch.at, H,
                                         cache.d ** -0.5 if scale is None else float(scale), int(window), lse.data_ptr(), zr, zh,
                                         float(decay), weights.data_ptr(), w.data_ptr(), size, handle)
        if status:
            _check(status)
        if check:
            _check(sp_workspace_status(w, handle))
        return weights

    return _on(device, stream, call)


def cache_choose(cache, batch, weights, budget, *, first=0, last=0, shared=False, kept=None, n_kept=None, ws=None, stream=None,
                 check=False):
    """Which `budget` tokens each sequence keeps: its first and last ones, and of those between the ones with the largest
    weights (ties to the lower token); all if it has no more.  Returns (kept int32 [B, H_kv, budget], ascending and then -1, and
    n_kept int64 [B]).  shared=True: one list for all heads, kept [B, 1, budget], by the maximum of their weights."""
    device, B, budget = cache.device, batch.c.B, int(budget)
    heads = 1 if shared else cache.H_kv
    _check_weights(weights, cache)
    _same_device(device, batch)
    if kept is not None:
        _check_ints(kept, "kept", (B, heads, budget), device)
    if n_kept is not None:
        _check_ints(n_kept, "n_kept", (B,), device, _torch.int64)

    def call(handle):
        k, n = kept, n_kept
        if k is None:
            k = _torch.empty(B, heads, max(budget, 0), dtype=_torch.int32, device=device)
        if n is None:
            n = _torch.empty(B, dtype=_torch.int64, device=device)
        w, size = _space(cache.ws_bytes, device, ws)
        status = lib().sp_cache_choose(cache.at, batch.at, weights.data_ptr(), 1 if shared else 0, budget, int(first), int(last),
                                       k.data_ptr(), k.stride(0), k.stride(1), n.data_ptr(), w.data_ptr(), size, handle)
        if status:
            _check(status)
        if check:
            _check(sp_workspace_status(w, handle))
        return k, n

    return _on(device, stream, call)


def cache_keep(cache, batch, kept, n_kept, *, drafted=False, to=None, weights=None, kv_len=None, ws=None, stream=None,
               check=False):
    """Keeps the listed tokens of each sequence, in order, and drops the others: kept int32 [B, most], or [B, H_kv, most] for a list
    a head, ascending, of which n_kept int64 [B] count (cache_choose's; select's positions of one prompt as [1, M]).  Returns
    the sequences' new lengths, int64 [B].  drafted=True: the lists count from the first new token, as tree_accept's, and the
    tokens before stay.  to int32 [B, width]: the kept tokens go to these pages, which are none of the listed tokens' own
    (default: to the front of their own, in place).  weights: the tokens' weights, moved along with them."""
    device, B = cache.device, batch.c.B
    if kept.dim() == 3:
        _check_ints(kept, "kept", (B, None, None), device)
        heads, most, seq, head = kept.shape[1], kept.shape[2], kept.stride(0), kept.stride(1)
    else:
        _check_ints(kept, "kept", (B, None), device)
        heads, most, seq, head = 1, kept.shape[1], kept.stride(0), 0
    _check_ints(n_kept, "n_kept", (B,), device, _torch.int64)
    if to is not None:
        _check_ints(to, "to", (B, None), device)
    if weights is not None:
        _check_weights(weights, cache)
    if kv_len is not None:
        _check_ints(kv_len, "kv_len", (B,), device, _torch.int64)
    _same_device(device, batch)

    def call(handle):
        n = kv_len
        if n is None:
            n = _torch.empty(B, dtype=_torch.int64, device=device)
        w, size = _space(cache.ws_bytes, device, ws)
        status = lib().sp_cache_keep(cache.at, batch.at, kept.data_ptr(), heads, seq, head, n_kept.data_ptr(), most,
                                     1 if drafted else 0, None if to is None else to.data_ptr(),
                                     0 if to is None else to.shape[1], 0 if to is None else _row_stride(to),
                                     None if weights is None else weights.data_ptr(), n.data_ptr(), w.data_ptr(), size, handle)
        if status:
            _check(status)
        if check:
            _check(sp_workspace_status(w, handle))
        return n

    return _on(device, stream, call)
