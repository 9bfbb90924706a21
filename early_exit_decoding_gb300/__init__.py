"""Python binding of libriver.so (River-LLM KV-shared exit river on GB300).

Argument marshalling only: every step of the decode/prefill path runs in the
library's CUDA kernels.  PyTorch supplies device memory (tensors) and
streams.  The binding fails loudly when libriver.so is missing: there is no
CPU fallback.

The ``rl_*`` functions mirror the C ABI in ``include/river.h`` one to one;
``Model``, ``KVCache`` and ``Policy`` are small conveniences on top of them.
"""
from __future__ import annotations

import ctypes
import operator
import os
import struct
from typing import Any, NamedTuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libriver.so")

RL_OK, RL_ERR_INVALID_ARG, RL_ERR_OOM, RL_ERR_CUDA, RL_ERR_CAPACITY, RL_ERR_STATE, \
    RL_ERR_DEVICE, RL_ERR_UNSUPPORTED = range(8)
RL_DEVERR_TOKEN, RL_DEVERR_CAPACITY, RL_DEVERR_SCHEDULE, RL_DEVERR_TIMEOUT = 1, 2, 4, 8
RL_EXIT_TAU, RL_EXIT_FORCED = 0, 1
RL_WQ, RL_WK, RL_WV, RL_WO, RL_WG, RL_WU, RL_WD = range(7)
LINEAR_NAMES = ("wq", "wk", "wv", "wo", "wg", "wu", "wd")

EXPORTS = (
    "rl_version", "rl_last_error", "rl_model_create", "rl_model_destroy",
    "rl_quantize_exit_layers", "rl_quantize_exit_layers_hqq", "rl_exit_layer_view", "rl_kv_cache_alloc", "rl_kv_cache_free",
    "rl_kv_view", "rl_kv_position", "rl_kv_set_position", "rl_kv_set_trace", "rl_prefill",
    "rl_decode_step", "rl_decode_step_host", "rl_sync", "rl_decode_kernel_count",
    "rl_kv_set_profiling", "rl_kv_profile", "rl_kv_timeline", "rl_lm_head_static", "rl_kv_set_decode_path",
    "rl_kv_decode_path", "rl_save_exit_layers", "rl_load_exit_layers", "rl_exit_kv_cosine",
    "rl_kv_set_wait_limit", "rl_debug_fail_allocations", "rl_debug_limit_waits", "rl_model_offload_backbone",
    "rl_model_memory", "rl_token_logprobs", "rl_window_attention", "rl_shared_prefix_workspace",
    "rl_shared_prefix_attention", "rl_kv_set_window", "rl_kv_share_prefix", "rl_prefill_score",
    "rl_packed_attention", "rl_kv4_append", "rl_kv4_read", "rl_kv4_attention_workspace", "rl_kv4_attention",
    "rl_sample",
)
RL_DT_F32, RL_DT_BF16, RL_DT_F16 = range(3)
RL_PATH_AUTO, RL_PATH_STEP, RL_PATH_FUSED, RL_PATH_GENERIC = range(4)
KERNEL_KINDS = ("embed", "qkv", "attention", "group_sums", "o_proj", "norm", "gate_up", "down",
                "layer_end", "lm_head", "argmax", "decode_step")


class rl_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_layers", "d_model", "n_q_heads", "n_kv_heads", "head_dim", "ffn_dim", "vocab",
        "group_size")] + [("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float)]


class rl_layer_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "wq", "wk", "wv", "wo", "wg", "wu", "wd", "g_attn", "g_ffn")]


class rl_weights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("lm_head", ctypes.c_void_p),
                ("g_final", ctypes.c_void_p), ("layers", ctypes.POINTER(rl_layer_weights))]


class rl_exit_policy(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("tau", ctypes.c_float),
                ("d_schedule", ctypes.c_void_p), ("schedule_len", ctypes.c_int32)]


class rl_attn_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "kv_dtype", "q_dtype", "batch", "q_len", "n_q_heads", "n_kv_heads", "head_dim",
        "kv_capacity")] + [("scale", ctypes.c_float)] + [(n, ctypes.c_int64 * 3) for n in (
            "q_stride", "out_stride", "k_stride", "v_stride")]


class rl_packed_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "dtype", "batch", "rows", "max_rows", "n_q_heads", "n_kv_heads", "head_dim")] + [
        ("scale", ctypes.c_float)] + [(n, ctypes.c_int64 * 2) for n in (
            "q_stride", "k_stride", "v_stride", "out_stride")]


class rl_kv4(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("page", ctypes.c_int32)] + [(n, ctypes.c_void_p) for n in (
        "k_codes", "k_scale", "v_codes", "v_scale")] + [
        ("code_stride", ctypes.c_int64 * 2), ("scale_stride", ctypes.c_int64 * 2), ("d_table", ctypes.c_void_p),
        ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int32)]


class rl_sampling(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_k", ctypes.c_int32), ("top_p", ctypes.c_float), ("min_p", ctypes.c_float)] + [
        (n, ctypes.c_void_p) for n in ("d_temperature", "d_top_k", "d_top_p", "d_min_p")]


class RiverError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"libriver status {status}: {msg}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built: run __graft_entry__.build() "
                          "(the CUDA library is required; there is no fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F, V = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, None
    PP = ctypes.POINTER(ctypes.c_void_p)
    PI = ctypes.POINTER(ctypes.c_int32)
    sig = {
        "rl_version": (ctypes.c_char_p, []),
        "rl_last_error": (ctypes.c_char_p, []),
        "rl_model_create": (I, [ctypes.POINTER(rl_config), ctypes.POINTER(rl_weights), P, PP]),
        "rl_model_destroy": (V, [P]),
        "rl_quantize_exit_layers": (I, [P, P]),
        "rl_quantize_exit_layers_hqq": (I, [P, I, ctypes.c_double, ctypes.c_double, ctypes.c_double, P]),
        "rl_exit_layer_view": (I, [P, I, I, PP, PP, PP, PI, PI]),
        "rl_kv_cache_alloc": (I, [P, I, I, PP]),
        "rl_kv_cache_free": (I, [P]),
        "rl_kv_view": (I, [P, I, PP, PP]),
        "rl_kv_position": (I, [P, PI, PI]),
        "rl_kv_set_position": (I, [P, I, I, P]),
        "rl_kv_set_trace": (I, [P, P]),
        "rl_prefill": (I, [P, P, P, I, I, ctypes.POINTER(rl_exit_policy), P, P, P, P, P]),
        "rl_decode_step": (I, [P, P, P, I, ctypes.POINTER(rl_exit_policy), P, P, P, P, P]),
        "rl_decode_step_host": (I, [P, P, P, I, ctypes.POINTER(rl_exit_policy), P, P, P, P, P]),
        "rl_sync": (I, [P, P, P]),
        "rl_decode_kernel_count": (I, [P, I]),
        "rl_kv_set_profiling": (I, [P, I]),
        "rl_kv_profile": (I, [P, P, I, PI, PI, PI, ctypes.POINTER(ctypes.c_float),
                              ctypes.POINTER(ctypes.c_double), PI]),
        "rl_kv_timeline": (I, [P, P, ctypes.c_int64, P, PI, PI, PI]),
        "rl_lm_head_static": (I, [P, P, I, P, P, P, P]),
        "rl_kv_set_decode_path": (I, [P, I]),
        "rl_kv_decode_path": (I, [P, I]),
        "rl_save_exit_layers": (I, [P, ctypes.c_char_p]),
        "rl_exit_kv_cosine": (I, [P, I, P, I, P, P]),
        "rl_kv_set_wait_limit": (I, [P, ctypes.c_int64]),
        "rl_model_offload_backbone": (I, [P, I, P]),
        "rl_model_memory": (I, [P, ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_uint64)]),
        "rl_debug_fail_allocations": (I, [ctypes.c_int64]),
        "rl_debug_limit_waits": (I, [ctypes.c_int64]),
        "rl_load_exit_layers": (I, [P, ctypes.c_char_p, P]),
        "rl_kv_set_window": (I, [P, I, I]),
        "rl_kv_share_prefix": (I, [P, I]),
        "rl_prefill_score": (I, [P, P, P, I, I, ctypes.POINTER(rl_exit_policy), P, P, P, P, P, P, I, P, P, P]),
        "rl_token_logprobs": (I, [P, I, I, I, ctypes.c_int64, P, I, I, P, P, P, P, P, P, P]),
        "rl_window_attention": (I, [ctypes.POINTER(rl_attn_desc), P, P, P, P, P, I, I, P, P, P, P]),
        "rl_shared_prefix_workspace": (I, [ctypes.POINTER(rl_attn_desc), I, ctypes.POINTER(ctypes.c_uint64)]),
        "rl_shared_prefix_attention": (I, [ctypes.POINTER(rl_attn_desc), P, P, P, I,
                                           ctypes.POINTER(ctypes.c_int64), P, P, P, P, P, P,
                                           ctypes.c_uint64, P, P]),
        "rl_packed_attention": (I, [ctypes.POINTER(rl_packed_desc), P, P, P, P, P, P, P, P]),
        "rl_kv4_append": (I, [ctypes.POINTER(rl_kv4), ctypes.POINTER(rl_packed_desc), P, P, P, P, P, P, I, P, P, P]),
        "rl_kv4_read": (I, [ctypes.POINTER(rl_kv4), ctypes.POINTER(rl_packed_desc), P, P, P, P, P, P]),
        "rl_kv4_attention_workspace": (I, [ctypes.POINTER(rl_packed_desc), ctypes.POINTER(ctypes.c_uint64)]),
        "rl_kv4_attention": (I, [ctypes.POINTER(rl_kv4), ctypes.POINTER(rl_packed_desc), P, P, P, P, P, P, ctypes.c_uint64, P, P]),
        "rl_sample": (I, [P, I, I, I, ctypes.c_int64, P, ctypes.POINTER(rl_sampling), P, P, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load()


def _check(status):
    if status != RL_OK:
        raise RiverError(status, _lib.rl_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# ----------------------------------------------------------------- C ABI, 1:1

def rl_version():
    return _lib.rl_version().decode()


def rl_last_error():
    return _lib.rl_last_error().decode()


def rl_model_create(cfg: rl_config, weights: rl_weights, stream=None):
    out = ctypes.c_void_p()
    _check(_lib.rl_model_create(ctypes.byref(cfg), ctypes.byref(weights), _stream(stream),
                                ctypes.byref(out)))
    return out


def rl_model_destroy(model):
    _lib.rl_model_destroy(model)


def rl_quantize_exit_layers(model, stream=None):
    _check(_lib.rl_quantize_exit_layers(model, _stream(stream)))


def rl_quantize_exit_layers_hqq(model, iters=20, lp_norm=0.7, beta=10.0, kappa=1.01, stream=None):
    _check(_lib.rl_quantize_exit_layers_hqq(model, int(iters), float(lp_norm), float(beta),
                                            float(kappa), _stream(stream)))


def rl_exit_kv_cosine(model, layer, d_h, B, d_cos, stream=None):
    _check(_lib.rl_exit_kv_cosine(model, int(layer), _ptr(d_h), int(B), _ptr(d_cos), _stream(stream)))


def rl_save_exit_layers(model, path):
    _check(_lib.rl_save_exit_layers(model, os.fsencode(path)))


def rl_load_exit_layers(model, path, stream=None):
    _check(_lib.rl_load_exit_layers(model, os.fsencode(path), _stream(stream)))


def rl_exit_layer_view(model, layer, which):
    q, s, z = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    n, k = ctypes.c_int32(), ctypes.c_int32()
    _check(_lib.rl_exit_layer_view(model, layer, which, ctypes.byref(q), ctypes.byref(s),
                                   ctypes.byref(z), ctypes.byref(n), ctypes.byref(k)))
    return q.value, s.value, z.value, n.value, k.value


def rl_kv_cache_alloc(model, max_batch, max_seq):
    out = ctypes.c_void_p()
    _check(_lib.rl_kv_cache_alloc(model, max_batch, max_seq, ctypes.byref(out)))
    return out


def rl_kv_cache_free(kv):
    _check(_lib.rl_kv_cache_free(kv))


def rl_kv_view(kv, layer):
    k, v = ctypes.c_void_p(), ctypes.c_void_p()
    _check(_lib.rl_kv_view(kv, layer, ctypes.byref(k), ctypes.byref(v)))
    return k.value, v.value


def rl_kv_position(kv):
    p, s = ctypes.c_int32(), ctypes.c_int32()
    _check(_lib.rl_kv_position(kv, ctypes.byref(p), ctypes.byref(s)))
    return p.value, s.value


def rl_kv_set_position(kv, pos, decode_step, stream=None):
    _check(_lib.rl_kv_set_position(kv, pos, decode_step, _stream(stream)))


def rl_kv_set_trace(kv, d_hidden):
    _check(_lib.rl_kv_set_trace(kv, _ptr(d_hidden)))


def rl_prefill(model, kv, d_tokens, B, T, policy, d_logits, d_next_token, d_exit_layer,
               d_min_cos, stream=None):
    _check(_lib.rl_prefill(model, kv, _ptr(d_tokens), B, T, ctypes.byref(policy), _ptr(d_logits),
                           _ptr(d_next_token), _ptr(d_exit_layer), _ptr(d_min_cos),
                           _stream(stream)))


def rl_decode_step(model, kv, d_tokens, B, policy, d_logits, d_next_token, d_exit_layer,
                   d_min_cos, stream=None):
    _check(_lib.rl_decode_step(model, kv, _ptr(d_tokens), B, ctypes.byref(policy),
                               _ptr(d_logits), _ptr(d_next_token), _ptr(d_exit_layer),
                               _ptr(d_min_cos), _stream(stream)))


def rl_decode_step_host(model, kv, h_tokens, B, policy, h_logits, h_next_token, h_exit_layer,
                        h_min_cos, stream=None):
    _check(_lib.rl_decode_step_host(model, kv, _ptr(h_tokens), B, ctypes.byref(policy),
                                    _ptr(h_logits), _ptr(h_next_token), _ptr(h_exit_layer),
                                    _ptr(h_min_cos), _stream(stream)))


def rl_sync(model, kv, stream=None):
    _check(_lib.rl_sync(model, kv, _stream(stream)))


def rl_decode_kernel_count(model, B):
    return int(_lib.rl_decode_kernel_count(model, B))


def rl_lm_head_static(model, d_h, B, d_logits, d_next_token=None, d_err=None, stream=None):
    """Final RMSNorm + LM head + greedy argmax of ``d_h [B][d]`` using only the
    library's static scratch (allocates nothing)."""
    _check(_lib.rl_lm_head_static(model, _ptr(d_h), B, _ptr(d_logits), _ptr(d_next_token),
                                  _ptr(d_err), _stream(stream)))


def rl_model_offload_backbone(model, first_layer, stream=None):
    _check(_lib.rl_model_offload_backbone(model, int(first_layer), _stream(stream)))


def rl_model_memory(model):
    """(device bytes, pinned host bytes) the model holds."""
    d, h = ctypes.c_uint64(), ctypes.c_uint64()
    _check(_lib.rl_model_memory(model, ctypes.byref(d), ctypes.byref(h)))
    return d.value, h.value


def rl_kv_set_wait_limit(kv, polls):
    """Test hook: grid-barrier / first GEMM-epilogue waits give up after
    ``polls`` polls (0 = the kernels' own limits)."""
    _check(_lib.rl_kv_set_wait_limit(kv, int(polls)))


def rl_debug_fail_allocations(after):
    """Test hook: the next ``after`` library allocations succeed, later ones
    fail (RL_ERR_OOM); negative switches it off."""
    _check(_lib.rl_debug_fail_allocations(int(after)))


def rl_debug_limit_waits(polls):
    """The many-row attention kernel's waits give up after ``polls`` polls; negative switches it off."""
    _check(_lib.rl_debug_limit_waits(int(polls)))


_INT32_MAX = 2**31 - 1


def _int32_of(n):
    """n for a C int32 that a larger one may stand for (ctypes keeps the low 32
    bits): what is beyond becomes the largest, what is negative -1."""
    return max(-1, min(n, _INT32_MAX))


def rl_kv_set_window(kv, window, sinks=0):
    _check(_lib.rl_kv_set_window(kv, _int32_of(int(window)), _int32_of(int(sinks))))


def rl_kv_share_prefix(kv, n):
    _check(_lib.rl_kv_share_prefix(kv, _int32_of(int(n))))


def rl_prefill_score(model, kv, d_tokens, B, T, policy, d_logits, d_next_token, d_exit_layer, d_min_cos,
                     d_logprob, d_entropy=None, top_k=0, d_top_ids=None, d_top_logprobs=None, stream=None):
    _check(_lib.rl_prefill_score(model, kv, _ptr(d_tokens), B, T, ctypes.byref(policy), _ptr(d_logits),
                                 _ptr(d_next_token), _ptr(d_exit_layer), _ptr(d_min_cos), _ptr(d_logprob),
                                 _ptr(d_entropy), top_k, _ptr(d_top_ids), _ptr(d_top_logprobs), _stream(stream)))


def rl_kv_set_decode_path(kv, path):
    _check(_lib.rl_kv_set_decode_path(kv, int(path)))


def rl_kv_decode_path(kv, B):
    return int(_lib.rl_kv_decode_path(kv, B))


def rl_kv_set_profiling(kv, enable):
    """0 off; 1 (or True) event records and the per-phase timeline; 2 also the
    per-CTA timeline of the step kernel (rl_kv_timeline)."""
    _check(_lib.rl_kv_set_profiling(kv, int(enable)))


def rl_kv_timeline(kv, stream=None):
    """Per-CTA timeline of the last profiled step: numpy uint64 array
    [phase][CTA][stamp] of globaltimer nanoseconds (0 = no such event)."""
    import numpy as np
    n_ph, n_cta, n_st = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    cap = 1 << 22
    buf = np.zeros(cap, dtype=np.uint64)
    _check(_lib.rl_kv_timeline(kv, _stream(stream), cap, buf.ctypes.data_as(ctypes.c_void_p),
                               ctypes.byref(n_ph), ctypes.byref(n_cta), ctypes.byref(n_st)))
    return buf[: n_ph.value * n_cta.value * n_st.value].reshape(n_ph.value, n_cta.value, n_st.value)


def rl_kv_profile(kv, stream=None, cap=1024):
    """List of (kind name, layer, path, ms, algorithmic bytes) of the last
    profiled decode step."""
    k = (ctypes.c_int32 * cap)()
    ly = (ctypes.c_int32 * cap)()
    pa = (ctypes.c_int32 * cap)()
    ms = (ctypes.c_float * cap)()
    by = (ctypes.c_double * cap)()
    n = ctypes.c_int32()
    _check(_lib.rl_kv_profile(kv, _stream(stream), cap, k, ly, pa, ms, by, ctypes.byref(n)))
    return [(KERNEL_KINDS[k[i]], ly[i], pa[i], ms[i], by[i]) for i in range(n.value)]


def rl_token_logprobs(d_logits, dtype, rows, vocab, row_stride, d_tokens, n_tok, top_k, d_lse,
                      d_entropy, d_logprob, d_top_ids, d_top_logprobs, d_err=None, stream=None):
    _check(_lib.rl_token_logprobs(_ptr(d_logits), dtype, rows, vocab, row_stride, _ptr(d_tokens), n_tok,
                                  top_k, _ptr(d_lse), _ptr(d_entropy), _ptr(d_logprob), _ptr(d_top_ids),
                                  _ptr(d_top_logprobs), _ptr(d_err), _stream(stream)))


def rl_window_attention(desc, d_q, d_k, d_v, d_kv_len, d_q_len, window, sinks, d_out, d_lse,
                        d_err=None, stream=None):
    _check(_lib.rl_window_attention(ctypes.byref(desc), _ptr(d_q), _ptr(d_k), _ptr(d_v), _ptr(d_kv_len),
                                    _ptr(d_q_len), _int32_of(window), _int32_of(sinks), _ptr(d_out), _ptr(d_lse), _ptr(d_err),
                                    _stream(stream)))


def rl_shared_prefix_workspace(desc, prefix_len):
    """Workspace bytes of rl_shared_prefix_attention."""
    n = ctypes.c_uint64()
    _check(_lib.rl_shared_prefix_workspace(ctypes.byref(desc), prefix_len, ctypes.byref(n)))
    return n.value


def rl_shared_prefix_attention(desc, d_q, d_k_prefix, d_v_prefix, prefix_len, prefix_stride, d_k, d_v,
                               d_kv_len, d_out, d_lse, d_ws, ws_bytes, d_err=None, stream=None):
    st = (ctypes.c_int64 * 4)(*prefix_stride)
    _check(_lib.rl_shared_prefix_attention(ctypes.byref(desc), _ptr(d_q), _ptr(d_k_prefix),
                                           _ptr(d_v_prefix), prefix_len, st, _ptr(d_k), _ptr(d_v),
                                           _ptr(d_kv_len), _ptr(d_out), _ptr(d_lse), _ptr(d_ws), ws_bytes,
                                           _ptr(d_err), _stream(stream)))


def rl_packed_attention(desc, d_q, d_k, d_v, d_start, d_out, d_lse, d_err=None, stream=None):
    _check(_lib.rl_packed_attention(ctypes.byref(desc), _ptr(d_q), _ptr(d_k), _ptr(d_v), _ptr(d_start), _ptr(d_out),
                                    _ptr(d_lse), _ptr(d_err), _stream(stream)))


def rl_kv4_append(cache, desc, d_start, d_kv_len, d_q, d_k, d_v, d_rope, rope_len, d_out, d_err=None, stream=None):
    _check(_lib.rl_kv4_append(ctypes.byref(cache), ctypes.byref(desc), _ptr(d_start), _ptr(d_kv_len), _ptr(d_q), _ptr(d_k),
                              _ptr(d_v), _ptr(d_rope), _int32_of(rope_len), _ptr(d_out), _ptr(d_err), _stream(stream)))


def rl_kv4_read(cache, desc, d_start, d_kv_len, d_k, d_v, d_err=None, stream=None):
    _check(_lib.rl_kv4_read(ctypes.byref(cache), ctypes.byref(desc), _ptr(d_start), _ptr(d_kv_len), _ptr(d_k), _ptr(d_v),
                            _ptr(d_err), _stream(stream)))


def rl_kv4_attention_workspace(desc):
    """Workspace bytes of rl_kv4_attention."""
    n = ctypes.c_uint64()
    _check(_lib.rl_kv4_attention_workspace(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def rl_kv4_attention(cache, desc, d_start, d_kv_len, d_q, d_out, d_lse, d_ws, ws_bytes, d_err=None, stream=None):
    _check(_lib.rl_kv4_attention(ctypes.byref(cache), ctypes.byref(desc), _ptr(d_start), _ptr(d_kv_len), _ptr(d_q),
                                 _ptr(d_out), _ptr(d_lse), _ptr(d_ws), ws_bytes, _ptr(d_err), _stream(stream)))


def rl_sample(d_logits, dtype, rows, vocab, row_stride, d_u, settings, d_token, d_logprob, stream=None):
    _check(_lib.rl_sample(_ptr(d_logits), dtype, rows, vocab, row_stride, _ptr(d_u), ctypes.byref(settings), _ptr(d_token),
                          _ptr(d_logprob), _stream(stream)))


# --------------------------------------------------------------- conveniences

class _DevArray:
    """Wraps a library-owned device buffer for torch.as_tensor (no copy)."""

    def __init__(self, ptr, shape, typestr):
        self.__cuda_array_interface__ = {
            "shape": tuple(shape), "typestr": typestr, "data": (ptr, False), "version": 3,
            "strides": None,
        }


class Policy:
    """Exit policy: ``Policy.tau(t)`` or ``Policy.forced(schedule_tensor)``
    (device int32, decode step i uses schedule[i % len], prefill schedule[0])."""

    def __init__(self, mode, tau=1.01, schedule=None):
        self.mode, self.tau, self.schedule = mode, float(tau), schedule

    @staticmethod
    def tau_(t):
        return Policy(RL_EXIT_TAU, t)

    @staticmethod
    def forced(schedule):
        return Policy(RL_EXIT_FORCED, 0.0, schedule)

    def c(self):
        s = self.schedule
        return rl_exit_policy(self.mode, self.tau, None if s is None else s.data_ptr(),
                              0 if s is None else int(s.numel()))


class Model:
    """A model on the current CUDA device built from a weight dict
    (``embed, lm_head, g_final, layers[{wq..wd, g_attn, g_ffn}]``, bf16 CUDA
    tensors, linear weights row-major [out][in])."""

    def __init__(self, shape, weights, stream=None):
        import torch
        self.shape = shape
        cfg = rl_config(shape.n_layers, shape.d_model, shape.n_q_heads, shape.n_kv_heads,
                        shape.head_dim, shape.ffn_dim, shape.vocab, shape.group_size,
                        shape.rms_eps, shape.rope_theta)
        layers = (rl_layer_weights * shape.n_layers)()
        keep = []
        for i, lw in enumerate(weights["layers"]):
            vals = []
            for n in ("wq", "wk", "wv", "wo", "wg", "wu", "wd", "g_attn", "g_ffn"):
                t = lw[n]
                assert t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous(), n
                keep.append(t)
                vals.append(t.data_ptr())
            layers[i] = rl_layer_weights(*vals)
        for n in ("embed", "lm_head", "g_final"):
            t = weights[n]
            assert t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous(), n
        w = rl_weights(weights["embed"].data_ptr(), weights["lm_head"].data_ptr(),
                       weights["g_final"].data_ptr(), layers)
        self.handle = rl_model_create(cfg, w, stream)

    def close(self):
        if getattr(self, "handle", None):
            rl_model_destroy(self.handle)
            self.handle = None

    __del__ = close

    def quantize_exit_layers(self, stream=None, method="rtn", **hqq):
        """Build the exit river: min-max rounding (``method="rtn"``) or with
        HQQ's zero-point refinement (``method="hqq"``; keyword settings
        iters, lp_norm, beta, kappa)."""
        if method == "hqq":
            rl_quantize_exit_layers_hqq(self.handle, stream=stream, **hqq)
        elif method == "rtn":
            rl_quantize_exit_layers(self.handle, stream)
        else:
            raise ValueError(f"unknown quantizer {method!r}")

    def save_exit_layers(self, path):
        """Write the exit river (published packing) to ``path``."""
        rl_save_exit_layers(self.handle, path)

    def load_exit_layers(self, path, stream=None):
        """Build the exit river from a file written by save_exit_layers."""
        rl_load_exit_layers(self.handle, path, stream)

    def offload_backbone(self, first_layer, stream=None):
        """Backbone weights of layers first_layer.. (0-based) to pinned host memory."""
        rl_model_offload_backbone(self.handle, first_layer, stream)

    def memory(self):
        """(device bytes, pinned host bytes) the model holds."""
        return rl_model_memory(self.handle)

    def exit_kv_cosine(self, layer, h, stream=None):
        """Cosine between the exit layer's and the backbone layer's K and V of
        residual rows ``h [B][d]`` (fp32 CUDA) entering ``layer`` (0-based):
        a tensor [B][2][n_kv_heads] (K, then V)."""
        import torch
        B = h.shape[0]
        out = torch.empty((B, 2, self.shape.n_kv_heads), dtype=torch.float32, device="cuda")
        rl_exit_kv_cosine(self.handle, layer, h.contiguous(), B, out, stream)
        return out

    def exit_layer_view(self, layer, which):
        """(qweight int32 [N][K/8], scales fp16 [N][G], zeros fp16 [N][G]) torch views."""
        import torch
        q, s, z, n, k = rl_exit_layer_view(self.handle, layer, which)
        g = (k + 127) // 128
        qt = torch.as_tensor(_DevArray(q, (n, k // 8), "<i4"), device="cuda")
        st = torch.as_tensor(_DevArray(s, (n, g), "<f2"), device="cuda")
        zt = torch.as_tensor(_DevArray(z, (n, g), "<f2"), device="cuda")
        return qt, st, zt

    def kv_cache_alloc(self, max_batch, max_seq):
        return KVCache(self, max_batch, max_seq)

    def kernel_count(self, B):
        return rl_decode_kernel_count(self.handle, B)


class KVCache:
    def __init__(self, model: Model, max_batch, max_seq):
        self.model = model
        self.max_batch, self.max_seq = max_batch, max_seq
        self.handle = rl_kv_cache_alloc(model.handle, max_batch, max_seq)
        self._trace = None

    def close(self):
        if getattr(self, "handle", None):
            rl_kv_cache_free(self.handle)
            self.handle = None

    __del__ = close

    def view(self, layer):
        """(K, V) torch views, bf16 [max_batch][Hkv][max_seq][hd]."""
        import torch
        S = self.model.shape
        k, v = rl_kv_view(self.handle, layer)
        shp = (self.max_batch, S.n_kv_heads, self.max_seq, S.head_dim)
        kt = torch.as_tensor(_DevArray(k, shp, "<i2"), device="cuda").view(torch.bfloat16)
        vt = torch.as_tensor(_DevArray(v, shp, "<i2"), device="cuda").view(torch.bfloat16)
        return kt, vt

    def position(self):
        return rl_kv_position(self.handle)

    def set_position(self, pos, decode_step=0, stream=None):
        rl_kv_set_position(self.handle, pos, decode_step, stream)

    def set_trace(self, t):
        self._trace = t
        rl_kv_set_trace(self.handle, t)

    def set_window(self, window, sinks=0):
        """Sliding-window attention with ``sinks`` first tokens that stay
        visible, from the next call on (0: off)."""
        rl_kv_set_window(self.handle, window, sinks)

    def share_prefix(self, n=None):
        """The first ``n`` positions of sequence 0 (None: all so far) serve
        every sequence of the later decode steps (0: off)."""
        rl_kv_share_prefix(self.handle, self.position()[0] if n is None else n)

    def set_decode_path(self, path):
        rl_kv_set_decode_path(self.handle, path)

    def decode_path(self, B):
        return rl_kv_decode_path(self.handle, B)

    def sync(self, stream=None):
        rl_sync(self.model.handle, self.handle, stream)


def _new(shape, dtype, device, stream):
    """A tensor taken on the stream that writes it (None: the current one):
    memory of another stream may still be in use there."""
    torch = _torch()
    if not isinstance(stream, torch.cuda.Stream):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _outputs(model, B, out, stream):
    torch = _torch()
    S = model.shape
    o = dict(out) if out else {}
    for key, shape, dtype in (("logits", (B, S.vocab), torch.float32), ("next_token", (B,), torch.int32),
                              ("exit_layer", (1,), torch.int32), ("min_cos", (S.n_layers,), torch.float32)):
        if key not in o:
            o[key] = _new(shape, dtype, "cuda", stream)
    return o


def prefill(model: Model, kv: KVCache, tokens, policy: Policy, out=None, stream=None):
    """tokens: CUDA int32 [B][T].  Returns a dict of output tensors."""
    B, T = tokens.shape
    o = _outputs(model, B, out, stream)
    rl_prefill(model.handle, kv.handle, tokens, B, T, policy.c(), o["logits"], o["next_token"],
               o["exit_layer"], o["min_cos"], stream)
    return o


def prefill_score(model: Model, kv: KVCache, tokens, policy: Policy, top_k=0, out=None, stream=None):
    """prefill that also scores the prompt: ``logprob [B][T]`` (of token t after
    the tokens before it, 0 for the first), ``entropy [B][T]`` and, for
    ``top_k`` > 0, ``top_ids`` and ``top_logprobs`` [B][T][top_k] of every
    position.  ``tokens``: CUDA int32 [B][T], contiguous; buffers present in
    ``out`` are used.  See rl_prefill_score."""
    torch = _torch()
    name = "prefill_score"
    if tokens.dim() != 2:
        _refuse(f"{name}: tokens must be [B][T]")
    B, T = tokens.shape
    _int32(name, "tokens", tokens, (B, T))
    _operands(name, (tokens,))
    S, f32, i32 = model.shape, torch.float32, torch.int32
    if not 0 <= top_k <= min(32, S.vocab):
        _refuse(f"{name}: top_k {top_k} outside [0, {min(32, S.vocab)}]")
    o = dict(out) if out else {}
    for n, shape, dt in (("logits", (B, S.vocab), f32), ("next_token", (B,), i32), ("exit_layer", (1,), i32),
                         ("min_cos", (S.n_layers,), f32), ("logprob", (B, T), f32), ("entropy", (B, T), f32)) + (
            (("top_ids", (B, T, top_k), i32), ("top_logprobs", (B, T, top_k), f32)) if top_k else ()):
        _buffer(o, n, shape, tokens, dt, stream, name)
    rl_prefill_score(model.handle, kv.handle, tokens, B, T, policy.c(), o["logits"], o["next_token"],
                     o["exit_layer"], o["min_cos"], o["logprob"], o["entropy"], top_k, o.get("top_ids"),
                     o.get("top_logprobs"), stream)
    return o


def decode_step(model: Model, kv: KVCache, tokens, policy: Policy, out=None, stream=None):
    """tokens: CUDA int32 [B].  Returns a dict of output tensors."""
    B = tokens.shape[0]
    o = _outputs(model, B, out, stream)
    rl_decode_step(model.handle, kv.handle, tokens, B, policy.c(), o["logits"], o["next_token"],
                   o["exit_layer"], o["min_cos"], stream)
    return o


_TORCH = []


def _torch():
    """The module (imported with the first use; the statement in every call cost
    the smallest calls 2 to 5 %)."""
    if not _TORCH:
        import torch
        _TORCH.append(torch)
    return _TORCH[0]


def _refuse(msg, status=RL_ERR_INVALID_ARG):
    raise RiverError(status, msg)


def _dtype_code(dtype):
    """RL_DT_* of a torch dtype; None for any other."""
    if not _DTYPES:
        torch = _torch()
        _DTYPES.update({torch.float32: RL_DT_F32, torch.bfloat16: RL_DT_BF16, torch.float16: RL_DT_F16})
    return _DTYPES.get(dtype)


_DTYPES = {}


def _operands(name, tensors):
    """The one CUDA device (index) of the tensors (None: absent), none of which
    may need a gradient or carry a tangent (the operators have no derivatives)."""
    torch = _torch()
    dev = tensors[0].get_device()
    grad, dual = torch.is_grad_enabled(), torch.autograd.forward_ad._current_level >= 0
    for t in tensors:
        if t is not None:
            if grad and t.requires_grad:
                _refuse(f"{name}: an operand requires a gradient; the operator has no backward pass", RL_ERR_UNSUPPORTED)
            if dual and torch.autograd.forward_ad.unpack_dual(t).tangent is not None:
                _refuse(f"{name}: an operand carries a tangent; the operator has no forward-mode derivative", RL_ERR_UNSUPPORTED)
            if t.get_device() != dev or dev < 0:
                _refuse(f"{name}: every operand must be on one CUDA device (found {t.device})")
    return dev


def _buffer(o, key, shape, like, dtype, stream, name):
    """``o[key]``, checked against (shape, dtype), or a new tensor put there
    (taken on the stream that writes it)."""
    t = o.get(key)
    if t is None:
        t = o[key] = _new(shape, dtype, like.device, stream)
    elif t.shape != shape or t.dtype != dtype or t.get_device() != like.get_device() or \
            (key != "out" and not t.is_contiguous()):
        _refuse(f"{name}: out[{key!r}] must be {dtype} {tuple(shape)} on {like.device}"
                + ("" if key == "out" else ", contiguous"))
    elif t.requires_grad and _torch().is_grad_enabled():
        _refuse(f"{name}: out[{key!r}] requires a gradient; the operator has no backward pass", RL_ERR_UNSUPPORTED)
    return t


def _run(dev, stream, fn, *args):
    """The library call ``fn(*args, stream)`` with device ``dev`` current;
    ``stream`` None: that device's current stream."""
    torch = _torch()
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _run(dev, stream, fn, *args)
    # (the raw handle: making a Stream object costs as much as a small launch)
    status = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if status != RL_OK:
        _check(status)


def _int32(name, key, t, shape):
    torch = _torch()
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        _refuse(f"{name}: {key} must be contiguous int32 {shape}")


def _whole(name, key, x):
    """x as an int; refused where it is none (a fraction is not cut off)."""
    try:
        n = int(x)
        if n == x:
            return n
    except (TypeError, ValueError, OverflowError):
        pass
    _refuse(f"{name}: {key} must be a whole number (found {x!r})")


def _addr(t):
    return None if t is None else t.data_ptr()


def token_logprobs(logits, tokens=None, top_k=0, out=None, err=None, stream=None):
    """Log-probabilities of given tokens, entropy and top alternatives of
    ``logits [R][V]`` (fp32, bf16 or fp16 CUDA, rows any stride apart).
    ``tokens``: int32 [R] or [R][n].  Returns a dict: ``lse`` and ``entropy``
    [R], ``logprob`` (tokens' shape), ``top_ids`` int32 and ``top_logprobs``
    [R][top_k]; buffers present in ``out`` are used.  ``err``: int32 [1] that
    collects RL_DEVERR_* bits.  See rl_token_logprobs."""
    torch = _torch()
    name = "token_logprobs"
    dt = _dtype_code(logits.dtype)
    if logits.dim() != 2 or dt is None or logits.numel() == 0 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        _refuse(f"{name}: logits must be fp32, bf16 or fp16 [R][V] with contiguous rows")
    R, V = logits.shape
    if R > _INT32_MAX or V > _INT32_MAX:
        _refuse(f"{name}: rows and vocabulary must be below 2^31", RL_ERR_UNSUPPORTED)
    dev = _operands(name, (logits, tokens, err))
    if not 0 <= top_k <= min(32, V):
        _refuse(f"{name}: top_k {top_k} outside [0, {min(32, V)}]")
    n = 0
    if tokens is not None:
        n = 1 if tokens.dim() == 1 else tokens.shape[-1]
        _int32(name, "tokens", tokens, (R,) if tokens.dim() == 1 else (R, n))
    if err is not None:
        _int32(name, "err", err, (1,))
    o = dict(out) if out else {}
    f32 = torch.float32
    lse = _buffer(o, "lse", (R,), logits, f32, stream, name).data_ptr()
    ent = _buffer(o, "entropy", (R,), logits, f32, stream, name).data_ptr()
    lp = ids = tlp = None
    if n:
        lp = _buffer(o, "logprob", tokens.shape, logits, f32, stream, name).data_ptr()
    if top_k:
        ids = _buffer(o, "top_ids", (R, top_k), logits, torch.int32, stream, name).data_ptr()
        tlp = _buffer(o, "top_logprobs", (R, top_k), logits, f32, stream, name).data_ptr()
    _run(dev, stream, _lib.rl_token_logprobs, logits.data_ptr(), dt, R, V, logits.stride(0) if R > 1 else V,
         tokens.data_ptr() if n else None, n, top_k, lse, ent, lp, ids, tlp, _addr(err))
    return o


def _strides(d, t):
    """Strides of the outer axes into the descriptor's field (of three: the
    middle one stays 0); an axis of one entry has no stride that matters."""
    s, n = t.stride(), t.shape
    d[0] = s[0] if n[0] > 1 else 0
    if len(n) == 4:
        d[1] = s[1] if n[1] > 1 else 0
    d[2] = s[-2] if n[-2] > 1 else 0


_PLANS = {}


_SHAPE_DTYPE = operator.attrgetter("shape", "dtype")


def _plan(name, scale, tensors, make):
    """What ``make()`` derives from the tensors' shapes, strides and types alone
    (their checks, the descriptor, a workspace's size), kept for calls of the
    same layout."""
    key = (name, scale, *map(_SHAPE_DTYPE, tensors), *map(_torch().Tensor.stride, tensors))
    p = _PLANS.get(key)
    if p is None:
        p = make()
        if len(_PLANS) >= 256:
            _PLANS.clear()
        _PLANS[key] = p
    return p


def _attn_desc(name, q, k, v, out, scale):
    """rl_attn_desc of q, out [B][T][Hq][hd] ([B][Hq][hd]: T is 1) and k, v
    [B][Hkv][S][hd]."""
    for t in (q, k, v, out):
        if t.dim() != (4 if t is k or t is v else q.dim()) or t.numel() == 0 or t.stride(-1) != 1:
            _refuse(f"{name}: q, k, v and out must have their axes, none empty, with a contiguous last one")
    B, Hq, hd = q.shape[0], q.shape[-2], q.shape[-1]
    T = q.shape[1] if q.dim() == 4 else 1
    _, Hkv, S, _ = k.shape
    if max(*q.shape, *k.shape) > _INT32_MAX:
        _refuse(f"{name}: sizes must be below 2^31", RL_ERR_UNSUPPORTED)
    qc, kc = _dtype_code(q.dtype), _dtype_code(k.dtype)
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != hd or v.dtype != k.dtype or out.dtype != k.dtype or \
            qc is None or kc is None:
        _refuse(f"{name}: q {tuple(q.shape)} {q.dtype}, k {tuple(k.shape)} {k.dtype}, v {tuple(v.shape)} {v.dtype} do not fit")
    if scale is not None and not scale > 0.0:
        _refuse(f"{name}: scale must be above 0")
    d = rl_attn_desc(kc, qc, B, T, Hq, Hkv, hd, S, 0.0 if scale is None else scale)
    if scale is not None and d.scale == 0.0:  # (which would stand for the default)
        _refuse(f"{name}: scale {scale} is 0 in fp32")
    _strides(d.q_stride, q)
    _strides(d.out_stride, out)
    _strides(d.k_stride, k)
    _strides(d.v_stride, v)
    return d


def window_attention(q, k, v, kv_len, window, sinks=0, q_len=None, scale=None, out=None, err=None, stream=None):
    """Causal attention over the last ``window`` keys and the first ``sinks``.
    ``q [B][T][Hq][hd]`` (k's type, or fp32), ``k``, ``v`` [B][Hkv][S][hd] bf16
    or fp16 (KVCache.view's layout), ``kv_len`` int32 [B], ``q_len`` int32 [B]
    or None (T each): the queries are the last q_len of a sequence's kv_len
    rows.  Returns a dict: ``out`` (q's shape, k's type) and ``lse`` fp32
    [B][T][Hq]; buffers present in ``out`` are used, their rows t >= q_len[b]
    left as they were.  See rl_window_attention."""
    torch = _torch()
    name = "window_attention"
    dev = _operands(name, (q, k, v, kv_len, q_len, err))
    if q.dim() != 4:
        _refuse(f"{name}: q must be [B][T][Hq][hd]")
    o = dict(out) if out else {}
    res = _buffer(o, "out", q.shape, q, k.dtype, stream, name)
    # (a new result's layout follows q's shape)
    d = _plan(name, scale, (q, k, v, res) if out else (q, k, v), lambda: _attn_desc(name, q, k, v, res, scale))
    B, T, Hq, _ = q.shape
    lse = _buffer(o, "lse", (B, T, Hq), q, torch.float32, stream, name)
    _int32(name, "kv_len", kv_len, (B,))
    if q_len is not None:
        _int32(name, "q_len", q_len, (B,))
    if err is not None:
        _int32(name, "err", err, (1,))
    _run(dev, stream, _lib.rl_window_attention, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), kv_len.data_ptr(),
         _addr(q_len), _int32_of(window), _int32_of(sinks), res.data_ptr(), lse.data_ptr(), _addr(err))
    return o


def shared_prefix_attention(q, k_prefix, v_prefix, k, v, kv_len, scale=None, out=None, workspace=None, err=None,
                            stream=None):
    """One decode step's attention of a batch behind one shared prefix.
    ``q [B][Hq][hd]``, ``k_prefix``, ``v_prefix`` [Hkv][P][hd], the sequences'
    own ``k``, ``v`` [B][Hkv][S][hd] with ``kv_len`` int32 [B] rows in use.
    Returns a dict: ``out`` [B][Hq][hd] (k's type), ``lse`` fp32 [B][Hq];
    buffers present in ``out`` are used.  ``workspace``: a uint8 tensor of
    rl_shared_prefix_workspace bytes; None takes one from PyTorch's allocator
    for this call.  See rl_shared_prefix_attention."""
    torch = _torch()
    name = "shared_prefix_attention"
    dev = _operands(name, (q, k_prefix, v_prefix, k, v, kv_len, workspace, err))
    if q.dim() != 3:
        _refuse(f"{name}: q must be [B][Hq][hd]")
    o = dict(out) if out else {}
    res = _buffer(o, "out", q.shape, q, k.dtype, stream, name)

    def make():
        d = _attn_desc(name, q, k, v, res, scale)
        if k_prefix.dim() != 3 or k_prefix.shape != v_prefix.shape or k_prefix.dtype != k.dtype or \
                v_prefix.dtype != k.dtype or k_prefix.shape[0] != d.n_kv_heads or k_prefix.shape[2] != d.head_dim or \
                k_prefix.stride(2) != 1 or v_prefix.stride(2) != 1:
            _refuse(f"{name}: k_prefix and v_prefix must be {k.dtype} [{d.n_kv_heads}][P][{d.head_dim}] with a contiguous last axis")
        if k_prefix.shape[1] > _INT32_MAX:
            _refuse(f"{name}: sizes must be below 2^31", RL_ERR_UNSUPPORTED)
        ps = (ctypes.c_int64 * 4)(*(t.stride(i) if t.shape[i] > 1 else 0 for t in (k_prefix, v_prefix) for i in (0, 1)))
        return d, ps, rl_shared_prefix_workspace(d, k_prefix.shape[1])

    d, ps, need = _plan(name, scale, (q, k, v, k_prefix, v_prefix, res) if out else (q, k, v, k_prefix, v_prefix), make)
    B, Hq, _ = q.shape
    lse = _buffer(o, "lse", (B, Hq), q, torch.float32, stream, name)
    _int32(name, "kv_len", kv_len, (B,))
    if err is not None:
        _int32(name, "err", err, (1,))
    if workspace is None:
        workspace = _buffer({}, "workspace", (need,), q, torch.uint8, stream, name)
    elif not workspace.is_contiguous():
        _refuse(f"{name}: workspace must be contiguous")
    _run(dev, stream, _lib.rl_shared_prefix_attention, d, q.data_ptr(), k_prefix.data_ptr(), v_prefix.data_ptr(),
         k_prefix.shape[1], ps, k.data_ptr(), v.data_ptr(), kv_len.data_ptr(), res.data_ptr(), lse.data_ptr(),
         workspace.data_ptr(), workspace.numel() * workspace.element_size(), _addr(err))
    return o


class KV4Cache(NamedTuple):
    """A paged cache held in 4 bits: ``k_codes``, ``v_codes`` uint8
    [pages][Hkv][page][hd / 2], ``k_scale``, ``v_scale`` bf16 or fp16
    [pages][Hkv][page][2] (step, minimum); views of a larger pool may have any
    page stride.  The kv4 functions also take such four tensors in a plain
    tuple.  See rl_kv4."""
    k_codes: Any
    k_scale: Any
    v_codes: Any
    v_scale: Any

    @staticmethod
    def alloc(n_pages, n_kv_heads, head_dim, page=64, dtype=None, device="cuda"):
        """A cache of zeros (dtype None: bf16)."""
        torch = _torch()
        codes, scale = (n_pages, n_kv_heads, page, head_dim // 2), (n_pages, n_kv_heads, page, 2)
        return KV4Cache(*(torch.zeros(s, dtype=t, device=device) for _ in "kv"
                          for s, t in ((codes, torch.uint8), (scale, dtype or torch.bfloat16))))


def rope_table(n, head_dim, theta, device="cuda"):
    """(cos, sin) of positions 0 .. n - 1 for kv4_append: fp32 [n][head_dim / 2][2],
    frequencies theta^(-2 i / head_dim) and angles in 64 bits."""
    torch = _torch()
    f = float(theta) ** (-2.0 * torch.arange(head_dim // 2, dtype=torch.float64, device=device) / head_dim)
    a = torch.arange(n, dtype=torch.float64, device=device)[:, None] * f
    return torch.stack([a.cos(), a.sin()], dim=-1).float()


def _packed_desc(name, dtype, heads, batch, rows, max_rows, scale, **tensors):
    """rl_packed_desc of packed tensors [rows][heads][hd] by their names (q, k, v, out; None: absent)."""
    d = rl_packed_desc()
    n_q, n_kv, hd = heads
    code = _dtype_code(dtype)
    if code is None:
        _refuse(f"{name}: bf16 or fp16 operands are needed (found {dtype})")
    if max(batch, rows, n_q, n_kv, hd) > _INT32_MAX:
        _refuse(f"{name}: sizes must be below 2^31", RL_ERR_UNSUPPORTED)
    if scale is not None and not scale > 0.0:
        _refuse(f"{name}: scale must be above 0")
    d.dtype, d.batch, d.rows, d.max_rows, d.n_q_heads, d.n_kv_heads, d.head_dim = code, batch, rows, _int32_of(_whole(name, "max_rows", max_rows)), n_q, n_kv, hd
    d.scale = 0.0 if scale is None else scale
    if scale is not None and d.scale == 0.0:  # (which would stand for the default)
        _refuse(f"{name}: scale {scale} is 0 in fp32")
    for key, t in tensors.items():
        if t is None:
            continue
        want = (rows, n_q if key in ("q", "out") else n_kv, hd)
        if t.shape != want or t.dtype != dtype or t.stride(2) != 1:
            _refuse(f"{name}: {key} must be {dtype} {want} with a contiguous last axis (found {t.dtype} {tuple(t.shape)})")
        s = getattr(d, key + "_stride")
        s[0] = t.stride(0) if rows > 1 else 0
        s[1] = t.stride(1) if want[1] > 1 else 0
    return d


def _kv4_desc(name, cache, table, dtype):
    """(rl_kv4 without its addresses, KV heads, head_dim) of a cache and a page table."""
    kc, km, vc, vm = cache
    torch = _torch()
    if kc.dim() != 4 or kc.dtype != torch.uint8 or kc.shape != vc.shape or vc.dtype != torch.uint8 or kc.numel() == 0 or \
            km.shape != (*kc.shape[:3], 2) or vm.shape != km.shape or km.dtype != vm.dtype or (dtype is not None and km.dtype != dtype):
        _refuse(f"{name}: the cache must be uint8 [pages][Hkv][page][hd / 2] codes and {dtype or 'bf16 or fp16'} [pages][Hkv][page][2] scales, k's and v's alike")
    n, heads, page, half = kc.shape
    for t, w in ((kc, half), (vc, half), (km, 2), (vm, 2)):
        if t.stride()[2:] != (w, 1) or (heads > 1 and t.stride(1) != page * w):
            _refuse(f"{name}: the cache's pages must be contiguous")
    if table.dim() != 2 or table.dtype != torch.int32 or table.numel() == 0 or (table.shape[1] > 1 and table.stride(1) != 1):
        _refuse(f"{name}: table must be int32 [B][pages] with contiguous rows")
    if max(n, heads, page, *table.shape) > _INT32_MAX:
        _refuse(f"{name}: sizes must be below 2^31", RL_ERR_UNSUPPORTED)
    # (what _kv4_with packs around a call's addresses)
    fixed = ([t.stride(0) if n > 1 else 0 for t in (kc, vc, km, vm)],
             table.stride(0) if table.shape[0] > 1 else table.shape[1], table.shape[1])
    return (n, page, *fixed), heads, 2 * half


_KV4_FORM = struct.Struct("@ii4P4qPqi0q")  # rl_kv4


def _kv4_with(c, cache, table):
    """rl_kv4 of _kv4_desc's values and this call's addresses."""
    kc, km, vc, vm = cache
    n, page, strides, table_stride, width = c
    return rl_kv4.from_buffer_copy(_KV4_FORM.pack(n, page, kc.data_ptr(), km.data_ptr(), vc.data_ptr(), vm.data_ptr(), *strides,
                                                  table.data_ptr(), table_stride, width))


def _spans(name, start, kv_len, batch, rows, err):
    if start is None:
        if rows != batch:
            _refuse(f"{name}: {rows} rows for {batch} sequences need start")
    else:
        _int32(name, "start", start, (batch + 1,))
    if kv_len is not None:
        _int32(name, "kv_len", kv_len, (batch,))
    if err is not None:
        _int32(name, "err", err, (1,))


def packed_attention(q, k, v, start, max_rows=None, scale=None, out=None, err=None, stream=None):
    """Causal attention of packed prompts: ``q [N][Hq][hd]``, ``k``, ``v``
    [N][Hkv][hd] bf16 or fp16, sequence b the rows ``start[b]`` .. ``start[b + 1]``
    (int32 [B + 1]).  ``max_rows``: no sequence has more (None: unknown; known,
    it saves time).  Returns a dict: ``out`` (q's shape and type) and ``lse``
    fp32 [N][Hq]; buffers present in ``out`` are used, their rows of no sequence
    left as they were.  See rl_packed_attention."""
    torch = _torch()
    name = "packed_attention"
    dev = _operands(name, (q, k, v, start, err))
    o = dict(out) if out else {}
    res = _buffer(o, "out", q.shape, q, q.dtype, stream, name)
    B = start.numel() - 1

    def make():
        if q.dim() != 3 or k.dim() != 3 or B < 1 or q.numel() == 0 or k.numel() == 0:
            _refuse(f"{name}: q, k, v must be [N][heads][hd], not empty, start [B + 1]")
        return _packed_desc(name, q.dtype, (q.shape[1], k.shape[1], q.shape[2]), B, q.shape[0], max_rows or 0, scale, q=q, k=k, v=v, out=res)

    d = _plan((name, B, max_rows), scale, (q, k, v, res) if out else (q, k, v), make)
    lse = _buffer(o, "lse", (d.rows, d.n_q_heads), q, torch.float32, stream, name)
    _spans(name, start, None, B, d.rows, err)
    _run(dev, stream, _lib.rl_packed_attention, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), start.data_ptr(), res.data_ptr(),
         lse.data_ptr(), _addr(err))
    return o


def kv4_append(cache, table, kv_len, k, v, q=None, rope=None, start=None, out=None, err=None, stream=None):
    """The sequences' new rows into a 4-bit cache, rotated on the way: ``k``,
    ``v`` [N][Hkv][hd] of the scales' type, packed by ``start`` (int32 [B + 1];
    None: one row each), the last of ``kv_len`` (int32 [B], the new ones
    counted).  ``table``: int32 [B][pages]; ``rope``: rope_table's, for q and k
    (None: no rotation).  Returns a dict, with ``q [N][Hq][hd]`` given ``q`` its
    rotated rows; a buffer present in ``out`` is used (q itself may be).  See
    rl_kv4_append."""
    torch = _torch()
    name = "kv4_append"
    dev = _operands(name, (k, v, q, table, kv_len, rope, start, err, *cache))
    o = dict(out) if out else {}
    B = kv_len.numel()
    res = None
    if q is not None:
        res = o.get("q")
        if res is None:
            res = o["q"] = _new(q.shape, q.dtype, q.device, stream)
        else:
            _operands(name, (k, res))

    def make():
        if k.dim() != 3 or k.numel() == 0 or B < 1:
            _refuse(f"{name}: k and v must be [N][Hkv][hd], not empty, kv_len [B]")
        if q is not None and (q.dim() != 3 or q.numel() == 0):
            _refuse(f"{name}: q must be [N][Hq][hd], not empty")
        c, heads, hd = _kv4_desc(name, cache, table, k.dtype)
        d = _packed_desc(name, k.dtype, (q.shape[1] if q is not None else heads, heads, hd), B, k.shape[0], 0, None, q=q, k=k, v=v, out=res)
        if table.shape[0] != B:
            _refuse(f"{name}: table must have a row for each of the {B} sequences")
        return c, d

    ts = (*cache, table, k, v) + (() if q is None else (q, res) if out else (q,))
    c, d = _plan((name, B, q is None), None, ts, make)
    _spans(name, start, kv_len, B, d.rows, err)
    n_rope = 0
    if rope is not None:
        if rope.dtype != torch.float32 or rope.dim() != 3 or rope.shape[0] < 1 or rope.shape[1:] != (d.head_dim // 2, 2) or not rope.is_contiguous():
            _refuse(f"{name}: rope must be contiguous fp32 [n][{d.head_dim // 2}][2]")
        n_rope = min(rope.shape[0], _INT32_MAX)
    _run(dev, stream, _lib.rl_kv4_append, _kv4_with(c, cache, table), d, _addr(start), kv_len.data_ptr(), _addr(q), k.data_ptr(),
         v.data_ptr(), _addr(rope), n_rope, _addr(res), _addr(err))
    return o


def kv4_read(cache, table, kv_len, start=None, rows=None, out=None, err=None, stream=None):
    """Rows of a 4-bit cache as values: of sequence b the last ``start[b + 1] -
    start[b]`` of its ``kv_len[b]`` rows (``start`` None: the last one), packed;
    ``rows``: how many there is room for (without ``start`` one a sequence).  Returns a
    dict: ``k``, ``v`` [rows][Hkv][hd] of the scales' type; buffers present in
    ``out`` are used, their rows of no sequence left as they were.  See rl_kv4_read."""
    name = "kv4_read"
    dev = _operands(name, (table, kv_len, start, err, *cache))
    B = kv_len.numel()
    if rows is None and start is not None:
        _refuse(f"{name}: start needs rows")
    N = B if rows is None else _whole(name, "rows", rows)

    def make():
        if not 1 <= N <= _INT32_MAX or B < 1:
            _refuse(f"{name}: rows must be in [1, 2^31), kv_len [B]")
        c, heads, hd = _kv4_desc(name, cache, table, None)
        if table.shape[0] != B:
            _refuse(f"{name}: table must have a row for each of the {B} sequences")
        new = _torch().empty((N, heads, hd), dtype=cache[1].dtype, device="meta")
        given = {x: new if o.get(x) is None else o[x] for x in ("k", "v")}
        if any(t.dim() != 3 for t in given.values()):
            _refuse(f"{name}: k and v must be [{N}][{heads}][{hd}]")
        return c, new.shape, _packed_desc(name, new.dtype, (heads, heads, hd), B, N, 0, None, **given)

    o = dict(out) if out else {}
    ts = [o[x] for x in ("k", "v") if o.get(x) is not None]
    for t in ts:
        _operands(name, (table, t))
    c, shape, d = _plan((name, B, N, o.get("k") is None, o.get("v") is None), None, (*cache, table, *ts), make)
    for x in ("k", "v"):
        if o.get(x) is None:
            o[x] = _new(shape, cache[1].dtype, table.device, stream)
    k, v = o["k"], o["v"]
    _spans(name, start, kv_len, B, N, err)
    _run(dev, stream, _lib.rl_kv4_read, _kv4_with(c, cache, table), d, _addr(start), kv_len.data_ptr(), k.data_ptr(), v.data_ptr(), _addr(err))
    return o


def kv4_attention(q, cache, table, kv_len, start=None, max_rows=None, scale=None, out=None, workspace=None, err=None, stream=None):
    """Attention of single tokens and drafts over a 4-bit cache: ``q [N][Hq][hd]``
    of the scales' type, packed by ``start`` (int32 [B + 1]; None: one row each),
    the last rows of ``kv_len`` (int32 [B]).  ``max_rows``: no sequence has more
    rows here (None: unknown; known, it saves time).  Returns a dict: ``out``
    (q's shape and type) and ``lse`` fp32 [N][Hq]; buffers present in ``out``
    are used, their rows of no sequence left as they were.  ``workspace``: a
    uint8 tensor of rl_kv4_attention_workspace bytes; None takes one from
    PyTorch's allocator for this call.  See rl_kv4_attention."""
    torch = _torch()
    name = "kv4_attention"
    dev = _operands(name, (q, table, kv_len, start, workspace, err, *cache))
    o = dict(out) if out else {}
    res = _buffer(o, "out", q.shape, q, q.dtype, stream, name)
    B = kv_len.numel()

    def make():
        if q.dim() != 3 or q.numel() == 0 or B < 1:
            _refuse(f"{name}: q must be [N][Hq][hd], not empty, kv_len [B]")
        c, heads, hd = _kv4_desc(name, cache, table, q.dtype)
        if table.shape[0] != B:
            _refuse(f"{name}: table must have a row for each of the {B} sequences")
        d = _packed_desc(name, q.dtype, (q.shape[1], heads, hd), B, q.shape[0], max_rows or 0, scale, q=q, out=res)
        return c, d, rl_kv4_attention_workspace(d)

    c, d, need = _plan((name, B, max_rows), scale, (*cache, table, q, res) if out else (*cache, table, q), make)
    lse = _buffer(o, "lse", (d.rows, d.n_q_heads), q, torch.float32, stream, name)
    _spans(name, start, kv_len, B, d.rows, err)
    if workspace is None:
        workspace = _new((need,), torch.uint8, q.device, stream)
    elif not workspace.is_contiguous():
        _refuse(f"{name}: workspace must be contiguous")
    _run(dev, stream, _lib.rl_kv4_attention, _kv4_with(c, cache, table), d, _addr(start), kv_len.data_ptr(), q.data_ptr(),
         res.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), _addr(err))
    return o


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None, stream=None):
    """Draws one token a row of ``logits [R][V]`` (as token_logprobs) with the
    random numbers ``u`` (fp32 [R] in [0, 1)).  Each setting is a number or a
    tensor [R] (fp32; top_k int32).  Returns a dict: ``token`` int32 [R] and
    ``logprob`` fp32 [R], of the token among those kept; buffers present in
    ``out`` are used.  See rl_sample."""
    torch = _torch()
    name = "sample"
    dt = _dtype_code(logits.dtype)
    if logits.dim() != 2 or dt is None or logits.numel() == 0 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        _refuse(f"{name}: logits must be fp32, bf16 or fp16 [R][V] with contiguous rows")
    R, V = logits.shape
    if R > _INT32_MAX or V > _INT32_MAX:
        _refuse(f"{name}: rows and vocabulary must be below 2^31", RL_ERR_UNSUPPORTED)
    s = rl_sampling()
    given = []
    for key, x in (("temperature", temperature), ("top_k", top_k), ("top_p", top_p), ("min_p", min_p)):
        if isinstance(x, torch.Tensor):
            if x.dtype != (torch.int32 if key == "top_k" else torch.float32) or x.shape != (R,) or not x.is_contiguous():
                _refuse(f"{name}: {key} must be a number or contiguous {'int32' if key == 'top_k' else 'fp32'} ({R},)")
            setattr(s, "d_" + key, x.data_ptr())
            given.append(x)
        else:
            setattr(s, key, _int32_of(_whole(name, key, x)) if key == "top_k" else float(x))
    dev = _operands(name, (logits, u, *given))
    if u.dtype != torch.float32 or u.shape != (R,) or not u.is_contiguous():
        _refuse(f"{name}: u must be contiguous fp32 ({R},)")
    o = dict(out) if out else {}
    token = _buffer(o, "token", (R,), logits, torch.int32, stream, name)
    lp = _buffer(o, "logprob", (R,), logits, torch.float32, stream, name)
    _run(dev, stream, _lib.rl_sample, logits.data_ptr(), dt, R, V, logits.stride(0) if R > 1 else V, u.data_ptr(), s,
         token.data_ptr(), lp.data_ptr())
    return o


def quantize_exit_layers(model: Model, stream=None):
    model.quantize_exit_layers(stream)


def kv_cache_alloc(model: Model, max_batch, max_seq):
    return model.kv_cache_alloc(max_batch, max_seq)


__all__ = [*EXPORTS, "Model", "KVCache", "Policy", "RiverError", "prefill", "decode_step",
           "quantize_exit_layers", "kv_cache_alloc", "prefill_score", "token_logprobs", "window_attention",
           "shared_prefix_attention", "rl_attn_desc", "packed_attention", "kv4_append", "kv4_read", "kv4_attention",
           "sample", "KV4Cache", "rope_table", "rl_packed_desc", "rl_kv4", "rl_sampling", "LIB_PATH"]
