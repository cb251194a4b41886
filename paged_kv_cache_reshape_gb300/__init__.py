"""Python binding of the GB300 PagedAttention step library (libpa_gb300.so).

Argument marshalling only: every function below forwards to the C entry
point of the same name declared in include/pa.h.  Tensors are passed by
`data_ptr()`; streams by `torch.cuda.Stream.cuda_stream`.  No computation
happens here, and there is no fallback: if the shared library is missing
or fails to load, every call raises.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa_gb300.so")

PA_OK, PA_INVALID_ARGUMENT, PA_NOT_SUPPORTED, PA_CUDA_ERROR, PA_DEVICE_DATA_ERROR = range(5)
STATUS_NAMES = {0: "PA_OK", 1: "PA_INVALID_ARGUMENT", 2: "PA_NOT_SUPPORTED", 3: "PA_CUDA_ERROR",
                4: "PA_DEVICE_DATA_ERROR"}

PA_DEVERR_CUM, PA_DEVERR_BLOCK_ID, PA_DEVERR_PAST = 1, 2, 4
PA_DEVERR_KV_BOUND, PA_DEVERR_Q_BOUND, PA_DEVERR_ROTARY_POS, PA_DEVERR_TIMEOUT = 8, 16, 32, 64
PA_DEVERR_SLOT = 128
PA_DEVERR_ACCEPTED = 256
PA_DEVERR_PAGES = 512

PA_OPT_SPLIT_KEYS, PA_OPT_NO_WINDOW_PRUNE, PA_OPT_KERNEL_TIMING, PA_OPT_DECODE_MAX_ROWS = 1, 2, 3, 4
PA_OPT_DECODE_ITEMS_PER_CTA = 5
PA_OPT_LATENT_TCGEN05 = 6
PA_OPT_PREFILL_SMS, PA_OPT_WAIT_PROBE = 7, 8
PA_SITE_DECODE, PA_SITE_COMBINE, PA_SITE_PREFILL, PA_SITE_PREFILL_PAIR, PA_SITE_LATENT, PA_SITE_LATENT_TC = (
    k << 8 for k in range(1, 7))
PA_SITE_TREE, PA_SITE_Q4 = 7 << 8, 8 << 8
PA_STEP_COUNTS = 6
STEP_COUNT_NAMES = ("n_dec", "n_pre", "n_comb", "split_keys", "pre_ctas", "dec_ctas")
PA_STAGE_WORKLIST, PA_STAGE_CACHE_WRITE, PA_STAGE_DECODE, PA_STAGE_PREFILL, PA_STAGE_COMBINE = range(5)
STAGES = ("worklist", "cache_write", "decode", "prefill", "combine")
PA_CACHE_FP16, PA_CACHE_INT8, PA_CACHE_FP8_E4M3, PA_CACHE_BF16 = 0, 1, 2, 3
PA_ACT_DEFAULT, PA_ACT_BF16 = 0, 1
PA_QUANT_NONE, PA_QUANT_PER_TENSOR, PA_QUANT_PER_CHANNEL = 0, 1, 2
PA_LAYOUT_SEPARATE, PA_LAYOUT_LATENT = 0, 1
PA_ROTARY_FP16, PA_ROTARY_BF16, PA_ROTARY_FP32 = 0, 1, 2
(PA_ROTARY_SCALE_NONE, PA_ROTARY_SCALE_LINEAR, PA_ROTARY_SCALE_BASE, PA_ROTARY_SCALE_BY_PARTS,
 PA_ROTARY_SCALE_BY_WAVELENGTH) = range(5)

EXPORTED = ("pa_config_init", "pa_validate_config", "pa_check_step", "pa_create", "pa_cache_write",
            "pa_forward", "pa_check_device_error", "pa_last_error_message", "pa_destroy",
            "pa_set_option", "pa_kernel_time_ms", "pa_last_launch_count", "pa_forward_no_alloc",
            "pa_cache_write_ex", "pa_forward_ex", "pa_last_wait_site", "pa_last_step_counts",
            "pa_rotary_config_init", "pa_rotary_steps", "pa_rotary", "pa_tree_create", "pa_tree_destroy",
            "pa_tree_write", "pa_tree_attention", "pa_tree_commit", "pa_tree_check_device_error",
            "pa_tree_last_error_message", "pa_q4_page_bytes", "pa_q4_create", "pa_q4_destroy", "pa_q4_write",
            "pa_q4_read", "pa_q4_attention", "pa_q4_check_device_error", "pa_q4_last_error_message",
            "pa_pages_create", "pa_pages_destroy", "pa_pages_copy", "pa_pages_fork", "pa_pages_resize",
            "pa_pages_compact", "pa_pages_check_device_error", "pa_pages_last_error_message")


class pa_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("num_heads", "kv_num_heads", "head_size", "block_size",
                                            "num_blocks", "max_blocks_per_seq")] + [
        ("scale", ctypes.c_float), ("softcap", ctypes.c_float)] + [
        (n, ctypes.c_int) for n in ("local_window_size", "do_rotary", "rotary_interleaved",
                                    "rotary_dim", "max_rotary_positions", "max_batch", "max_tokens",
                                    "max_query_len_bound", "max_kv_len_bound", "cache_dtype",
                                    "k_quant_type", "v_quant_type", "packed_qkv", "qk_norm")] + [
        ("qk_norm_epsilon", ctypes.c_float)] + [
        (n, ctypes.c_int) for n in ("kv_cache_layout", "v_head_size", "rotary_offset", "act_dtype")]


class pa_extra_inputs(ctypes.Structure):
    _fields_ = [("head_sink", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("slot_mapping", ctypes.c_void_p), ("q_norm_weight", ctypes.c_void_p),
                ("k_norm_weight", ctypes.c_void_p)]


class pa_rotary_scaling(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int)] + [(n, ctypes.c_double) for n in ("base", "factor", "original_positions",
                                                                         "low", "high")]


class pa_rotary_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("head_size", "rotary_dim", "rotary_offset", "interleaved", "dtype")] + [
        ("attention_factor", ctypes.c_float), ("conjugate", ctypes.c_int)]


class pa_tree_inputs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("positions", "tree_mask", "distance_slopes", "head_sink")]


class pa_pages_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("block_size", "num_blocks", "max_blocks_per_seq", "max_rows")] + [
        ("page_bytes", ctypes.c_int64)]


class PAError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status
        self.message = message


_lib = None


def lib():
    """The loaded library (builds nothing; call build() first)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; run paged_kv_cache_reshape_gb300.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        CFG = ctypes.POINTER(pa_config)
        L.pa_config_init.argtypes = [CFG]
        L.pa_validate_config.argtypes = [CFG, ctypes.c_char_p, S]
        L.pa_check_step.argtypes = [CFG, I, P, P, P, P, P, P, P, P, I, I, P, P, P, ctypes.c_char_p, S]
        L.pa_create.argtypes = [CFG, ctypes.POINTER(P)]
        L.pa_cache_write.argtypes = [P, P, P, P, P, P, P, P, I, I, P, P, P]
        L.pa_forward.argtypes = [P, P, P, P, P, P, P, P, P, I, I, P, P, P, P]
        L.pa_check_device_error.argtypes = [P, ctypes.POINTER(I)]
        L.pa_last_error_message.argtypes = [P]
        L.pa_destroy.argtypes = [P]
        L.pa_set_option.argtypes = [P, I, I]
        L.pa_kernel_time_ms.argtypes = [P, I, ctypes.POINTER(ctypes.c_float)]
        L.pa_forward_no_alloc.argtypes = [CFG, P, P, P, P, P, P, P, P, I, I, P, P, P, P, P]
        X = ctypes.POINTER(pa_extra_inputs)
        L.pa_cache_write_ex.argtypes = [P, P, P, P, P, P, P, P, I, I, P, P, X, P]
        L.pa_forward_ex.argtypes = [P, P, P, P, P, P, P, P, P, I, I, P, P, X, P, P]
        L.pa_last_launch_count.argtypes = [P]
        L.pa_last_wait_site.argtypes = [P]
        L.pa_last_step_counts.argtypes = [P, ctypes.POINTER(I)]
        L64, RC = ctypes.c_int64, ctypes.POINTER(pa_rotary_config)
        L.pa_rotary_config_init.argtypes = [RC]
        L.pa_rotary_steps.argtypes = [ctypes.POINTER(pa_rotary_scaling), I, ctypes.POINTER(ctypes.c_uint64),
                                      ctypes.POINTER(ctypes.c_float)]
        L.pa_rotary.argtypes = [RC, P, P, I, I, P, L64, P, L64, I, P, L64, P, L64, P]
        L.pa_tree_create.argtypes = [CFG, I, ctypes.POINTER(P)]
        L.pa_tree_destroy.argtypes = [P]
        L.pa_tree_write.argtypes = [P, RC, P, P, P, L64, P, L64, P, L64, P, P, P, P, P, P, I, I, P]
        L.pa_tree_attention.argtypes = [P, P, P, P, P, P, P, I, I, ctypes.POINTER(pa_tree_inputs), P, P]
        L.pa_tree_commit.argtypes = [P, P, P, I, P, P, P, P, I, I, P, P]
        L.pa_tree_check_device_error.argtypes = [P, ctypes.POINTER(I)]
        L.pa_tree_last_error_message.argtypes = [P]
        L.pa_q4_page_bytes.argtypes = [I, I]
        L.pa_q4_create.argtypes = [CFG, I, ctypes.POINTER(P)]
        L.pa_q4_destroy.argtypes = [P]
        L.pa_q4_write.argtypes = [P, P, L64, P, L64, P, P, P, P, P, I, I, P]
        L.pa_q4_read.argtypes = [P, P, P, P, P, P, I, I, P, L64, P, L64, P]
        L.pa_q4_attention.argtypes = [P, P, P, P, P, P, P, I, I, P, P, P]
        L.pa_q4_check_device_error.argtypes = [P, ctypes.POINTER(I)]
        L.pa_q4_last_error_message.argtypes = [P]
        L.pa_pages_create.argtypes = [ctypes.POINTER(pa_pages_config), ctypes.POINTER(P)]
        L.pa_pages_destroy.argtypes = [P]
        L.pa_pages_copy.argtypes = [P, P, I, P, P, I, P]
        L.pa_pages_fork.argtypes = [P, P, I, P, P, I, P, I, P, P, P, P, P]
        L.pa_pages_resize.argtypes = [P, P, I, P, P, P, I, P, P, P]
        L.pa_pages_compact.argtypes = [P, P, I, P, I, P, P, P, P, P]
        L.pa_pages_check_device_error.argtypes = [P, ctypes.POINTER(I)]
        L.pa_pages_last_error_message.argtypes = [P]
        others = dict(pa_config_init=None, pa_rotary_config_init=None, pa_q4_page_bytes=L64,
                      pa_last_error_message=ctypes.c_char_p, pa_tree_last_error_message=ctypes.c_char_p,
                      pa_q4_last_error_message=ctypes.c_char_p, pa_pages_last_error_message=ctypes.c_char_p)
        for n in EXPORTED:
            getattr(L, n).restype = others.get(n, I)
        _lib = L
    return _lib


def build(force: bool = False):
    from . import builder as _b
    return _b.build(force=force)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(status, handle=None):
    if status != PA_OK:
        msg = lib().pa_last_error_message(handle).decode()
        raise PAError(status, msg)


def make_config(num_heads, kv_num_heads, head_size, block_size, num_blocks, max_blocks_per_seq,
                max_batch, max_tokens, scale=0.0, softcap=0.0, local_window_size=-1, do_rotary=0,
                rotary_interleaved=0, rotary_dim=0, max_rotary_positions=0, max_query_len_bound=0,
                max_kv_len_bound=0, cache_dtype=0, k_quant_type=0, v_quant_type=0, packed_qkv=0,
                qk_norm=0, qk_norm_epsilon=1e-6, kv_cache_layout=0, v_head_size=0,
                rotary_offset=0, act_dtype=0) -> pa_config:
    c = pa_config()
    lib().pa_config_init(ctypes.byref(c))
    for k, v in dict(num_heads=num_heads, kv_num_heads=kv_num_heads, head_size=head_size,
                     block_size=block_size, num_blocks=num_blocks,
                     max_blocks_per_seq=max_blocks_per_seq, max_batch=max_batch,
                     max_tokens=max_tokens, scale=scale, softcap=softcap,
                     local_window_size=local_window_size, do_rotary=do_rotary,
                     rotary_interleaved=rotary_interleaved, rotary_dim=rotary_dim,
                     max_rotary_positions=max_rotary_positions,
                     max_query_len_bound=max_query_len_bound,
                     max_kv_len_bound=max_kv_len_bound, cache_dtype=cache_dtype,
                     k_quant_type=k_quant_type, v_quant_type=v_quant_type, packed_qkv=packed_qkv,
                     qk_norm=qk_norm, qk_norm_epsilon=qk_norm_epsilon, kv_cache_layout=kv_cache_layout,
                     v_head_size=v_head_size, rotary_offset=rotary_offset, act_dtype=act_dtype).items():
        setattr(c, k, v)
    return c


def pa_validate_config(cfg: pa_config):
    buf = ctypes.create_string_buffer(512)
    st = lib().pa_validate_config(ctypes.byref(cfg), buf, 512)
    return st, buf.value.decode()


def pa_check_step(cfg: pa_config, for_forward, query, key, value, key_cache, value_cache,
                  block_table, cumulative_sequence_lengths, past_sequence_lengths, batch,
                  token_count, cos_cache, sin_cache, output):
    """Host-only argument check; pointer arguments are plain integers (or None)."""
    buf = ctypes.create_string_buffer(512)
    vp = lambda x: None if x is None else ctypes.c_void_p(x)
    st = lib().pa_check_step(ctypes.byref(cfg), for_forward, vp(query), vp(key), vp(value),
                             vp(key_cache), vp(value_cache), vp(block_table),
                             vp(cumulative_sequence_lengths), vp(past_sequence_lengths), batch,
                             token_count, vp(cos_cache), vp(sin_cache), vp(output), buf, 512)
    return st, buf.value.decode()


def pa_create(cfg: pa_config):
    h = ctypes.c_void_p()
    _check(lib().pa_create(ctypes.byref(cfg), ctypes.byref(h)))
    return h


def pa_destroy(h):
    _check(lib().pa_destroy(h))


def pa_set_option(h, option, value):
    _check(lib().pa_set_option(h, option, value), h)


def pa_cache_write(h, key, value, key_cache, value_cache, block_table,
                   cumulative_sequence_lengths, past_sequence_lengths, batch, token_count,
                   cos_cache=None, sin_cache=None, stream=None):
    _check(lib().pa_cache_write(h, _ptr(key), _ptr(value), _ptr(key_cache), _ptr(value_cache),
                                _ptr(block_table), _ptr(cumulative_sequence_lengths),
                                _ptr(past_sequence_lengths), batch, token_count, _ptr(cos_cache),
                                _ptr(sin_cache), ctypes.c_void_p(stream or 0)), h)


def pa_forward(h, query, key, value, key_cache, value_cache, block_table,
               cumulative_sequence_lengths, past_sequence_lengths, batch, token_count,
               cos_cache, sin_cache, output, stream=None):
    _check(lib().pa_forward(h, _ptr(query), _ptr(key), _ptr(value), _ptr(key_cache),
                            _ptr(value_cache), _ptr(block_table),
                            _ptr(cumulative_sequence_lengths), _ptr(past_sequence_lengths),
                            batch, token_count, _ptr(cos_cache), _ptr(sin_cache), _ptr(output),
                            ctypes.c_void_p(stream or 0)), h)


def _extra(head_sink=None, k_scale=None, v_scale=None, slot_mapping=None, q_norm_weight=None,
           k_norm_weight=None):
    if all(v is None for v in (head_sink, k_scale, v_scale, slot_mapping, q_norm_weight, k_norm_weight)):
        return None
    x = pa_extra_inputs()
    x.q_norm_weight = None if q_norm_weight is None else q_norm_weight.data_ptr()
    x.k_norm_weight = None if k_norm_weight is None else k_norm_weight.data_ptr()
    x.head_sink = None if head_sink is None else head_sink.data_ptr()
    x.k_scale = None if k_scale is None else k_scale.data_ptr()
    x.v_scale = None if v_scale is None else v_scale.data_ptr()
    x.slot_mapping = None if slot_mapping is None else slot_mapping.data_ptr()
    return ctypes.byref(x)


def pa_cache_write_ex(h, key, value, key_cache, value_cache, block_table,
                      cumulative_sequence_lengths, past_sequence_lengths, batch, token_count,
                      cos_cache=None, sin_cache=None, head_sink=None, k_scale=None, v_scale=None,
                      slot_mapping=None, q_norm_weight=None, k_norm_weight=None, stream=None):
    _check(lib().pa_cache_write_ex(h, _ptr(key), _ptr(value), _ptr(key_cache), _ptr(value_cache),
                                   _ptr(block_table), _ptr(cumulative_sequence_lengths),
                                   _ptr(past_sequence_lengths), batch, token_count, _ptr(cos_cache),
                                   _ptr(sin_cache),
                                   _extra(head_sink, k_scale, v_scale, slot_mapping, q_norm_weight, k_norm_weight),
                                   ctypes.c_void_p(stream or 0)), h)


def pa_forward_ex(h, query, key, value, key_cache, value_cache, block_table,
                  cumulative_sequence_lengths, past_sequence_lengths, batch, token_count,
                  cos_cache, sin_cache, output, head_sink=None, k_scale=None, v_scale=None,
                  slot_mapping=None, q_norm_weight=None, k_norm_weight=None, stream=None):
    _check(lib().pa_forward_ex(h, _ptr(query), _ptr(key), _ptr(value), _ptr(key_cache),
                               _ptr(value_cache), _ptr(block_table),
                               _ptr(cumulative_sequence_lengths), _ptr(past_sequence_lengths),
                               batch, token_count, _ptr(cos_cache), _ptr(sin_cache),
                               _extra(head_sink, k_scale, v_scale, slot_mapping, q_norm_weight, k_norm_weight),
                               _ptr(output),
                               ctypes.c_void_p(stream or 0)), h)


def pa_forward_no_alloc(cfg: pa_config, query, key, value, key_cache, value_cache, block_table,
                        cumulative_sequence_lengths, past_sequence_lengths, batch, token_count,
                        cos_cache, sin_cache, output, device_error=None, stream=None):
    """The whole step without a handle or any device allocation (scratch in a
    static device array); see include/pa.h for its limits and sharing rules."""
    _check(lib().pa_forward_no_alloc(ctypes.byref(cfg), _ptr(query), _ptr(key), _ptr(value),
                                     _ptr(key_cache), _ptr(value_cache), _ptr(block_table),
                                     _ptr(cumulative_sequence_lengths),
                                     _ptr(past_sequence_lengths), batch, token_count,
                                     _ptr(cos_cache), _ptr(sin_cache), _ptr(output),
                                     _ptr(device_error), ctypes.c_void_p(stream or 0)))


def pa_check_device_error(h) -> int:
    code = ctypes.c_int(0)
    st = lib().pa_check_device_error(h, ctypes.byref(code))
    if st not in (PA_OK, PA_DEVICE_DATA_ERROR):
        _check(st, h)
    return code.value


def pa_kernel_time_ms(h, stage) -> float:
    ms = ctypes.c_float(-1.0)
    _check(lib().pa_kernel_time_ms(h, stage, ctypes.byref(ms)), h)
    return ms.value


def pa_last_launch_count(h) -> int:
    return lib().pa_last_launch_count(h)


def pa_last_wait_site(h) -> int:
    return lib().pa_last_wait_site(h)


def pa_last_step_counts(h) -> dict:
    out = (ctypes.c_int * PA_STEP_COUNTS)()
    _check(lib().pa_last_step_counts(h, out), h)
    return dict(zip(STEP_COUNT_NAMES, list(out)))


def pa_last_error_message(h=None) -> str:
    return lib().pa_last_error_message(h).decode()


class PagedAttention:
    """A handle bound to one layer configuration (owns the device workspace)."""

    def __init__(self, cfg: pa_config):
        self.cfg = cfg
        self.handle = pa_create(cfg)

    @classmethod
    def for_step(cls, step: dict, max_batch: Optional[int] = None, max_tokens: Optional[int] = None,
                 **bounds):
        cos = step.get("cos_cache")
        cfg = make_config(step["num_heads"], step["kv_num_heads"], step["head_size"],
                          step["block_size"], step["num_blocks"], step["max_blocks_per_seq"],
                          max_batch or step["batch"], max_tokens or max(step["token_count"], 1),
                          scale=step["scale"], softcap=step["softcap"],
                          local_window_size=step["local_window_size"],
                          do_rotary=step["do_rotary"],
                          rotary_interleaved=step["rotary_interleaved"],
                          rotary_dim=step.get("rotary_dim", 0) or 0,
                          max_rotary_positions=0 if cos is None else cos.shape[0],
                          cache_dtype=step.get("cache_dtype", 0),
                          k_quant_type=step.get("quant_type", 0), v_quant_type=step.get("quant_type", 0),
                          packed_qkv=int(step.get("key") is None),
                          kv_cache_layout=step.get("kv_cache_layout", 0), v_head_size=step.get("v_head_size", 0),
                          rotary_offset=step.get("rotary_offset", 0),
                          act_dtype=PA_ACT_BF16 if step.get("act_bf16") else PA_ACT_DEFAULT,
                          qk_norm=int(step.get("q_norm_weight") is not None),
                          qk_norm_epsilon=step.get("qk_norm_epsilon", 1e-6), **bounds)
        return cls(cfg)

    def forward(self, step: dict, output, stream=None):
        pa_forward_ex(self.handle, step["query"], step["key"], step["value"], step["key_cache"],
                      step["value_cache"], step["block_table"], step["cumulative_sequence_lengths"],
                      step["past_sequence_lengths"], step["batch"], step["token_count"],
                      step.get("cos_cache"), step.get("sin_cache"), output,
                      head_sink=step.get("head_sink"), k_scale=step.get("k_scale"),
                      v_scale=step.get("v_scale"), slot_mapping=step.get("slot_mapping"),
                      q_norm_weight=step.get("q_norm_weight"), k_norm_weight=step.get("k_norm_weight"),
                      stream=stream)

    def cache_write(self, step: dict, stream=None):
        pa_cache_write_ex(self.handle, step["key"], step["value"], step["key_cache"],
                          step["value_cache"], step["block_table"],
                          step["cumulative_sequence_lengths"], step["past_sequence_lengths"],
                          step["batch"], step["token_count"], step.get("cos_cache"),
                          step.get("sin_cache"), head_sink=step.get("head_sink"),
                          k_scale=step.get("k_scale"), v_scale=step.get("v_scale"),
                          slot_mapping=step.get("slot_mapping"), q_norm_weight=step.get("q_norm_weight"),
                          k_norm_weight=step.get("k_norm_weight"), stream=stream)

    def set_option(self, option, value):
        pa_set_option(self.handle, option, value)

    def device_error(self) -> int:
        return pa_check_device_error(self.handle)

    def kernel_time_ms(self, stage) -> float:
        return pa_kernel_time_ms(self.handle, stage)

    def last_launch_count(self) -> int:
        return pa_last_launch_count(self.handle)

    def last_wait_site(self) -> int:
        return pa_last_wait_site(self.handle)

    def last_step_counts(self) -> dict:
        return pa_last_step_counts(self.handle)

    def close(self):
        if self.handle is not None:
            pa_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- speculative decoding: trees of drafted tokens (include/pa.h)


def make_rotary_config(head_size, rotary_dim=0, rotary_offset=0, interleaved=0, dtype=PA_ROTARY_FP16,
                       attention_factor=1.0, conjugate=0) -> pa_rotary_config:
    rc = pa_rotary_config()
    lib().pa_rotary_config_init(ctypes.byref(rc))
    rc.head_size, rc.rotary_dim, rc.rotary_offset, rc.interleaved = head_size, rotary_dim, rotary_offset, interleaved
    rc.dtype, rc.attention_factor, rc.conjugate = dtype, attention_factor, conjugate
    return rc


def pa_rotary_steps(rotary_dim, type=PA_ROTARY_SCALE_NONE, base=10000.0, factor=1.0, original_positions=0.0,
                    low=1.0, high=4.0):
    """(steps, attention_factor): the phase steps as a list of rotary_dim / 2
    whole numbers in [0, 2^64).  As a tensor they are int64 (the same bits):
    rotary_steps_tensor()."""
    sc = pa_rotary_scaling(type, base, factor, original_positions, low, high)
    steps, m = (ctypes.c_uint64 * max(rotary_dim // 2, 1))(), ctypes.c_float(0.0)
    _check(lib().pa_rotary_steps(ctypes.byref(sc), rotary_dim, steps, ctypes.byref(m)))
    return list(steps)[:rotary_dim // 2], m.value


def rotary_steps_tensor(steps, device="cuda"):
    """Phase steps as the int64 device tensor that pa_rotary and pa_tree_write take."""
    import torch
    return torch.tensor([v - (1 << 64) if v >> 63 else v for v in steps], dtype=torch.int64, device=device)


def _row_stride(t, token_count):
    stride = t.stride()
    if len(stride) != 2 or stride[1] != 1:
        raise PAError(PA_INVALID_ARGUMENT, "rows must be 2-D with contiguous columns")
    if stride[0] == 0 and token_count > 1:  # (an expanded row; in the C call 0 means dense rows)
        raise PAError(PA_INVALID_ARGUMENT, "rows must not share memory (a row stride of 0)")
    return stride[0]


def _gaps():
    raise PAError(PA_INVALID_ARGUMENT, "tensors must be contiguous (save rows of Q, K and V in pa_rotary and "
                                       "pa_tree_write)")


_types = None  # torch's int32, float16 and bfloat16, once a call has tensors


def _torch_types():
    global _types
    if _types is None:
        import torch
        _types = (torch.int32, torch.float16, torch.bfloat16)
    return _types


def _not_int32():
    raise PAError(PA_INVALID_ARGUMENT, "tables, lengths, ids and counts must be int32")


def _optional(t):
    if t is None:
        return None
    if not t.is_contiguous():
        _gaps()
    return t.data_ptr()


def pa_rotary(rc, steps, positions, token_count, num_heads, query, query_out, kv_num_heads=0, key=None,
              key_out=None, stream=None):
    """Rotates the rows of query [T, num_heads * D] and key; row strides are the tensors' own."""
    if not (steps.is_contiguous() and positions.is_contiguous()):
        _gaps()
    st = (_lib or lib()).pa_rotary(
        rc, steps.data_ptr(), positions.data_ptr(), token_count,
        num_heads, query.data_ptr() if num_heads else None, _row_stride(query, token_count) if num_heads else 0,
        query_out.data_ptr() if num_heads else None, _row_stride(query_out, token_count) if num_heads else 0,
        kv_num_heads, key.data_ptr() if kv_num_heads else None, _row_stride(key, token_count) if kv_num_heads else 0,
        key_out.data_ptr() if kv_num_heads else None, _row_stride(key_out, token_count) if kv_num_heads else 0, stream)
    if st:
        _check(st)


def _tree_check(status, h):
    if status != PA_OK:
        raise PAError(status, lib().pa_tree_last_error_message(h).decode())


def pa_tree_create(cfg: pa_config, max_draft_tokens):
    h = ctypes.c_void_p()
    _tree_check(lib().pa_tree_create(ctypes.byref(cfg), max_draft_tokens, ctypes.byref(h)), None)
    return h


def pa_tree_destroy(h):
    _tree_check(lib().pa_tree_destroy(h), None)


def pa_tree_write(h, rc, steps, positions, query, key, value, query_out, key_cache, value_cache, block_table,
                  cumulative_sequence_lengths, past_sequence_lengths, batch, token_count, stream=None):
    # (checked in one expression: the host's time bounds the smallest steps)
    if not (steps.is_contiguous() and positions.is_contiguous() and query_out.is_contiguous()
            and key_cache.is_contiguous() and value_cache.is_contiguous() and block_table.is_contiguous()
            and cumulative_sequence_lengths.is_contiguous() and past_sequence_lengths.is_contiguous()):
        _gaps()
    st = (_lib or lib()).pa_tree_write(
        h, rc, steps.data_ptr(), positions.data_ptr(), query.data_ptr(), _row_stride(query, token_count),
        key.data_ptr(), _row_stride(key, token_count), value.data_ptr(), _row_stride(value, token_count),
        query_out.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), block_table.data_ptr(),
        cumulative_sequence_lengths.data_ptr(), past_sequence_lengths.data_ptr(), batch, token_count, stream)
    if st:
        _tree_check(st, h)


def pa_tree_attention(h, query, key_cache, value_cache, block_table, cumulative_sequence_lengths,
                      past_sequence_lengths, batch, token_count, output, positions=None, tree_mask=None,
                      distance_slopes=None, head_sink=None, stream=None):
    if not (query.is_contiguous() and output.is_contiguous() and key_cache.is_contiguous()
            and value_cache.is_contiguous() and block_table.is_contiguous()
            and cumulative_sequence_lengths.is_contiguous() and past_sequence_lengths.is_contiguous()):
        _gaps()
    x = pa_tree_inputs(_optional(positions), _optional(tree_mask), _optional(distance_slopes), _optional(head_sink))
    st = (_lib or lib()).pa_tree_attention(
        h, query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), block_table.data_ptr(),
        cumulative_sequence_lengths.data_ptr(), past_sequence_lengths.data_ptr(), batch, token_count, x,
        output.data_ptr(), stream)
    if st:
        _tree_check(st, h)


class layer_pools:
    """The pools of a model's layers as pa_tree_commit takes them (holds the tensors)."""

    def __init__(self, key_caches, value_caches):
        self.tensors = (list(key_caches), list(value_caches))
        if len(self.tensors[0]) != len(self.tensors[1]):
            raise PAError(PA_INVALID_ARGUMENT, "key_caches and value_caches must have one pool per layer each")
        self.num_layers = len(self.tensors[0])
        if not all(t.is_contiguous() for ts in self.tensors for t in ts):
            _gaps()
        self.keys, self.values = ((ctypes.c_void_p * self.num_layers)(*[t.data_ptr() for t in ts])
                                  for ts in self.tensors)


def pa_tree_commit(h, layers, block_table, past_sequence_lengths, accepted, accepted_count, batch, new_past=None,
                   stream=None):
    """accepted [batch, max_accepted] int32 (contiguous), accepted_count [batch]; layers: a layer_pools."""
    if not (block_table.is_contiguous() and past_sequence_lengths.is_contiguous() and accepted.is_contiguous()
            and accepted_count.is_contiguous()):
        _gaps()
    st = (_lib or lib()).pa_tree_commit(
        h, layers.keys, layers.values, layers.num_layers, block_table.data_ptr(), past_sequence_lengths.data_ptr(),
        accepted.data_ptr(), accepted_count.data_ptr(), accepted.shape[1], batch, _optional(new_past), stream)
    if st:
        _tree_check(st, h)


def pa_tree_check_device_error(h) -> int:
    code = ctypes.c_int(0)
    st = lib().pa_tree_check_device_error(h, ctypes.byref(code))
    if st not in (PA_OK, PA_DEVICE_DATA_ERROR):
        _tree_check(st, h)
    return code.value


class PagedTree:
    """A handle for trees of drafted tokens over one layer configuration (owns the device workspace)."""

    def __init__(self, cfg: pa_config, max_draft_tokens: int):
        self.handle = None
        self.cfg, self.max_draft_tokens = cfg, max_draft_tokens
        self.handle = pa_tree_create(cfg, max_draft_tokens)

    def write(self, *args, **kw):
        pa_tree_write(self.handle, *args, **kw)

    def attention(self, *args, **kw):
        pa_tree_attention(self.handle, *args, **kw)

    def commit(self, *args, **kw):
        pa_tree_commit(self.handle, *args, **kw)

    def device_error(self) -> int:
        return pa_tree_check_device_error(self.handle)

    def close(self):
        if self.handle is not None:
            pa_tree_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- pools held in 4 bits (include/pa.h)


def pa_q4_page_bytes(block_size, head_size) -> int:
    """Bytes of a page's share of one kv head; 0 for sizes that are not built."""
    return lib().pa_q4_page_bytes(block_size, head_size)


def q4_pool(cfg: pa_config, device="cuda"):
    """An empty 4-bit pool of a layer: uint8 [num_blocks, kv_num_heads, page bytes], every value 0."""
    import torch
    size = pa_q4_page_bytes(cfg.block_size, cfg.head_size)
    if not size:
        raise PAError(PA_NOT_SUPPORTED, "4-bit pools are built for head_size 64, 128 and 256 and a block_size that is "
                                        "a power of two >= 16")
    return torch.zeros(cfg.num_blocks, cfg.kv_num_heads, size, dtype=torch.uint8, device=device)


def _q4_check(status, h):
    if status != PA_OK:
        raise PAError(status, lib().pa_q4_last_error_message(h).decode())


def pa_q4_create(cfg: pa_config, first_tokens=0):
    h = ctypes.c_void_p()
    _q4_check(lib().pa_q4_create(ctypes.byref(cfg), first_tokens, ctypes.byref(h)), None)
    return h


def pa_q4_destroy(h):
    _q4_check(lib().pa_q4_destroy(h), None)


def _q4_args(rows, other_rows, token_count, key_cache, value_cache, block_table, cumulative_sequence_lengths,
             past_sequence_lengths, batch, sizes):
    """What the C calls cannot see: gaps, types and sizes (sizes: of a PagedQ4's configuration)."""
    i32 = (_types or _torch_types())[0]
    if not (key_cache.is_contiguous() and value_cache.is_contiguous() and block_table.is_contiguous()
            and cumulative_sequence_lengths.is_contiguous() and past_sequence_lengths.is_contiguous()):
        _gaps()
    if not (block_table.dtype is i32 and cumulative_sequence_lengths.dtype is i32
            and past_sequence_lengths.dtype is i32):
        _not_int32()
    if cumulative_sequence_lengths.numel() <= batch or past_sequence_lengths.numel() < batch:
        raise PAError(PA_INVALID_ARGUMENT, f"cumulative_sequence_lengths must have batch + 1 = {batch + 1} entries, "
                                           f"past_sequence_lengths {batch}")
    if sizes:
        columns, pool_bytes, kind, width = sizes
        if key_cache.nbytes != pool_bytes or value_cache.nbytes != pool_bytes:
            raise PAError(PA_INVALID_ARGUMENT, f"pools must have {pool_bytes} bytes")
        shape = block_table.shape
        if len(shape) != 2 or shape[1] != columns or shape[0] < batch:
            raise PAError(PA_INVALID_ARGUMENT, f"block_table must have {columns} columns and a row for each of the "
                                               f"{batch} sequences")
        if not (rows.dtype is kind and other_rows.dtype is kind):
            raise PAError(PA_INVALID_ARGUMENT, f"rows must be {kind}")
        if rows.numel() < token_count * width or other_rows.numel() < token_count * width:
            raise PAError(PA_INVALID_ARGUMENT, f"{token_count} rows of {width} values are needed")


def pa_q4_write(h, key, value, key_cache, value_cache, block_table, cumulative_sequence_lengths,
                past_sequence_lengths, batch, token_count, stream=None, sizes=None):
    """Rows of key and value [T, kv_num_heads * head_size] (their own row strides) into the pools."""
    _q4_args(key, value, token_count, key_cache, value_cache, block_table, cumulative_sequence_lengths,
             past_sequence_lengths, batch, sizes)
    st = (_lib or lib()).pa_q4_write(
        h, key.data_ptr(), _row_stride(key, token_count), value.data_ptr(), _row_stride(value, token_count),
        key_cache.data_ptr(), value_cache.data_ptr(), block_table.data_ptr(), cumulative_sequence_lengths.data_ptr(),
        past_sequence_lengths.data_ptr(), batch, token_count, stream)
    if st:
        _q4_check(st, h)


def pa_q4_read(h, key_cache, value_cache, block_table, cumulative_sequence_lengths, past_sequence_lengths, batch,
               token_count, key_out, value_out, stream=None, sizes=None):
    """The values held in slots past + j, to rows of key_out and value_out (their own row strides)."""
    _q4_args(key_out, value_out, token_count, key_cache, value_cache, block_table, cumulative_sequence_lengths,
             past_sequence_lengths, batch, sizes)
    st = (_lib or lib()).pa_q4_read(
        h, key_cache.data_ptr(), value_cache.data_ptr(), block_table.data_ptr(),
        cumulative_sequence_lengths.data_ptr(), past_sequence_lengths.data_ptr(), batch, token_count,
        key_out.data_ptr(), _row_stride(key_out, token_count), value_out.data_ptr(),
        _row_stride(value_out, token_count), stream)
    if st:
        _q4_check(st, h)


def pa_q4_attention(h, query, key_cache, value_cache, block_table, cumulative_sequence_lengths,
                    past_sequence_lengths, batch, token_count, output, head_sink=None, stream=None, sizes=None):
    if not (query.is_contiguous() and output.is_contiguous()):
        _gaps()
    _q4_args(query, output, token_count, key_cache, value_cache, block_table, cumulative_sequence_lengths,
             past_sequence_lengths, batch, sizes)
    st = (_lib or lib()).pa_q4_attention(
        h, query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), block_table.data_ptr(),
        cumulative_sequence_lengths.data_ptr(), past_sequence_lengths.data_ptr(), batch, token_count,
        _optional(head_sink), output.data_ptr(), stream)
    if st:
        _q4_check(st, h)


def pa_q4_check_device_error(h) -> int:
    code = ctypes.c_int(0)
    st = lib().pa_q4_check_device_error(h, ctypes.byref(code))
    if st not in (PA_OK, PA_DEVICE_DATA_ERROR):
        _q4_check(st, h)
    return code.value


class PagedQ4:
    """A handle for pools held in 4 bits over one layer configuration (owns the device workspace)."""

    def __init__(self, cfg: pa_config, first_tokens: int = 0):
        self.handle = None
        self.cfg, self.first_tokens = cfg, first_tokens
        self.handle = pa_q4_create(cfg, first_tokens)
        kind = _torch_types()[2 if cfg.cache_dtype == PA_CACHE_BF16 else 1]
        pool_bytes = cfg.num_blocks * cfg.kv_num_heads * pa_q4_page_bytes(cfg.block_size, cfg.head_size)
        self.row_sizes = (cfg.max_blocks_per_seq, pool_bytes, kind, cfg.kv_num_heads * cfg.head_size)
        self.query_sizes = (*self.row_sizes[:3], cfg.num_heads * cfg.head_size)

    def pool(self, device="cuda"):
        return q4_pool(self.cfg, device)

    def write(self, key, value, key_cache, value_cache, block_table, cumulative_sequence_lengths,
              past_sequence_lengths, batch, token_count, stream=None):
        pa_q4_write(self.handle, key, value, key_cache, value_cache, block_table, cumulative_sequence_lengths,
                    past_sequence_lengths, batch, token_count, stream, self.row_sizes)

    def read(self, key_cache, value_cache, block_table, cumulative_sequence_lengths, past_sequence_lengths, batch,
             token_count, key_out, value_out, stream=None):
        pa_q4_read(self.handle, key_cache, value_cache, block_table, cumulative_sequence_lengths,
                   past_sequence_lengths, batch, token_count, key_out, value_out, stream, self.row_sizes)

    def attention(self, query, key_cache, value_cache, block_table, cumulative_sequence_lengths,
                  past_sequence_lengths, batch, token_count, output, head_sink=None, stream=None):
        if head_sink is not None and (head_sink.dtype is not self.query_sizes[2]
                                      or head_sink.numel() < self.cfg.num_heads):
            raise PAError(PA_INVALID_ARGUMENT, f"head_sink must be {self.query_sizes[2]}, a value for each head")
        pa_q4_attention(self.handle, query, key_cache, value_cache, block_table, cumulative_sequence_lengths,
                        past_sequence_lengths, batch, token_count, output, head_sink, stream, self.query_sizes)

    def device_error(self) -> int:
        return pa_q4_check_device_error(self.handle)

    def close(self):
        if self.handle is not None:
            pa_q4_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- the pages of a cache (include/pa.h)


def _pages_check(status, h):
    if status != PA_OK:
        raise PAError(status, lib().pa_pages_last_error_message(h).decode())


def pa_pages_create(block_size, num_blocks, max_blocks_per_seq, max_rows, page_bytes):
    h, c = ctypes.c_void_p(), pa_pages_config(block_size, num_blocks, max_blocks_per_seq, max_rows, page_bytes)
    _pages_check(lib().pa_pages_create(ctypes.byref(c), ctypes.byref(h)), None)
    return h


def pa_pages_destroy(h):
    _pages_check(lib().pa_pages_destroy(h), None)


class page_pools:
    """Pools as the pa_pages_* calls take them (holds the tensors): the first dimension counts the pages."""

    def __init__(self, pools):
        self.tensors = list(pools)
        if not all(t.is_contiguous() for t in self.tensors):
            _gaps()
        self.num_pools = len(self.tensors)
        self.pages = {(t.shape[0], t.numel() * t.element_size()) for t in self.tensors}
        if len(self.pages) > 1:
            raise PAError(PA_INVALID_ARGUMENT, "pools must have the same pages")
        self.pointers = (ctypes.c_void_p * max(1, self.num_pools))(*[t.data_ptr() for t in self.tensors])


def pa_pages_copy(h, pools, src, dst, stream=None):
    """Page dst[i] of every pool receives page src[i]; pools: a page_pools."""
    if not (src.is_contiguous() and dst.is_contiguous()):
        _gaps()
    i32 = (_types or _torch_types())[0]
    if not (src.dtype is i32 and dst.dtype is i32):
        _not_int32()
    if src.numel() != dst.numel():
        raise PAError(PA_INVALID_ARGUMENT, "src and dst must have the same length")
    st = (_lib or lib()).pa_pages_copy(h, pools.pointers, pools.num_pools, src.data_ptr(), dst.data_ptr(),
                                       src.numel(), stream)
    if st:
        _pages_check(st, h)


def pa_pages_fork(h, pools, block_table, lengths, parent, ref_count, new_block_table, new_lengths, new_ref_count,
                  stream=None):
    """Row i of new_block_table continues row parent[i] of block_table (-1: an empty row)."""
    if not (block_table.is_contiguous() and lengths.is_contiguous() and parent.is_contiguous()
            and ref_count.is_contiguous() and new_block_table.is_contiguous() and new_lengths.is_contiguous()
            and new_ref_count.is_contiguous()):
        _gaps()
    i32 = (_types or _torch_types())[0]
    if not (block_table.dtype is i32 and lengths.dtype is i32 and parent.dtype is i32 and ref_count.dtype is i32
            and new_block_table.dtype is i32 and new_lengths.dtype is i32 and new_ref_count.dtype is i32):
        _not_int32()
    rows, new_rows = block_table.shape[0], new_block_table.shape[0]
    if lengths.numel() != rows or parent.numel() != new_rows or new_lengths.numel() != new_rows:
        raise PAError(PA_INVALID_ARGUMENT, "lengths must have block_table's rows, parent and new_lengths "
                                           "new_block_table's")
    st = (_lib or lib()).pa_pages_fork(
        h, pools.pointers, pools.num_pools, block_table.data_ptr(), lengths.data_ptr(), rows, parent.data_ptr(),
        new_rows, ref_count.data_ptr(), new_block_table.data_ptr(), new_lengths.data_ptr(), new_ref_count.data_ptr(),
        stream)
    if st:
        _pages_check(st, h)


def pa_pages_resize(h, pools, block_table, lengths, delta, new_lengths, ref_count, stream=None):
    """Rows of block_table become lengths + delta positions long, in place."""
    if not (block_table.is_contiguous() and lengths.is_contiguous() and delta.is_contiguous()
            and new_lengths.is_contiguous() and ref_count.is_contiguous()):
        _gaps()
    i32 = (_types or _torch_types())[0]
    if not (block_table.dtype is i32 and lengths.dtype is i32 and delta.dtype is i32 and new_lengths.dtype is i32
            and ref_count.dtype is i32):
        _not_int32()
    rows = block_table.shape[0]
    if lengths.numel() != rows or delta.numel() != rows or new_lengths.numel() != rows:
        raise PAError(PA_INVALID_ARGUMENT, "lengths, delta and new_lengths must have block_table's rows")
    st = (_lib or lib()).pa_pages_resize(
        h, pools.pointers, pools.num_pools, block_table.data_ptr(), lengths.data_ptr(), delta.data_ptr(), rows,
        new_lengths.data_ptr(), ref_count.data_ptr(), stream)
    if st:
        _pages_check(st, h)


def pa_pages_compact(h, pools, block_table, ref_count, new_block_table, new_ref_count, pages_in_use, stream=None):
    """Moves the pages in use to the front; block_table and ref_count may be written in place."""
    if not (block_table.is_contiguous() and ref_count.is_contiguous() and new_block_table.is_contiguous()
            and new_ref_count.is_contiguous() and pages_in_use.is_contiguous()):
        _gaps()
    i32 = (_types or _torch_types())[0]
    if not (block_table.dtype is i32 and ref_count.dtype is i32 and new_block_table.dtype is i32
            and new_ref_count.dtype is i32 and pages_in_use.dtype is i32):
        _not_int32()
    if block_table.shape != new_block_table.shape:
        raise PAError(PA_INVALID_ARGUMENT, "block_table and new_block_table must have the same shape")
    st = (_lib or lib()).pa_pages_compact(
        h, pools.pointers, pools.num_pools, block_table.data_ptr(), block_table.shape[0], ref_count.data_ptr(),
        new_block_table.data_ptr(), new_ref_count.data_ptr(), pages_in_use.data_ptr(), stream)
    if st:
        _pages_check(st, h)


def pa_pages_check_device_error(h) -> int:
    code = ctypes.c_int(0)
    st = lib().pa_pages_check_device_error(h, ctypes.byref(code))
    if st not in (PA_OK, PA_DEVICE_DATA_ERROR):
        _pages_check(st, h)
    return code.value


class CachePages:
    """A handle for the pages of a cache: copies, forks, growth and release, compaction."""

    def __init__(self, block_size, num_blocks, max_blocks_per_seq, max_rows, page_bytes):
        self.handle = None
        self.num_blocks, self.max_blocks_per_seq, self.page_bytes = num_blocks, max_blocks_per_seq, page_bytes
        self.pages = {(num_blocks, num_blocks * page_bytes)}
        self.handle = pa_pages_create(block_size, num_blocks, max_blocks_per_seq, max_rows, page_bytes)

    def _own(self, pools, tables=(), counts=()):
        """The C calls take these sizes from the handle."""
        if pools.pages and pools.pages != self.pages:
            raise PAError(PA_INVALID_ARGUMENT, f"pools must have {self.num_blocks} pages of {self.page_bytes} bytes")
        for t in tables:
            shape = t.shape
            if len(shape) != 2 or shape[1] != self.max_blocks_per_seq:
                raise PAError(PA_INVALID_ARGUMENT, f"block tables must have {self.max_blocks_per_seq} columns")
        for t in counts:
            if t.numel() != self.num_blocks:
                raise PAError(PA_INVALID_ARGUMENT, f"ref_count must have {self.num_blocks} entries")

    def copy(self, pools, src, dst, stream=None):
        self._own(pools)
        pa_pages_copy(self.handle, pools, src, dst, stream)

    def fork(self, pools, block_table, lengths, parent, ref_count, new_block_table, new_lengths, new_ref_count,
             stream=None):
        self._own(pools, (block_table, new_block_table), (ref_count, new_ref_count))
        pa_pages_fork(self.handle, pools, block_table, lengths, parent, ref_count, new_block_table, new_lengths,
                      new_ref_count, stream)

    def resize(self, pools, block_table, lengths, delta, new_lengths, ref_count, stream=None):
        self._own(pools, (block_table,), (ref_count,))
        pa_pages_resize(self.handle, pools, block_table, lengths, delta, new_lengths, ref_count, stream)

    def compact(self, pools, block_table, ref_count, new_block_table, new_ref_count, pages_in_use, stream=None):
        self._own(pools, (block_table, new_block_table), (ref_count, new_ref_count))
        pa_pages_compact(self.handle, pools, block_table, ref_count, new_block_table, new_ref_count, pages_in_use,
                         stream)

    def device_error(self) -> int:
        return pa_pages_check_device_error(self.handle)

    def close(self):
        if self.handle is not None:
            pa_pages_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
