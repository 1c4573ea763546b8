"""ctypes binding of libpi.so (include/pi.h), argument marshalling only.

Every function here forwards device pointers of torch tensors to the C ABI; all
arithmetic happens in the library's HIP kernels. There is no fallback: if
libpi.so is missing or fails to load, :func:`lib` raises.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_double, c_float, c_int32, c_int64, c_void_p

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpi.so")

PI_OK, PI_ERR_INVALID, PI_ERR_UNSUPPORTED, PI_ERR_OOM, PI_ERR_HIP = range(5)
KERNEL_CLASSES = ("stage1", "stage2", "truemask", "up", "down", "reduce")
ACT = {"relu": 0, "reglu": 1, "sqrelu": 2}
WTYPE = {"f32": 0, "f16": 1, "q4_0": 2}
MASK_MODE = {"union": 0, "per_token": 1}
DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


class FfnDesc(ctypes.Structure):
    _fields_ = [
        ("d", c_int32), ("ffn", c_int32), ("rank", c_int32), ("act", c_int32), ("wtype", c_int32),
        ("threshold", c_float),
        ("w_up", c_void_p), ("w_gate", c_void_p), ("w_down_t", c_void_p),
        ("s_up", c_void_p), ("s_gate", c_void_p), ("s_down", c_void_p),
        ("b", c_void_p), ("p_w1", c_void_p), ("p_w2", c_void_p), ("p_b", c_void_p),
        ("neuron_table", c_void_p), ("hot_prefix", c_int32), ("y_center", c_void_p),
    ]


class StackDump(ctypes.Structure):
    _fields_ = [("x", c_void_p), ("mask", c_void_p), ("idx", c_void_p), ("n", c_void_p), ("y", c_void_p),
                ("ffn_stride", c_int32)]


class KvDesc(ctypes.Structure):
    _fields_ = [("dtype", c_int32), ("heads", c_int32), ("head_dim", c_int32), ("pages", c_int32),
                ("page_tokens", c_int32), ("k", c_void_p), ("v", c_void_p),
                ("page_stride", c_int64), ("token_stride", c_int64), ("head_stride", c_int64)]


class AppendArgs(ctypes.Structure):
    _fields_ = [("k_new", c_void_p), ("v_new", c_void_p), ("kv_batch", c_int64), ("kv_node", c_int64),
                ("kv_head", c_int64), ("table", c_void_p), ("table_stride", c_int64), ("table_width", c_int32),
                ("ctx_len", c_void_p), ("nodes", c_void_p), ("n", c_void_p), ("len_out", c_void_p),
                ("B", c_int32), ("N", c_int32)]


class AttnArgs(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("q_batch", c_int64), ("q_node", c_int64), ("q_head", c_int64),
                ("k_new", c_void_p), ("v_new", c_void_p), ("kv_batch", c_int64), ("kv_node", c_int64),
                ("kv_head", c_int64), ("tree", c_void_p), ("table", c_void_p), ("table_stride", c_int64),
                ("table_width", c_int32), ("ctx_len", c_void_p), ("out", c_void_p), ("out_batch", c_int64),
                ("out_node", c_int64), ("out_head", c_int64), ("B", c_int32), ("N", c_int32)]


class VerifyArgs(ctypes.Structure):
    _fields_ = [("logits", c_void_p), ("dtype", c_int32), ("logits_batch", c_int64), ("logits_node", c_int64),
                ("q", c_void_p), ("q_batch", c_int64), ("q_node", c_int64), ("tokens", c_void_p),
                ("parents", c_void_p), ("u", c_void_p), ("u_next", c_void_p), ("temperature", c_void_p),
                ("nodes", c_void_p), ("out", c_void_p), ("n", c_void_p), ("B", c_int32), ("N", c_int32)]


class NormArgs(ctypes.Structure):
    _fields_ = [("x", c_void_p), ("res", c_void_p), ("res_out", c_void_p), ("x_dtype", c_int32),
                ("res_dtype", c_int32), ("x_stride", c_int64), ("res_stride", c_int64), ("res_out_stride", c_int64),
                ("w", c_void_p), ("eps", c_float), ("q", c_void_p), ("q_stride", c_int64), ("scale", c_void_p),
                ("y", c_void_p), ("y_dtype", c_int32), ("y_stride", c_int64), ("T", c_int32), ("d", c_int32)]


class LinearDesc(ctypes.Structure):
    _fields_ = [("N", c_int32), ("K", c_int32), ("w", c_void_p), ("w_stride", c_int64), ("w_scale", c_void_p),
                ("bias", c_void_p), ("max_tokens", c_int32)]


class Kv4Desc(ctypes.Structure):
    _fields_ = [("dtype", c_int32), ("heads", c_int32), ("head_dim", c_int32), ("pages", c_int32),
                ("page_tokens", c_int32), ("k", c_void_p), ("v", c_void_p),
                ("page_stride", c_int64), ("token_stride", c_int64), ("head_stride", c_int64),
                ("k_scale", c_void_p), ("v_scale", c_void_p),
                ("scale_page_stride", c_int64), ("scale_token_stride", c_int64), ("scale_head_stride", c_int64)]


class ReadArgs(ctypes.Structure):
    _fields_ = [("table", c_void_p), ("table_stride", c_int64), ("table_width", c_int32), ("ctx_len", c_void_p),
                ("start", c_void_p), ("cu", c_void_p), ("k_out", c_void_p), ("v_out", c_void_p),
                ("out_row", c_int64), ("out_head", c_int64), ("B", c_int32), ("rows", c_int32)]


class PromptArgs(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("q_row", c_int64), ("q_head", c_int64), ("k", c_void_p),
                ("k_row", c_int64), ("k_head", c_int64), ("v", c_void_p), ("v_row", c_int64), ("v_head", c_int64),
                ("out", c_void_p), ("out_row", c_int64), ("out_head", c_int64), ("cu_q", c_void_p), ("cu_k", c_void_p), ("B", c_int32), ("q_rows", c_int32),
                ("k_rows", c_int32)]


class RopeArgs(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("k", c_void_p), ("q_row", c_int64), ("q_head", c_int64), ("k_row", c_int64),
                ("k_head", c_int64), ("q_out", c_void_p), ("k_out", c_void_p), ("q_out_row", c_int64),
                ("q_out_head", c_int64), ("k_out_row", c_int64), ("k_out_head", c_int64), ("x_dtype", c_int32),
                ("y_dtype", c_int32), ("q_w", c_void_p), ("k_w", c_void_p), ("eps", c_float), ("pos", c_void_p),
                ("inv_freq", c_void_p), ("rot", c_int32), ("interleaved", c_int32), ("T", c_int32),
                ("heads", c_int32), ("kv_heads", c_int32), ("head_dim", c_int32)]


_SIGS = {
    "pi_abi_version": (c_int32, []),
    "pi_status_str": (ctypes.c_char_p, [c_int32]),
    "pi_last_error": (ctypes.c_char_p, [c_void_p]),
    "pi_ctx_create": (c_int32, [c_int32, c_void_p, c_int32, c_int32, c_int32, c_int32, POINTER(c_void_p)]),
    "pi_ctx_destroy": (None, [c_void_p]),
    "pi_ctx_set_stream": (c_int32, [c_void_p, c_void_p]),
    "pi_ctx_set_mask_mode": (c_int32, [c_void_p, c_int32]),
    "pi_ffn_create": (c_int32, [c_void_p, POINTER(FfnDesc), POINTER(c_void_p)]),
    "pi_ffn_destroy": (None, [c_void_p]),
    "pi_predict": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_void_p]),
    "pi_sparse_ffn": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_void_p]),
    "pi_layer": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_void_p]),
    "pi_layer_noalloc": (c_int32, [c_int32, c_void_p, POINTER(FfnDesc), c_void_p, c_int32, c_void_p, c_void_p,
                                   c_void_p, c_void_p]),
    "pi_q4_dequant": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_void_p]),
    "pi_compact": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_float, c_void_p, c_void_p, c_void_p]),
    "pi_glue": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_int32, c_void_p]),
    "pi_stack_run": (c_int32, [c_void_p, POINTER(c_void_p), c_int32, c_void_p, c_int32, c_int32, c_void_p,
                               c_void_p, c_int32]),
    "pi_stack_run_dump": (c_int32, [c_void_p, POINTER(c_void_p), c_int32, c_void_p, c_int32, c_int32, c_void_p,
                                    c_void_p, POINTER(StackDump)]),
    "pi_stack_profile": (c_int32, [c_void_p, POINTER(c_void_p), c_int32, c_void_p, c_int32, c_int32, c_void_p,
                                   c_void_p, POINTER(c_double), POINTER(c_int64)]),
    "pi_hot_first_order": (c_int32, [POINTER(c_double), c_int32, POINTER(c_int32)]),
    "pi_permute_rows": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_int64]),
    "pi_kv_create": (c_int32, [c_void_p, POINTER(KvDesc), POINTER(c_void_p)]),
    "pi_kv_destroy": (None, [c_void_p]),
    "pi_kv4_create": (c_int32, [c_void_p, POINTER(Kv4Desc), POINTER(c_void_p)]),
    "pi_kv_read": (c_int32, [c_void_p, c_void_p, POINTER(ReadArgs)]),
    "pi_prompt_create": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_int32, c_int32, c_int32, c_float, POINTER(c_void_p)]),
    "pi_prompt_destroy": (None, [c_void_p]),
    "pi_prompt_attention": (c_int32, [c_void_p, c_void_p, POINTER(PromptArgs)]),
    "pi_qk_norm_rope": (c_int32, [c_void_p, POINTER(RopeArgs)]),
    "pi_kv_append": (c_int32, [c_void_p, c_void_p, POINTER(AppendArgs)]),
    "pi_attn_create": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_int32, c_float, POINTER(c_void_p)]),
    "pi_attn_destroy": (None, [c_void_p]),
    "pi_tree_attention": (c_int32, [c_void_p, c_void_p, POINTER(AttnArgs)]),
    "pi_verifier_create": (c_int32, [c_void_p, c_int32, c_int32, c_int32, POINTER(c_void_p)]),
    "pi_verifier_destroy": (None, [c_void_p]),
    "pi_verify": (c_int32, [c_void_p, c_void_p, POINTER(VerifyArgs)]),
    "pi_add_rmsnorm": (c_int32, [c_void_p, POINTER(NormArgs)]),
    "pi_linear_create": (c_int32, [c_void_p, POINTER(LinearDesc), POINTER(c_void_p)]),
    "pi_linear_destroy": (None, [c_void_p]),
    "pi_linear_q8": (c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_int32, c_void_p, c_int32, c_int64]),
}

_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded library. Raises if libpi.so has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first (python -m activation_sparse_ffn_layer_amd.build)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


class PiError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{lib().pi_status_str(status).decode()}: {msg}")
        self.status = status


def _ptr(t):
    """Device pointer of a tensor (or None)."""
    if t is None:
        return None
    return c_void_p(t.data_ptr())
