"""ctypes binding of libgemma3attn.so: same names as the C ABI in include/gemma3_attn.h.

The functions here only marshal arguments (tensor -> device pointer, torch's
current CUDA stream -> cudaStream_t) and turn a non-zero status into an
exception.  All computation runs in the library's CUDA kernels; there is no
fallback: if the library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os

from .build import LIB

c_int, c_long, c_double, c_float, c_size_t, c_void_p = (
    ctypes.c_int, ctypes.c_long, ctypes.c_double, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p)

GEMMA3_OK = 0
GEMMA3_ERR_TIMEOUT = -5
GEMMA3_ERR_BAD_INPUT = -7
GEMMA3_LOCAL_SLIDING, GEMMA3_GLOBAL = 0, 1
GEMMA3_BF16, GEMMA3_F16, GEMMA3_F32 = 0, 1, 2
GEMMA3_CACHE8_BLOCK = 64
GEMMA3_TREE_MAX = 64
MODEL_SIZES = {"270M": 0, "1B": 1, "4B": 2, "12B": 3, "27B": 4}


class gemma3_attn_dims(ctypes.Structure):
    _fields_ = [("B", c_int), ("T", c_int), ("D", c_int), ("H", c_int), ("H_kv", c_int),
                ("d_h", c_int)]


class gemma3_block_weights(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in (
        "Wq", "Wkv", "Wo", "gamma_q", "gamma_k", "gamma_pre_attn", "gamma_post_attn",
        "gamma_pre_ffn", "gamma_post_ffn", "W_gating", "W_down")]


class gemma3_paged_batch(ctypes.Structure):
    _fields_ = [(n, c_int) for n in ("B", "M", "T_max", "page_size", "n_pages", "max_pages")] + [
        (n, c_void_p) for n in ("lens", "row_start", "parents", "page_table")]


# name -> (restype, argtypes); mirrors include/gemma3_attn.h
SIGNATURES = {
    "gemma3_layer_attn_type": (c_int, [c_int, c_int]),
    "gemma3_layer_config": (c_int, [c_int, c_int, c_int, ctypes.POINTER(c_int),
                                    ctypes.POINTER(c_int), ctypes.POINTER(c_double),
                                    ctypes.POINTER(c_double)]),
    "gemma3_query_scale": (c_int, [c_int, c_int, c_int, c_int, ctypes.POINTER(c_float)]),
    "gemma3_attn_workspace_size": (c_int, [ctypes.POINTER(gemma3_attn_dims),
                                           ctypes.POINTER(c_size_t)]),
    "gemma3_attn_forward": (c_int, [ctypes.POINTER(gemma3_attn_dims), c_void_p, c_void_p, c_void_p,
                                    c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int,
                                    c_double, c_double, c_float, c_void_p, c_void_p, c_size_t,
                                    c_void_p]),
    "gemma3_attn_forward_noalloc": (c_int, [ctypes.POINTER(gemma3_attn_dims), c_void_p, c_void_p,
                                            c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                            c_void_p, c_int, c_int, c_double, c_double, c_float,
                                            c_void_p, c_void_p]),
    "gemma3_attn_noalloc_max_scratch": (c_size_t, []),
    "gemma3_block_attn_workspace_size": (c_int, [ctypes.POINTER(gemma3_attn_dims),
                                                 ctypes.POINTER(c_size_t)]),
    "gemma3_block_attn_forward": (c_int, [ctypes.POINTER(gemma3_attn_dims), c_void_p, c_int,
                                          c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                          c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int,
                                          c_int, c_double, c_double, c_float, c_void_p, c_size_t,
                                          c_void_p]),
    "gemma3_block_ffn_workspace_size": (c_int, [c_int, c_int, c_int, ctypes.POINTER(c_size_t)]),
    "gemma3_block_ffn_forward": (c_int, [c_int, c_int, c_int, c_void_p, c_void_p, c_void_p,
                                         c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                         c_void_p]),
    "gemma3_block_workspace_size": (c_int, [ctypes.POINTER(gemma3_attn_dims), c_int,
                                            ctypes.POINTER(c_size_t)]),
    "gemma3_block_forward": (c_int, [ctypes.POINTER(gemma3_attn_dims), c_int, c_void_p, c_int,
                                     c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_int, c_int, c_double, c_double,
                                     c_float, c_void_p, c_size_t, c_void_p]),
    "gemma3_model_workspace_size": (c_int, [ctypes.POINTER(gemma3_attn_dims), c_int, c_int,
                                            ctypes.POINTER(c_size_t)]),
    "gemma3_model_forward": (c_int, [ctypes.POINTER(gemma3_attn_dims), c_int, c_int, c_int, c_int,
                                     c_void_p, c_void_p, c_void_p, c_void_p,
                                     ctypes.POINTER(gemma3_block_weights), c_void_p, c_void_p,
                                     c_void_p, c_size_t, c_void_p]),
    "gemma3_embed": (c_int, [c_void_p, c_void_p, c_int, c_int, c_int, c_float, c_void_p,
                             c_void_p]),
    "gemma3_attn_cached_workspace_size": (c_int, [ctypes.POINTER(gemma3_attn_dims), c_int,
                                                  ctypes.POINTER(c_size_t)]),
    "gemma3_attn_forward_cached": (c_int, [ctypes.POINTER(gemma3_attn_dims), c_int, c_int,
                                           c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                           c_void_p, c_void_p, c_void_p, c_int, c_int, c_double,
                                           c_double, c_float, c_void_p, c_void_p, c_void_p,
                                           c_void_p, c_void_p, c_size_t, c_void_p]),
    "gemma3_kv_cache_write": (c_int, [c_void_p, c_void_p, c_long, c_void_p, c_void_p, c_int,
                                      c_int, c_int, c_int, c_int, c_int, c_void_p, c_void_p,
                                      c_void_p, c_void_p]),
    "gemma3_cached_attention_workspace_size": (c_int, [c_int, c_int, c_int, c_int, c_int, c_int,
                                                       ctypes.POINTER(c_size_t)]),
    "gemma3_cached_attention": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                        c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int,
                                        c_int, c_int, c_int, c_int, c_void_p, c_size_t,
                                        c_void_p]),
    "gemma3_kv_cache8_write": (c_int, [c_void_p, c_void_p, c_long, c_void_p, c_void_p] +
                               [c_int] * 6 + [c_void_p] * 6),
    "gemma3_kv_cache8_read": (c_int, [c_void_p] * 4 + [c_int] * 6 +
                              [c_void_p, c_void_p, c_long, c_void_p]),
    "gemma3_cached8_attention_workspace_size": (c_int, [c_int] * 7 + [ctypes.POINTER(c_size_t)]),
    "gemma3_cached8_attention": (c_int, [c_void_p] * 9 + [c_int, c_void_p] + [c_int] * 8 +
                                 [c_void_p, c_size_t, c_void_p]),
    "gemma3_kv_cache8_evict": (c_int, [c_void_p] * 6 + [c_int] * 7 + [c_void_p] * 7 +
                               [c_int, c_void_p]),
    "gemma3_attn_cached8_workspace_size": (c_int, [ctypes.POINTER(gemma3_attn_dims), c_int, c_int,
                                                   ctypes.POINTER(c_size_t)]),
    "gemma3_attn_forward_cached8": (c_int, [ctypes.POINTER(gemma3_attn_dims), c_int, c_int] +
                                    [c_void_p] * 8 + [c_int, c_int, c_double, c_double, c_float] +
                                    [c_void_p] * 8 + [c_size_t, c_void_p]),
    "gemma3_paged_positions": (c_int, [ctypes.POINTER(gemma3_paged_batch), c_void_p, c_void_p]),
    "gemma3_paged_append": (c_int, [ctypes.POINTER(gemma3_paged_batch), c_void_p, c_long, c_void_p,
                                    c_long, c_void_p, c_void_p, c_long, c_void_p, c_void_p, c_int,
                                    c_int, c_int, c_double, c_double, c_float, c_void_p, c_void_p,
                                    c_void_p]),
    "gemma3_paged_attention_workspace_size": (c_int, [ctypes.POINTER(gemma3_paged_batch), c_int,
                                                      c_int, c_int, ctypes.POINTER(c_size_t)]),
    "gemma3_paged_attention": (c_int, [ctypes.POINTER(gemma3_paged_batch)] + [c_void_p] * 4 +
                               [c_int] * 5 + [c_void_p, c_size_t, c_void_p]),
    "gemma3_paged_commit": (c_int, [ctypes.POINTER(gemma3_paged_batch), c_void_p, c_void_p, c_int,
                                    c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p]),
    "gemma3_attn_paged_workspace_size": (c_int, [ctypes.POINTER(gemma3_paged_batch)] +
                                         [c_int] * 4 + [ctypes.POINTER(c_size_t)]),
    "gemma3_attn_forward_paged": (c_int, [ctypes.POINTER(gemma3_paged_batch)] + [c_int] * 4 +
                                  [c_void_p] * 6 + [c_int, c_int, c_double, c_double, c_float] +
                                  [c_void_p] * 4 + [c_size_t, c_void_p]),
    "gemma3_geglu": (c_int, [c_void_p, c_long, c_void_p, c_long, c_void_p, c_long, c_int, c_int,
                             c_int, c_int, c_void_p]),
    "gemma3_linear": (c_int, [c_void_p, c_long, c_void_p, c_long, c_void_p, c_long, c_int, c_int,
                              c_int, c_int, c_int, c_int, c_void_p, c_int, c_void_p]),
    "gemma3_qkv_proj_norm_rope": (c_int, [c_void_p, c_long, c_void_p, c_void_p, c_void_p,
                                          c_void_p, c_int, c_int, c_int, c_int, c_int, c_int,
                                          c_void_p, c_void_p, c_void_p, c_double, c_double,
                                          c_float, c_void_p, c_int, c_void_p]),
    "gemma3_linear_qk_norm_rope": (c_int, [c_void_p, c_long, c_void_p, c_long, c_void_p, c_long,
                                           c_int, c_int, c_int, c_int, c_void_p, c_void_p, c_int,
                                           c_int, c_double, c_double, c_float, c_void_p]),
    "gemma3_cast_bf16_f16": (c_int, [c_void_p, c_void_p, c_size_t, c_void_p]),
    "gemma3_qk_norm_rope": (c_int, [c_void_p, c_long, c_void_p, c_long, c_void_p, c_void_p,
                                    c_void_p, c_int, c_int, c_int, c_int, c_double, c_double,
                                    c_float, c_void_p]),
    "gemma3_flash_attention": (c_int, [c_void_p, c_void_p, c_void_p, c_long, c_void_p, c_int,
                                       c_void_p, c_int, c_int, c_int, c_int, c_int, c_int,
                                       c_void_p, c_void_p]),
    "gemma3_rmsnorm": (c_int, [c_void_p, c_int, c_void_p, c_void_p, c_int, c_int, c_int,
                               c_void_p, c_int, c_void_p]),
    "gemma3_postnorm_residual": (c_int, [c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_int,
                                         c_int, c_void_p, c_int, c_void_p]),
    "gemma3_attn_check_status": (c_int, [c_void_p]),
    "gemma3_last_device_status": (c_int, []),
    "gemma3_set_gemm_tile_rows": (c_int, [c_int]),
    "gemma3_strerror": (ctypes.c_char_p, [c_int]),
    "gemma3_selftest_wait_timeout": (c_int, [ctypes.c_longlong, c_void_p]),
}

_lib = None


class Gemma3Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: status {status} ({strerror(status)})")


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(
                f"{LIB} is missing: build it with transformer_attention_gb300.build.build() "
                "(nvcc, sm_103a); there is no CPU fallback")
        handle = ctypes.CDLL(LIB)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def strerror(status: int) -> str:
    return lib().gemma3_strerror(status).decode()


def _check(fn: str, status: int) -> int:
    if status < 0:
        raise Gemma3Error(fn, status)
    return status


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on the GPU")
    return t.data_ptr()


_raw_stream = None       # () -> the current stream's cudaStream_t
_device = None           # () -> the current device's index


def _bind_torch():
    """The current stream and device by the calls that torch's own generated
    code uses (0.2 us where building a Stream object takes 3.3, more than the
    launch of a small kernel), or by the public ones where those are missing."""
    global _raw_stream, _device
    import torch
    torch.cuda.current_stream()              # initialises CUDA
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    dev = getattr(torch._C, "_cuda_getDevice", None)
    _device = dev or torch.cuda.current_device
    if raw is None:
        _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    else:
        _raw_stream = lambda: raw(_device())  # noqa: E731


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is None:
            _bind_torch()
        return _raw_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _here(*tensors):
    """Device pointers of the tensors (None and integers as they are), which
    must all live on the current device: the kernels run there."""
    if _device is None:
        _bind_torch()
    dev, out = _device(), []
    for t in tensors:
        if t is None or t.__class__ is int:
            out.append(t)
        elif t.get_device() != dev:
            raise ValueError("tensor arguments must live on the current GPU")
        else:
            out.append(t.data_ptr())
    return out


def _dims(B, T, D, H, H_kv, d_h):
    return gemma3_attn_dims(B, T, D, H, H_kv, d_h)


# ---------------------------------------------------------------- same-name wrappers
def gemma3_layer_attn_type(layer: int, num_layers: int) -> int:
    return _check("gemma3_layer_attn_type", lib().gemma3_layer_attn_type(layer, num_layers))


def gemma3_layer_config(layer: int, num_layers: int, model_size: str):
    t, w, base, scale = c_int(), c_int(), c_double(), c_double()
    _check("gemma3_layer_config", lib().gemma3_layer_config(
        layer, num_layers, MODEL_SIZES[model_size], ctypes.byref(t), ctypes.byref(w),
        ctypes.byref(base), ctypes.byref(scale)))
    return t.value, w.value, base.value, scale.value


def gemma3_query_scale(model_size: str, D: int, H: int, d_h: int) -> float:
    a = c_float()
    _check("gemma3_query_scale",
           lib().gemma3_query_scale(MODEL_SIZES[model_size], D, H, d_h, ctypes.byref(a)))
    return a.value


def gemma3_attn_workspace_size(B, T, D, H, H_kv, d_h) -> int:
    n = c_size_t()
    d = _dims(B, T, D, H, H_kv, d_h)
    _check("gemma3_attn_workspace_size", lib().gemma3_attn_workspace_size(ctypes.byref(d),
                                                                          ctypes.byref(n)))
    return n.value


def gemma3_block_attn_workspace_size(B, T, D, H, H_kv, d_h) -> int:
    n = c_size_t()
    d = _dims(B, T, D, H, H_kv, d_h)
    _check("gemma3_block_attn_workspace_size",
           lib().gemma3_block_attn_workspace_size(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def gemma3_attn_forward(dims, x, segment_pos, pad_lens, Wq, Wkv, Wo, gamma_q, gamma_k,
                        attn_type, window, rope_base, rope_scale, query_scale, out, workspace,
                        workspace_bytes, stream=None):
    d = _dims(*dims)
    return _check("gemma3_attn_forward", lib().gemma3_attn_forward(
        ctypes.byref(d), _ptr(x), _ptr(segment_pos), _ptr(pad_lens), _ptr(Wq), _ptr(Wkv),
        _ptr(Wo), _ptr(gamma_q), _ptr(gamma_k), attn_type, window, rope_base, rope_scale,
        query_scale, _ptr(out), _ptr(workspace), workspace_bytes, _stream(stream)))


def gemma3_attn_forward_noalloc(dims, x, segment_pos, pad_lens, Wq, Wkv, Wo, gamma_q, gamma_k,
                                attn_type, window, rope_base, rope_scale, query_scale, out,
                                stream=None):
    """gemma3_attn_forward without a workspace: for callers that cannot
    allocate device memory; uses the library's fixed per-device scratch."""
    d = _dims(*dims)
    return _check("gemma3_attn_forward_noalloc", lib().gemma3_attn_forward_noalloc(
        ctypes.byref(d), _ptr(x), _ptr(segment_pos), _ptr(pad_lens), _ptr(Wq), _ptr(Wkv),
        _ptr(Wo), _ptr(gamma_q), _ptr(gamma_k), attn_type, window, rope_base, rope_scale,
        query_scale, _ptr(out), _stream(stream)))


def gemma3_attn_noalloc_max_scratch() -> int:
    return lib().gemma3_attn_noalloc_max_scratch()


def gemma3_block_attn_forward(dims, x, x_dtype, y, segment_pos, pad_lens, Wq, Wkv, Wo, gamma_q,
                              gamma_k, gamma_pre, gamma_post, attn_type, window, rope_base,
                              rope_scale, query_scale, workspace, workspace_bytes, stream=None):
    d = _dims(*dims)
    return _check("gemma3_block_attn_forward", lib().gemma3_block_attn_forward(
        ctypes.byref(d), _ptr(x), x_dtype, _ptr(y), _ptr(segment_pos), _ptr(pad_lens), _ptr(Wq),
        _ptr(Wkv), _ptr(Wo), _ptr(gamma_q), _ptr(gamma_k), _ptr(gamma_pre), _ptr(gamma_post),
        attn_type, window, rope_base, rope_scale, query_scale, _ptr(workspace), workspace_bytes,
        _stream(stream)))


def gemma3_block_ffn_workspace_size(M, D, D_ff) -> int:
    n = c_size_t()
    _check("gemma3_block_ffn_workspace_size",
           lib().gemma3_block_ffn_workspace_size(M, D, D_ff, ctypes.byref(n)))
    return n.value


def gemma3_block_ffn_forward(M, D, D_ff, h, y, gamma_pre_ffn, gamma_post_ffn, W_gating, W_down,
                             workspace, workspace_bytes, stream=None):
    return _check("gemma3_block_ffn_forward", lib().gemma3_block_ffn_forward(
        M, D, D_ff, _ptr(h), _ptr(y), _ptr(gamma_pre_ffn), _ptr(gamma_post_ffn), _ptr(W_gating),
        _ptr(W_down), _ptr(workspace), workspace_bytes, _stream(stream)))


def gemma3_block_workspace_size(dims, D_ff) -> int:
    n = c_size_t()
    d = _dims(*dims)
    _check("gemma3_block_workspace_size",
           lib().gemma3_block_workspace_size(ctypes.byref(d), D_ff, ctypes.byref(n)))
    return n.value


def gemma3_block_forward(dims, D_ff, x, x_dtype, y, segment_pos, pad_lens, Wq, Wkv, Wo, gamma_q,
                         gamma_k, gamma_pre_attn, gamma_post_attn, gamma_pre_ffn, gamma_post_ffn,
                         W_gating, W_down, attn_type, window, rope_base, rope_scale, query_scale,
                         workspace, workspace_bytes, stream=None):
    d = _dims(*dims)
    return _check("gemma3_block_forward", lib().gemma3_block_forward(
        ctypes.byref(d), D_ff, _ptr(x), x_dtype, _ptr(y), _ptr(segment_pos), _ptr(pad_lens),
        _ptr(Wq), _ptr(Wkv), _ptr(Wo), _ptr(gamma_q), _ptr(gamma_k), _ptr(gamma_pre_attn),
        _ptr(gamma_post_attn), _ptr(gamma_pre_ffn), _ptr(gamma_post_ffn), _ptr(W_gating),
        _ptr(W_down), attn_type, window, rope_base, rope_scale, query_scale, _ptr(workspace),
        workspace_bytes, _stream(stream)))


def gemma3_model_workspace_size(dims, D_ff, V) -> int:
    n = c_size_t()
    d = _dims(*dims)
    _check("gemma3_model_workspace_size",
           lib().gemma3_model_workspace_size(ctypes.byref(d), D_ff, V, ctypes.byref(n)))
    return n.value


def gemma3_model_forward(dims, D_ff, V, num_layers, model_size, tokens, segment_pos, pad_lens, E,
                         layers, gamma_final, logits, workspace, workspace_bytes, stream=None):
    """``layers``: a sequence of dicts of device tensors keyed by the
    gemma3_block_weights field names; ``model_size``: "270M" .. "27B"."""
    d = _dims(*dims)
    arr = (gemma3_block_weights * max(1, num_layers))()
    for i, L in enumerate(layers):
        for name, _ in gemma3_block_weights._fields_:
            setattr(arr[i], name, _ptr(L[name]))
    return _check("gemma3_model_forward", lib().gemma3_model_forward(
        ctypes.byref(d), D_ff, V, num_layers, MODEL_SIZES[model_size], _ptr(tokens),
        _ptr(segment_pos), _ptr(pad_lens), _ptr(E), arr, _ptr(gamma_final), _ptr(logits),
        _ptr(workspace), workspace_bytes, _stream(stream)))


def gemma3_embed(tokens, E, V, D, M, scale, x, stream=None):
    return _check("gemma3_embed", lib().gemma3_embed(_ptr(tokens), _ptr(E), V, D, M, scale,
                                                     _ptr(x), _stream(stream)))


def gemma3_attn_cached_workspace_size(dims, S) -> int:
    n = c_size_t()
    d = _dims(*dims)
    _check("gemma3_attn_cached_workspace_size",
           lib().gemma3_attn_cached_workspace_size(ctypes.byref(d), S, ctypes.byref(n)))
    return n.value


def gemma3_attn_forward_cached(dims, S, end_index, x, segment_pos, pad_lens, Wq, Wkv, Wo,
                               gamma_q, gamma_k, attn_type, window, rope_base, rope_scale,
                               query_scale, K_cache, V_cache, pos_cache, out, workspace,
                               workspace_bytes, stream=None):
    d = _dims(*dims)
    return _check("gemma3_attn_forward_cached", lib().gemma3_attn_forward_cached(
        ctypes.byref(d), S, end_index, _ptr(x), _ptr(segment_pos), _ptr(pad_lens), _ptr(Wq),
        _ptr(Wkv), _ptr(Wo), _ptr(gamma_q), _ptr(gamma_k), attn_type, window, rope_base,
        rope_scale, query_scale, _ptr(K_cache), _ptr(V_cache), _ptr(pos_cache), _ptr(out),
        _ptr(workspace), workspace_bytes, _stream(stream)))


def gemma3_kv_cache_write(K_rows, V_rows, ld_rows, segment_pos, pad_lens, B, T, S, end_index,
                          H_kv, d_h, K_cache, V_cache, pos_cache, stream=None):
    return _check("gemma3_kv_cache_write", lib().gemma3_kv_cache_write(
        _ptr(K_rows), _ptr(V_rows), ld_rows, _ptr(segment_pos), _ptr(pad_lens), B, T, S,
        end_index, H_kv, d_h, _ptr(K_cache), _ptr(V_cache), _ptr(pos_cache), _stream(stream)))


def gemma3_cached_attention_workspace_size(B, T, S, H, H_kv, d_h) -> int:
    n = c_size_t()
    _check("gemma3_cached_attention_workspace_size", lib().gemma3_cached_attention_workspace_size(
        B, T, S, H, H_kv, d_h, ctypes.byref(n)))
    return n.value


def gemma3_cached_attention(Q, K_cache, V_cache, pos_cache, segment_pos, pad_lens, O, o_dtype, B,
                            T, S, end_index, H, H_kv, d_h, window, workspace, workspace_bytes,
                            stream=None):
    return _check("gemma3_cached_attention", lib().gemma3_cached_attention(
        _ptr(Q), _ptr(K_cache), _ptr(V_cache), _ptr(pos_cache), _ptr(segment_pos),
        _ptr(pad_lens), _ptr(O), o_dtype, B, T, S, end_index, H, H_kv, d_h, window,
        _ptr(workspace), workspace_bytes, _stream(stream)))


def gemma3_kv_cache8_write(K_rows, V_rows, ld_rows, segment_pos, pad_lens, B, T, S, end_index,
                           H_kv, d_h, K8, V8, K_scale, V_scale, pos_cache, stream=None):
    kr, vr, sp, pl, *cache = _here(K_rows, V_rows, segment_pos, pad_lens, K8, V8, K_scale, V_scale,
                                   pos_cache)
    return _check("gemma3_kv_cache8_write", lib().gemma3_kv_cache8_write(
        kr, vr, ld_rows, sp, pl, B, T, S, end_index, H_kv, d_h, *cache, _stream(stream)))


def gemma3_kv_cache8_read(K8, V8, K_scale, V_scale, B, S, first, n, H_kv, d_h, K_rows, V_rows,
                          ld_rows, stream=None):
    k8, v8, ks, vs, kr, vr = _here(K8, V8, K_scale, V_scale, K_rows, V_rows)
    return _check("gemma3_kv_cache8_read", lib().gemma3_kv_cache8_read(
        k8, v8, ks, vs, B, S, first, n, H_kv, d_h, kr, vr, ld_rows, _stream(stream)))


def gemma3_cached8_attention_workspace_size(B, T, S, H, H_kv, d_h, with_weights=False) -> int:
    n = c_size_t()
    _check("gemma3_cached8_attention_workspace_size",
           lib().gemma3_cached8_attention_workspace_size(B, T, S, H, H_kv, d_h,
                                                         int(with_weights), ctypes.byref(n)))
    return n.value


def gemma3_cached8_attention(Q, K8, V8, K_scale, V_scale, pos_cache, segment_pos, pad_lens, O,
                             o_dtype, weight_sum, B, T, S, end_index, H, H_kv, d_h, window,
                             workspace, workspace_bytes, stream=None):
    *ins, w, ws = _here(Q, K8, V8, K_scale, V_scale, pos_cache, segment_pos, pad_lens, O,
                        weight_sum, workspace)
    return _check("gemma3_cached8_attention", lib().gemma3_cached8_attention(
        *ins, o_dtype, w, B, T, S, end_index, H, H_kv, d_h, window, ws, workspace_bytes,
        _stream(stream)))


def gemma3_kv_cache8_evict(K8, V8, K_scale, V_scale, pos_cache, weight_sum, B, S, end_index, H_kv,
                           d_h, keep, recent, K8_dst, V8_dst, K_scale_dst, V_scale_dst, pos_dst,
                           weight_dst, kept, S_dst, stream=None):
    src = _here(K8, V8, K_scale, V_scale, pos_cache, weight_sum)
    dst = _here(K8_dst, V8_dst, K_scale_dst, V_scale_dst, pos_dst, weight_dst, kept)
    return _check("gemma3_kv_cache8_evict", lib().gemma3_kv_cache8_evict(
        *src, B, S, end_index, H_kv, d_h, keep, recent, *dst, S_dst, _stream(stream)))


def gemma3_attn_cached8_workspace_size(dims, S, with_weights=False) -> int:
    n = c_size_t()
    d = _dims(*dims)
    _check("gemma3_attn_cached8_workspace_size",
           lib().gemma3_attn_cached8_workspace_size(ctypes.byref(d), S, int(with_weights),
                                                    ctypes.byref(n)))
    return n.value


def gemma3_attn_forward_cached8(dims, S, end_index, x, segment_pos, pad_lens, Wq, Wkv, Wo,
                                gamma_q, gamma_k, attn_type, window, rope_base, rope_scale,
                                query_scale, K8, V8, K_scale, V_scale, pos_cache, weight_sum, out,
                                workspace, workspace_bytes, stream=None):
    d = _dims(*dims)
    ins = _here(x, segment_pos, pad_lens, Wq, Wkv, Wo, gamma_q, gamma_k)
    outs = _here(K8, V8, K_scale, V_scale, pos_cache, weight_sum, out, workspace)
    return _check("gemma3_attn_forward_cached8", lib().gemma3_attn_forward_cached8(
        ctypes.byref(d), S, end_index, *ins, attn_type, window, rope_base, rope_scale,
        query_scale, *outs, workspace_bytes, _stream(stream)))


class PagedBatch:
    """A gemma3_paged_batch over device tensors, which it keeps alive: lens [B],
    row_start [B + 1], page_table [B, max_pages] and parents [rows] or None,
    all int32, contiguous and on one GPU.  Their contents may change between
    calls; the sizes may not."""

    def __init__(self, lens, row_start, page_table, *, rows, T_max, page_size, n_pages,
                 parents=None):
        import torch
        B = lens.shape[0] if lens.dim() == 1 else -1
        pages = page_table.shape[1] if page_table.dim() == 2 else -1
        for name, t, shape in (("lens", lens, (B,)), ("row_start", row_start, (B + 1,)),
                               ("page_table", page_table, (B, pages)), ("parents", parents, (rows,))):
            if t is None and name == "parents":
                continue
            if tuple(t.shape) != shape or t.dtype != torch.int32 or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape}")
        self.tensors = (lens, row_start, parents, page_table)
        self.device = lens.get_device()
        if any(t is not None and t.get_device() != self.device for t in self.tensors):
            raise ValueError("a batch's tensors must live on one device")
        self.sizes = (B, rows, T_max, page_size, n_pages, pages)
        if any(not -2 ** 31 <= n < 2 ** 31 for n in self.sizes):   # (ctypes would cut them off)
            raise ValueError("a batch's sizes must fit 32 bits")
        self.struct = gemma3_paged_batch(*self.sizes, *(
            None if t is None else t.data_ptr() for t in self.tensors))

    def ref(self):
        """A reference to the struct, its arrays on the current device."""
        if _device is None:
            _bind_torch()
        if self.device != _device():
            raise ValueError("the batch's tensors must live on the current GPU")
        return ctypes.byref(self.struct)

    def sizes_ref(self):
        return ctypes.byref(self.struct)


def gemma3_paged_positions(batch, segment_pos, stream=None):
    pos, = _here(segment_pos)
    return _check("gemma3_paged_positions", lib().gemma3_paged_positions(
        batch.ref(), pos, _stream(stream)))


def gemma3_paged_append(batch, Q, ldq, Q_out, ldqo, K, V, ldkv, gamma_q, gamma_k, H, H_kv, d_h,
                        rope_base, rope_scale, query_scale, K_pages, V_pages, stream=None):
    q, qo, k, v, gq, gk, kp, vp = _here(Q, Q_out, K, V, gamma_q, gamma_k, K_pages, V_pages)
    return _check("gemma3_paged_append", lib().gemma3_paged_append(
        batch.ref(), q, ldq, qo, ldqo, k, v, ldkv, gq, gk, H, H_kv, d_h, rope_base, rope_scale,
        query_scale, kp, vp, _stream(stream)))


def gemma3_paged_attention_workspace_size(batch, H, H_kv, d_h) -> int:
    n = c_size_t()
    _check("gemma3_paged_attention_workspace_size", lib().gemma3_paged_attention_workspace_size(
        batch.sizes_ref(), H, H_kv, d_h, ctypes.byref(n)))
    return n.value


def gemma3_paged_attention(batch, Q, K_pages, V_pages, O, o_dtype, H, H_kv, d_h, window, workspace,
                           workspace_bytes, stream=None):
    q, kp, vp, o, ws = _here(Q, K_pages, V_pages, O, workspace)
    return _check("gemma3_paged_attention", lib().gemma3_paged_attention(
        batch.ref(), q, kp, vp, o, o_dtype, H, H_kv, d_h, window, ws, workspace_bytes,
        _stream(stream)))


def gemma3_paged_commit(batch, accepted, counts, num_layers, H_kv, d_h, K_pages, V_pages, new_lens,
                        stream=None):
    ac, co, kp, vp, nl = _here(accepted, counts, K_pages, V_pages, new_lens)
    return _check("gemma3_paged_commit", lib().gemma3_paged_commit(
        batch.ref(), ac, co, num_layers, H_kv, d_h, kp, vp, nl, _stream(stream)))


def gemma3_attn_paged_workspace_size(batch, D, H, H_kv, d_h) -> int:
    n = c_size_t()
    _check("gemma3_attn_paged_workspace_size", lib().gemma3_attn_paged_workspace_size(
        batch.sizes_ref(), D, H, H_kv, d_h, ctypes.byref(n)))
    return n.value


def gemma3_attn_forward_paged(batch, D, H, H_kv, d_h, x, Wq, Wkv, Wo, gamma_q, gamma_k, attn_type,
                              window, rope_base, rope_scale, query_scale, K_pages, V_pages, out,
                              workspace, workspace_bytes, stream=None):
    ins = _here(x, Wq, Wkv, Wo, gamma_q, gamma_k)
    outs = _here(K_pages, V_pages, out, workspace)
    return _check("gemma3_attn_forward_paged", lib().gemma3_attn_forward_paged(
        batch.ref(), D, H, H_kv, d_h, *ins, attn_type, window, rope_base, rope_scale, query_scale,
        *outs, workspace_bytes, _stream(stream)))


def gemma3_geglu(A, lda, W_gating, ldw, Z, ldz, M, D_ff, K, in_dtype, stream=None):
    return _check("gemma3_geglu", lib().gemma3_geglu(
        _ptr(A), lda, _ptr(W_gating), ldw, _ptr(Z), ldz, M, D_ff, K, in_dtype, _stream(stream)))


def gemma3_linear(A, lda, W, ldw, C, ldc, M, N, K, in_dtype, out_dtype, max_ctas=0,
                  stream=None, pad_lens=None, seg_T=0):
    return _check("gemma3_linear", lib().gemma3_linear(
        _ptr(A), lda, _ptr(W), ldw, _ptr(C), ldc, M, N, K, in_dtype, out_dtype, max_ctas,
        _ptr(pad_lens), seg_T, _stream(stream)))


def gemma3_qkv_proj_norm_rope(x, ldx, Wq, Wkv, Q, KV, M, D, H, H_kv, d_h, in_dtype, gamma_q,
                              gamma_k, pos, rope_base, rope_scale, query_scale, stream=None,
                              pad_lens=None, seg_T=0):
    return _check("gemma3_qkv_proj_norm_rope", lib().gemma3_qkv_proj_norm_rope(
        _ptr(x), ldx, _ptr(Wq), _ptr(Wkv), _ptr(Q), _ptr(KV), M, D, H, H_kv, d_h, in_dtype,
        _ptr(gamma_q), _ptr(gamma_k), _ptr(pos), rope_base, rope_scale, query_scale,
        _ptr(pad_lens), seg_T, _stream(stream)))


def gemma3_linear_qk_norm_rope(A, lda, W, ldw, C, ldc, M, N, K, in_dtype, gamma, pos, d_h, n_norm,
                               rope_base, rope_scale, scale, stream=None):
    return _check("gemma3_linear_qk_norm_rope", lib().gemma3_linear_qk_norm_rope(
        _ptr(A), lda, _ptr(W), ldw, _ptr(C), ldc, M, N, K, in_dtype, _ptr(gamma), _ptr(pos), d_h,
        n_norm, rope_base, rope_scale, scale, _stream(stream)))


def gemma3_cast_bf16_f16(src, dst, n, stream=None):
    return _check("gemma3_cast_bf16_f16", lib().gemma3_cast_bf16_f16(_ptr(src), _ptr(dst), n,
                                                                      _stream(stream)))


def gemma3_qk_norm_rope(Q, ldq, K, ldk, gamma_q, gamma_k, pos, M, H, H_kv, d_h, rope_base,
                        rope_scale, query_scale, stream=None):
    return _check("gemma3_qk_norm_rope", lib().gemma3_qk_norm_rope(
        _ptr(Q), ldq, _ptr(K), ldk, _ptr(gamma_q), _ptr(gamma_k), _ptr(pos), M, H, H_kv, d_h,
        rope_base, rope_scale, query_scale, _stream(stream)))


def gemma3_flash_attention(Q, K, V, ldkv, O, o_dtype, pad_lens, B, T, H, H_kv, d_h, window,
                           scratch=None, stream=None):
    """scratch: a 256-byte device tensor for the dynamic work order, or None
    for the fixed assignment."""
    return _check("gemma3_flash_attention", lib().gemma3_flash_attention(
        _ptr(Q), _ptr(K), _ptr(V), ldkv, _ptr(O), o_dtype, _ptr(pad_lens), B, T, H, H_kv, d_h,
        window, _ptr(scratch), _stream(stream)))


def gemma3_rmsnorm(x, x_dtype, gamma, u, u_dtype, M, D, stream=None, pad_lens=None, seg_T=0):
    return _check("gemma3_rmsnorm", lib().gemma3_rmsnorm(_ptr(x), x_dtype, _ptr(gamma), _ptr(u),
                                                         u_dtype, M, D, _ptr(pad_lens), seg_T,
                                                         _stream(stream)))


def gemma3_postnorm_residual(a, x, x_dtype, gamma, y, M, D, stream=None, pad_lens=None, seg_T=0):
    return _check("gemma3_postnorm_residual", lib().gemma3_postnorm_residual(
        _ptr(a), _ptr(x), x_dtype, _ptr(gamma), _ptr(y), M, D, _ptr(pad_lens), seg_T,
        _stream(stream)))


def gemma3_attn_check_status(stream=None) -> int:
    """Synchronises the stream and returns the library status (raises on error)."""
    return _check("gemma3_attn_check_status", lib().gemma3_attn_check_status(_stream(stream)))


def gemma3_last_device_status() -> int:
    return lib().gemma3_last_device_status()


def gemma3_set_gemm_tile_rows(rows: int) -> int:
    """Rows per projection-GEMM tile for later calls (0 chosen per call, 128
    or 256); returns the previous setting."""
    return _check("gemma3_set_gemm_tile_rows", lib().gemma3_set_gemm_tile_rows(rows))


def gemma3_selftest_wait_timeout(timeout_ns: int, stream=None) -> int:
    """Returns the raw status (GEMMA3_ERR_TIMEOUT expected); never raises on it."""
    return lib().gemma3_selftest_wait_timeout(timeout_ns, _stream(stream))
