"""Gemma 3 attention-block forward pass on one GB300 (sm_103a).

The compute lives in libgemma3attn.so (CUDA kernels behind the C ABI of
include/gemma3_attn.h).  ``_lib`` binds that ABI under the same names;
the helpers below only allocate outputs and workspaces with torch, on the
stream of the call, and call it.
"""
from __future__ import annotations

import contextlib

from ._lib import (  # noqa: F401  (re-exported C-ABI names)
    GEMMA3_BF16, GEMMA3_F16, GEMMA3_F32, GEMMA3_GLOBAL, GEMMA3_LOCAL_SLIDING, Gemma3Error,
    gemma3_attn_cached_workspace_size, gemma3_attn_check_status, gemma3_attn_forward,
    gemma3_attn_forward_cached, gemma3_attn_workspace_size, gemma3_cached_attention,
    gemma3_cached_attention_workspace_size, gemma3_kv_cache_write,
    GEMMA3_CACHE8_BLOCK, gemma3_attn_cached8_workspace_size, gemma3_attn_forward_cached8,
    gemma3_cached8_attention, gemma3_cached8_attention_workspace_size, gemma3_kv_cache8_evict,
    gemma3_kv_cache8_read, gemma3_kv_cache8_write,
    GEMMA3_TREE_MAX, PagedBatch, gemma3_attn_forward_paged, gemma3_attn_paged_workspace_size,
    gemma3_paged_append, gemma3_paged_attention, gemma3_paged_attention_workspace_size,
    gemma3_paged_commit, gemma3_paged_positions,
    gemma3_block_attn_forward, gemma3_block_attn_workspace_size, gemma3_block_ffn_forward,
    gemma3_block_ffn_workspace_size, gemma3_block_forward, gemma3_block_workspace_size,
    gemma3_cast_bf16_f16, gemma3_geglu,
    gemma3_flash_attention,
    gemma3_last_device_status, gemma3_layer_attn_type, gemma3_layer_config, gemma3_linear,
    gemma3_linear_qk_norm_rope, gemma3_qkv_proj_norm_rope, gemma3_embed, gemma3_model_forward, gemma3_model_workspace_size,
    GEMMA3_ERR_BAD_INPUT,
    gemma3_postnorm_residual, gemma3_qk_norm_rope, gemma3_query_scale, gemma3_rmsnorm,
    gemma3_selftest_wait_timeout, gemma3_set_gemm_tile_rows, lib)

__all__ = ["attention_forward", "attention_forward_cached", "attention_forward_cached8",
           "attention_forward_paged", "block_attention_forward", "block_forward",
           "commit_paged_cache", "evict_kv_cache8", "model_forward", "new_kv_cache",
           "new_kv_cache8", "new_paged_cache", "paged_batch", "linear", "lib"]


def _on(stream):
    """The context in which torch allocates and fills on ``stream``, as the
    call launched on it will use it: memory of the current stream could still
    be filled, or be handed out again, while that call runs."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _empty_ws(nbytes: int, device):
    import torch
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def attention_forward(x, segment_pos, pad_lens, Wq, Wkv, Wo, gamma_q, gamma_k, *, H, H_kv,
                      attn_type, window, rope_base, rope_scale, query_scale, out=None,
                      workspace=None, stream=None):
    """One attention layer: x [B,T,D] bf16 (CUDA) -> out [B,T,D] bf16.

    attn_type: GEMMA3_LOCAL_SLIDING or GEMMA3_GLOBAL.  pad_lens may be None.
    """
    import torch
    B, T, D = x.shape
    d_h = gamma_q.shape[0]
    dims = (B, T, D, H, H_kv, d_h)
    ws_bytes = gemma3_attn_workspace_size(*dims)
    with _on(stream):
        if workspace is None:
            workspace = _empty_ws(ws_bytes, x.device)
        if out is None:
            out = torch.empty((B, T, D), dtype=torch.bfloat16, device=x.device)
    gemma3_attn_forward(dims, x, segment_pos, pad_lens, Wq, Wkv, Wo, gamma_q, gamma_k, attn_type,
                        window, rope_base, rope_scale, query_scale, out, workspace,
                        workspace.numel(), stream)
    return out


def new_kv_cache(B, S, H_kv, d_h, device):
    """An empty KV cache of S slots per row: (K_cache, V_cache) [B, S, H_kv,
    d_h] fp16 and pos_cache [B, S] int32, every stored position -1."""
    import torch
    K = torch.zeros((B, S, H_kv, d_h), dtype=torch.float16, device=device)
    V = torch.zeros_like(K)
    pos = torch.full((B, S), -1, dtype=torch.int32, device=device)
    return K, V, pos


def attention_forward_cached(x, segment_pos, pad_lens, cache, end_index, Wq, Wkv, Wo, gamma_q,
                             gamma_k, *, H, H_kv, attn_type, window, rope_base, rope_scale,
                             query_scale, out=None, workspace=None, stream=None):
    """One attention layer over x [B,T,D] bf16, new tokens written to slots
    [end_index, end_index + T) of ``cache`` = (K_cache, V_cache, pos_cache)
    from new_kv_cache (updated in place).  Returns out [B,T,D] bf16."""
    import torch
    B, T, D = x.shape
    d_h = gamma_q.shape[0]
    K_cache, V_cache, pos_cache = cache
    S = pos_cache.shape[1]
    dims = (B, T, D, H, H_kv, d_h)
    ws_bytes = gemma3_attn_cached_workspace_size(dims, S)
    with _on(stream):
        if workspace is None:
            workspace = _empty_ws(ws_bytes, x.device)
        if out is None:
            out = torch.empty((B, T, D), dtype=torch.bfloat16, device=x.device)
    gemma3_attn_forward_cached(dims, S, end_index, x, segment_pos, pad_lens, Wq, Wkv, Wo,
                               gamma_q, gamma_k, attn_type, window, rope_base, rope_scale,
                               query_scale, K_cache, V_cache, pos_cache, out, workspace,
                               workspace.numel(), stream)
    return out


def new_kv_cache8(B, S, H_kv, d_h, device):
    """An empty 8-bit KV cache of S slots per row: (K8, V8) [B, S, H_kv, d_h]
    e4m3, (K_scale, V_scale) [B, ceil(S / 64), H_kv] fp32 and pos_cache [B, S]
    int32, every stored position -1."""
    import torch
    nb = -(-S // GEMMA3_CACHE8_BLOCK)
    K8 = torch.zeros((B, S, H_kv, d_h), dtype=torch.uint8, device=device)
    V8 = torch.zeros_like(K8)
    K_scale = torch.zeros((B, nb, H_kv), dtype=torch.float32, device=device)
    pos = torch.full((B, S), -1, dtype=torch.int32, device=device)
    return (K8.view(torch.float8_e4m3fn), V8.view(torch.float8_e4m3fn), K_scale,
            torch.zeros_like(K_scale), pos)


def _check_cache8(cache, B, H_kv, d_h, weight_sum):
    """ValueError unless ``cache`` is an 8-bit cache of these sizes in the
    layout of new_kv_cache8 (the kernels see addresses only), and weight_sum
    None or [B, S] fp32.  Returns S."""
    import torch
    K8, V8, K_scale, V_scale, pos = cache
    S = pos.shape[-1]
    num, sc = (B, S, H_kv, d_h), (B, -(-S // GEMMA3_CACHE8_BLOCK), H_kv)
    f32 = torch.float32
    for name, t, shape, dtypes in (
            ("K8", K8, num, (torch.float8_e4m3fn, torch.uint8)),
            ("V8", V8, num, (torch.float8_e4m3fn, torch.uint8)),
            ("K_scale", K_scale, sc, (f32,)), ("V_scale", V_scale, sc, (f32,)),
            ("pos_cache", pos, (B, S), (torch.int32,)),
            ("weight_sum", weight_sum, (B, S), (f32,))):
        if t is None and name == "weight_sum":
            continue
        if t.shape != shape or t.dtype not in dtypes or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtypes[0]} tensor of shape {shape}")
    return S


def attention_forward_cached8(x, segment_pos, pad_lens, cache, end_index, Wq, Wkv, Wo, gamma_q,
                              gamma_k, *, H, H_kv, attn_type, window, rope_base, rope_scale,
                              query_scale, weight_sum=None, out=None, workspace=None,
                              stream=None):
    """attention_forward_cached over an 8-bit cache from new_kv_cache8 (updated
    in place).  weight_sum [B, S] fp32, if given, gains the probabilities that
    every slot received.  Returns out [B,T,D] bf16."""
    import torch
    B, T, D = x.shape
    d_h = gamma_q.shape[0]
    K8, V8, K_scale, V_scale, pos_cache = cache
    S = _check_cache8(cache, B, H_kv, d_h, weight_sum)
    dims = (B, T, D, H, H_kv, d_h)
    ws_bytes = gemma3_attn_cached8_workspace_size(dims, S, weight_sum is not None)
    with _on(stream):
        if workspace is None:
            workspace = _empty_ws(ws_bytes, x.device)
        if out is None:
            out = torch.empty((B, T, D), dtype=torch.bfloat16, device=x.device)
    gemma3_attn_forward_cached8(dims, S, end_index, x, segment_pos, pad_lens, Wq, Wkv, Wo,
                                gamma_q, gamma_k, attn_type, window, rope_base, rope_scale,
                                query_scale, K8, V8, K_scale, V_scale, pos_cache, weight_sum, out,
                                workspace, workspace.numel(), stream)
    return out


def evict_kv_cache8(cache, weight_sum, end_index, keep, recent, *, into=None, S=None,
                    stream=None):
    """The ``keep`` slots of an 8-bit cache that matter most: those of its last
    ``recent`` slots and the heaviest others by weight_sum, moved in order to
    the front of another cache.  Returns (cache, weight_sum [B, S], kept
    [B, keep] int32, the slots they came from, -1 for none); the next
    end_index is ``keep``.  ``into``: (cache, weight_sum) to fill, else new
    ones of ``S`` slots (default: as many as before).  What it makes belongs
    to ``stream`` (default: the current one)."""
    import torch
    K8, V8, K_scale, V_scale, pos = cache
    B, S0, H_kv, d_h = K8.shape
    _check_cache8(cache, B, H_kv, d_h, weight_sum)
    with _on(stream):
        if into is None:
            S = S0 if S is None else S
            into = (new_kv_cache8(B, S, H_kv, d_h, K8.device),
                    torch.zeros((B, S), dtype=torch.float32, device=K8.device))
        dst, w_dst = into
        _check_cache8(dst, B, H_kv, d_h, w_dst)
        kept = torch.empty((B, keep), dtype=torch.int32, device=K8.device)
    gemma3_kv_cache8_evict(K8, V8, K_scale, V_scale, pos, weight_sum, B, S0, end_index, H_kv, d_h,
                           keep, recent, *dst, w_dst, kept, dst[4].shape[1], stream)
    return dst, w_dst, kept


def new_paged_cache(num_layers, n_pages, page_size, H_kv, d_h, device):
    """An empty paged KV cache of num_layers layers: (K_pages, V_pages)
    [num_layers, n_pages, page_size, H_kv, d_h] fp16."""
    import torch
    K = torch.zeros((num_layers, n_pages, page_size, H_kv, d_h), dtype=torch.float16,
                    device=device)
    return K, torch.zeros_like(K)


def paged_batch(lens, row_start, page_table, *, rows, T_max, page_size, n_pages, parents=None):
    """The batch that the paged calls take (PagedBatch): sequence b's slots [0,
    lens[b]) are filled, its new tokens are rows [row_start[b], row_start[b +
    1]) of packed arrays of ``rows`` rows, at most ``T_max`` of them, and its
    slots lie in the pages page_table[b] of a pool of ``n_pages``.  parents
    [rows] (T_max <= 64): drafted trees."""
    return PagedBatch(lens, row_start, page_table, rows=rows, T_max=T_max, page_size=page_size,
                      n_pages=n_pages, parents=parents)


def _check_pages(cache, layers, batch, H_kv, d_h):
    """ValueError unless ``cache`` is a pair of contiguous fp16 pools of these sizes."""
    import torch
    _, _, _, page_size, n_pages, _ = batch.sizes
    shape = layers + (n_pages, page_size, H_kv, d_h)
    for name, t in zip(("K_pages", "V_pages"), cache):
        if tuple(t.shape) != shape or t.dtype != torch.float16 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp16 tensor of shape {shape}")


def attention_forward_paged(x, batch, cache, Wq, Wkv, Wo, gamma_q, gamma_k, *, H, H_kv, attn_type,
                            window, rope_base, rope_scale, query_scale, out=None, workspace=None,
                            stream=None):
    """One attention layer over the packed rows x [rows, D] bf16 of a paged
    batch.  ``cache``: the layer's (K_pages, V_pages) [n_pages, page_size,
    H_kv, d_h], which gain the new tokens.  Returns out [rows, D] bf16, 0 in
    rows behind the last sequence."""
    import torch
    M, D = x.shape
    d_h = gamma_q.shape[0]
    if M != batch.sizes[1]:
        raise ValueError(f"x has {M} rows, the batch {batch.sizes[1]}")
    _check_pages(cache, (), batch, H_kv, d_h)
    ws_bytes = gemma3_attn_paged_workspace_size(batch, D, H, H_kv, d_h)
    with _on(stream):
        if workspace is None:
            workspace = _empty_ws(ws_bytes, x.device)
        if out is None:
            out = torch.empty((M, D), dtype=torch.bfloat16, device=x.device)
    gemma3_attn_forward_paged(batch, D, H, H_kv, d_h, x, Wq, Wkv, Wo, gamma_q, gamma_k, attn_type,
                              window, rope_base, rope_scale, query_scale, *cache, out, workspace,
                              workspace.numel(), stream)
    return out


def commit_paged_cache(batch, cache, accepted=None, counts=None, *, new_lens=None, stream=None):
    """After a step over a paged batch: of each sequence's new tokens those
    numbered accepted[b, :counts[b]] (ascending; default: the first counts[b],
    or all) become its next filled slots in every layer of ``cache`` =
    (K_pages, V_pages) [num_layers, n_pages, page_size, H_kv, d_h].  Returns
    the new lens [B] int32, in a tensor that is not the batch's."""
    import torch
    K, V = cache
    L, _, _, H_kv, d_h = K.shape
    B, _, T_max = batch.sizes[:3]
    _check_pages(cache, (L,), batch, H_kv, d_h)
    for name, t, shape in (("accepted", accepted, (B, T_max)), ("counts", counts, (B,)),
                           ("new_lens", new_lens, (B,))):
        if t is not None and (tuple(t.shape) != shape or t.dtype != torch.int32 or
                              not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape}")
    if new_lens is None:
        with _on(stream):
            new_lens = torch.empty(B, dtype=torch.int32, device=K.device)
    gemma3_paged_commit(batch, accepted, counts, L, H_kv, d_h, K, V, new_lens, stream)
    return new_lens


def block_attention_forward(x, segment_pos, pad_lens, Wq, Wkv, Wo, gamma_q, gamma_k, gamma_pre,
                            gamma_post, *, H, H_kv, attn_type, window, rope_base, rope_scale,
                            query_scale, y=None, workspace=None, stream=None):
    """y = x + RMSNorm_post(Attn(RMSNorm_pre(x))); x bf16 or fp32, y fp32 (may be x)."""
    import torch
    B, T, D = x.shape
    d_h = gamma_q.shape[0]
    dims = (B, T, D, H, H_kv, d_h)
    ws_bytes = gemma3_block_attn_workspace_size(*dims)
    with _on(stream):
        if workspace is None:
            workspace = _empty_ws(ws_bytes, x.device)
        if y is None:
            y = torch.empty((B, T, D), dtype=torch.float32, device=x.device)
    x_dtype = GEMMA3_F32 if x.dtype == torch.float32 else GEMMA3_BF16
    gemma3_block_attn_forward(dims, x, x_dtype, y, segment_pos, pad_lens, Wq, Wkv, Wo, gamma_q,
                              gamma_k, gamma_pre, gamma_post, attn_type, window, rope_base,
                              rope_scale, query_scale, workspace, workspace.numel(), stream)
    return y


def block_forward(x, segment_pos, pad_lens, Wq, Wkv, Wo, gamma_q, gamma_k, gamma_pre_attn,
                  gamma_post_attn, gamma_pre_ffn, gamma_post_ffn, W_gating, W_down, *, H, H_kv,
                  attn_type, window, rope_base, rope_scale, query_scale, y=None,
                  workspace=None, stream=None):
    """The whole block: y = h + FFN sandwich(h), h = x + attention sandwich(x).
    x bf16 or fp32 [B,T,D]; y fp32 (may be x); W_gating [2,D_ff,D], W_down [D,D_ff]."""
    import torch
    B, T, D = x.shape
    d_h = gamma_q.shape[0]
    D_ff = W_gating.shape[1]
    dims = (B, T, D, H, H_kv, d_h)
    ws_bytes = gemma3_block_workspace_size(dims, D_ff)
    with _on(stream):
        if workspace is None:
            workspace = _empty_ws(ws_bytes, x.device)
        if y is None:
            y = torch.empty((B, T, D), dtype=torch.float32, device=x.device)
    x_dtype = GEMMA3_F32 if x.dtype == torch.float32 else GEMMA3_BF16
    gemma3_block_forward(dims, D_ff, x, x_dtype, y, segment_pos, pad_lens, Wq, Wkv, Wo, gamma_q,
                         gamma_k, gamma_pre_attn, gamma_post_attn, gamma_pre_ffn, gamma_post_ffn,
                         W_gating, W_down, attn_type, window, rope_base, rope_scale, query_scale,
                         workspace, workspace.numel(), stream)
    return y


def model_forward(tokens, segment_pos, pad_lens, E, layers, gamma_final, *, H, H_kv, D_ff,
                  model_size, logits=None, workspace=None, stream=None):
    """The model: tokens [B,T] int32 -> logits [B,T,V] fp32 (read-out through
    E [V,D] bf16).  ``layers``: list of dicts of device tensors (Wq, Wkv, Wo,
    gamma_q, gamma_k, gamma_pre_attn, gamma_post_attn, gamma_pre_ffn,
    gamma_post_ffn, W_gating [2,D_ff,D], W_down [D,D_ff])."""
    import torch
    B, T = tokens.shape
    V, D = E.shape
    d_h = layers[0]["gamma_q"].shape[0] if layers else 256
    dims = (B, T, D, H, H_kv, d_h)
    ws_bytes = gemma3_model_workspace_size(dims, D_ff, V)
    with _on(stream):
        if workspace is None:
            workspace = _empty_ws(ws_bytes, tokens.device)
        if logits is None:
            logits = torch.empty((B, T, V), dtype=torch.float32, device=tokens.device)
    gemma3_model_forward(dims, D_ff, V, len(layers), model_size, tokens, segment_pos, pad_lens,
                         E, layers, gamma_final, logits, workspace, workspace.numel(), stream)
    return logits


def linear(A, W, out_dtype=None, max_ctas=0, stream=None):
    """C = A @ W^T on the tcgen05 GEMM (A [M,K], W [N,K], both bf16 or both f16)."""
    import torch
    out_dtype = out_dtype or torch.bfloat16
    code = {torch.bfloat16: GEMMA3_BF16, torch.float16: GEMMA3_F16, torch.float32: GEMMA3_F32}
    if A.dtype != W.dtype or A.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("A and W must both be bf16 or both f16")
    M, K = A.shape
    N = W.shape[0]
    with _on(stream):
        C = torch.empty((M, N), dtype=out_dtype, device=A.device)
    gemma3_linear(A, A.stride(0), W, W.stride(0), C, C.stride(0), M, N, K, code[A.dtype],
                  code[out_dtype], max_ctas, stream)
    return C
