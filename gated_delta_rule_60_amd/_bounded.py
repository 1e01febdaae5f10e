"""Attention over a bounded part of the past (a sliding window and the first
positions of a sequence), what keeps a cache bounded, and their gradients: the
binding of the ``attn_window_*`` entry points of libkda.so, of
``attn_prefill_weights``, ``attn_weighed_decode`` and ``kv_evict``
(include/kda.h).

As in ``_attn``: the functions named like the C symbols take raw device
pointers and a stream handle; the ``*_t`` functions take torch tensors.
"""
from __future__ import annotations

from ._attn import (KVPages, _cache_shape, _gpu, _layers, _need, _on_stream, _pages_args, _prompt_args, _requests,
                    _scale, _tokens, _workspace)
from ._lib import _check, _dtype_code, load


# What an int32 argument of the C ABI can take: ctypes would cut a larger number to its lowest 32 bits.  Compared in
# place (a call is some 10 us in all).
_LEAST, _MOST = -(1 << 31), (1 << 31) - 1


def _too_large(**values):
    name, x = next((n, x) for n, x in values.items() if not _LEAST <= x <= _MOST)
    raise ValueError(f"{name} does not fit in 32 bits: {x}")


# ---------------------------------------------------------------------------
# C ABI, one to one
# ---------------------------------------------------------------------------
def attn_window_prefill(q, k, v, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride, k_stride, v_stride, window, sinks,
                        scale, dtype, o, lse, stream) -> int:
    if not (_LEAST <= window <= _MOST and _LEAST <= sinks <= _MOST):
        _too_large(window=window, sinks=sinks)
    return load().attn_window_prefill(q, k, v, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride, k_stride, v_stride,
                                      window, sinks, scale, dtype, o, lse, stream)


def attn_window_prefill_backward(q, k, v, o, lse, d_o, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride, k_stride,
                                 v_stride, window, sinks, scale, dtype, d_q, d_k_out, d_v_out, workspace,
                                 workspace_bytes, stream) -> int:
    if not (_LEAST <= window <= _MOST and _LEAST <= sinks <= _MOST):
        _too_large(window=window, sinks=sinks)
    return load().attn_window_prefill_backward(q, k, v, o, lse, d_o, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride,
                                               k_stride, v_stride, window, sinks, scale, dtype, d_q, d_k_out, d_v_out,
                                               workspace, workspace_bytes, stream)


def attn_window_prefill_backward_workspace_size(N, T_tot, H_q, H_kv, d_k, d_v, window, sinks, dtype) -> int:
    if not (_LEAST <= window <= _MOST and _LEAST <= sinks <= _MOST):
        return 0
    return int(load().attn_window_prefill_backward_workspace_size(N, T_tot, H_q, H_kv, d_k, d_v, window, sinks, dtype))


def attn_window_decode(q, k_cache, v_cache, block_table, ctx_lens, cu_q, N, T_q, H_q, H_kv, d_k, d_v, n_pages, page_size,
                       max_pages, q_stride, window, sinks, scale, dtype, o, lse, workspace, workspace_bytes, stream) -> int:
    if not (_LEAST <= window <= _MOST and _LEAST <= sinks <= _MOST):
        _too_large(window=window, sinks=sinks)
    return load().attn_window_decode(q, k_cache, v_cache, block_table, ctx_lens, cu_q, N, T_q, H_q, H_kv, d_k, d_v, n_pages,
                                     page_size, max_pages, q_stride, window, sinks, scale, dtype, o, lse, workspace,
                                     workspace_bytes, stream)


def attn_window_decode_workspace_size(N, T_q, H_q, H_kv, d_v, page_size, max_pages, window, sinks) -> int:
    if not (_LEAST <= window <= _MOST and _LEAST <= sinks <= _MOST):
        return 0
    return int(load().attn_window_decode_workspace_size(N, T_q, H_q, H_kv, d_v, page_size, max_pages, window, sinks))


def attn_weighed_decode(q, k_cache, v_cache, block_table, ctx_lens, N, H_q, H_kv, d_k, d_v, n_pages, page_size, max_pages,
                        q_stride, scale, dtype, o, lse, weights, workspace, workspace_bytes, stream) -> int:
    return load().attn_weighed_decode(q, k_cache, v_cache, block_table, ctx_lens, N, H_q, H_kv, d_k, d_v, n_pages, page_size,
                                      max_pages, q_stride, scale, dtype, o, lse, weights, workspace, workspace_bytes, stream)


def attn_weighed_decode_workspace_size(N, H_q, H_kv, d_v, page_size, max_pages) -> int:
    return int(load().attn_weighed_decode_workspace_size(N, H_q, H_kv, d_v, page_size, max_pages))


def attn_prefill_weights(q, k, lse, cu_seqlens, N, T_tot, H_q, H_kv, d_k, q_stride, k_stride, rows, scale, dtype, weights,
                         width, workspace, workspace_bytes, stream) -> int:
    if not (_LEAST <= rows <= _MOST and _LEAST <= width <= _MOST):
        _too_large(rows=rows, width=width)
    return load().attn_prefill_weights(q, k, lse, cu_seqlens, N, T_tot, H_q, H_kv, d_k, q_stride, k_stride, rows, scale,
                                       dtype, weights, width, workspace, workspace_bytes, stream)


def attn_prefill_weights_workspace_size(N, T_tot, H_q, H_kv, rows) -> int:
    if not _LEAST <= rows <= _MOST:
        return 0
    return int(load().attn_prefill_weights_workspace_size(N, T_tot, H_q, H_kv, rows))


def kv_evict(block_table, lens, held, refs, free_list, n_free, n_rows, n_pages, page_size, max_pages, rows, n, k_cache,
             v_cache, n_layers, H_kv, d_k, d_v, dtype, weights, budget, recent, sinks, status, stream) -> int:
    if not (_LEAST <= budget <= _MOST and _LEAST <= recent <= _MOST and _LEAST <= sinks <= _MOST):
        _too_large(budget=budget, recent=recent, sinks=sinks)
    return load().kv_evict(block_table, lens, held, refs, free_list, n_free, n_rows, n_pages, page_size, max_pages, rows, n,
                           k_cache, v_cache, n_layers, H_kv, d_k, d_v, dtype, weights, budget, recent, sinks, status, stream)


# ---------------------------------------------------------------------------
# torch conveniences (marshalling only)
# ---------------------------------------------------------------------------
def attn_window_prefill_t(q, k, v, cu_seqlens=None, *, window, sinks=0, scale=None, o=None, lse=None, stream=None):
    """Causal softmax attention with a sliding window over packed prompts:
    position i sees the last ``window`` positions (itself among them) and the
    first ``sinks`` ones of its sequence.  Returns (o, lse); tensors as for
    ``attn_prefill_t``."""
    return _on_stream(stream, _gpu(q, "q"), _window_prefill_on, q, k, v, cu_seqlens, window, sinks, scale, o, lse)


def _window_prefill_on(q, k, v, cu_seqlens, window, sinks, scale, o, lse, stream):
    import torch
    dev = q.device
    cu_seqlens, N, T, Hq, Hkv, dk, dv, strides, code = _prompt_args(q, k, v, cu_seqlens)
    if o is None:
        o = torch.empty((T, Hq, dv), dtype=q.dtype, device=dev)
    else:
        _need(o, "o", (T, Hq, dv), q.dtype, dev)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    else:
        _need(lse, "lse", (T, Hq), torch.float32, dev)
    _check(attn_window_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), N, T, Hq, Hkv, dk, dv,
                               *strides, window, sinks, _scale(scale, dk), code, o.data_ptr(), lse.data_ptr(), stream))
    return o, lse


def attn_window_prefill_backward_t(q, k, v, o, lse, d_o, cu_seqlens=None, *, window, sinks=0, scale=None, workspace=None,
                                   stream=None):
    """Backward of ``attn_window_prefill_t`` (of the same window and sinks):
    gradients (d_q, d_k, d_v), shaped and typed like q, k and v.
    ``workspace``: optional uint8 device tensor of at least
    ``attn_window_prefill_backward_workspace_size(...)`` bytes."""
    return _on_stream(stream, _gpu(q, "q"), _window_backward_on, q, k, v, o, lse, d_o, cu_seqlens, window, sinks, scale,
                      workspace)


def _window_backward_on(q, k, v, o, lse, d_o, cu_seqlens, window, sinks, scale, workspace, stream):
    import torch
    dev = q.device
    cu_seqlens, N, T, Hq, Hkv, dk, dv, strides, code = _prompt_args(q, k, v, cu_seqlens)
    _need(o, "o", (T, Hq, dv), q.dtype, dev)
    _need(lse, "lse", (T, Hq), torch.float32, dev)
    _need(d_o, "d_o", (T, Hq, dv), q.dtype, dev)
    d_q = torch.empty((T, Hq, dk), dtype=q.dtype, device=dev)
    d_k = torch.empty((T, Hkv, dk), dtype=q.dtype, device=dev)
    d_v = torch.empty((T, Hkv, dv), dtype=q.dtype, device=dev)
    need = attn_window_prefill_backward_workspace_size(N, T, Hq, Hkv, dk, dv, window, sinks, code)
    ws = _workspace(workspace, need, dev)
    _check(attn_window_prefill_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                        d_o.data_ptr(), cu_seqlens.data_ptr(), N, T, Hq, Hkv, dk, dv, *strides, window,
                                        sinks, _scale(scale, dk), code, d_q.data_ptr(), d_k.data_ptr(), d_v.data_ptr(),
                                        ws.data_ptr(), ws.numel(), stream))
    return d_q, d_k, d_v


def attn_window_decode_t(q, k_cache, v_cache, block_table, ctx_lens, cu_q=None, *, window, sinks=0, scale=None, o=None,
                         lse=None, workspace=None, stream=None):
    """Attention of new tokens with a sliding window and sinks over a paged
    cache; returns (o, lse).

    Token j of sequence n stands at position ctx_lens[n] + j and sees the last
    ``window`` positions (itself among them) and the first ``sinks`` ones.
    Tensors as for ``attn_tree_decode_t``.  ``workspace``: optional uint8
    device tensor of ``attn_window_decode_workspace_size`` bytes."""
    return _on_stream(stream, _gpu(q, "q"), _window_decode_on, q, k_cache, v_cache, block_table, ctx_lens, cu_q, window,
                      sinks, scale, o, lse, workspace)


def _decode_args(q, k_cache, v_cache, block_table, ctx_lens, o, lse):
    """Checks of a step over a paged cache; returns (device, N, T, H_q, H_kv, d_k, d_v, pages, page size, pages a row,
    stride of q, dtype code, o, lse)."""
    import torch
    dev = q.device
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q must be [tokens, heads, size] and block_table [N, max_pages]")
    T, Hq, dk = q.shape
    code = _dtype_code(q)
    P, ps, Hkv, dk_cache, dv = _cache_shape(k_cache, v_cache, q.dtype, dev)
    if dk_cache != dk:
        raise ValueError(f"k_cache holds keys of {dk_cache}, q has {dk}")
    N, MP = ctx_lens.shape[0], block_table.shape[1]
    qs = _tokens(q, "q", (T, Hq, dk), q.dtype, dev)
    _need(block_table, "block_table", (N, MP), torch.int32, dev)
    _need(ctx_lens, "ctx_lens", (N,), torch.int32, dev)
    if o is None:
        o = torch.empty((T, Hq, dv), dtype=q.dtype, device=dev)
    else:
        _need(o, "o", (T, Hq, dv), q.dtype, dev)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    else:
        _need(lse, "lse", (T, Hq), torch.float32, dev)
    return dev, N, T, Hq, Hkv, dk, dv, P, ps, MP, qs, code, o, lse


def _window_decode_on(q, k_cache, v_cache, block_table, ctx_lens, cu_q, window, sinks, scale, o, lse, workspace, stream):
    import torch
    dev, N, T, Hq, Hkv, dk, dv, P, ps, MP, qs, code, o, lse = _decode_args(q, k_cache, v_cache, block_table, ctx_lens, o, lse)
    if cu_q is None:
        if T != N:
            raise ValueError(f"without cu_q there is one token per sequence: {T} tokens, {N} sequences")
        cu_q = torch.arange(N + 1, dtype=torch.int32, device=dev)
    _need(cu_q, "cu_q", (N + 1,), torch.int32, dev)
    ws = _workspace(workspace, attn_window_decode_workspace_size(N, T, Hq, Hkv, dv, ps, MP, window, sinks), dev)
    _check(attn_window_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                              ctx_lens.data_ptr(), cu_q.data_ptr(), N, T, Hq, Hkv, dk, dv, P, ps, MP, qs, window, sinks,
                              _scale(scale, dk), code, o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), stream))
    return o, lse


def attn_weighed_decode_t(q, k_cache, v_cache, block_table, ctx_lens, weights, *, scale=None, o=None, lse=None,
                          workspace=None, stream=None):
    """One token per sequence over a paged cache, as ``attn_tree_decode_t``;
    its attention weights, summed over the query heads of a key head, are added
    to ``weights`` (fp32 [N, H_kv, max_pages * page_size]; a position's is at
    its number).  Returns (o, lse).  ``workspace``: optional uint8 device
    tensor of ``attn_weighed_decode_workspace_size`` bytes."""
    return _on_stream(stream, _gpu(q, "q"), _weighed_decode_on, q, k_cache, v_cache, block_table, ctx_lens, weights, scale,
                      o, lse, workspace)


def _weighed_decode_on(q, k_cache, v_cache, block_table, ctx_lens, weights, scale, o, lse, workspace, stream):
    import torch
    dev, N, T, Hq, Hkv, dk, dv, P, ps, MP, qs, code, o, lse = _decode_args(q, k_cache, v_cache, block_table, ctx_lens, o, lse)
    if T != N:
        raise ValueError(f"there is one token per sequence: {T} tokens, {N} sequences")
    _need(weights, "weights", (N, Hkv, MP * ps), torch.float32, dev)
    ws = _workspace(workspace, attn_weighed_decode_workspace_size(N, Hq, Hkv, dv, ps, MP), dev)
    _check(attn_weighed_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                               ctx_lens.data_ptr(), N, Hq, Hkv, dk, dv, P, ps, MP, qs, _scale(scale, dk), code,
                               o.data_ptr(), lse.data_ptr(), weights.data_ptr(), ws.data_ptr(), ws.numel(), stream))
    return o, lse


def attn_prefill_weights_t(q, k, lse, cu_seqlens=None, *, weights, rows=None, scale=None, workspace=None, stream=None):
    """How much attention each position of the packed prompts has drawn from
    the last ``rows`` rows of its sequence (None: all), summed over the query
    heads of a key head, into ``weights`` (fp32 [N, H_kv, width], written in
    full, zero behind a sequence).  q, k, cu_seqlens, scale as for
    ``attn_prefill_t``, and its lse.  Returns ``weights``.  ``workspace``:
    optional uint8 device tensor of ``attn_prefill_weights_workspace_size``
    bytes."""
    return _on_stream(stream, _gpu(q, "q"), _prefill_weights_on, q, k, lse, cu_seqlens, weights, rows, scale, workspace)


def _prefill_weights_on(q, k, lse, cu_seqlens, weights, rows, scale, workspace, stream):
    import torch
    dev = q.device
    if weights.dim() != 3:
        raise ValueError("weights must be [N, H_kv, width]")
    cu_seqlens, N, T, Hq, Hkv, dk, _, strides, code = _prompt_args(q, k, k, cu_seqlens)
    _need(lse, "lse", (T, Hq), torch.float32, dev)
    width = weights.shape[2]
    _need(weights, "weights", (N, Hkv, width), torch.float32, dev)
    rows = max(T, 1) if rows is None else min(rows, max(T, 1))
    need = attn_prefill_weights_workspace_size(N, T, Hq, Hkv, rows)
    ws, size = None, 0  # few rows need none
    if need or workspace is not None:
        buf = _workspace(workspace, need, dev)
        ws, size = buf.data_ptr(), buf.numel()
    _check(attn_prefill_weights(q.data_ptr(), k.data_ptr(), lse.data_ptr(), cu_seqlens.data_ptr(), N, T, Hq, Hkv, dk,
                                strides[0], strides[1], rows, _scale(scale, dk), code, weights.data_ptr(), width, ws, size,
                                stream))
    return weights


def kv_evict_t(pages: KVPages, rows, k_cache, v_cache, weights=None, *, budget, recent, sinks=0, stream=None):
    """Rows ``rows`` (int32 [n]) with more than ``budget`` positions keep the
    first ``sinks``, the last ``recent`` and, by layer and key head, those
    between with the largest ``weights`` (fp32 [n_layers, rows, H_kv,
    max_pages * page_size]; None if budget = sinks + recent).  What is kept
    moves together in the caches and the weights; pages behind the budget go
    back.  Returns status int32 [n]: 0 done, 2 refused (a row that shares a
    page among them)."""
    return _on_stream(stream, _gpu(pages.table, "table"), _kv_evict_on, pages, rows, k_cache, v_cache, weights, budget,
                      recent, sinks)


def _kv_evict_on(pages, rows, k_cache, v_cache, weights, budget, recent, sinks, stream):
    import torch
    dev, args = _pages_args(pages)
    n = _requests(dev, rows=rows)
    code, L, P, ps, Hkv, dk, dv = _layers(k_cache, v_cache, dev)
    if (P, ps) != (args[7], args[8]):
        raise ValueError(f"the caches have {P} pages of {ps} positions, the bookkeeping {args[7]} of {args[8]}")
    if weights is not None:
        _need(weights, "weights", (L,) * (k_cache.dim() == 5) + (args[6], Hkv, args[9] * ps), torch.float32, dev)
    status = torch.empty(n, dtype=torch.int32, device=dev)
    _check(kv_evict(*args, rows.data_ptr(), n, k_cache.data_ptr(), v_cache.data_ptr(), L, Hkv, dk, dv, code,
                    weights.data_ptr() if weights is not None else None, budget, recent, sinks, status.data_ptr(), stream))
    return status
