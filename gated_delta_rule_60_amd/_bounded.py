"""Attention over a bounded part of the past (a sliding window and the first
positions of a sequence), what keeps a cache bounded, and their gradients: the
binding of the ``attn_window_*`` entry points of libkda.so (include/kda.h).

As in ``_attn``: the functions named like the C symbols take raw device
pointers and a stream handle; the ``*_t`` functions take torch tensors.
"""
from __future__ import annotations

from ._attn import _gpu, _need, _on_stream, _prompt_args, _scale, _workspace
from ._lib import _check, load


# ---------------------------------------------------------------------------
# C ABI, one to one
# ---------------------------------------------------------------------------
def attn_window_prefill(q, k, v, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride, k_stride, v_stride, window, sinks,
                        scale, dtype, o, lse, stream) -> int:
    return load().attn_window_prefill(q, k, v, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride, k_stride, v_stride,
                                      window, sinks, scale, dtype, o, lse, stream)


def attn_window_prefill_backward(q, k, v, o, lse, d_o, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride, k_stride,
                                 v_stride, window, sinks, scale, dtype, d_q, d_k_out, d_v_out, workspace,
                                 workspace_bytes, stream) -> int:
    return load().attn_window_prefill_backward(q, k, v, o, lse, d_o, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride,
                                               k_stride, v_stride, window, sinks, scale, dtype, d_q, d_k_out, d_v_out,
                                               workspace, workspace_bytes, stream)


def attn_window_prefill_backward_workspace_size(N, T_tot, H_q, H_kv, d_k, d_v, window, sinks, dtype) -> int:
    return int(load().attn_window_prefill_backward_workspace_size(N, T_tot, H_q, H_kv, d_k, d_v, window, sinks, dtype))


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
