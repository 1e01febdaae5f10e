"""Softmax attention over packed prompts and over a paged cache, and the
cache's page operations: the binding of the ``attn_*`` and ``kv_*`` entry
points of libkda.so (include/kda.h).

As in ``_lib``: the functions named like the C symbols take raw device
pointers and a stream handle; the ``*_t`` functions take torch tensors, check
shapes, types and devices, allocate outputs, and call the C ABI on ``stream``
(torch's current stream by default).  Every arithmetic step runs in the
library's HIP kernels; there is no fallback of any kind.
"""
from __future__ import annotations

import dataclasses
import math
from typing import Any

from ._lib import _check, _dtype_code, _stream_of, load


# ---------------------------------------------------------------------------
# C ABI, one to one
# ---------------------------------------------------------------------------
def attn_prefill(q, k, v, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride, k_stride, v_stride, scale, dtype,
                 o, lse, stream) -> int:
    return load().attn_prefill(q, k, v, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride, k_stride, v_stride,
                               scale, dtype, o, lse, stream)


def attn_prefill_backward(q, k, v, o, lse, d_o, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride, k_stride,
                          v_stride, scale, dtype, d_q, d_k_out, d_v_out, workspace, workspace_bytes, stream) -> int:
    return load().attn_prefill_backward(q, k, v, o, lse, d_o, cu_seqlens, N, T_tot, H_q, H_kv, d_k, d_v, q_stride,
                                        k_stride, v_stride, scale, dtype, d_q, d_k_out, d_v_out, workspace,
                                        workspace_bytes, stream)


def attn_prefill_backward_workspace_size(N, T_tot, H_q, H_kv, d_k, d_v, dtype) -> int:
    return int(load().attn_prefill_backward_workspace_size(N, T_tot, H_q, H_kv, d_k, d_v, dtype))


def attn_tree_decode(q, k_cache, v_cache, block_table, ctx_lens, cu_q, tree_mask, N, T_q, H_q, H_kv, d_k, d_v, n_pages,
                     page_size, max_pages, q_stride, scale, dtype, o, lse, workspace, workspace_bytes, stream) -> int:
    return load().attn_tree_decode(q, k_cache, v_cache, block_table, ctx_lens, cu_q, tree_mask, N, T_q, H_q, H_kv, d_k,
                                   d_v, n_pages, page_size, max_pages, q_stride, scale, dtype, o, lse, workspace,
                                   workspace_bytes, stream)


def attn_tree_decode_workspace_size(N, T_q, H_q, H_kv, d_v, page_size, max_pages) -> int:
    return int(load().attn_tree_decode_workspace_size(N, T_q, H_q, H_kv, d_v, page_size, max_pages))


def kv_reserve(block_table, lens, held, refs, free_list, n_free, n_rows, n_pages, page_size, max_pages, rows, n_tokens,
               n, status, stream) -> int:
    return load().kv_reserve(block_table, lens, held, refs, free_list, n_free, n_rows, n_pages, page_size, max_pages,
                             rows, n_tokens, n, status, stream)


def kv_free(block_table, lens, held, refs, free_list, n_free, n_rows, n_pages, page_size, max_pages, rows, n,
            stream) -> int:
    return load().kv_free(block_table, lens, held, refs, free_list, n_free, n_rows, n_pages, page_size, max_pages, rows,
                          n, stream)


def kv_fork(block_table, lens, held, refs, free_list, n_free, n_rows, n_pages, page_size, max_pages, src, dst, n,
            k_cache, v_cache, n_layers, H_kv, d_k, d_v, dtype, status, stream) -> int:
    return load().kv_fork(block_table, lens, held, refs, free_list, n_free, n_rows, n_pages, page_size, max_pages, src,
                          dst, n, k_cache, v_cache, n_layers, H_kv, d_k, d_v, dtype, status, stream)


def kv_append(k, v, k_cache, v_cache, block_table, lens, cu_new, N, T_new, n_layers, H_kv, d_k, d_v, n_pages, page_size,
              max_pages, dtype, stream) -> int:
    return load().kv_append(k, v, k_cache, v_cache, block_table, lens, cu_new, N, T_new, n_layers, H_kv, d_k, d_v,
                            n_pages, page_size, max_pages, dtype, stream)


def kv_compact(k_cache, v_cache, block_table, lens, accepted, cu_accepted, N, A_tot, n_layers, H_kv, d_k, d_v, n_pages,
               page_size, max_pages, dtype, new_lens, stream) -> int:
    return load().kv_compact(k_cache, v_cache, block_table, lens, accepted, cu_accepted, N, A_tot, n_layers, H_kv, d_k,
                             d_v, n_pages, page_size, max_pages, dtype, new_lens, stream)


# ---------------------------------------------------------------------------
# torch conveniences (marshalling only)
# ---------------------------------------------------------------------------
# A call's own cost counts where its kernels take microseconds: on the current
# device and stream it enters no context, and a dense tensor is checked by one
# comparison of each property.
def _on_stream(stream, dev, body, *args):
    """body(*args, stream handle) with outputs and temporaries allocated under that stream."""
    import torch
    if stream is None and dev.index == torch.cuda.current_device():
        return body(*args, torch._C._cuda_getCurrentRawStream(dev.index))  # 0.1 us; current_stream() is 1.8
    st = _stream_of(stream, dev)
    with torch.cuda.device(dev), torch.cuda.stream(st):
        return body(*args, st.cuda_stream)


def _need(t, name, shape, dtype, device):
    """A dense tensor of this shape, type and device."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _gpu(t, name):
    if not t.is_cuda:
        raise ValueError(f"the attention and cache calls run on a GPU device; {name} is on the CPU")
    return t.device


def _tokens(t, name, shape, dtype, device) -> int:
    """Check a [tokens, heads, size] tensor whose tokens are contiguous blocks;
    returns the elements between tokens."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    n, h, d = shape
    s = t.stride()
    if n == 0:
        return h * d
    if (d > 1 and s[2] != 1) or (h > 1 and s[1] != d):
        raise ValueError(f"the heads of a token of {name} must be contiguous (strides {s})")
    return s[0] if n > 1 else h * d


def _scale(scale, d_k) -> float:
    return 1.0 / math.sqrt(d_k) if scale is None else float(scale)


def _prompt_args(q, k, v, cu_seqlens):
    """Checks shared by the forward and backward; returns (cu_seqlens, N, T, H_q, H_kv, d_k, d_v, strides, dtype code)."""
    import torch
    dev = q.device
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [tokens, heads, size]")
    T, Hq, dk = q.shape
    Hkv, dv = k.shape[1], v.shape[2]
    code = _dtype_code(q)
    if cu_seqlens is None:
        # made on the device: nothing is copied from the host, so the call can be captured
        cu_seqlens = torch.arange(0, 2 * T, T, dtype=torch.int32, device=dev) if T else torch.zeros(2, dtype=torch.int32, device=dev)
    N = cu_seqlens.shape[0] - 1
    dt = q.dtype
    strides = (_tokens(q, "q", (T, Hq, dk), dt, dev), _tokens(k, "k", (T, Hkv, dk), dt, dev),
               _tokens(v, "v", (T, Hkv, dv), dt, dev))
    _need(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
    return cu_seqlens, N, T, Hq, Hkv, dk, dv, strides, code


def attn_prefill_t(q, k, v, cu_seqlens=None, *, scale=None, o=None, lse=None, stream=None):
    """Causal softmax attention over packed prompts; returns (o, lse).

    q: [T, H_q, d_k]; k: [T, H_kv, d_k]; v: [T, H_kv, d_v] (bf16 or fp32, one
    type; slices of a fused projection are taken as they are); cu_seqlens:
    int32 [N + 1] on the device (None = one sequence); ``scale``: 1 / sqrt(d_k)
    if None.  o: [T, H_q, d_v] in q's dtype; lse: [T, H_q] fp32."""
    return _on_stream(stream, _gpu(q, "q"), _attn_prefill_on, q, k, v, cu_seqlens, scale, o, lse)


def _attn_prefill_on(q, k, v, cu_seqlens, scale, o, lse, stream):
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
    _check(attn_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), N, T, Hq, Hkv, dk, dv,
                        *strides, _scale(scale, dk), code, o.data_ptr(), lse.data_ptr(), stream))
    return o, lse


def _workspace(workspace, need, dev):
    import torch
    if workspace is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    if workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on q's device")
    return workspace


def attn_prefill_backward_t(q, k, v, o, lse, d_o, cu_seqlens=None, *, scale=None, workspace=None, stream=None):
    """Backward of ``attn_prefill_t``: gradients (d_q, d_k, d_v), shaped and
    typed like q, k and v, of a loss given d_o = dL/do and the forward's o and
    lse.  ``workspace``: optional uint8 device tensor of at least
    ``attn_prefill_backward_workspace_size(...)`` bytes."""
    return _on_stream(stream, _gpu(q, "q"), _attn_backward_on, q, k, v, o, lse, d_o, cu_seqlens, scale, workspace)


def _attn_backward_on(q, k, v, o, lse, d_o, cu_seqlens, scale, workspace, stream):
    import torch
    dev = q.device
    cu_seqlens, N, T, Hq, Hkv, dk, dv, strides, code = _prompt_args(q, k, v, cu_seqlens)
    _need(o, "o", (T, Hq, dv), q.dtype, dev)
    _need(lse, "lse", (T, Hq), torch.float32, dev)
    _need(d_o, "d_o", (T, Hq, dv), q.dtype, dev)
    d_q = torch.empty((T, Hq, dk), dtype=q.dtype, device=dev)
    d_k = torch.empty((T, Hkv, dk), dtype=q.dtype, device=dev)
    d_v = torch.empty((T, Hkv, dv), dtype=q.dtype, device=dev)
    ws = _workspace(workspace, attn_prefill_backward_workspace_size(N, T, Hq, Hkv, dk, dv, code), dev)
    _check(attn_prefill_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), d_o.data_ptr(),
                                 cu_seqlens.data_ptr(), N, T, Hq, Hkv, dk, dv, *strides, _scale(scale, dk), code,
                                 d_q.data_ptr(), d_k.data_ptr(), d_v.data_ptr(), ws.data_ptr(), ws.numel(), stream))
    return d_q, d_k, d_v


def attn_tree_masks(parents):
    """The masks of drafted trees: ``parents`` is one list per sequence with
    every token's parent (an earlier token's number in the sequence, or -1 at
    the root); a token sees its ancestors and itself.  Returns an int64 tensor
    [tokens] on the host (bit j: drafted position j), for ``attn_tree_decode_t``."""
    import torch
    masks = []
    for tree in parents:
        if len(tree) > 64:
            raise ValueError(f"a drafted tree holds at most 64 tokens, got {len(tree)}")
        seen = []
        for j, p in enumerate(tree):
            if not -1 <= p < j:
                raise ValueError(f"the parent of token {j} must be an earlier token or -1, got {p}")
            seen.append((1 << j) | (seen[p] if p >= 0 else 0))
        masks += [m - (1 << 64) if m >> 63 else m for m in seen]
    return torch.tensor(masks, dtype=torch.int64)


def _cache_shape(k_cache, v_cache, dtype, device):
    if k_cache.dim() != 4 or v_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must be [n_pages, page_size, H_kv, d]")
    P, ps, Hkv, dk = k_cache.shape
    dv = v_cache.shape[3]
    _need(k_cache, "k_cache", (P, ps, Hkv, dk), dtype, device)
    _need(v_cache, "v_cache", (P, ps, Hkv, dv), dtype, device)
    return P, ps, Hkv, dk, dv


def attn_tree_decode_t(q, k_cache, v_cache, block_table, ctx_lens, cu_q=None, tree_mask=None, *, scale=None, o=None,
                       lse=None, workspace=None, stream=None):
    """Attention of drafted tokens over a paged cache; returns (o, lse).

    q: [T, H_q, d_k]; k_cache: [n_pages, page_size, H_kv, d_k] and v_cache:
    [n_pages, page_size, H_kv, d_v] of q's dtype, which already hold the
    drafted tokens' keys and values behind ctx_lens (``kv_append_t``);
    block_table: int32 [N, max_pages]; ctx_lens: int32 [N]; cu_q: int32
    [N + 1] (None: one token per sequence); tree_mask: int64 [T], bit j of a
    token's mask set if it sees drafted position j (None: the ones up to
    itself; ``attn_tree_masks`` builds it).  ``workspace``: optional uint8
    device tensor of ``attn_tree_decode_workspace_size`` bytes."""
    return _on_stream(stream, _gpu(q, "q"), _attn_tree_on, q, k_cache, v_cache, block_table, ctx_lens, cu_q, tree_mask,
                      scale, o, lse, workspace)


def _attn_tree_on(q, k_cache, v_cache, block_table, ctx_lens, cu_q, tree_mask, scale, o, lse, workspace, stream):
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
    if cu_q is None:
        if T != N:
            raise ValueError(f"without cu_q there is one token per sequence: {T} tokens, {N} sequences")
        cu_q = torch.arange(N + 1, dtype=torch.int32, device=dev)
    qs = _tokens(q, "q", (T, Hq, dk), q.dtype, dev)
    _need(block_table, "block_table", (N, MP), torch.int32, dev)
    _need(ctx_lens, "ctx_lens", (N,), torch.int32, dev)
    _need(cu_q, "cu_q", (N + 1,), torch.int32, dev)
    if tree_mask is not None:
        _need(tree_mask, "tree_mask", (T,), torch.int64, dev)
    if o is None:
        o = torch.empty((T, Hq, dv), dtype=q.dtype, device=dev)
    else:
        _need(o, "o", (T, Hq, dv), q.dtype, dev)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    else:
        _need(lse, "lse", (T, Hq), torch.float32, dev)
    ws = _workspace(workspace, attn_tree_decode_workspace_size(N, T, Hq, Hkv, dv, ps, MP), dev)
    _check(attn_tree_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                            ctx_lens.data_ptr(), cu_q.data_ptr(), tree_mask.data_ptr() if tree_mask is not None else None,
                            N, T, Hq, Hkv, dk, dv, P, ps, MP, qs, _scale(scale, dk), code, o.data_ptr(), lse.data_ptr(),
                            ws.data_ptr(), ws.numel(), stream))
    return o, lse


# ---------------------------------------------------------------------------
# pages of the cache
# ---------------------------------------------------------------------------
@dataclasses.dataclass
class KVPages:
    """The bookkeeping of a paged cache: int32 device tensors, shared by all
    layers (``kv_pages`` makes an empty one).

    table [rows, max_pages]: a row's pages, -1 behind them; lens [rows]: its
    committed positions; held [rows]: its pages; refs [n_pages]: rows that
    hold a page; free [n_pages]: free pages, the first n_free [1] of them."""
    table: Any
    lens: Any
    held: Any
    refs: Any
    free: Any
    n_free: Any
    page_size: int


def kv_pages(n_rows: int, max_pages: int, n_pages: int, page_size: int, device="cuda") -> KVPages:
    """The bookkeeping of an empty cache: every page free, every row unused."""
    import torch
    z = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)  # noqa: E731
    return KVPages(table=z(n_rows, max_pages) - 1, lens=z(n_rows), held=z(n_rows), refs=z(n_pages),
                   free=torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device=device),
                   n_free=z(1) + n_pages, page_size=page_size)


def _pages_args(p: KVPages):
    """Check the six tensors; returns (device, the C calls' leading arguments)."""
    import torch
    t = p.table
    dev = _gpu(t, "table")
    if t.dim() != 2 or p.refs.dim() != 1:
        raise ValueError("table must be [rows, max_pages] and refs [n_pages]")
    (R, MP), P = t.shape, p.refs.shape[0]
    for x, name, shape in ((t, "table", (R, MP)), (p.lens, "lens", (R,)), (p.held, "held", (R,)),
                           (p.refs, "refs", (P,)), (p.free, "free", (P,)), (p.n_free, "n_free", (1,))):
        _need(x, name, shape, torch.int32, dev)
    return dev, (t.data_ptr(), p.lens.data_ptr(), p.held.data_ptr(), p.refs.data_ptr(), p.free.data_ptr(),
                 p.n_free.data_ptr(), R, P, int(p.page_size), MP)


def _requests(dev, **lists):
    import torch
    n = None
    for name, t in lists.items():
        n = t.shape[0] if n is None else n
        _need(t, name, (n,), torch.int32, dev)
    return n


def _layers(k_cache, v_cache, device):
    """(dtype code, n_layers, n_pages, page_size, H_kv, d_k, d_v) of [n_layers, n_pages, page_size,
    H_kv, d] caches ([n_pages, page_size, H_kv, d]: one layer)."""
    if k_cache.dim() not in (4, 5) or v_cache.dim() != k_cache.dim():
        raise ValueError("k_cache and v_cache must both be [n_layers, n_pages, page_size, H_kv, d] or one layer of it")
    shape, dv = k_cache.shape, v_cache.shape[-1]
    _need(k_cache, "k_cache", shape, k_cache.dtype, device)
    _need(v_cache, "v_cache", (*shape[:-1], dv), k_cache.dtype, device)
    return (_dtype_code(k_cache), shape[0] if len(shape) == 5 else 1, *shape[-4:], dv)


def kv_reserve_t(pages: KVPages, rows, n_tokens, *, stream=None):
    """Pages for ``n_tokens[i]`` more positions of row ``rows[i]`` (int32 [n]).
    Returns status int32 [n]: 0 done, 1 no pages left, 2 refused."""
    return _on_stream(stream, _gpu(pages.table, "table"), _kv_reserve_on, pages, rows, n_tokens)


def _kv_reserve_on(pages, rows, n_tokens, stream):
    import torch
    dev, args = _pages_args(pages)
    n = _requests(dev, rows=rows, n_tokens=n_tokens)
    status = torch.empty(n, dtype=torch.int32, device=dev)
    _check(kv_reserve(*args, rows.data_ptr(), n_tokens.data_ptr(), n, status.data_ptr(), stream))
    return status


def kv_free_t(pages: KVPages, rows, *, stream=None) -> None:
    """Rows ``rows`` (int32 [n]) give up their pages and become unused."""
    return _on_stream(stream, _gpu(pages.table, "table"), _kv_free_on, pages, rows)


def _kv_free_on(pages, rows, stream):
    dev, args = _pages_args(pages)
    n = _requests(dev, rows=rows)
    _check(kv_free(*args, rows.data_ptr(), n, stream))


def kv_fork_t(pages: KVPages, src, dst, k_cache, v_cache, *, stream=None):
    """Row ``dst[i]`` (unused) becomes a continuation of row ``src[i]`` (int32
    [n]): full pages shared, the last one copied in every layer of the caches.
    Returns status as ``kv_reserve_t`` does."""
    return _on_stream(stream, _gpu(pages.table, "table"), _kv_fork_on, pages, src, dst, k_cache, v_cache)


def _kv_fork_on(pages, src, dst, k_cache, v_cache, stream):
    import torch
    dev, args = _pages_args(pages)
    n = _requests(dev, src=src, dst=dst)
    code, L, P, ps, Hkv, dk, dv = _layers(k_cache, v_cache, dev)
    if (P, ps) != (args[7], args[8]):
        raise ValueError(f"the caches have {P} pages of {ps} positions, the bookkeeping {args[7]} of {args[8]}")
    status = torch.empty(n, dtype=torch.int32, device=dev)
    _check(kv_fork(*args, src.data_ptr(), dst.data_ptr(), n, k_cache.data_ptr(), v_cache.data_ptr(), L, Hkv, dk, dv, code,
                   status.data_ptr(), stream))
    return status


def kv_append_t(k, v, k_cache, v_cache, block_table, lens, cu_new=None, *, stream=None) -> None:
    """Keys and values of new tokens into the cache: k [n_layers, T, H_kv, d_k]
    and v [n_layers, T, H_kv, d_v] (one layer: [T, H_kv, d] with the caches of
    that layer), token j of sequence n to position lens[n] + j through row n of
    block_table; cu_new int32 [N + 1] (None: one token per sequence).  lens is
    left as it is."""
    return _on_stream(stream, _gpu(k, "k"), _kv_append_on, k, v, k_cache, v_cache, block_table, lens, cu_new)


def _kv_append_on(k, v, k_cache, v_cache, block_table, lens, cu_new, stream):
    import torch
    dev = k.device
    code, L, P, ps, Hkv, dk, dv = _layers(k_cache, v_cache, dev)
    lead = (L,) if k_cache.dim() == 5 else ()
    if k.dim() != 3 + len(lead) or block_table.dim() != 2:
        raise ValueError("k must be [n_layers, T, H_kv, d_k] (one layer: [T, H_kv, d_k]) and block_table [N, max_pages]")
    T, N, MP = k.shape[len(lead)], lens.shape[0], block_table.shape[1]
    if cu_new is None:
        if T != N:
            raise ValueError(f"without cu_new there is one token per sequence: {T} tokens, {N} sequences")
        cu_new = torch.arange(N + 1, dtype=torch.int32, device=dev)
    _need(k, "k", lead + (T, Hkv, dk), k_cache.dtype, dev)
    _need(v, "v", lead + (T, Hkv, dv), k_cache.dtype, dev)
    _need(block_table, "block_table", (N, MP), torch.int32, dev)
    _need(lens, "lens", (N,), torch.int32, dev)
    _need(cu_new, "cu_new", (N + 1,), torch.int32, dev)
    _check(kv_append(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                     lens.data_ptr(), cu_new.data_ptr(), N, T, L, Hkv, dk, dv, P, ps, MP, code, stream))


def kv_compact_t(k_cache, v_cache, block_table, lens, accepted, cu_accepted, *, new_lens=None, stream=None):
    """The accepted drafted tokens of every sequence move together behind its
    committed positions (all layers): ``accepted`` int32 [A], their numbers in
    the draft, rising, packed by ``cu_accepted`` int32 [N + 1].  Returns the
    new lengths, int32 [N]."""
    return _on_stream(stream, _gpu(k_cache, "k_cache"), _kv_compact_on, k_cache, v_cache, block_table, lens, accepted,
                      cu_accepted, new_lens)


def _kv_compact_on(k_cache, v_cache, block_table, lens, accepted, cu_accepted, new_lens, stream):
    import torch
    dev = k_cache.device
    code, L, P, ps, Hkv, dk, dv = _layers(k_cache, v_cache, dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [N, max_pages]")
    N, MP, A = lens.shape[0], block_table.shape[1], accepted.shape[0]
    _need(block_table, "block_table", (N, MP), torch.int32, dev)
    _need(lens, "lens", (N,), torch.int32, dev)
    _need(accepted, "accepted", (A,), torch.int32, dev)
    _need(cu_accepted, "cu_accepted", (N + 1,), torch.int32, dev)
    if new_lens is None:
        new_lens = torch.empty(N, dtype=torch.int32, device=dev)
    else:
        _need(new_lens, "new_lens", (N,), torch.int32, dev)
    _check(kv_compact(k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), lens.data_ptr(),
                      accepted.data_ptr(), cu_accepted.data_ptr(), N, A, L, Hkv, dk, dv, P, ps, MP, code,
                      new_lens.data_ptr(), stream))
    return new_lens
