"""Windowed attention in 64 bits with bounds for every element: the reference
of tests/attn_ref.py over the pairs that a window and sinks leave."""
from __future__ import annotations

import torch

import attn_ref


def seen(n, window, sinks, first=0):
    """[n - first, n]: whether row first + i of a sequence sees key j."""
    i, j = torch.arange(first, n)[:, None], torch.arange(n)[None]
    return (j <= i) & ((i - j < window) | (j < sinks))


def prefill(q, k, v, lens, window, sinks, scale, d_o=None):
    """As attn_ref.prefill.  Keys that no row of a head sees do not count."""
    dtype, groups = q.dtype, q.shape[1] // k.shape[1]
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    d_o = None if d_o is None else d_o.detach().cpu().double()
    shape = dict(o=(*q.shape[:2], v.shape[2]), lse=q.shape[:2], d_q=q.shape, d_k=k.shape, d_v=v.shape)
    names = ("o", "lse") if d_o is None else tuple(shape)
    out = {x: (torch.zeros(shape[x], dtype=torch.float64), torch.zeros(shape[x], dtype=torch.float64)) for x in names}
    a = 0
    for n in lens:
        mask = seen(n, window, sinks)
        for h in range(q.shape[1] if n else 0):
            g = h // groups
            r = attn_ref.attend(q[a:a + n, h], k[a:a + n, g], v[a:a + n, g], mask, scale, dtype,
                                None if d_o is None else d_o[a:a + n, h])
            for x in names:
                at = g if x in ("d_k", "d_v") else h  # shared heads: values and bounds add up
                out[x][0][a:a + n, at] += r[x][0]
                out[x][1][a:a + n, at] += r[x][1]
        a += n
    return out
