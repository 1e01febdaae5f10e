"""Softmax attention in 64 bits, on the CPU, and how far a kernel may be from
it: bounds worked out element by element from the roundings the kernels make.

u = half a step of the storage type (bf16 2^-8, fp32 2^-24); e = 2^-24.

* a score s = scale q.k is summed in fp32: off by at most
  (d_k + 4) e scale sum |q||k| (the sum's n e, the products, scale, log2 e);
  its difference from the maximum rounds once more, e |s - m|, and the
  hardware's 2^x is off by one step, 2 e.  E: the row's largest such sum,
  twice, since the row's statistic carries the same error.
* p exp'd from it: relative 2 E; rounded to bf16 before the product: u more.
  o = sum p v in fp32: (n + 8) e of sum p |v|, then one rounding u |o|.
* the gradients alike; D = do.o meets the stored o, off by what o may be.
* what lies below the smallest normal number of either type, t = 2^-126, is
  taken for zero on the way: p is off by t more, ds = p (dp - D) by
  t (|dp - D| + 1), and each output by t and what these weigh in its sum.
  (A weight e^-91 met dp - D ~ 1: ds = 2^-131, d_k = -1e-40 came out as 0.)
"""
from __future__ import annotations

import math

import torch

E24 = 2.0 ** -24
TINY = 2.0 ** -126


def half_step(dtype) -> float:
    return float(torch.finfo(dtype).eps) / 2


def _score_error(q, k, s, seen, scale):
    """[L, 1]: E of each row (0 where it sees nothing)."""
    size = (q.abs() @ k.abs().T) * scale
    m = torch.where(seen, s, -math.inf).amax(-1, keepdim=True)
    gap = torch.where(seen, (s - m).abs(), 0.0)
    e = (q.shape[-1] + 4) * E24 * size + 2 * E24 * (gap + m.abs().nan_to_num(0, 0, 0)) + 2 * E24
    return torch.where(seen, e, 0.0).amax(-1, keepdim=True)


def attend(q, k, v, seen, scale, dtype, d_o=None):
    """One head.  q [L, d_k], k [S, d_k], v [S, d_v] (64 bits), seen [L, S].
    Returns a dict of name -> (value, bound); d_q, d_k and d_v too with d_o."""
    u, n = half_step(dtype), k.shape[0]
    up = u if dtype == torch.bfloat16 else 0.0  # what p and ds are rounded to before a product
    some = seen.any(-1, keepdim=True)
    s = (q @ k.T) * scale
    x = torch.where(seen, s, -math.inf)
    lse = torch.logsumexp(x, -1, keepdim=True)
    p = torch.where(seen, torch.exp(s - torch.where(some, lse, 0.0)), 0.0)
    vz = torch.where(seen.any(0)[:, None], v, 0.0) if not torch.isfinite(v).all() else v
    o = p @ vz
    E = 2 * _score_error(q, k, s, seen, scale)
    sums = (n + 8) * E24
    o_bound = (up + 2 * E + sums) * (p @ vz.abs()) * 1.01 + u * o.abs() + TINY * (1 + vz.abs().sum(0))
    out = dict(o=(o, o_bound), lse=(lse[:, 0], (E + sums)[:, 0] + 4 * E24 * lse[:, 0].abs().nan_to_num(0, 0, 0)))
    if d_o is None:
        return out
    sums_q = (q.shape[0] + 8) * E24
    dp, D = d_o @ v.T, (d_o * o).sum(-1, keepdim=True)
    e_dp = (v.shape[-1] + 2) * E24 * (d_o.abs() @ v.abs().T)
    e_D = (d_o.abs() * o_bound).sum(-1, keepdim=True) + (v.shape[-1] + 2) * E24 * (d_o * o).abs().sum(-1, keepdim=True)
    ds = p * (dp - D)
    e_ds = (ds.abs() * (2 * E + up) + p * (e_dp + e_D)) * 1.01 + TINY * ((dp - D).abs() + 1)
    d_q, d_k, d_v = scale * ds @ k, scale * ds.T @ q, p.T @ d_o
    out["d_q"] = (d_q, scale * (e_ds @ k.abs() + sums * (ds.abs() @ k.abs())) + u * d_q.abs() + TINY)
    out["d_k"] = (d_k, scale * (e_ds.T @ q.abs() + sums_q * (ds.abs().T @ q.abs())) + u * d_k.abs() + TINY)
    out["d_v"] = (d_v, (p * (up + 2 * E) + TINY).T @ d_o.abs() * 1.01 + sums_q * (p.T @ d_o.abs()) + u * d_v.abs() + TINY)
    return out


def prefill(q, k, v, lens, scale, d_o=None):
    """Packed causal attention with grouped heads; tensors of any type on any
    device.  Returns name -> (value, bound), laid out like the kernels'."""
    dtype, groups = q.dtype, q.shape[1] // k.shape[1]
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    d_o = None if d_o is None else d_o.detach().cpu().double()
    shape = dict(o=(*q.shape[:2], v.shape[2]), lse=q.shape[:2], d_q=q.shape, d_k=k.shape, d_v=v.shape)
    names = ("o", "lse") if d_o is None else tuple(shape)
    out = {x: (torch.zeros(shape[x], dtype=torch.float64), torch.zeros(shape[x], dtype=torch.float64)) for x in names}
    a = 0
    for n in lens:
        seen = torch.tril(torch.ones(n, n, dtype=torch.bool))
        for h in range(q.shape[1] if n else 0):
            g = h // groups
            r = attend(q[a:a + n, h], k[a:a + n, g], v[a:a + n, g], seen, scale, dtype,
                       None if d_o is None else d_o[a:a + n, h])
            for x in names:
                at = g if x in ("d_k", "d_v") else h  # shared heads: values and bounds add up
                out[x][0][a:a + n, at] += r[x][0]
                out[x][1][a:a + n, at] += r[x][1]
        a += n
    return out


def check(got, want, what=""):
    """got within want's bound everywhere; infinities equal."""
    value, bound = want
    got = got.detach().cpu().double()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    if not value.numel():
        return
    fine = torch.isfinite(value)
    assert torch.equal(got[~fine], value[~fine]), f"{what}: infinite values differ"
    assert torch.isfinite(got[fine]).all(), f"{what}: not finite"
    ratio = ((got - value).abs()[fine] / (bound[fine] + 1e-300)).max() if fine.any() else torch.zeros(())
    print(f"    {what}: at {float(ratio):.3f} of its bound", flush=True)
    assert ratio <= 1, f"{what}: {float(ratio):.3f} times its bound"
