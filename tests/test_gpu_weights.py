"""Accumulated attention weights against a 64-bit reference."""
import math
import random

import pytest
import torch

import attn_ref
import gated_delta_rule_60_amd as kda
from attn_ref import E24, TINY
from test_gpu_attn_tree import Case as TreeCase

pytestmark = pytest.mark.gpu


def weights_of(q, k, seen, scale, lse=None):
    """One head: (sum over the rows of exp(s - lse), bound) for every key.  A score is off by E (attn_ref);
    lse by E, its sum's n e and four of its own steps; exp2's argument is rounded once more from lse log2 e,
    and the sum over the rows adds n e."""
    s = (q @ k.T) * scale
    x = torch.where(seen, s, -math.inf)
    full = torch.logsumexp(x, -1, keepdim=True) if lse is None else lse[:, None]
    p = torch.where(seen, torch.exp(s - torch.where(torch.isfinite(full), full, 0.0)), 0.0)
    E = 2 * attn_ref._score_error(q, k, s, seen, scale)
    sums = (k.shape[0] + 8) * E24
    off = p * (3 * E + sums + 8 * E24 * full.abs().nan_to_num(0, 0, 0)) * 1.01 + TINY
    value = p.sum(0)
    return value, off.sum(0) + (q.shape[0] + 8) * E24 * value


class Case(TreeCase):
    def __init__(self, ctx, hq, hkv, dk, dv, page, dtype, seed=0):
        super().__init__(ctx, [1] * len(ctx), hq, hkv, dk, dv, page, dtype, seed, tree=None)
        g = torch.Generator().manual_seed(seed + 1)
        self.weights = torch.rand(len(ctx), hkv, self.table.shape[1] * page, generator=g).cuda()

    def call(self, **kw):
        return kda.attn_weighed_decode_t(self.q, self.k, self.v, self.table, self.lens, self.weights, **kw)

    def check_weights(self, before, steps=1, scale=None):
        s = 1 / math.sqrt(self.q.shape[-1]) if scale is None else scale
        k, q, before = self.k.cpu(), self.q.cpu().double(), before.cpu().double()
        value, bound = before.clone(), torch.zeros_like(before)
        for n, at in enumerate(self.rows):
            pg, rw = (torch.tensor(x, dtype=torch.long) for x in zip(*at))
            kn = k[pg, rw].double()
            seen = torch.ones(1, len(at), dtype=torch.bool)
            for h in range(self.hq):
                g = h // (self.hq // self.hkv)
                v, b = weights_of(q[n:n + 1, h], kn[:, g], seen, s)
                value[n, g, :len(at)] += steps * v
                bound[n, g, :len(at)] += steps * b
            bound[n, :, :len(at)] += steps * (self.hq // self.hkv) * E24 * value[n, :, :len(at)]
        attn_ref.check(self.weights, (value, bound + TINY), "weights")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (20, 1), (40, 1), (100, 1)])
def test_decode_head_sizes(dtype, dk, dv, hq, hkv):
    c = Case([70, 0, 133], hq, hkv, dk, dv, 16, dtype, seed=dk + dv)
    before = c.weights.clone()
    c.check()
    c.check_weights(before)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (8, 1), (6, 2), (24, 8), (5, 1), (130, 1)])
def test_decode_head_groups(dtype, hq, hkv):
    c = Case([40, 65, 3], hq, hkv, 32, 64, 32, dtype, seed=hq)
    before = c.weights.clone()
    c.check()
    c.check_weights(before)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 2, 16, 64, 256, 4096])
def test_decode_pages_and_context_lengths(dtype, page):
    c = Case([0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500, 1022, 1023, 1024, 1025], 2, 1, 64, 64, page, dtype, seed=page)
    before = c.weights.clone()
    c.check()
    c.check_weights(before)
    for n, x in enumerate(c.ctx):  # what lies behind the token stays
        assert torch.equal(c.weights[n, :, x + 1:], before[n, :, x + 1:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_long_contexts_and_many_sequences(dtype):
    for ctx, hq, hkv in (([9000, 20, 3000], 8, 2), ([random.Random(1).randrange(200) for _ in range(290)], 2, 1)):
        c = Case(ctx, hq, hkv, 64, 32, 64, dtype, seed=len(ctx))
        before = c.weights.clone()
        c.check()
        c.check_weights(before)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 1e-3])
def test_decode_scales(dtype, scale):
    c = Case([200, 33], 4, 2, 64, 32, 16, dtype, seed=11)
    before = c.weights.clone()
    c.check(scale=scale)
    c.check_weights(before, scale=scale)


def test_decode_without_pages_and_statistics():
    """Positions without a page weigh nothing; lse may be left out; o is attn_tree_decode's."""
    c = Case([60, 40], 4, 2, 64, 64, 16, "bf16", seed=2)
    c.table[0, 1], c.table[1] = -1, -1
    before = c.weights.clone()
    o, lse = c.call()
    tree = kda.attn_tree_decode_t(c.q, c.k, c.v, c.table, c.lens)
    assert torch.equal(o, tree[0]) and torch.equal(lse, tree[1])
    added = c.weights.clone()
    assert torch.equal(added[0, :, 16:32], before[0, :, 16:32]) and torch.equal(added[1], before[1])
    assert (added[0, :, :16] >= before[0, :, :16]).all() and (o[1] == 0).all()
    c.weights.copy_(before)
    o2 = torch.empty_like(o)
    ws = torch.empty(kda.attn_weighed_decode_workspace_size(2, 4, 2, 64, 16, c.table.shape[1]), dtype=torch.uint8, device="cuda")
    assert kda.attn_weighed_decode(
        c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.table.data_ptr(), c.lens.data_ptr(), 2, 4, 2, 64, 64, c.k.shape[0], 16,
        c.table.shape[1], 256, 1 / 8, kda.KDA_DTYPE_BF16, o2.data_ptr(), None, c.weights.data_ptr(), ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream().cuda_stream) == kda.KDA_OK
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(c.weights, added)


def test_decode_a_full_row():
    """ctx at the table's room and past it: the token's own position is not in the cache."""
    c = Case([63, 31], 2, 1, 32, 32, 16, "f32", seed=3)
    c.lens.copy_(torch.tensor([64, 2 ** 31 - 1], dtype=torch.int32))
    o, lse = c.call()
    tree = kda.attn_tree_decode_t(c.q, c.k, c.v, c.table, c.lens)
    assert torch.equal(o[0], tree[0][0]) and torch.equal(lse[0], tree[1][0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_streams_graph_replays_and_the_same_bits(dtype):
    c = Case([300, 2000], 8, 2, 64, 64, 16, dtype, seed=5)
    start = c.weights.clone()
    first = c.call()
    once = c.weights.clone()
    c.weights.copy_(start)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = c.call(stream=side)
    side.synchronize()
    assert torch.equal(once, c.weights) and all(torch.equal(x, y) for x, y in zip(first, second))
    c.weights.copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = c.call()
    c.weights.copy_(start)
    want = start.clone()
    for n in range(4):
        c.lens.copy_(torch.tensor([20 + 90 * n, 5 + 600 * n], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        eager = kda.attn_weighed_decode_t(c.q, c.k, c.v, c.table, c.lens, want)
        torch.cuda.synchronize()
        assert torch.equal(want, c.weights) and all(torch.equal(x, y) for x, y in zip(kept, eager)), f"replay {n}"


def test_decode_refusals():
    c = Case([30], 2, 1, 32, 32, 16, "f32")
    with pytest.raises(ValueError, match="weights must have shape"):
        kda.attn_weighed_decode_t(c.q, c.k, c.v, c.table, c.lens, c.weights[:, :, :-1])
    with pytest.raises(TypeError, match="weights must be"):
        kda.attn_weighed_decode_t(c.q, c.k, c.v, c.table, c.lens, c.weights.double())
    with pytest.raises(ValueError, match="one token per sequence"):
        kda.attn_weighed_decode_t(torch.cat([c.q, c.q]), c.k, c.v, c.table, c.lens, c.weights)
    with pytest.raises(kda.KDAError, match="workspace smaller"):
        c.call(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
