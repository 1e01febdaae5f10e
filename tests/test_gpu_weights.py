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


def test_decode_more_positions_than_workgroups_take_at_once():
    """Many sequences in a wide table: a row's positions go to its workgroups in turns."""
    c = Case([random.Random(2).randrange(60) for _ in range(600)] + [6000, 4095, 4096], 8, 8, 32, 32, 64, "bf16", seed=1)
    before = c.weights.clone()
    c.check()
    c.check_weights(before)
    for n, x in enumerate(c.ctx):
        assert torch.equal(c.weights[n, :, x + 1:], before[n, :, x + 1:])


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


def test_decode_scores_below_the_range_weigh_nothing():
    """Finite queries and keys whose scores pass -2^128, by the product or only by the scale: a row without another
    score has a statistic of -infinity, and weighs nothing."""
    for size, scale in ((1e20, 1 / 8), (1e19, 10.0)):
        c = Case([60, 40], 4, 2, 64, 64, 16, "bf16", seed=4)
        c.q[1, :, 0] = size
        pages = c.table[1][c.table[1] >= 0].long()
        c.k[pages] = 0
        c.k[pages, :, :, 0] = -size
        before = c.weights.clone()
        c.call(scale=scale)
        torch.cuda.synchronize()
        assert torch.equal(c.weights[1], before[1]), f"{size} {scale}"
        assert c.weights[0].isfinite().all()


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


# ---------------------------------------------------------------------------
# prompts
# ---------------------------------------------------------------------------
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _prompt(lens, hq, hkv, dk, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    t = sum(lens)
    q, k = ((spread * torch.randn(t, h, dk, generator=g)).to(DT[dtype]).cuda() for h in (hq, hkv))
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32).cuda()
    # the row statistics, rounded from 64 bits
    lse = torch.zeros(t, hq, dtype=torch.float64)
    a = 0
    for n in lens:
        for h in range(hq if n else 0):
            s = q[a:a + n, h].cpu().double() @ k[a:a + n, h // (hq // hkv)].cpu().double().T / math.sqrt(dk)
            lse[a:a + n, h] = torch.logsumexp(torch.where(torch.ones(n, n).tril() > 0, s, -math.inf), -1)
        a += n
    return q, k, lse.float().cuda(), cu


def _check_prompt(lens, hq, hkv, dk, dtype, rows=None, width=None, seed=0, spread=1.0):
    q, k, lse, cu = _prompt(lens, hq, hkv, dk, dtype, seed, spread)
    width = max(lens) + 3 if width is None else width
    weights = torch.full((len(lens), hkv, width), float("nan"), device="cuda")
    assert kda.attn_prefill_weights_t(q, k, lse, cu, weights=weights, rows=rows) is weights
    torch.cuda.synchronize()
    value, bound = (torch.zeros(len(lens), hkv, width, dtype=torch.float64) for _ in range(2))
    a = 0
    for n, length in enumerate(lens):
        first = 0 if rows is None else max(0, length - rows)
        seen = torch.ones(length, length, dtype=torch.bool).tril()[first:]
        for h in range(hq if length else 0):
            g = h // (hq // hkv)
            v, b = weights_of(q[a + first:a + length, h].cpu().double(), k[a:a + length, g].cpu().double(), seen,
                              1 / math.sqrt(dk), lse[a + first:a + length, h].cpu().double())
            m = min(length, width)
            value[n, g, :m] += v[:m]
            bound[n, g, :m] += b[:m]
        # the heads of a group are summed on
        bound[n] += (hq // hkv) * E24 * value[n]
        a += length
    attn_ref.check(weights, (value, bound), f"{dtype} weights")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (5, 1), (9, 3)])
def test_prompt_head_sizes_and_groups(dtype, dk, hq, hkv):
    _check_prompt([70, 331], hq, hkv, dk, dtype, seed=dk + hq)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [2], [31, 32, 33], [63, 64, 65], [127, 128, 129], [1, 0, 0, 5, 1], [0, 300, 0],
                                  [255, 256, 257, 513], [1] * 70, [3, 130] * 40])
@pytest.mark.parametrize("rows", [1, 17, 32, 64, 100, None])
def test_prompt_lengths_and_rows(dtype, lens, rows):
    _check_prompt(lens, 2, 1, 64, dtype, rows=rows, seed=len(lens))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [1, 100, 256, 257, 1024, 5000])
def test_prompt_widths(dtype, width):
    """Narrower than a sequence: what lies past it is left out."""
    _check_prompt([300, 1, 700], 2, 2, 32, dtype, width=width, seed=width)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_longer_sequences(dtype):
    _check_prompt([2100, 777], 4, 2, 128, dtype, seed=5)
    _check_prompt([2100, 777], 8, 1, 128, dtype, rows=64, seed=6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_peaked_rows(dtype):
    _check_prompt([200, 33], 2, 2, 64, dtype, seed=11, spread=3.0)


def test_prompt_every_row_gives_one():
    """All rows: a row's weights sum to one, so the positions' sum to the rows times heads of the group."""
    q, k, lse, cu = _prompt([400], 6, 2, 64, "f32", 3)
    w = kda.attn_prefill_weights_t(q, k, lse, cu, weights=torch.empty(1, 2, 400, device="cuda"))
    assert ((w.double().sum(-1) - 3 * 400).abs() < 1200 * (400 + 400 + 64) * 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_from_the_passes_own_statistics(dtype):
    lens = [200, 61]
    q, k, lse, cu = _prompt(lens, 4, 2, 64, dtype, 8)
    _, own = kda.attn_prefill_t(q, k, k, cu)
    a, b = (kda.attn_prefill_weights_t(q, k, x, cu, weights=torch.empty(2, 2, 200, device="cuda")) for x in (lse, own))
    torch.cuda.synchronize()
    # either lse is within 64 + 200 + 8 roundings of exact, twice
    assert ((a - b).abs() <= 2 * (64 + 200 + 8 + 40) * 2.0 ** -24 * 2 * (a + 1e-30)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_padding_neighbours_and_later_tokens(dtype):
    q, k, lse, cu = _prompt([170, 50, 190], 2, 1, 64, dtype, 13)
    call = lambda: kda.attn_prefill_weights_t(q, k, lse, cu, weights=torch.full((3, 1, 256), 7.0, device="cuda"))  # noqa: E731
    want = call()
    q[170:220], k[170:220], lse[170:220] = float("nan"), float("inf"), float("nan")
    got = call()
    assert torch.equal(got[[0, 2]], want[[0, 2]]) and (got[1, :, 50:] == 0).all()
    # a key that is not finite: the others of its sequence keep theirs
    k[100, 0, 3] = float("nan")
    got = call()
    keep = [j for j in range(256) if j != 100]
    assert torch.equal(got[0][:, keep], want[0][:, keep]) and torch.isnan(got[0][:, 100]).all()
    # rows past the last sequence do not count, whatever they hold
    cu2 = torch.tensor([0, 170], dtype=torch.int32).cuda()
    lse[170:], q[170:] = float("nan"), float("inf")
    k[100, 0, 3] = 0.5
    w1 = kda.attn_prefill_weights_t(q, k, lse, cu2, weights=torch.empty(1, 1, 256, device="cuda"))
    w2 = kda.attn_prefill_weights_t(q[:170], k[:170], lse[:170], weights=torch.empty(1, 1, 256, device="cuda"))
    torch.cuda.synchronize()
    value, bound = torch.zeros(1, 256, dtype=torch.float64), torch.zeros(1, 256, dtype=torch.float64)
    for h in range(2):
        x, y = weights_of(q[:170, h].cpu().double(), k[:170, 0].cpu().double(), torch.ones(170, 170, dtype=torch.bool).tril(), 1 / 8,
                          lse[:170, h].cpu().double())
        value[0, :170] += x
        bound[0, :170] += y + 2 * E24 * x
    for w in (w1, w2):
        attn_ref.check(w[0], (value, bound), "weights")


def test_prompt_streams_graph_replays_slices_and_the_same_bits():
    fused = torch.randn(500, 8 * 64, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    q, k = fused[:, :256].view(500, 4, 64), fused[:, 256:384].view(500, 2, 64)
    cu = torch.tensor([0, 330, 500], dtype=torch.int32).cuda()
    _, lse = kda.attn_prefill_t(q, k, k, cu)
    call = lambda **kw: kda.attn_prefill_weights_t(q, k, lse, cu, weights=torch.empty(2, 2, 400, device="cuda"), **kw)  # noqa: E731
    want = call()
    assert torch.equal(want, kda.attn_prefill_weights_t(q.contiguous(), k.contiguous(), lse, cu, weights=torch.empty(2, 2, 400, device="cuda")))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(stream=side)
    side.synchronize()
    assert torch.equal(want, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = call(rows=50)
    for n in range(3):
        lse.add_(0.5 * n)
        kept.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, call(rows=50)), f"replay {n}"


def test_prompt_no_tokens():
    q, k = (torch.empty(0, h, 64, device="cuda") for h in (4, 2))
    w = kda.attn_prefill_weights_t(q, k, torch.empty(0, 4, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"),
                                   weights=torch.full((2, 2, 300), 7.0, device="cuda"))
    torch.cuda.synchronize()
    assert (w == 0).all()


def test_prompt_no_tokens_in_a_wide_table():
    q, k = (torch.empty(0, h, 64, device="cuda") for h in (4, 2))
    w = kda.attn_prefill_weights_t(q, k, torch.empty(0, 4, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"),
                                   weights=torch.full((2, 2, 50000), 7.0, device="cuda"))
    torch.cuda.synchronize()
    assert (w == 0).all()


def test_prompt_offsets_past_32_bits():
    stride, t = 1 << 16, 33000
    fused = torch.zeros(t, stride, dtype=torch.bfloat16, device="cuda")
    fused[:, :384] = torch.randn(t, 384, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    q, k = fused[:, :256].view(t, 2, 128), fused[:, 256:384].view(t, 1, 128)
    lse = torch.full((t, 2), 5.0, device="cuda")
    cu = torch.tensor([0, 32800, 33000], dtype=torch.int32).cuda()
    w = kda.attn_prefill_weights_t(q, k, lse, cu, weights=torch.empty(2, 1, 256, device="cuda"))
    torch.cuda.synchronize()
    value, bound = torch.zeros(1, 256, dtype=torch.float64), torch.zeros(1, 256, dtype=torch.float64)
    for h in range(2):
        x, y = weights_of(q[32800:, h].cpu().double(), k[32800:, 0].cpu().double(), torch.ones(200, 200, dtype=torch.bool).tril(),
                          1 / math.sqrt(128), lse[32800:, h].cpu().double())
        value[0, :200] += x
        bound[0, :200] += y + 2 * E24 * x
    attn_ref.check(w[1], (value, bound), "weights")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size,scale", [(1e20, 1 / 8), (1e19, 10.0)])
def test_prompt_scores_below_the_range_weigh_nothing(dtype, size, scale):
    """The first keys' scores pass -2^128, by the product or only by the scale: their rows have a statistic of
    -infinity and weigh nothing, and the later rows do not see them."""
    gone, n = 100, 300
    g = torch.Generator().manual_seed(12)
    q, k, v = (0.1 * torch.randn(n, h, 64, generator=g) for h in (2, 1, 1))
    q[:, :, 0], k[:gone, :, 0], k[gone:, :, 0] = size, -size, 0.0
    q, k, v = (x.to(DT[dtype]).cuda() for x in (q, k, v))
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    _, lse = kda.attn_prefill_t(q, k, v, cu, scale=scale)
    w = kda.attn_prefill_weights_t(q, k, lse, cu, weights=torch.empty(1, 1, n, device="cuda"), scale=scale)
    torch.cuda.synchronize()
    assert (lse[:gone] == -math.inf).all() and (w[0, 0, :gone] == 0).all()
    value, bound = torch.zeros(n - gone, dtype=torch.float64), torch.zeros(n - gone, dtype=torch.float64)
    for h in range(2):
        x, y = weights_of(q[gone:, h].cpu().double(), k[gone:, 0].cpu().double(), torch.ones(n - gone, n - gone, dtype=torch.bool).tril(), scale)
        value += x
        bound += y + 2 * E24 * x
    attn_ref.check(w[0, 0, gone:], (value, bound), "weights")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 63, 350, 640, 699])
@pytest.mark.parametrize("lens", [[700, 40], [700, 40] + [64] * 150])
def test_prompt_rows_that_are_not_a_number(dtype, at, lens):
    """A NaN query: every key that its row sees is NaN, and the later ones and the other sequences keep their bits.
    A NaN key: the rows from its own on are NaN, and with them every key of the sequence.  (A statistic of NaN
    read as the lowest finite number gave keys an infinite weight, the heaviest.)"""
    g = torch.Generator().manual_seed(at)
    q, k = (torch.randn(sum(lens), h, 64, generator=g).to(DT[dtype]).cuda() for h in (2, 1))
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32).cuda()

    def call(q, k):
        _, lse = kda.attn_prefill_t(q, k, k, cu)
        return kda.attn_prefill_weights_t(q, k, lse, cu, weights=torch.empty(len(lens), 1, 700, device="cuda")), lse

    want, _ = call(q, k)
    q2, k2 = q.clone(), k.clone()
    q2[at, 1, 5] = k2[at, 0, 5] = float("nan")
    got, lse = call(q2, k)
    torch.cuda.synchronize()
    assert torch.isnan(lse[at, 1]) and torch.isnan(lse).sum() == 1
    assert torch.isnan(got[0, 0, :at + 1]).all()
    assert torch.equal(got[0, 0, at + 1:], want[0, 0, at + 1:]) and torch.equal(got[1:], want[1:])
    got, lse = call(q, k2)
    torch.cuda.synchronize()
    assert torch.isnan(lse[at:700]).all() and not torch.isnan(lse[:at]).any()
    assert torch.isnan(got[0, 0]).all() and torch.equal(got[1:], want[1:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 100, 300])
def test_decode_rows_that_are_not_a_number(dtype, at):
    """A NaN key or query: NaN for every position that the row sees, as for a prompt's; the positions behind it, the
    other sequences and key heads keep theirs."""
    c = Case([300, 40], 4, 2, 64, 32, 16, dtype, seed=9)
    before = c.weights.clone()
    c.call()
    want = c.weights.clone()
    k, q = c.k.clone(), c.q.clone()
    page, row = c.rows[0][at]
    for poison in ("key", "query"):
        c.k.copy_(k), c.q.copy_(q), c.weights.copy_(before)
        if poison == "key":
            c.k[page, row, 1, 7] = float("nan")
        else:
            c.q[0, 3, 7] = float("nan")
        c.call()
        torch.cuda.synchronize()
        assert torch.isnan(c.weights[0, 1, :301]).all(), poison
        assert torch.equal(c.weights[0, 1, 301:], before[0, 1, 301:])
        assert torch.equal(c.weights[0, 0], want[0, 0]) and torch.equal(c.weights[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_keys_of_minus_infinity_weigh_nothing(dtype):
    """A key whose scores are all -infinity (an infinite element that every query meets with a positive one)."""
    n, at = 300, 100
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn(n, h, 64, generator=g).to(DT[dtype]).cuda() for h in (2, 1))
    q[:, :, 5], k[at, 0, 5] = 1.0, -math.inf
    _, lse = kda.attn_prefill_t(q, k, k[..., 32:].contiguous())
    w = kda.attn_prefill_weights_t(q, k, lse, weights=torch.empty(1, 1, n, device="cuda"))
    c = Case([n], 2, 1, 64, 32, 16, dtype, seed=4)
    c.weights.zero_()
    c.q[..., 5] = 1.0
    page, row = c.rows[0][at]
    c.k[page, row, 0, 5] = -math.inf
    c.call()
    torch.cuda.synchronize()
    for x, m in ((w, n), (c.weights, n + 1)):
        assert x[0, 0, at] == 0 and x[0, 0, :m].isfinite().all()
        assert (x[0, 0, :m] > 0).sum() == m - 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [200, 700, 2100, 70001])
@pytest.mark.parametrize("rows", [17, None])
def test_prompt_tables_of_many_sequences(dtype, width, rows):
    """All rows (in parts) and few, more sequences than a look-up's round, and a table narrower and much wider than they
    are."""
    lens = [40] * 70 + [0, 1, 2100, 300]
    assert (kda.attn_prefill_weights_workspace_size(len(lens), sum(lens), 8, 2, rows or sum(lens)) > 0) == (rows is None)
    _check_prompt(lens, 8, 2, 64, dtype, rows=rows, width=width, seed=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [1, 255, 4095, 4096, 4097, 8193, 12289])
@pytest.mark.parametrize("before", [0, 30])
def test_prompt_a_wide_table_is_zero_behind_its_sequences(dtype, width, before):
    """Written in full, whatever stood there; rows before the first sequence do not count."""
    lens = [256, 257, 0, 40, 511]
    q, k, lse, _ = _prompt([before] + lens, 4, 2, 32, dtype, width)
    cu = torch.tensor([before, *(before + torch.tensor(lens).cumsum(0)).tolist()], dtype=torch.int32).cuda()
    guard = torch.full((5 * 2 * width + 2 * 64,), 7.0, device="cuda")
    w = guard[64:-64].view(5, 2, width)
    w.fill_(float("nan"))
    kda.attn_prefill_weights_t(q, k, lse, cu, weights=w, rows=9)
    torch.cuda.synchronize()
    assert (guard[:64] == 7).all() and (guard[-64:] == 7).all()
    for n, length in enumerate(lens):
        m = min(length, width)
        assert (w[n, :, m:] == 0).all() and (w[n, :, :m] > 0).all()


def test_prompt_more_rows_than_there_are():
    """All of them, whatever the number."""
    q, k, lse, cu = _prompt([300, 40], 4, 2, 64, "bf16", 3)
    call = lambda **kw: kda.attn_prefill_weights_t(q, k, lse, cu, weights=torch.empty(2, 2, 320, device="cuda"), **kw)  # noqa: E731
    want = call()
    for rows in (340, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 7, 10 ** 15):
        assert torch.equal(call(rows=rows), want), rows


def test_prompt_parts_at_once_and_replayed():
    """A long prompt's rows go to several workgroups, with a workspace: two calls at once, and replays."""
    q, k, v = (torch.randn(4096, h, 64, generator=torch.Generator().manual_seed(h)).bfloat16().cuda() for h in (8, 2, 3))
    v = v[:, :2].contiguous()
    cu = torch.tensor([0, 4000, 4096], dtype=torch.int32).cuda()
    assert kda.attn_prefill_weights_workspace_size(2, 4096, 8, 2, 4096) > 0
    _, lse = kda.attn_prefill_t(q, k, v, cu)
    call = lambda rows, **kw: kda.attn_prefill_weights_t(q, k, lse, cu, weights=torch.empty(2, 2, 4096, device="cuda"), rows=rows, **kw)  # noqa: E731
    want = [call(rows) for rows in (None, 3000)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(4):
        for i, rows in enumerate((None, 3000)):
            got[i].append(call(rows, stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = call(None)
    for n in range(3):
        lse.add_(0.25 * n)
        kept.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, call(None)), f"replay {n}"


def test_prompt_refusals():
    q, k, lse, cu = _prompt([20], 4, 2, 32, "f32", 1)
    w = torch.empty(1, 2, 32, device="cuda")
    with pytest.raises(ValueError, match="lse must have shape"):
        kda.attn_prefill_weights_t(q, k, lse[:10], cu, weights=w)
    with pytest.raises(ValueError, match="weights must have shape"):
        kda.attn_prefill_weights_t(q, k, lse, cu, weights=torch.empty(2, 2, 32, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        kda.attn_prefill_weights_t(q, k, lse, cu, weights=w[..., :20])
    with pytest.raises(kda.KDAError, match="rows"):
        kda.attn_prefill_weights_t(q, k, lse, cu, weights=w, rows=0)
