"""Attention of drafted tokens over a paged cache against a 64-bit reference."""
import math
import random

import pytest
import torch

import attn_ref
import gated_delta_rule_60_amd as kda

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Case:
    """A cache with shuffled pages, drafted tokens and their trees.  What no
    row may read (rest of the last pages, unused pages) is NaN."""

    def __init__(self, ctx, draft, hq, hkv, dk, dv, page, dtype, seed=0, tree="random", spare=3):
        rng = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.draft, self.page, self.hq, self.hkv = ctx, draft, page, hq, hkv
        t = sum(draft)
        need = [-(-(a + d) // page) for a, d in zip(ctx, draft)]
        total, wide = sum(need) + spare, max(max(need), 1)
        ids = list(range(total))
        rng.shuffle(ids)
        self.rows = []  # (page, row) of each sequence's positions
        table = torch.full((len(ctx), wide), -1, dtype=torch.int32)
        k = torch.full((total, page, hkv, dk), float("nan"))
        v = torch.full((total, page, hkv, dv), float("nan"))
        for n, m in enumerate(need):
            mine = [ids.pop() for _ in range(m)]
            table[n, :m] = torch.tensor(mine, dtype=torch.int32)
            length = ctx[n] + draft[n]
            at = [(mine[p // page], p % page) for p in range(length)]
            self.rows.append(at)
            if length:
                pg, rw = (torch.tensor(x) for x in zip(*at))
                k[pg, rw] = torch.randn(length, hkv, dk, generator=g)
                v[pg, rw] = torch.randn(length, hkv, dv, generator=g)
        self.q = torch.randn(t, hq, dk, generator=g).to(DT[dtype]).cuda()
        self.k, self.v = k.to(DT[dtype]).cuda(), v.to(DT[dtype]).cuda()
        self.table = table.cuda()
        self.lens = torch.tensor(ctx, dtype=torch.int32).cuda()
        self.cu = torch.tensor([0] + torch.tensor(draft).cumsum(0).tolist(), dtype=torch.int32).cuda()
        parents = [[(j - 1 if tree == "chain" else rng.randrange(-1, j)) for j in range(d)] for d in draft]
        self.mask = None if tree is None else kda.attn_tree_masks(parents).cuda()

    def call(self, **kw):
        return kda.attn_tree_decode_t(self.q, self.k, self.v, self.table, self.lens, self.cu, self.mask, **kw)

    def want(self, scale=None, gone=()):
        """gone: (sequence, position) pairs that no row sees."""
        t, hq, dv = self.q.shape[0], self.hq, self.v.shape[-1]
        out = {"o": (torch.zeros(t, hq, dv, dtype=torch.float64), torch.zeros(t, hq, dv, dtype=torch.float64)),
               "lse": (torch.zeros(t, hq, dtype=torch.float64), torch.zeros(t, hq, dtype=torch.float64))}
        s = 1 / math.sqrt(self.q.shape[-1]) if scale is None else scale
        k, v, q = self.k.cpu(), self.v.cpu(), self.q.cpu().double()
        mask = None if self.mask is None else [m & ((1 << 64) - 1) for m in self.mask.tolist()]
        a = 0
        for n, d in enumerate(self.draft):
            length = len(self.rows[n])
            if d == 0:
                continue
            pg, rw = (torch.tensor(x, dtype=torch.long) for x in zip(*self.rows[n]))
            kn, vn = k[pg, rw].double(), v[pg, rw].double()
            seen = torch.zeros(d, length, dtype=torch.bool)
            seen[:, :self.ctx[n]] = True
            for t_ in range(d):
                for j in range(d):
                    seen[t_, self.ctx[n] + j] = j <= t_ if mask is None else j < 64 and (mask[a + t_] >> j) & 1 == 1
            for m, p in gone:
                if m == n:
                    seen[:, p] = False
            kn, vn = (torch.where(torch.isfinite(x), x, 0.0) for x in (kn, vn))
            for h in range(hq):
                g = h // (hq // self.hkv)
                r = attn_ref.attend(q[a:a + d, h], kn[:, g], vn[:, g], seen, s, self.q.dtype)
                for name in out:
                    out[name][0][a:a + d, h] = r[name][0]
                    out[name][1][a:a + d, h] = r[name][1]
            a += d
        return out

    def check(self, got=None, **kw):
        o, lse = self.call(scale=kw.get("scale")) if got is None else got
        torch.cuda.synchronize()
        want = self.want(**kw)
        attn_ref.check(o, want["o"], "o")
        attn_ref.check(lse, want["lse"], "lse")


# rows of a key head: up to 16, 32, 64 and 128 a pass, and several passes
DRAFTS = [[1, 1, 1], [8, 5, 11], [16, 2, 25], [64, 40, 33]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("draft", DRAFTS)
def test_head_sizes(dtype, dk, dv, draft):
    Case([70, 0, 133], draft, 4, 2, dk, dv, 16, dtype, seed=dk + dv).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (8, 1), (6, 2), (24, 8), (5, 1)])
def test_head_groups(dtype, hq, hkv):
    Case([40, 65, 3], [1, 5, 64], hq, hkv, 32, 64, 32, dtype, seed=hq).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 2, 16, 64, 256, 4096])
@pytest.mark.parametrize("tree", ["random", "chain", None])
def test_pages_and_context_lengths(dtype, page, tree):
    ctx = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500]
    Case(ctx, [1 + i % 3 for i in range(len(ctx))], 2, 1, 64, 64, page, dtype, seed=page, tree=tree).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("draft", DRAFTS)
def test_long_contexts_are_cut_and_joined(dtype, draft):
    Case([9000, 20, 4100], draft, 4, 1, 64, 32, 64, dtype, seed=3).check()


# chunks: one a compute unit (made larger until they fit), two, four; joined by one group of threads
# a row or by eight
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ctx,hq,hkv", [
    ([3000], 4, 1), ([2600, 3100], 2, 1), ([5000], 8, 4), ([700 + 611 * n for n in range(7)], 8, 8),
    ([90 + 377 * n % 1500 for n in range(24)], 8, 8), ([64 * n for n in range(17)], 64, 64),
])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_chunks_of_few_and_many_sequences(dtype, ctx, hq, hkv, dv):
    Case(ctx, [1 + n % 3 for n in range(len(ctx))], hq, hkv, 32, dv, 16, dtype, seed=dv).check()


def test_many_sequences():
    rng = random.Random(1)
    ctx = [rng.randrange(0, 700) for _ in range(150)]
    Case(ctx, [rng.choice([0, 1, 1, 2]) for _ in ctx], 4, 2, 32, 32, 16, "bf16", seed=8).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_chain_longer_than_a_mask(dtype):
    """Without a mask any number of tokens: a piece of a prompt over its cached beginning."""
    Case([37, 300], [150, 70], 2, 1, 64, 64, 16, dtype, tree=None).check()


def test_the_chain_is_causal_attention():
    c = Case([0, 0], [60, 64], 4, 2, 64, 64, 32, "bf16", tree=None)
    o, lse = c.call()
    k, v = (torch.cat([x[tuple(torch.tensor(i) for i in zip(*r))] for r in c.rows]) for x in (c.k, c.v))
    o2, lse2 = kda.attn_prefill_t(c.q, k, v, c.cu)
    assert (o.float() - o2.float()).abs().max() <= 2 ** -6 * o2.float().abs().max()
    assert (lse - lse2).abs().max() <= 2 ** -18


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing(dtype):
    c = Case([0, 10, 0], [20, 3, 2], 2, 1, 32, 32, 16, dtype)
    c.mask[0] = 0
    c.mask[7] = 0
    c.mask[23] = 0
    o, lse = c.call()
    for t in (0, 7, 23):
        assert (o[t] == 0).all() and (lse[t] == -math.inf).all()
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_mask_bits_behind_the_draft_count_as_clear(dtype):
    c = Case([5, 30], [3, 64], 2, 1, 32, 64, 16, dtype)
    want = c.call()
    c.mask[:3] |= ~7
    got = c.call()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.mask[:] = -1  # everything there is
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("draft", [[1, 2], [6, 12], [20, 30], [64, 50]])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_drafted_values_that_a_row_does_not_see(dtype, draft, bad):
    """A drafted key or value that is not finite reaches the rows that see it, and no other."""
    c = Case([33, 100], draft, 4, 2, 64, 64, 16, dtype, seed=5)
    want = c.call()
    a, j = draft[0], draft[1] - 1  # the second sequence, its last token
    pg, rw = c.rows[1][100 + j]
    sees = torch.tensor([(m >> j) & 1 == 1 for m in c.mask.tolist()]).cuda()
    sees[:a] = False
    assert sees.any()
    v = c.v.clone()
    c.v[pg, rw, 1, 5] = bad
    o, lse = c.call()
    assert torch.equal(lse, want[1]) and torch.equal(o[~sees], want[0][~sees])
    assert torch.equal(o[:, :2], want[0][:, :2])
    hit = o[sees][:, 2:, 5].float()
    assert torch.isnan(hit).all() if bad != bad else (hit == bad).all()
    rest = [i for i in range(64) if i != 5]
    assert torch.equal(o[..., rest], want[0][..., rest])
    c.v = v
    c.k[pg, rw, 1, 5] = bad
    o, lse = c.call()
    assert torch.equal(o[~sees], want[0][~sees]) and torch.equal(lse[~sees], want[1][~sees])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_committed_values_reach_every_row(dtype):
    c = Case([100, 60], [5, 30], 2, 1, 64, 64, 16, dtype)
    for p in (0, 40, 98):
        v = c.v.clone()
        pg, rw = c.rows[0][p]
        c.v[pg, rw, 0, 3] = float("nan")
        o, _ = c.call()
        assert torch.isnan(o[:5, :, 3]).all() and torch.isfinite(o[5:]).all()
        c.v = v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("draft", [[1, 1], [40, 40]])
def test_positions_without_a_page_are_not_seen(dtype, draft):
    c = Case([90, 70], draft, 2, 1, 64, 32, 16, dtype, seed=2)
    for entry in (-1, -2 ** 31, c.k.shape[0], 2 ** 31 - 1):
        t = c.table.clone()
        c.table[0, 2] = entry
        c.check(gone=[(0, p) for p in range(32, 48)])
        c.table = t


def test_lengths_outside_the_table_are_clamped():
    c = Case([30, 16], [2, 1], 2, 1, 32, 32, 16, "bf16", tree=None)
    want = c.call()
    c.lens[0] = 10 ** 9  # all positions of the table: here its two pages
    o, lse = c.call()
    torch.cuda.synchronize()
    assert torch.equal(o[2], want[0][2]) and torch.isfinite(o).all()
    c.lens[0] = -5
    o, lse = c.call()
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_last_token_stay(dtype):
    c = Case([20, 300], [3, 2], 2, 1, 64, 64, 16, dtype)
    q = torch.cat([c.q, torch.full((4, 2, 64), float("nan"), dtype=c.q.dtype, device="cuda")])
    mask = torch.cat([c.mask, torch.full((4,), -1, device="cuda")])
    o = torch.full((9, 2, 64), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((9, 2), 7.0, device="cuda")
    kda.attn_tree_decode_t(q, c.k, c.v, c.table, c.lens, c.cu, mask, o=o, lse=lse)
    assert (o[5:] == 7).all() and (lse[5:] == 7).all()
    c.check(got=(o[:5], lse[:5]))


def test_one_token_a_sequence_needs_no_offsets():
    c = Case([20, 300, 0], [1, 1, 1], 4, 2, 64, 64, 16, "bf16", tree=None)
    o, lse = c.call()
    o2, lse2 = kda.attn_tree_decode_t(c.q, c.k, c.v, c.table, c.lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    c.check()


def test_queries_as_a_slice():
    c = Case([20, 300], [3, 9], 4, 2, 64, 64, 16, "bf16")
    want = c.call()
    wide = torch.randn(12, 8, 64, device="cuda").bfloat16()
    wide[:, 2:6] = c.q
    o, lse = kda.attn_tree_decode_t(wide[:, 2:6], c.k, c.v, c.table, c.lens, c.cu, c.mask)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("draft", DRAFTS)
def test_streams_and_replays_while_the_sequences_grow(dtype, draft):
    c = Case([3000, 1500, 100], draft, 4, 2, 64, 64, 32, dtype, tree=None)
    want = c.call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.call(stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = c.call()
    for n in range(4):
        o.fill_(float("nan"))
        lse.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        o2, lse2 = c.call()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2), f"replay {n}"
        c.lens -= torch.tensor([700, 333, 25], dtype=torch.int32).cuda()  # other lengths, same launch


def test_two_calls_at_once_with_their_own_workspaces():
    a = Case([5000, 900], [1, 1], 8, 2, 64, 64, 32, "bf16", seed=1)
    b = Case([4000, 7000], [9, 4], 8, 2, 64, 64, 32, "bf16", seed=2)
    wa, wb = a.call(), b.call()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ga, gb = [], []
    for _ in range(5):
        ga.append(a.call(stream=s1))
        gb.append(b.call(stream=s2))
    torch.cuda.synchronize()
    assert all(torch.equal(x[0], wa[0]) and torch.equal(x[1], wa[1]) for x in ga)
    assert all(torch.equal(x[0], wb[0]) and torch.equal(x[1], wb[1]) for x in gb)


def test_offsets_past_32_bits():
    """Pages 2^31 elements and more into the cache."""
    pages, page, hkv, d = 33000, 64, 8, 128  # 2.16e9 elements, 4.3 GB
    k = torch.zeros(pages, page, hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    for x in (k, v):
        x[-4:] = torch.randn(4, page, hkv, d, generator=g, device="cuda")
    q = torch.randn(2, 16, d, generator=g, device="cuda").bfloat16()
    table = torch.tensor([[pages - 2, pages - 4, pages - 1, pages - 3]], dtype=torch.int32).cuda()
    lens, cu = torch.tensor([200], dtype=torch.int32).cuda(), torch.tensor([0, 2], dtype=torch.int32).cuda()
    o, lse = kda.attn_tree_decode_t(q, k, v, table, lens, cu)
    small = torch.tensor([[2, 0, 3, 1]], dtype=torch.int32).cuda()
    o2, lse2 = kda.attn_tree_decode_t(q, k[-4:].clone(), v[-4:].clone(), small, lens, cu)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.isfinite(o).all() and (o != 0).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("draft", [[2, 1], [9, 5], [40, 30]])
def test_clamped_lengths_are_those_of_the_table(dtype, draft):
    """A length past the table is all its positions, with no drafted one behind them; a negative one is
    zero, and the drafted tokens lie at positions 0, 1, ..."""
    d, page = draft[0], 16
    c = Case([3 * page - d % page, 16], draft, 2, 1, 32, 64, page, dtype, tree=None)
    room = c.table.shape[1] * page
    assert len(c.rows[0]) == room  # every position of the table has a key
    pg, rw = (torch.tensor(x) for x in zip(*c.rows[0]))
    k, v = c.k.cpu()[pg, rw, 0].double(), c.v.cpu()[pg, rw, 0].double()
    for given, clamped in ((10 ** 9, room), (2 ** 31 - 1, room), (room + 1, room), (-5, 0), (-2 ** 31, 0)):
        c.lens[0] = given
        o, lse = c.call()
        c.lens[0] = clamped
        o2, lse2 = c.call()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2), given
        seen = torch.arange(room)[None] < (room if clamped else torch.arange(1, d + 1)[:, None])
        for h in range(2):
            r = attn_ref.attend(c.q[:d, h].cpu().double(), k, v, seen.expand(d, room), 1 / math.sqrt(32), DT[dtype])
            attn_ref.check(o[:d, h], r["o"], f"length {given}")
            attn_ref.check(lse[:d, h], r["lse"], f"length {given} lse")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [257, 600])
def test_more_than_256_sequences(dtype, n):
    """The look-up keeps the work of 256 sequences; the rest, long ones that are cut and joined among
    them, come 64 at a time."""
    rng = random.Random(n)
    ctx = [rng.randrange(0, 100) for _ in range(n)]
    ctx[3], ctx[256], ctx[n - 1] = 3000, 5000, 2000
    draft = [rng.choice([0, 1, 1, 2]) for _ in range(n)]
    draft[3] = draft[256] = draft[n - 1] = 1
    Case(ctx, draft, 4, 2, 32, 32, 16, dtype, seed=n).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("few,most", [(17, 31), (40, 64)])  # 64 and 128 rows a pass
def test_more_than_64_sequences_of_wide_drafts(dtype, few, most):
    rng = random.Random(most)
    n = 150
    ctx = [rng.randrange(0, 60) for _ in range(n)]
    ctx[0], ctx[64], ctx[n - 1] = 1500, 4000, 2500
    draft = [rng.randrange(few, most + 1) for _ in range(n)]
    draft[7], draft[70], draft[130] = 0, 1, 0
    Case(ctx, draft, 2, 1, 32, 32, 16, dtype, seed=most).check()


def test_one_wide_tree_among_many_decode_rows():
    """The rows of a pass come from the batch's average: the tree takes several passes."""
    rng = random.Random(3)
    ctx = [rng.randrange(0, 300) for _ in range(100)]
    ctx[40] = 1900
    Case(ctx, [64 if n == 40 else 1 for n in range(100)], 8, 2, 64, 64, 32, "bf16", seed=4).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("draft", DRAFTS)
def test_scores_below_the_range_weigh_nothing(dtype, draft):
    """Finite queries and keys whose products pass -2^128 in 32 bits: a weight of zero."""
    c = Case([300, 20, 133], draft, 4, 2, 64, 64, 16, dtype, seed=7)
    c.q[:, :, 0] = 1e20
    c.k[..., 0] = 0.0
    for p in range(140):
        pg, rw = c.rows[0][p]
        c.k[pg, rw, :, 0] = -1e20
    c.check(gone=[(0, p) for p in range(140)])


def test_torch_helper_refusals():
    c = Case([20], [2], 4, 2, 32, 32, 16, "f32")
    with pytest.raises(ValueError, match="one token per sequence"):
        kda.attn_tree_decode_t(c.q, c.k, c.v, c.table, c.lens)
    with pytest.raises(TypeError, match="tree_mask"):
        kda.attn_tree_decode_t(c.q, c.k, c.v, c.table, c.lens, c.cu, c.mask.int())
    with pytest.raises(ValueError, match="k_cache"):
        kda.attn_tree_decode_t(c.q[..., :16].contiguous(), c.k, c.v, c.table, c.lens, c.cu, c.mask)
    with pytest.raises(kda.KDAError, match="page_size"):
        kda.attn_tree_decode_t(c.q, c.k[:, :12].contiguous(), c.v[:, :12].contiguous(), c.table, c.lens, c.cu, c.mask)
    with pytest.raises(kda.KDAError, match="workspace smaller"):
        kda.attn_tree_decode_t(c.q, c.k, c.v, c.table.repeat(1, 50), c.lens, c.cu, c.mask,
                               workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
