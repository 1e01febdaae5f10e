"""Attention of new tokens with a sliding window and sinks over a paged cache
against a 64-bit reference."""
import math
import random

import pytest
import torch

import attn_ref
import gated_delta_rule_60_amd as kda
from test_gpu_attn_tree import Case as TreeCase

pytestmark = pytest.mark.gpu


class Case(TreeCase):
    """What no token sees is NaN, and a page that holds nothing seen is taken off the table."""

    def __init__(self, ctx, draft, window, sinks, hq, hkv, dk, dv, page, dtype, seed=0, clear=True):
        super().__init__(ctx, draft, hq, hkv, dk, dv, page, dtype, seed, tree=None)
        self.window, self.sinks = window, sinks
        if not clear:
            return
        table = self.table.cpu()
        for n, at in enumerate(self.rows):
            used = self.seen(n).any(0)
            for p, (pg, rw) in enumerate(at):
                if not used[p]:
                    self.k[pg, rw] = self.v[pg, rw] = float("nan")
            for i in range(-(-len(at) // page)):
                if not used[i * page:(i + 1) * page].any():
                    table[n, i] = random.Random(n).choice([-1, 1 << 30, -5])
        self.table = table.cuda()

    def seen(self, n):
        i = self.ctx[n] + torch.arange(self.draft[n])[:, None]
        j = torch.arange(len(self.rows[n]))[None]
        return (j <= i) & ((i - j < self.window) | (j < self.sinks))

    def call(self, **kw):
        return kda.attn_window_decode_t(self.q, self.k, self.v, self.table, self.lens, self.cu, window=self.window,
                                        sinks=self.sinks, **kw)

    def want(self, scale=None):
        t, hq, dv = self.q.shape[0], self.hq, self.v.shape[-1]
        out = {"o": [torch.zeros(t, hq, dv, dtype=torch.float64) for _ in range(2)],
               "lse": [torch.zeros(t, hq, dtype=torch.float64) for _ in range(2)]}
        s = 1 / math.sqrt(self.q.shape[-1]) if scale is None else scale
        k, v, q = self.k.cpu(), self.v.cpu(), self.q.cpu().double()
        a = 0
        for n, d in enumerate(self.draft):
            if d == 0:
                continue
            pg, rw = (torch.tensor(x, dtype=torch.long) for x in zip(*self.rows[n]))
            kn, vn = (torch.where(torch.isfinite(x[pg, rw]), x[pg, rw], 0.0).double() for x in (k, v))
            for h in range(hq):
                g = h // (hq // self.hkv)
                r = attn_ref.attend(q[a:a + d, h], kn[:, g], vn[:, g], self.seen(n), s, self.q.dtype)
                for name in out:
                    for i in range(2):
                        out[name][i][a:a + d, h] = r[name][i]
            a += d
        return out


# rows of a key head: up to 16, 32, 64 and 128 a pass, and several passes
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("draft", [[1, 1, 1], [8, 5, 11], [16, 2, 25], [64, 40, 33]])
def test_head_sizes(dtype, dk, dv, draft):
    Case([170, 0, 333], draft, 70, 5, 4, 2, dk, dv, 16, dtype, seed=dk + dv).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (8, 1), (6, 2), (24, 8), (5, 1)])
def test_head_groups(dtype, hq, hkv):
    Case([140, 65, 3], [1, 5, 64], 33, 3, hq, hkv, 32, 64, 32, dtype, seed=hq).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 64, 100, 128, 129, 300, 1 << 30])
@pytest.mark.parametrize("sinks", [0, 1, 4, 32, 50, 256])
def test_windows_and_sinks(dtype, window, sinks):
    ctx = [0, 1, 31, 32, 33, 64, 127, 128, 129, 400]
    Case(ctx, [1 + i % 3 for i in range(len(ctx))], window, sinks, 2, 1, 64, 64, 16, dtype, seed=sinks + window % 999).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 2, 16, 64, 256, 4096])
@pytest.mark.parametrize("draft", [1, 40])
def test_pages_and_context_lengths(dtype, page, draft):
    ctx = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500]
    Case(ctx, [draft] * len(ctx), 40, 4, 2, 1, 64, 32, page, dtype, seed=page).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,draft", [(16, 300), (100, 130), (400, 257)])
def test_more_new_tokens_than_the_window(dtype, window, draft):
    """A piece of a prompt over the cache: every pass of rows walks its own part of the keys."""
    Case([90, 0, 700], [draft, 3, draft], window, 3, 4, 1, 64, 64, 32, dtype, seed=window).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_contexts_in_chunks(dtype):
    Case([9000, 20], [1, 2], 4000, 20, 8, 2, 128, 128, 64, dtype, seed=4).check()
    Case([7000], [7], 3000, 200, 2, 1, 64, 128, 16, dtype, seed=5).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences(dtype):
    r = random.Random(3)
    Case([r.randrange(300) for _ in range(290)], [r.randrange(3) for _ in range(290)], 50, 4, 2, 1, 32, 32, 16, dtype, seed=6).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_window_as_long_as_the_context(dtype):
    """The plain chain of attn_tree_decode, within both kernels' bounds."""
    c = Case([90, 33, 0], [3, 1, 20], 200, 0, 4, 2, 64, 64, 16, dtype, clear=False)
    o, lse = kda.attn_tree_decode_t(c.q, c.k, c.v, c.table, c.lens, c.cu)
    want = c.want()
    attn_ref.check(o, want["o"], "tree o")
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 2, 3, 4, 60, 79, 80, 81, 99, 100, 102])
def test_rows_that_do_not_see_a_position(dtype, at):
    """Positions 100 to 104 are new, with a window of 20 and 3 sinks: NaN and infinite keys and values reach
    the tokens that see them and no other."""
    c = Case([100], [5], 20, 3, 2, 1, 64, 64, 16, dtype, clear=False)
    want, lse_want = c.call()
    sees = c.seen(0)[:, at].cuda()
    pg, rw = c.rows[0][at]
    k, v = c.k.clone(), c.v.clone()
    for bad in (float("nan"), float("inf"), -float("inf")):
        c.k, c.v = k.clone(), v.clone()
        c.v[pg, rw, 0, 5] = bad
        o, lse = c.call()
        assert torch.equal(o[~sees], want[~sees]) and torch.equal(lse, lse_want)
        if bad != bad:
            assert torch.isnan(o[sees][..., 5]).all()
        else:
            assert (o[sees][..., 5].float() == bad).all()
        rest = [i for i in range(64) if i != 5]
        assert torch.equal(o[..., rest], want[..., rest])
        c.v = v
        c.k[pg, rw, 0, 9] = bad
        o, lse = c.call()
        assert torch.equal(o[~sees], want[~sees]) and torch.equal(lse[~sees], lse_want[~sees])


def test_rows_that_see_nothing():
    c = Case([50, 40], [1, 1], 8, 2, 2, 1, 32, 32, 16, "bf16", clear=False)
    c.table[0] = -1
    o, lse = c.call()
    torch.cuda.synchronize()
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all() and torch.isfinite(o[1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_last_sequence_and_clamped_lengths(dtype):
    c = Case([60, 33], [2, 1], 25, 4, 2, 1, 32, 32, 16, dtype)
    q = torch.cat([c.q, torch.full((4, 2, 32), float("nan"), dtype=c.q.dtype, device="cuda")])
    o = torch.full((7, 2, 32), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((7, 2), 7.0, device="cuda")
    kda.attn_window_decode_t(q, c.k, c.v, c.table, c.lens, c.cu, window=25, sinks=4, o=o, lse=lse)
    assert (o[3:] == 7).all() and (lse[3:] == 7).all()
    c.check((o[:3], lse[:3]))
    # lengths past the table's room: the tokens' own positions are not in the cache, their window's last ones are
    room = c.table.shape[1] * 16
    far = torch.tensor([2 ** 31 - 1, -9], dtype=torch.int32).cuda()
    o1, _ = kda.attn_window_decode_t(c.q, c.k, c.v, c.table, far, c.cu, window=25, sinks=4)
    o2, _ = kda.attn_window_decode_t(c.q, c.k, c.v, c.table, torch.tensor([room, 0], dtype=torch.int32).cuda(), c.cu, window=25, sinks=4)
    torch.cuda.synchronize()
    assert torch.equal(o1.isnan(), o2.isnan()) and torch.equal(o1.nan_to_num(), o2.nan_to_num())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_queries_streams_and_graph_replays_while_the_sequences_grow(dtype):
    c = Case([300, 90], [1, 1], 64, 4, 4, 2, 64, 64, 16, dtype, clear=False)
    want = c.call()
    wide = torch.zeros(2, 640, dtype=c.q.dtype, device="cuda")
    wide[:, 64:320] = c.q.view(2, 256)
    q, c.q = c.q, wide[:, 64:320].view(2, 4, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.call(stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    c.q = q
    c.lens.fill_(20)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = c.call()
    for n in range(4):
        c.lens.copy_(torch.tensor([20 + 70 * n, 5 + 20 * n], dtype=torch.int32))
        for x in kept:
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        eager = c.call()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(kept, eager)), f"replay {n}"


def test_prompt_then_decode_is_the_longer_prompt():
    """Keys and values of a prompt in the cache, the next tokens by the decode step: the rows that the longer
    prompt's pass gives, within both bounds."""
    lens, new, hq, hkv, d, page = [200, 61], 3, 4, 2, 64, 16
    g = torch.Generator().manual_seed(8)
    total = [n + new for n in lens]
    q, k, v = (torch.randn(sum(total), h, d, generator=g).bfloat16().cuda() for h in (hq, hkv, hkv))
    cu = torch.tensor([0, total[0], sum(total)], dtype=torch.int32).cuda()
    o, lse = kda.attn_window_prefill_t(q, k, v, cu, window=50, sinks=4)
    pages = kda.kv_pages(2, 20, 40, page)
    kc, vc = (torch.zeros(40, page, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rows = torch.arange(2, dtype=torch.int32, device="cuda")
    assert (kda.kv_reserve_t(pages, rows, torch.tensor(total, dtype=torch.int32).cuda()) == 0).all()
    kda.kv_append_t(k, v, kc, vc, pages.table, pages.lens, cu)
    pages.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    at = torch.cat([torch.arange(a + n, a + n + new) for a, n in ((0, lens[0]), (total[0], lens[1]))]).cuda()
    o2, lse2 = kda.attn_window_decode_t(q[at], kc, vc, pages.table, pages.lens, torch.tensor([0, 3, 6], dtype=torch.int32).cuda(),
                                        window=50, sinks=4)
    import window_ref
    want = window_ref.prefill(q, k, v, total, 50, 4, 1 / 8)
    for name, x, y in (("o", o, o2), ("lse", lse, lse2)):
        attn_ref.check(x, want[name], name)
        attn_ref.check(y, [w[at.cpu()] for w in want[name]], name)


def test_offsets_past_32_bits():
    """Pages 2^31 elements and more into the cache."""
    n_pages, page, d = 140000, 64, 128  # 1.15e9 positions x ... : 2.3e9 elements of keys
    kc = torch.zeros(n_pages, page, 2, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn(1, 4, d, generator=g, device="cuda").bfloat16()
    table = torch.arange(n_pages - 3, n_pages, dtype=torch.int32, device="cuda").view(1, 3)
    for x in (kc, vc):
        x[-3:] = torch.randn(3, page, 2, d, generator=g, device="cuda").bfloat16()
    o, lse = kda.attn_window_decode_t(q, kc, vc, table, torch.tensor([150], dtype=torch.int32).cuda(), window=70, sinks=3)
    k, v = (x[-3:].reshape(192, 2, d)[:151].cpu().double() for x in (kc, vc))
    j = torch.arange(151)
    seen = ((150 - j < 70) | (j < 3))[None]
    for h in range(4):
        r = attn_ref.attend(q[:, h].cpu().double(), k[:, h // 2], v[:, h // 2], seen, 1 / math.sqrt(d), torch.bfloat16)
        attn_ref.check(o[:, h], r["o"], "o")
        attn_ref.check(lse[:, h], r["lse"], "lse")


def test_two_steps_at_once_over_one_cache():
    """A windowed and a weighed step read one cache on two streams, each with its own workspace and outputs."""
    c = Case([3000, 90, 700], [1, 1, 1], 100, 4, 8, 2, 64, 64, 16, "bf16", clear=False)
    weights = torch.zeros(3, 2, c.table.shape[1] * 16, device="cuda")
    weighed = lambda **kw: kda.attn_weighed_decode_t(c.q, c.k, c.v, c.table, c.lens, weights, **kw)  # noqa: E731
    want, other = c.call(), weighed()
    torch.cuda.synchronize()
    once = weights.clone()
    weights.zero_()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(4):
        got.append((c.call(stream=streams[0]), weighed(stream=streams[1])))
    torch.cuda.synchronize()
    for x, y in got:
        assert all(torch.equal(a, b) for a, b in zip(x, want)) and all(torch.equal(a, b) for a, b in zip(y, other))
    total = torch.zeros_like(once)
    for _ in range(4):
        total += once
    assert torch.equal(weights, total)


def test_torch_helper_refusals():
    c = Case([30], [1], 8, 2, 2, 1, 32, 32, 16, "f32", clear=False)
    with pytest.raises(kda.KDAError, match="window"):
        kda.attn_window_decode_t(c.q, c.k, c.v, c.table, c.lens, c.cu, window=0)
    with pytest.raises(kda.KDAError, match="sinks"):
        kda.attn_window_decode_t(c.q, c.k, c.v, c.table, c.lens, c.cu, window=3, sinks=-1)
    with pytest.raises(ValueError, match="one token per sequence"):
        kda.attn_window_decode_t(torch.cat([c.q, c.q]), c.k, c.v, c.table, c.lens, window=3)
    with pytest.raises(kda.KDAError, match="workspace smaller"):
        kda.attn_window_decode_t(c.q, c.k, c.v, torch.zeros(1, 100, dtype=torch.int32, device="cuda"), c.lens, c.cu, window=1000,
                                 workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
