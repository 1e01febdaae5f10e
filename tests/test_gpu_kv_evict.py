"""Eviction from the paged cache against a model of it on the host, request by
request, and a run of it with the calls that make and read the weights."""
import math
import random

import pytest
import torch

import attn_ref
import gated_delta_rule_60_amd as kda
from test_gpu_kv_pages import DT, Model as Pages, i32

pytestmark = pytest.mark.gpu


class Model(Pages):
    """With weights [layers, rows, heads, positions]; rows of given lengths."""

    def __init__(self, lens, page, layers=2, hkv=2, dk=32, dv=64, dtype="bf16", seed=0, spare=3, room=2, extra=0):
        most = max(-(-x // page) for x in lens) + room
        super().__init__(len(lens) + extra, most, sum(-(-x // page) for x in lens) + spare, page, layers, hkv, dk, dv, dtype, seed)
        assert self.reserve(range(len(lens)), lens) == [0] * len(lens)
        self.lens[:len(lens)] = lens
        g = torch.Generator().manual_seed(seed + 1)
        self.w = torch.randn(layers, self.rows, hkv, most * page, generator=g).mul(2).exp()
        self.w *= torch.rand(self.w.shape, generator=g) > 0.1
        for n, x in enumerate(self.lens):
            self.w[:, n, :, x:] = 0

    def upload(self):
        self.dw = self.w.cuda()
        return super().upload()

    def evict(self, rows, budget, recent, sinks):
        status, seen = [], set()
        for r in rows:
            again = r in seen
            seen.add(r)
            ok = 0 <= r < self.rows and not again and self.lens[r] <= self.held[r] * self.page
            ok = ok and all(0 <= p < self.n_pages and self.refs[p] == 1 for p in self.table[r][:self.held[r]])
            status.append(0 if ok else 2)
            n = self.lens[r] if ok else 0
            if n <= budget:
                continue
            front = budget - recent
            at = [(self.table[r][p // self.page], p % self.page) for p in range(n)]
            pg, rw = (torch.tensor(x) for x in zip(*at))
            for layer in range(self.w.shape[0]):
                for h in range(self.w.shape[2]):
                    w = self.w[layer, r, h].tolist()
                    key = lambda p: (-(w[p] if w[p] == w[p] else -math.inf), w[p] != w[p], p)  # noqa: E731
                    best = sorted(range(sinks, n - recent), key=key)[:front - sinks]
                    late = iter(sorted(p for p in best if p >= front))
                    kept = set(best)
                    src = [p if p < sinks or p in kept else next(late) for p in range(front)] + list(range(n - recent, n))
                    assert next(late, None) is None
                    src = torch.tensor(src, dtype=torch.long)
                    for c in (self.k, self.v):
                        c[layer, pg[:budget], rw[:budget], h] = c[layer, pg[src], rw[src], h].clone()
                    self.w[layer, r, h, :budget] = self.w[layer, r, h, src].clone()
                    self.w[layer, r, h, budget:n] = 0
            need = -(-budget // self.page)
            for j in range(need, self.held[r]):
                p = self.table[r][j]
                self.refs[p], self.table[r][j] = 0, -1
                self.free[self.n] = p
                self.n += 1
            self.held[r], self.lens[r] = need, budget
        return status

    def call(self, rows, budget, recent, sinks, weights=True, **kw):
        return kda.kv_evict_t(self.pages, i32(rows), self.dk, self.dv, self.dw if weights else None, budget=budget, recent=recent,
                              sinks=sinks, **kw)

    def check(self, rows, budget, recent, sinks, weights=True):
        status = self.call(rows, budget, recent, sinks, weights)
        torch.cuda.synchronize()
        before = self.w.clone()
        assert status.tolist() == self.evict(rows, budget, recent, sinks)
        if not weights:
            self.w = before
        self.same()

    def same(self):
        p = self.pages
        assert p.table.tolist() == self.table and p.lens.tolist() == self.lens and p.held.tolist() == self.held
        assert p.refs.tolist() == self.refs and int(p.n_free) == self.n and p.free.tolist()[:self.n] == self.free[:self.n]
        assert torch.equal(self.dw.cpu().nan_to_num(nan=-7.0), self.w.nan_to_num(nan=-7.0))
        assert torch.equal(self.dk.cpu(), self.k) and torch.equal(self.dv.cpu(), self.v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_head_sizes(dtype, dk, dv):
    Model([200, 90, 41], 16, hkv=3, dk=dk, dv=dv, dtype=dtype, seed=dk + dv).upload().check([0, 1, 2], 64, 20, 4)


@pytest.mark.parametrize("budget,recent,sinks", [
    (1, 0, 0), (1, 1, 0), (1, 0, 1), (10, 0, 0), (10, 10, 0), (10, 0, 10), (64, 1, 0), (64, 63, 0), (64, 60, 4), (64, 30, 33),
    (64, 30, 34), (100, 16, 1), (199, 50, 4), (200, 50, 4), (201, 50, 4), (5000, 100, 4)])
@pytest.mark.parametrize("page", [1, 16, 64])
def test_budgets(budget, recent, sinks, page):
    Model([200, 199, 201, 1, 64, 65, 100], page, seed=budget).upload().check([3, 0, 6, 5, 4, 2, 1], budget, recent, sinks)


@pytest.mark.parametrize("lens,budget,recent,sinks", [
    ([9000, 8193, 100], 1024, 256, 4),      # long lists, and a few chosen far behind
    ([20000], 9000, 1, 0),                  # more moves than a list holds
    ([30001], 20011, 9000, 7),              # most stay; the last ones overlap their new places
    ([5000], 4999, 3000, 0),                # one too many
    ([4500], 4436, 1000, 16)])
def test_long_rows(lens, budget, recent, sinks):
    Model(lens, 64, layers=1, hkv=2, dk=32, dv=32, seed=budget).upload().check(list(range(len(lens))), budget, recent, sinks)


def test_all_moves_of_a_long_row_come_from_behind():
    """The chosen ones all lie behind the front, in more than two lists; and none does."""
    for late in (True, False):
        m = Model([40000], 128, layers=1, hkv=1, dk=32, dv=32, seed=1)
        m.w[..., :40000] = torch.rand(40000, generator=torch.Generator().manual_seed(3))
        m.w[..., 25000:40000] += 10 if late else -10
        m.upload().check([0], 19000, 1000, 0)


@pytest.mark.parametrize("values", ["equal", "two", "zeros", "special"])
def test_ties_go_to_the_lower_position(values):
    m = Model([3000, 300], 16, layers=2, hkv=1, dk=32, dv=32, seed=4)
    r = torch.Generator().manual_seed(5)
    w = m.w[:, :, :, :]
    if values == "equal":
        w.fill_(0.25)
    elif values == "two":
        w.copy_((torch.rand(w.shape, generator=r) > 0.5).float() + 1)
    elif values == "zeros":
        w.zero_()
        w[..., 1::2] = -0.0  # the same weight as zero
    else:
        w.copy_(torch.randn(w.shape, generator=r))
        pick = torch.randint(0, 12, w.shape, generator=r)
        for i, x in enumerate((float("nan"), float("inf"), -float("inf"), 1e-42, -1e-42, 3.4e38, -float("nan"))):
            w[pick == i] = x
    for n, x in enumerate(m.lens):
        w[:, n, :, x:] = 0
    m.upload().check([1, 0], 200, 40, 4)


def test_without_weights_the_first_and_last_stay():
    Model([500, 60, 64, 65], 16, seed=2).upload().check([0, 1, 2, 3], 64, 60, 4, weights=False)
    Model([500, 60], 32, seed=2).upload().check([0, 1], 40, 40, 0, weights=False)


def test_requests_that_are_refused():
    m = Model([200, 150, 90, 80, 70, 60], 16, seed=6, spare=20, extra=3)
    assert m.fork([1], [6]) == [0]       # rows 1 and 6 share pages
    m.lens[2] = 16 * m.held[2] + 1       # fewer pages than positions
    m.table[3][1] = 10 ** 6              # no page
    m.lens[4] = -3
    m.upload()
    rows = [0, 0, -1, 9, 1, 6, 2, 3, 4, 5, 7, 10 ** 9]
    status = m.call(rows, 40, 10, 2)
    torch.cuda.synchronize()
    m.lens[4] = 70  # the model's own rule for a negative length
    want = m.evict([r for r in rows if r != 4], 40, 10, 2)
    want.insert(rows.index(4), 2)
    assert status.tolist() == want == [0, 2, 2, 2, 2, 2, 2, 2, 2, 0, 0, 2]
    m.lens[4] = -3
    m.same()


def test_many_requests():
    r = random.Random(3)
    m = Model([r.randrange(1, 200) for _ in range(1000)], 16, layers=1, hkv=1, dk=32, dv=32, seed=7)
    rows = list(range(1000))
    r.shuffle(rows)
    m.upload().check(rows + rows[:24], 50, 20, 2)


@pytest.mark.parametrize("seed", range(6))
def test_random_sequences_of_calls(seed):
    """Rows grow, are evicted, freed and forked in turn."""
    r = random.Random(seed)
    page = r.choice([1, 4, 16, 32])
    m = Model([r.randrange(1, 300) for _ in range(6)], page, layers=r.randint(1, 3), hkv=r.randint(1, 3), dk=32, dv=32,
              dtype=r.choice(["bf16", "f32"]), seed=seed, spare=700 // page, room=300 // page, extra=2).upload()
    for _ in range(12):
        what = r.choice(["evict", "evict", "grow", "free", "fork"])
        rows = r.sample(range(8), r.randint(1, 8))
        if what == "evict":
            sinks, recent = r.randint(0, 5), r.randint(0, 60)
            m.check(rows, max(1, sinks + recent + r.randint(0, 100)), recent, sinks)
        elif what == "grow":
            more = [r.randrange(0, 100) for _ in rows]
            status = kda.kv_reserve_t(m.pages, i32(rows), i32(more)).tolist()
            assert status == m.reserve(rows, more)
            for x, n, s in zip(rows, more, status):
                if s == 0:
                    m.w[:, x, :, m.lens[x]:m.lens[x] + n] = r.random()
                    m.lens[x] += n
            m.pages.lens.copy_(i32(m.lens))
            m.dw.copy_(m.w)
        elif what == "free":
            kda.kv_free_t(m.pages, i32(rows[:2]))
            m.release(rows[:2])
        else:
            src, dst = rows[:len(rows) // 2], rows[len(rows) // 2:][:len(rows) // 2]
            got = kda.kv_fork_t(m.pages, i32(src), i32(dst), m.dk, m.dv).tolist()
            assert got == m.fork(src, dst)
    m.same()


def test_one_layer_and_another_stream():
    m = Model([200, 90], 16, layers=1, seed=8).upload()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    status = kda.kv_evict_t(m.pages, i32([1, 0]), m.dk[0], m.dv[0], m.dw[0], budget=50, recent=20, sinks=2, stream=side)
    side.synchronize()
    assert status.tolist() == m.evict([1, 0], 50, 20, 2)
    m.same()


def test_no_requests():
    m = Model([20], 16, seed=8).upload()
    assert m.call([], 4, 1, 1).numel() == 0
    torch.cuda.synchronize()
    m.same()


def test_graph_replays_while_the_rows_grow():
    """The step that evicts is captured once; what it does depends on the lengths it finds."""
    m = Model([300, 40, 90], 16, seed=9, spare=60, room=20).upload()
    rows, more = i32([0, 1, 2]), i32([30, 30, 30])

    def step():
        a = kda.kv_reserve_t(m.pages, rows, more)
        m.pages.lens.add_(30)
        return a, kda.kv_evict_t(m.pages, rows, m.dk, m.dv, m.dw, budget=64, recent=24, sinks=3)

    def model():
        a = m.reserve([0, 1, 2], [30] * 3)
        m.lens = [x + 30 for x in m.lens]
        return a, m.evict([0, 1, 2], 64, 24, 3)

    step()
    torch.cuda.synchronize()
    model()
    m.same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for n in range(4):
        fresh = torch.rand(m.w.shape, generator=torch.Generator().manual_seed(n)) * (m.w == 0)
        for x in (m.w, m.dw):
            x.add_(fresh.to(x.device))
        graph.replay()
        torch.cuda.synchronize()
        assert [x.tolist() for x in kept] == list(model()), f"replay {n}"
        m.same()


def test_offsets_past_32_bits():
    """Pages 2^31 elements and more into the caches, and weights of rows that far."""
    n_pages, page, hkv, d = 70000, 64, 4, 128  # 2.3e9 elements of keys
    kc, vc = (torch.zeros(n_pages, page, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pages = kda.kv_pages(3, 1 << 20, n_pages, page)  # 64 M positions a row: weights of 8e8 elements
    w = torch.zeros(3, hkv, 64 << 20, device="cuda")
    last = list(range(n_pages - 5, n_pages))
    pages.table[2, :5] = i32(last)
    pages.lens[2], pages.held[2] = 300, 5
    pages.refs[n_pages - 5:] = 1
    pages.free[:n_pages - 5] = torch.arange(n_pages - 5, dtype=torch.int32, device="cuda")
    pages.n_free.fill_(n_pages - 5)
    g = torch.Generator(device="cuda").manual_seed(5)
    for x in (kc, vc):
        x[-5:] = torch.randn(5, page, hkv, d, generator=g, device="cuda").bfloat16()
    w[2, :, :300] = torch.rand(hkv, 300, generator=g, device="cuda")
    k0, w0 = kc[-5:].reshape(320, hkv, d)[:300].clone(), w[2, :, :300].clone()
    assert kda.kv_evict_t(pages, i32([2]), kc, vc, w, budget=100, recent=30, sinks=2).tolist() == [0]
    for h in range(hkv):
        best = w0[h, 2:270].argsort(descending=True)[:68] + 2
        kept = sorted(best.tolist())
        late = iter([p for p in kept if p >= 70])
        src = [p if p < 2 or p in set(kept) else next(late) for p in range(70)] + list(range(270, 300))
        src = torch.tensor(src, device="cuda")
        assert torch.equal(kc[-5:].reshape(320, hkv, d)[:100, h], k0[src, h]) and torch.equal(w[2, h, :100], w0[h, src])
        assert (w[2, h, 100:300] == 0).all()
    assert int(pages.lens[2]) == 100 and int(pages.held[2]) == 2 and int(pages.n_free) == n_pages - 2


def test_refusals():
    m = Model([40], 16, seed=1).upload()
    with pytest.raises(kda.KDAError, match="budget"):
        m.call([0], 0, 0, 0)
    with pytest.raises(kda.KDAError, match="budget"):
        m.call([0], 10, 8, 3)
    with pytest.raises(kda.KDAError, match="without weights"):
        m.call([0], 10, 6, 3, weights=False)
    with pytest.raises(ValueError, match="weights must have shape"):
        kda.kv_evict_t(m.pages, i32([0]), m.dk, m.dv, m.dw[..., :-1], budget=10, recent=2)
    with pytest.raises(ValueError, match="bookkeeping"):
        kda.kv_evict_t(m.pages, i32([0]), m.dk[:, 1:].contiguous(), m.dv[:, 1:].contiguous(), m.dw, budget=10, recent=2)
    m.same()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("streaming", [False, True])
def test_a_prompt_and_steps_over_a_bounded_cache(dtype, streaming):
    """As a server would: the prompt's pass, its weights, its keys and values into the cache, eviction down to the
    budget, then steps that append a token, attend, add their weights up and evict again.  On the host every head
    keeps its own list of positions; each step is held against attention over that list, in 64 bits.  `streaming`:
    no weights, the first and the last positions only."""
    hq, hkv, d, page, lens, steps = 4, 2, 32, 16, [150, 47, 90], 40
    sinks, recent = 3, 20
    budget = sinks + recent + (0 if streaming else 25)
    g = torch.Generator().manual_seed(12)
    r = lambda t, h: torch.randn(t, h, d, generator=g).to(DT[dtype]).cuda()  # noqa: E731
    t, N = sum(lens), len(lens)
    q, k, v = r(t, hq), r(t, hkv), r(t, hkv)
    cu = i32([0, *torch.tensor(lens).cumsum(0).tolist()])
    pages = kda.kv_pages(N, 12, 60, page)
    kc, vc = (torch.zeros(1, 60, page, hkv, d, dtype=DT[dtype], device="cuda") for _ in range(2))
    weights = torch.zeros(1, N, hkv, 12 * page, device="cuda")
    rows, one = i32(range(N)), i32([1] * N)
    o, lse = kda.attn_prefill_t(q, k, v, cu)
    assert (kda.kv_reserve_t(pages, rows, i32(lens)) == 0).all()
    kda.kv_append_t(k[None], v[None], kc, vc, pages.table, pages.lens, cu)
    kda.attn_prefill_weights_t(q, k, lse, cu, weights=weights[0])
    pages.lens.copy_(i32(lens))
    # the host's: all keys and values by sequence, and every head's positions in the cache's order
    at = [0, *torch.tensor(lens).cumsum(0).tolist()]
    keys = [k[a:b].cpu().double() for a, b in zip(at, at[1:])]
    values = [v[a:b].cpu().double() for a, b in zip(at, at[1:])]
    order = [[list(range(n)) for _ in range(hkv)] for n in lens]

    def evict():
        before = weights[0].tolist()
        status = kda.kv_evict_t(pages, rows, kc, vc, None if streaming else weights, budget=budget, recent=recent, sinks=sinks)
        assert status.tolist() == [0] * N
        front = budget - recent
        for n in range(N):
            for h in range(hkv):
                x = order[n][h]
                if len(x) <= budget:
                    continue
                w = before[n][h]
                best = sorted(range(sinks, len(x) - recent), key=lambda p: (-w[p], p))[:front - sinks]
                late = iter(sorted(p for p in best if p >= front))
                src = [p if p < sinks or p in best else next(late) for p in range(front)]
                order[n][h] = [x[p] for p in src] + x[len(x) - recent:]

    evict()
    for step in range(steps):
        q, k, v = r(N, hq), r(N, hkv), r(N, hkv)
        assert (kda.kv_reserve_t(pages, rows, one) == 0).all()
        kda.kv_append_t(k[None], v[None], kc, vc, pages.table, pages.lens)
        if streaming and step % 2:
            o, lse = kda.attn_window_decode_t(q, kc[0], vc[0], pages.table, pages.lens, window=recent, sinks=sinks)
        else:
            o, lse = kda.attn_weighed_decode_t(q, kc[0], vc[0], pages.table, pages.lens, weights[0])
        for n in range(N):
            keys[n], values[n] = torch.cat([keys[n], k[n:n + 1].cpu().double()]), torch.cat([values[n], v[n:n + 1].cpu().double()])
            for h in range(hkv):
                order[n][h].append(len(keys[n]) - 1)
            for h in range(hq):
                x = order[n][h // 2]
                if streaming and step % 2:
                    x = [p for i, p in enumerate(x) if i < sinks or i >= len(x) - recent]
                want = attn_ref.attend(q[n:n + 1, h].cpu().double(), keys[n][x, h // 2], values[n][x, h // 2],
                                       torch.ones(1, len(x), dtype=torch.bool), 1 / math.sqrt(d), DT[dtype])
                value, bound = want["o"]
                assert ((o[n, h].cpu().double() - value[0]).abs() <= bound[0]).all(), (step, n, h)
        pages.lens.add_(1)
        if step % 7 == 6:
            evict()
            assert pages.lens.tolist() == [min(len(order[n][0]), budget) for n in range(N)]
    assert int(pages.n_free) == 60 - int(pages.held.sum())
