"""The cache's page operations against a model of them on the host, request by
request, and a run of them with the attention that reads the cache."""
import math
import random

import pytest
import torch

import attn_ref
import gated_delta_rule_60_amd as kda

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32).cuda()


class Model:
    """The six arrays as lists, and caches of whole numbers (exact in bf16)."""

    def __init__(self, rows, max_pages, n_pages, page, layers=2, hkv=1, dk=32, dv=64, dtype="bf16", seed=0):
        self.rng = random.Random(seed)
        self.page, self.max_pages, self.n_pages, self.rows = page, max_pages, n_pages, rows
        self.table = [[-1] * max_pages for _ in range(rows)]
        self.lens, self.held, self.refs = [0] * rows, [0] * rows, [0] * n_pages
        self.free = list(range(n_pages))
        self.rng.shuffle(self.free)
        self.n = n_pages
        g = torch.Generator().manual_seed(seed)
        self.k, self.v = (torch.randint(-100, 100, (layers, n_pages, page, hkv, d), generator=g).to(DT[dtype]) for d in (dk, dv))

    def upload(self):
        self.pages = kda.KVPages(torch.tensor(self.table, dtype=torch.int32).cuda(), i32(self.lens), i32(self.held),
                                 i32(self.refs), i32(self.free), i32([self.n]), self.page)
        self.dk, self.dv = self.k.cuda(), self.v.cuda()
        return self

    # the operations, one request after another
    def reserve(self, rows, more):
        status, short, seen = [], False, set()
        for r, t in zip(rows, more):
            again = r in seen
            seen.add(r)  # the first request of a row counts, also where it is refused
            if not 0 <= r < self.rows or again or t < 0:
                status.append(2)
                continue
            pages = -(-(self.lens[r] + t) // self.page)
            if pages > self.max_pages:
                status.append(2)
                continue
            need = max(0, pages - self.held[r])
            if need and (short or need > self.n):
                short = True
                status.append(1)
                continue
            for _ in range(need):
                self.n -= 1
                p = self.free[self.n]
                self.refs[p] = 1
                self.table[r][self.held[r]] = p
                self.held[r] += 1
            status.append(0)
        return status

    def release(self, rows):
        seen, freed = set(), []
        for r in rows:
            if not 0 <= r < self.rows or r in seen:
                continue
            seen.add(r)
            freed += self.table[r][:self.held[r]]
            for j in range(self.held[r]):
                self.table[r][j] = -1
            self.held[r] = self.lens[r] = 0
        for p in freed:
            self.refs[p] -= 1
        for p in dict.fromkeys(freed):
            if self.refs[p] == 0:
                self.free[self.n] = p
                self.n += 1

    def fork(self, src, dst):
        status, short, seen, before = [], False, set(), list(self.held)
        for a, b in zip(src, dst):
            ok = 0 <= a < self.rows and 0 <= b < self.rows and a not in dst and b not in seen
            seen.add(b)
            full, used = divmod(self.lens[a], self.page) if ok else (0, 0)
            if not ok or before[b] or full + (used > 0) > self.held[a]:
                status.append(2)
                continue
            if used and (short or self.n == 0):
                short = True
                status.append(1)
                continue
            for j in range(full):
                self.table[b][j] = self.table[a][j]
                self.refs[self.table[a][j]] += 1
            if used:
                self.n -= 1
                p, q = self.free[self.n], self.table[a][full]
                self.refs[p] = 1
                self.table[b][full] = p
                self.k[:, p, :used] = self.k[:, q, :used]
                self.v[:, p, :used] = self.v[:, q, :used]
            self.lens[b], self.held[b] = self.lens[a], full + (used > 0)
            status.append(0)
        return status

    def place(self, n, pos):
        if self.lens[n] < 0 or pos // self.page >= self.max_pages:
            return None
        p = self.table[n][pos // self.page]
        return (p, pos % self.page) if 0 <= p < self.n_pages else None

    def append(self, k, v, counts):
        t = 0
        for n, c in enumerate(counts):
            for j in range(c):
                at = self.place(n, self.lens[n] + j)
                if at:
                    self.k[:, at[0], at[1]], self.v[:, at[0], at[1]] = k[:, t], v[:, t]
                t += 1

    def compact(self, accepted):
        out = []
        for n, acc in enumerate(accepted):
            done, last = 0, -1
            for i, x in enumerate(acc):
                a, b = self.place(n, self.lens[n] + x) if x >= i and x > last else None, self.place(n, self.lens[n] + i)
                if a is None or b is None:
                    break
                for c in (self.k, self.v):
                    c[:, b[0], b[1]] = c[:, a[0], a[1]]
                done, last = done + 1, x
            out.append(self.lens[n] + done)
        return out

    def check(self, data=True):
        p = self.pages
        torch.cuda.synchronize()
        assert p.table.tolist() == self.table
        assert p.lens.tolist() == self.lens and p.held.tolist() == self.held
        assert p.refs.tolist() == self.refs and int(p.n_free) == self.n
        assert p.free.tolist()[:self.n] == self.free[:self.n]
        if data:
            assert torch.equal(self.dk.cpu(), self.k) and torch.equal(self.dv.cpu(), self.v)


def filled(seed=0, rows=12, used=6, page=16, max_pages=9, n_pages=60, dtype="bf16", **kw):
    m = Model(rows, max_pages, n_pages, page, dtype=dtype, seed=seed, **kw)
    m.reserve(range(used), [m.rng.randrange(0, page * (max_pages - 2)) for _ in range(used)])
    for r in range(used):
        m.lens[r] = m.rng.randrange(0, m.held[r] * page + 1)
    return m.upload()


@pytest.mark.parametrize("seed", range(6))
def test_reserve(seed):
    m = filled(seed)
    rows = [m.rng.randrange(-1, 13) for _ in range(20)]
    more = [m.rng.choice([0, 1, 15, 16, 17, 60, 200, -1]) for _ in rows]
    status = kda.kv_reserve_t(m.pages, i32(rows), i32(more))
    assert status.tolist() == m.reserve(rows, more)
    assert {0, 2} <= set(status.tolist())
    m.check()


def test_reserve_when_pages_run_out():
    m = filled(1, n_pages=30)
    left = m.n
    rows, more = [6, 7, 8, 9, 0], [16 * left - 20, 10, 60, 1, 0]
    status = kda.kv_reserve_t(m.pages, i32(rows), i32(more))
    assert status.tolist() == m.reserve(rows, more)
    m.check()
    rows = list(range(6, 12))
    status = kda.kv_reserve_t(m.pages, i32(rows), i32([100] * 6))
    want = m.reserve(rows, [100] * 6)
    assert status.tolist() == want and 1 in want
    m.check()


@pytest.mark.parametrize("seed", range(4))
def test_free(seed):
    m = filled(seed)
    m.fork([0, 0, 1, 2], [6, 7, 8, 9])
    m.upload()
    rows = [6, 0, 6, 50, -1, 7, 2]
    kda.kv_free_t(m.pages, i32(rows))
    m.release(rows)
    m.check()
    rows = list(range(12))
    kda.kv_free_t(m.pages, i32(rows))
    m.release(rows)
    m.check()
    assert m.n == m.n_pages and sorted(m.free) == list(range(m.n_pages))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 4, 16, 64])
def test_fork(dtype, page):
    m = filled(page, page=page, dtype=dtype, hkv=3)
    m.lens[1] = page * (m.lens[1] // page)  # ends with a page: nothing to copy
    m.lens[2] = 0                           # nothing at all
    m.upload()
    src, dst = [0, 0, 1, 2, 3, 4], [6, 7, 8, 9, 10, 11]
    status = kda.kv_fork_t(m.pages, i32(src), i32(dst), m.dk, m.dv)
    assert status.tolist() == m.fork(src, dst) == [0] * 6
    m.check()


def test_fork_refuses_request_by_request():
    m = filled(3)
    m.held[5] = 0  # row 5: positions without pages
    m.lens[5] = 20
    m.upload()
    src = [0, 0, 6, 1, 7, 5, 12, 2, -1, 3, 4]
    dst = [6, 6, 7, 0, 8, 9, 9, 12, 9, 10, 11]  # twice; of a row being made; held; no pages; outside
    status = kda.kv_fork_t(m.pages, i32(src), i32(dst), m.dk, m.dv)
    want = m.fork(src, dst)
    assert status.tolist() == want and want.count(2) >= 6
    m.check()


def test_fork_when_pages_run_out():
    m = filled(2, n_pages=60)
    for r in range(6):
        m.lens[r] = max(1, m.lens[r] // 16 * 16 - 3) if m.held[r] else 0
    keep = 2
    m.n = keep
    m.upload()
    src, dst = [r for r in range(6) if m.lens[r]], []
    dst = list(range(6, 6 + len(src)))
    status = kda.kv_fork_t(m.pages, i32(src), i32(dst), m.dk, m.dv)
    want = m.fork(src, dst)
    assert status.tolist() == want and want.count(1) == len(src) - keep
    m.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layers", [1, 2, 5, 9])
def test_append(dtype, layers):
    m = filled(7, layers=layers, dtype=dtype, hkv=2)
    m.table[3][0] = -1       # a page that is not there
    m.lens[4] = -2           # and a row without a length
    m.upload()
    counts = [5, 0, 40, 20, 3, 200, 1, 0, 0, 0, 0, 2]  # past the pages, past the table
    t = sum(counts)
    k, v = (torch.randint(-99, 99, (layers, t + 3, 2, d)).to(DT[dtype]) for d in (32, 64))
    cu = i32([0] + torch.tensor(counts).cumsum(0).tolist())
    kda.kv_append_t(k.cuda(), v.cuda(), m.dk, m.dv, m.pages.table, m.pages.lens, cu)  # three tokens behind the last
    m.append(k, v, counts)
    m.check()


def test_append_to_more_than_64_sequences():
    m = filled(13, rows=200, used=190, n_pages=1600, layers=2)
    counts = [m.rng.choice([0, 0, 1, 2, 7]) for _ in range(200)]
    counts[63] = counts[64] = counts[127] = counts[128] = 3
    t = sum(counts)
    k, v = (torch.randint(-99, 99, (2, t + 2, 1, d)).bfloat16() for d in (32, 64))
    cu = i32([0] + torch.tensor(counts).cumsum(0).tolist())
    kda.kv_append_t(k.cuda(), v.cuda(), m.dk, m.dv, m.pages.table, m.pages.lens, cu)  # two tokens behind the last
    m.append(k, v, counts)
    m.check()


def test_append_one_layer_and_one_token_each():
    m = filled(9, layers=3)
    k, v = torch.randint(-9, 9, (12, 1, 32)).bfloat16(), torch.randint(-9, 9, (12, 1, 64)).bfloat16()
    kda.kv_append_t(k.cuda(), v.cuda(), m.dk[1], m.dv[1], m.pages.table, m.pages.lens)
    torch.cuda.synchronize()
    one = filled(9, layers=3)
    one.append(k[None].repeat(3, 1, 1, 1), v[None].repeat(3, 1, 1, 1), [1] * 12)
    m.k[1], m.v[1] = one.k[1], one.v[1]
    m.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seed", range(4))
def test_compact(dtype, seed):
    m = filled(seed, dtype=dtype, rows=8, used=8, hkv=2)
    acc = []
    for n in range(8):
        room = m.held[n] * 16 - m.lens[n]
        acc.append(sorted(m.rng.sample(range(room), m.rng.randrange(0, room + 1))) if room else [])
    acc[1] = list(range(m.held[1] * 16 - m.lens[1]))     # all of them: nothing moves
    acc[2] = [0, 3, 2, 5]                                # does not rise
    acc[3] = [1, 10 ** 6, 2]                             # outside
    acc[4] = [-1]
    acc[5] = [2, 2]                                      # twice
    cu = i32([0] + torch.tensor([len(x) for x in acc]).cumsum(0).tolist())
    flat = i32([x for a in acc for x in a] + [0, 1])     # two behind the last sequence's
    new = kda.kv_compact_t(m.dk, m.dv, m.pages.table, m.pages.lens, flat, cu)
    assert new.tolist() == m.compact(acc)
    m.check()


def test_compact_of_hundreds():
    """More accepted tokens than one round of the kernel takes."""
    m = Model(2, 80, 150, 16, layers=2, seed=4)
    m.reserve([0, 1], [1200, 1000])
    m.lens = [33, 0]
    m.upload()
    acc = [sorted(m.rng.sample(range(1100), 700)), sorted(m.rng.sample(range(1000), 513))]
    new = kda.kv_compact_t(m.dk, m.dv, m.pages.table, m.pages.lens, i32(acc[0] + acc[1]), i32([0, 700, 1213]))
    assert new.tolist() == m.compact(acc) == [733, 513]
    m.check()


def test_a_long_random_run():
    """The calls in any order keep to the model, and no page is lost."""
    m = Model(40, 12, 160, 8, layers=1, seed=11).upload()
    rng = m.rng
    for step in range(60):
        op = rng.choice(["reserve", "reserve", "free", "fork", "fork"])
        some = [rng.randrange(40) for _ in range(rng.randrange(1, 30))]
        if op == "reserve":
            more = [rng.randrange(0, 50) for _ in some]
            assert kda.kv_reserve_t(m.pages, i32(some), i32(more)).tolist() == m.reserve(some, more), step
            for r in set(some):  # the sequences grow into their pages
                m.lens[r] = rng.randrange(m.lens[r], m.held[r] * 8 + 1) if m.held[r] * 8 > m.lens[r] else m.lens[r]
            m.pages.lens.copy_(i32(m.lens))
        elif op == "free":
            kda.kv_free_t(m.pages, i32(some[:6]))
            m.release(some[:6])
        else:
            dst = [rng.randrange(40) for _ in some]
            assert kda.kv_fork_t(m.pages, i32(some), i32(dst), m.dk, m.dv).tolist() == m.fork(some, dst), step
        m.check(data=step % 10 == 9)
    held = {p for r in range(40) for p in m.table[r][:m.held[r]]}
    assert held.isdisjoint(m.free[:m.n]) and len(held) + m.n == m.n_pages


def test_many_requests_and_pages():
    m = Model(1100, 40, 20000, 1, layers=1, dk=32, dv=32, seed=2)
    rows = list(range(1024))
    more = [m.rng.randrange(0, 40) for _ in rows]
    m.upload()
    assert kda.kv_reserve_t(m.pages, i32(rows), i32(more)).tolist() == m.reserve(rows, more)
    m.check(data=False)
    kda.kv_free_t(m.pages, i32(rows[::-1]))
    m.release(rows[::-1])
    m.check(data=False)


@pytest.mark.parametrize("keep", [0, 5])
def test_free_of_shared_pages_in_several_rounds(keep):
    """More entries than a round of the kernel takes (8192), the same pages in all of them, rows with
    pages of their own in between; with some continuations kept their pages stay."""
    m = Model(320, 40, 700, 1, layers=1, dk=32, dv=32, seed=3)
    m.reserve([0, 1, 2], [40, 39, 40])
    m.lens[:3] = [40, 39, 40]
    dst = list(range(3, 303))
    assert m.fork([i % 3 for i in range(300)], dst) == [0] * 300
    own = list(range(303, 317))
    assert m.reserve(own, [30] * 14) == [0] * 14
    m.upload()
    rows = dst[keep:] + [0, 1, 2]
    m.rng.shuffle(rows)
    for i, r in enumerate(own):
        rows.insert(22 * i + 3, r)
    rows += rows[:4]  # twice
    assert sum(m.held[r] for r in set(rows)) > 8192 + 3000
    kda.kv_free_t(m.pages, i32(rows))
    m.release(rows)
    m.check(data=False)
    assert m.n == 700 - (119 if keep else 0)


def test_nothing_asked():
    m = filled(0)
    none = torch.zeros(0, dtype=torch.int32).cuda()
    assert kda.kv_reserve_t(m.pages, none, none).numel() == 0
    kda.kv_free_t(m.pages, none)
    assert kda.kv_fork_t(m.pages, none, none, m.dk, m.dv).numel() == 0
    m.check()


def test_replays():
    m = filled(5)
    src, dst = i32([0, 1, 2]), i32([6, 7, 8])
    kda.kv_fork_t(m.pages, src, dst, m.dk, m.dv)
    m.fork([0, 1, 2], [6, 7, 8])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kv_free_t(m.pages, dst)
        status = kda.kv_fork_t(m.pages, src, dst, m.dk, m.dv)
    for n in range(4):
        graph.replay()
        torch.cuda.synchronize()
        m.release([6, 7, 8])
        assert status.tolist() == m.fork([0, 1, 2], [6, 7, 8])
        m.check()
        m.dk.mul_(1)


def test_offsets_past_32_bits():
    layers, pages, page = 2, 17000, 64  # each layer 1.1e9 elements of keys
    k = torch.zeros(layers, pages, page, 8, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(layers, pages, page, 8, 32, dtype=torch.bfloat16, device="cuda")
    p = kda.kv_pages(4, 4, pages, page)
    new_k, new_v = torch.randn(layers, 70, 8, 128, device="cuda").bfloat16(), torch.randn(layers, 70, 8, 32, device="cuda").bfloat16()
    p.free.copy_(torch.arange(pages, dtype=torch.int32))  # the last pages first
    row = i32([0])
    assert kda.kv_reserve_t(p, row, i32([70])).tolist() == [0]
    one = lambda x: x[:1].contiguous()  # noqa: E731
    kda.kv_append_t(new_k, new_v, k, v, one(p.table), one(p.lens), i32([0, 70]))
    p.lens[0] = 70
    assert kda.kv_fork_t(p, row, i32([2]), k, v).tolist() == [0]
    lens = kda.kv_compact_t(k, v, one(p.table), i32([60]), i32([1, 4, 9]), i32([0, 3]))
    torch.cuda.synchronize()
    a, b = pages - 1, pages - 2
    assert p.table[0, :2].tolist() == [a, b] and p.table[2, :2].tolist() == [a, pages - 3]
    assert torch.equal(k[:, pages - 3, :6], new_k[:, 64:]) and torch.equal(v[:, pages - 3, :6], new_v[:, 64:])
    assert lens.tolist() == [63]
    assert torch.equal(k[:, a, 60:63], new_k[:, [61, 64, 69]]) and torch.equal(v[:, a, 60:63], new_v[:, [61, 64, 69]])
    assert (k[:, :100] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_drafting_over_a_cache_gives_whole_prompt_attention(dtype):
    """Prompts, their pages, a drafted tree, what of it is accepted, a fork, and
    a token on each branch: every output is that of attention over the whole
    sequence so far."""
    g = torch.Generator().manual_seed(6)
    hq, hkv, dk, dv, page, scale = 4, 2, 64, 32, 16, 1 / 8
    rnd = lambda t, h, d: torch.randn(t, h, d, generator=g).to(DT[dtype]).cuda()  # noqa: E731
    prompts = [37, 0, 90]
    p = kda.kv_pages(6, 12, 60, page)
    kc = torch.full((60, page, hkv, dk), float("nan"), dtype=DT[dtype], device="cuda")
    vc = torch.full((60, page, hkv, dv), float("nan"), dtype=DT[dtype], device="cuda")
    three = lambda x: x[:3].contiguous()  # noqa: E731
    cu = i32([0, 37, 37, 127])
    q, k, v = rnd(127, hq, dk), rnd(127, hkv, dk), rnd(127, hkv, dv)
    o, lse = kda.attn_prefill_t(q, k, v, cu, scale=scale)
    want = attn_ref.prefill(q, k, v, prompts, scale)
    attn_ref.check(o, want["o"], "prompt")
    assert kda.kv_reserve_t(p, i32([0, 1, 2]), i32(prompts)).tolist() == [0, 0, 0]
    kda.kv_append_t(k, v, kc, vc, three(p.table), three(p.lens), cu)
    p.lens[:3] = i32(prompts)
    so_far = [(k[:37], v[:37]), (k[:0], v[:0]), (k[37:], v[37:])]

    # a drafted tree on each: what a token sees are its ancestors
    trees = [[-1, 0, 0, 1, 2], [-1, 0, 1], [-1, -1, 1, 2, 2, 4]]
    cu = i32([0, 5, 8, 14])
    q, k, v = rnd(14, hq, dk), rnd(14, hkv, dk), rnd(14, hkv, dv)
    assert kda.kv_reserve_t(p, i32([0, 1, 2]), i32([5, 3, 6])).tolist() == [0, 0, 0]
    kda.kv_append_t(k, v, kc, vc, three(p.table), three(p.lens), cu)
    o, lse = kda.attn_tree_decode_t(q, kc, vc, three(p.table), three(p.lens), cu, kda.attn_tree_masks(trees).cuda(),
                                    scale=scale)
    paths, a = [], 0
    for n, tree in enumerate(trees):
        for t in range(len(tree)):
            path = [t]
            while tree[path[0]] >= 0:
                path.insert(0, tree[path[0]])
            rows = [a + x for x in path]
            kk, vv = torch.cat([so_far[n][0], k[rows]]), torch.cat([so_far[n][1], v[rows]])
            for h in range(hq):
                r = attn_ref.attend(q[a + t:a + t + 1, h].cpu().double(), kk[:, h // 2].cpu().double(),
                                    vv[:, h // 2].cpu().double(), torch.ones(1, kk.shape[0], dtype=torch.bool), scale, DT[dtype])
                attn_ref.check(o[a + t:a + t + 1, h], r["o"], f"sequence {n} token {t}")
        a += len(tree)
    # the last token's path is accepted
    paths = [[0, 2, 4], [0, 1, 2], [1, 2, 4, 5]]
    lens = kda.kv_compact_t(kc, vc, three(p.table), three(p.lens), i32(sum(paths, [])), i32([0, 3, 6, 10]))
    assert lens.tolist() == [40, 3, 94]
    p.lens[:3] = lens
    for n, (base, path) in enumerate(zip((0, 5, 8), paths)):
        rows = [base + x for x in path]
        so_far[n] = (torch.cat([so_far[n][0], k[rows]]), torch.cat([so_far[n][1], v[rows]]))

    # two continuations of the third, and a token on all five rows
    assert kda.kv_fork_t(p, i32([2, 2]), i32([3, 4]), kc, vc).tolist() == [0, 0]
    so_far += [so_far[2], so_far[2]]
    five = lambda x: x[:5].contiguous()  # noqa: E731
    for _ in range(20):  # across a page
        q, k, v = rnd(5, hq, dk), rnd(5, hkv, dk), rnd(5, hkv, dv)
        assert kda.kv_reserve_t(p, i32(range(5)), i32([1] * 5)).tolist() == [0] * 5
        kda.kv_append_t(k, v, kc, vc, five(p.table), five(p.lens))
        o, lse = kda.attn_tree_decode_t(q, kc, vc, five(p.table), five(p.lens), scale=scale)
        p.lens[:5] += 1
        so_far = [(torch.cat([x, k[n:n + 1]]), torch.cat([y, v[n:n + 1]])) for n, (x, y) in enumerate(so_far)]
    for n, (x, y) in enumerate(so_far):
        whole = x.shape[0]
        qq = torch.zeros(whole, hq, dk, dtype=DT[dtype], device="cuda")
        qq[-1] = q[n]
        want = attn_ref.prefill(qq, x, y, [whole], scale)
        attn_ref.check(o[n], tuple(z[-1] for z in want["o"]), f"row {n}")
        attn_ref.check(lse[n], tuple(z[-1] for z in want["lse"]), f"row {n} lse")
    kda.kv_free_t(p, i32([4, 2, 0, 3, 1]))
    torch.cuda.synchronize()
    assert int(p.n_free) == 60 and sorted(p.free.tolist()) == list(range(60)) and (p.refs == 0).all()


def test_torch_helper_refusals():
    m = filled(0)
    with pytest.raises(TypeError, match="rows must be"):
        kda.kv_free_t(m.pages, i32([0]).long())
    with pytest.raises(ValueError, match="n_tokens"):
        kda.kv_reserve_t(m.pages, i32([0, 1]), i32([1]))
    with pytest.raises(ValueError, match="bookkeeping"):
        kda.kv_fork_t(m.pages, i32([0]), i32([6]), m.dk[:, :5].contiguous(), m.dv[:, :5].contiguous())
    with pytest.raises(ValueError, match="one token per sequence"):
        kda.kv_append_t(m.dk[:, 0], m.dv[:, 0], m.dk, m.dv, m.pages.table, m.pages.lens)
    with pytest.raises(kda.KDAError, match="must not be lens"):
        kda.kv_compact_t(m.dk, m.dv, m.pages.table, m.pages.lens, i32([0]), i32([0] * 12 + [1]), new_lens=m.pages.lens)
    with pytest.raises(kda.KDAError, match="1024"):
        kda.kv_free_t(m.pages, torch.zeros(1025, dtype=torch.int32).cuda())
    with pytest.raises(kda.KDAError, match="page_size"):
        kda.kv_free_t(kda.KVPages(m.pages.table, m.pages.lens, m.pages.held, m.pages.refs, m.pages.free, m.pages.n_free, 12),
                      i32([0]))
