"""The softmax-attention operators and the paged cache, as a program uses them.

Five kinds of pass:

  prompt  causal attention over whole packed prompts (the forward of a full-attention layer)
  train   the same with its backward pass: the gradients of q, k and v
  tree    attention of drafted tokens over a paged cache; one drafted token is the plain decode step
  accept  room for drafted tokens, their keys and values into the cache, and the accepted ones moved together
  fork    last step's continuations dropped, and new ones made of the chosen sequences (a step of a beam search)

Where ``own`` is false the passes are elementary torch operations in 32 bits; where it is true they are the
calls of gated_delta_rule_60_amd.
"""
import math
import random

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


def _ints(text):
    return [int(x) for x in str(text).split(",")]


def _text(values):
    return ",".join(str(int(x)) for x in values)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    r = random.Random(5)
    batch = _text(int(math.exp(r.uniform(math.log(300), math.log(4000)))) for _ in range(256))
    beams = _text(int(math.exp(r.uniform(math.log(200), math.log(3900)))) for _ in range(32))
    return [
        # a short prompt of a small fp32 model: a launch is all it should cost
        dict(name="prompt_t256_h2_d32_f32", kind="prompt", dtype="f32", lens="256", hq=2, hkv=2, dk=32, dv=32),
        # the packed batch of eight prompts that the delta-attention prefill is measured on, grouped heads
        dict(name="prompt_varlen8_32k_h32_d128", kind="prompt", dtype="bf16",
             lens="5416,2822,7999,7811,1485,2381,2454,2309", hq=32, hkv=8, dk=128, dv=128),
        # one long document
        dict(name="prompt_t16384_h16_d128", kind="prompt", dtype="bf16", lens="16384", hq=16, hkv=2, dk=128, dv=128),
        # a gradient check's or small fp32 model's step, ragged down to one token
        dict(name="train_ragged_h8_d64_f32", kind="train", dtype="f32", lens="1,77,300,33,513", hq=8, hkv=2, dk=64, dv=64),
        # a training step's micro-batch: packed documents
        dict(name="train_varlen4_16k_h32_d128", kind="train", dtype="bf16", lens="4096,2822,7811,1485", hq=32, hkv=8,
             dk=128, dv=128),
        # one user's next token: latency
        dict(name="decode_n1_h32_d128", kind="tree", dtype="bf16", ctx="1023", draft="1", hq=32, hkv=8, dk=128, dv=128,
             page=16),
        # a full serving batch, one token each
        dict(name="decode_n256_h32_d128", kind="tree", dtype="bf16", ctx=batch, draft=_text([1] * 256), hq=32, hkv=8,
             dk=128, dv=128, page=64),
        # drafted trees over long and short contexts, one context empty
        dict(name="tree_n12_32k_h32_d128", kind="tree", dtype="bf16",
             ctx="32700,1000,17,8191,0,20011,4096,12345,640,2500,30001,777", draft="16,64,7,32,48,16,33,64,1,21,16,12",
             hq=32, hkv=8, dk=128, dv=128, page=32),
        # the cache's own work around such a step: a small model, and all layers of a larger one
        dict(name="accept_n3_l4_d64_f32", kind="accept", dtype="f32", lens="33,640,5", draft="8,5,1", layers=4, hkv=2,
             dk=64, dv=64, page=16),
        dict(name="accept_n64_l8_d128", kind="accept", dtype="bf16", lens=beams + "," + beams, draft=_text([16, 33, 64, 7] * 16),
             layers=8, hkv=8, dk=128, dv=128, page=32),
        # four beams of one sequence, and a batch of them
        dict(name="fork_n2_l4_d64_f32", kind="fork", dtype="f32", lens="100,17", children=4, layers=4, hkv=2, dk=64,
             dv=64, page=16),
        dict(name="fork_n32_l8_d128", kind="fork", dtype="bf16", lens=beams, children=128, layers=8, hkv=8, dk=128,
             dv=128, page=64),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    kind = rng.choice(["prompt", "prompt", "train", "train", "tree", "tree", "accept", "fork"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([g for g in (1, 2, 3, 4, 8) if hkv * g <= 32])
    c = dict(kind=kind, dtype=dtype, dk=rng.choice([32, 64, 128]), dv=rng.choice([32, 64, 128]), hkv=hkv)
    if kind in ("prompt", "train"):
        n = _spread(rng, 1, 16)
        c.update(hq=hq, lens=_text(_spread(rng, 1, 8192) for _ in range(n)))
    elif kind == "tree":
        n = _spread(rng, 1, 128)
        most = rng.choice([1, 1, 8, 64])
        c.update(hq=hq, ctx=_text(_spread(rng, 1, 16000) - 1 for _ in range(n)),
                 draft=_text(rng.randint(1, most) for _ in range(n)), page=rng.choice([16, 32, 64, 128]))
    else:
        n = _spread(rng, 1, 64)
        c.update(lens=_text(_spread(rng, 1, 4000) for _ in range(n)), layers=rng.randint(1, 8),
                 page=rng.choice([16, 32, 64]))
        if kind == "accept":
            c.update(draft=_text(rng.randint(1, 64) for _ in range(n)))
        else:
            c.update(children=_spread(rng, 1, 128))
    return c


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["kind"]] = max(most.get(c["kind"], (0, 0)), (w["flops"] * (16 if c["dtype"] == "f32" else 1), _held(c)))
    while True:
        c = _draw(rng)
        f, b = work(c)["flops"] * (16 if c["dtype"] == "f32" else 1), _held(c)
        if f <= most[c["kind"]][0] and b <= most[c["kind"]][1]:
            return c


def _pairs(lens):
    return sum(x * (x + 1) // 2 for x in lens)


def _held(c):
    """Bytes that the inputs (for prompts also the plain form's largest score matrix) take."""
    if c["kind"] in ("prompt", "train"):
        lens = _ints(c["lens"])
        return max(lens) ** 2 * c["hq"] * 4 + sum(lens) * (c["hq"] + c["hkv"]) * (c["dk"] + c["dv"]) * _SIZE[c["dtype"]]
    if c["kind"] == "tree":
        ctx, draft = _ints(c["ctx"]), _ints(c["draft"])
        room = max(a + b for a, b in zip(ctx, draft)) * len(ctx)  # the plain form pads to the longest
        return room * c["hkv"] * (c["dk"] + c["dv"]) * 4 + max(draft) * room * c["hq"] * 4
    tokens = sum(_ints(c["lens"])) + 64 * c.get("children", len(_ints(c["lens"])))
    return tokens * c["layers"] * c["hkv"] * (c["dk"] + c["dv"]) * _SIZE[c["dtype"]]


def _accepted(n):
    """How many of n drafted tokens the cases accept."""
    return (n + 2) // 3


def work(c):
    es = _SIZE[c["dtype"]]
    if c["kind"] in ("prompt", "train"):
        lens = _ints(c["lens"])
        t, pairs = sum(lens), _pairs(lens)
        q_like, kv = c["hq"] * (c["dk"] + c["dv"]), c["hkv"] * (c["dk"] + c["dv"])
        fwd_b, fwd_f = t * (q_like + kv) * es, 2 * pairs * c["hq"] * (c["dk"] + c["dv"])
        if c["kind"] == "prompt":
            return {"bytes": fwd_b + 4 * t * c["hq"], "flops": fwd_f}
        # d_o is read too, d_q, d_k and d_v are written; five products a pair
        more = t * (q_like + kv) * es
        return {"bytes": fwd_b + more, "flops": fwd_f + 2 * pairs * c["hq"] * (3 * c["dk"] + 2 * c["dv"])}
    if c["kind"] == "tree":
        ctx, draft = _ints(c["ctx"]), _ints(c["draft"])
        tokens, kv = sum(draft), c["hkv"] * (c["dk"] + c["dv"]) * es
        pairs = sum(a * d + d * (d + 1) // 2 for a, d in zip(ctx, draft))
        return {"bytes": (sum(ctx) + tokens) * kv + tokens * c["hq"] * ((c["dk"] + c["dv"]) * es + 4),
                "flops": 2 * pairs * c["hq"] * (c["dk"] + c["dv"])}
    row = c["layers"] * c["hkv"] * (c["dk"] + c["dv"]) * es
    if c["kind"] == "accept":
        draft = _ints(c["draft"])
        return {"bytes": 2 * row * (sum(draft) + sum(_accepted(d) for d in draft)), "flops": 0}
    lens, page = _ints(c["lens"]), c["page"]
    part = sum(lens[i % len(lens)] % page for i in range(c["children"]))
    ids = sum(-(-lens[i % len(lens)] // page) for i in range(c["children"]))
    return {"bytes": 2 * row * part + 4 * 8 * ids, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


class _State:
    pass


def _i32(values, dev):
    return torch.tensor(list(values), dtype=torch.int32, device=dev)


def _offsets(lens):
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    return at


def prepare(case, seed):
    s, dev = _State(), _device()
    s.case, s.kind = case, case["kind"]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = random.Random(seed)
    dt = _DTYPE[case["dtype"]]
    rand = lambda *shape: torch.randn(*shape, generator=gen, device=dev, dtype=dt)  # noqa: E731
    dk, dv, hkv = case["dk"], case["dv"], case["hkv"]
    s.scale = 1.0 / math.sqrt(dk)
    if s.kind in ("prompt", "train"):
        s.lens = _ints(case["lens"])
        t = sum(s.lens)
        s.cu = _i32(_offsets(s.lens), dev)
        s.q, s.k, s.v = rand(t, case["hq"], dk), rand(t, hkv, dk), rand(t, hkv, dv)
        s.do = rand(t, case["hq"], dv) if s.kind == "train" else None
        return s
    s.page = case["page"]
    if s.kind == "tree":
        ctx, draft = _ints(case["ctx"]), _ints(case["draft"])
        s.cu = _i32(_offsets(draft), dev)
        s.lens = _i32(ctx, dev)
        s.draft = draft
        # which sequence a drafted token belongs to, and its number in the draft
        s.seq = torch.tensor([n for n, d in enumerate(draft) for _ in range(d)], device=dev)
        s.num = torch.tensor([j for d in draft for j in range(d)], device=dev)
        masks = []
        for d in draft:  # a random tree: every token's parent is an earlier one, the first is the root
            seen = []
            for j in range(d):
                seen.append((1 << j) | (seen[rng.randrange(j)] if j else 0))
            masks += [m - (1 << 64) if m >> 63 else m for m in seen]
        s.mask = torch.tensor(masks, dtype=torch.int64, device=dev)
        pages = [-(-(a + d) // s.page) for a, d in zip(ctx, draft)]
        total, wide = sum(pages) + 3, max(pages)
        ids = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
        s.table = torch.full((len(ctx), wide), -1, dtype=torch.int32, device=dev)
        held = torch.arange(wide, device=dev) < torch.tensor(pages, device=dev)[:, None]
        s.table[held] = ids[: sum(pages)]
        s.q = rand(sum(draft), case["hq"], dk)
        s.k, s.v = rand(total, s.page, hkv, dk), rand(total, s.page, hkv, dv)
        return s
    # a cache of all layers: rows with their pages, and the free ones
    lens = _ints(case["lens"])
    kids = case.get("children", 0)
    draft = _ints(case["draft"])[: len(lens)] if s.kind == "accept" else [0] * len(lens)
    rows = len(lens) + kids
    wide = max(-(-(a + d) // s.page) for a, d in zip(lens, draft)) + 1
    held = [-(-a // s.page) for a in lens]
    total = sum(held) + kids + sum(-(-d // s.page) + 1 for d in draft) + 5
    ids = list(range(total))
    rng.shuffle(ids)
    table, refs = [[-1] * wide for _ in range(rows)], [0] * total
    all_lens, all_held = list(lens) + [0] * kids, list(held) + [0] * kids
    for n, h in enumerate(held):
        for p in range(h):
            table[n][p] = ids.pop()
            refs[table[n][p]] = 1
    if s.kind == "fork":
        s.src = [rng.randrange(len(lens)) if kids > len(lens) else i % len(lens) for i in range(kids)]
        for i in range(kids):  # last step's continuations: full pages shared, the last one their own
            n, r = i % len(lens), len(lens) + i
            all_lens[r], all_held[r] = lens[n], held[n]
            for p in range(held[n]):
                table[r][p] = table[n][p] if (p + 1) * s.page <= lens[n] else ids.pop()
                refs[table[r][p]] += 1
        s.children = _i32(range(len(lens), rows), dev)
        s.src = _i32(s.src, dev)
    else:
        s.rows = _i32(range(rows), dev)
        s.need = _i32(draft, dev)
        s.cu = _i32(_offsets(draft), dev)
        s.seq = torch.tensor([n for n, d in enumerate(draft) for _ in range(d)], device=dev)
        s.num = torch.tensor([j for d in draft for j in range(d)], device=dev)
        taken = [sorted(rng.sample(range(d), _accepted(d))) for d in draft]
        s.taken = _i32([j for x in taken for j in x], dev)
        s.cu_taken = _i32(_offsets([len(x) for x in taken]), dev)
        s.taken_seq = torch.tensor([n for n, x in enumerate(taken) for _ in x], device=dev)
        s.taken_num = torch.tensor([i for x in taken for i in range(len(x))], device=dev)
        s.new_k = rand(case["layers"], sum(draft), hkv, dk)
        s.new_v = rand(case["layers"], sum(draft), hkv, dv)
    s.k, s.v = rand(case["layers"], total, s.page, hkv, dk), rand(case["layers"], total, s.page, hkv, dv)
    s.table, s.refs = torch.tensor(table, dtype=torch.int32, device=dev), _i32(refs, dev)
    s.lens, s.held = _i32(all_lens, dev), _i32(all_held, dev)
    s.free = torch.zeros(total, dtype=torch.int32, device=dev)
    s.free[: len(ids)] = _i32(ids, dev)
    s.n_free = _i32([len(ids)], dev)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _heads_first(x, groups):
    """[L, H, d] -> [H / groups, groups * L, d] in 32 bits: the query heads of a key head one after another."""
    length, h, d = x.shape
    return x.float().view(length, h // groups, groups, d).permute(1, 2, 0, 3).reshape(h // groups, groups * length, d)


def _tokens_first(x, length):
    """The way back."""
    h, rows, d = x.shape
    return x.view(h, rows // length, length, d).permute(2, 0, 1, 3).reshape(length, h * (rows // length), d)


def _scores(q, k, length, scale):
    """Scaled causal scores of one sequence, [key heads, groups * L, L]; -inf where masked."""
    s = torch.matmul(q, k.transpose(1, 2)).mul_(scale)
    later = torch.ones(length, length, dtype=torch.bool, device=q.device).triu_(1)
    s.view(s.shape[0], -1, length, length).masked_fill_(later, float("-inf"))
    return s


def _prompt(s, backward):
    groups = s.case["hq"] // s.case["hkv"]
    parts = []
    at = _offsets(s.lens)
    for a, b in zip(at, at[1:]):  # sequence by sequence: scores of all heads at once
        if a == b:
            continue
        n = b - a
        q, k, v = _heads_first(s.q[a:b], groups), _heads_first(s.k[a:b], 1), _heads_first(s.v[a:b], 1)
        p = _scores(q, k, n, s.scale)
        m = p.amax(-1, keepdim=True)
        p = p.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        p = p.div_(total)
        o = torch.matmul(p, v)
        out = [_tokens_first(o, n).to(s.q.dtype)]
        if backward:
            do = _heads_first(s.do[a:b], groups)
            d_v = torch.matmul(p.transpose(1, 2), do)
            ds = torch.matmul(do, v.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
            d_q = torch.matmul(ds, k).mul_(s.scale)
            d_k = torch.matmul(ds.transpose(1, 2), q).mul_(s.scale)
            out += [_tokens_first(d_q, n).to(s.q.dtype), _tokens_first(d_k, n).to(s.q.dtype),
                    _tokens_first(d_v, n).to(s.q.dtype)]
        else:
            out.append(_tokens_first(m + total.log(), n)[..., 0])
        parts.append(out)
    return [torch.cat(x) for x in zip(*parts)]


def _tree(s):
    c = s.case
    groups, most, n = c["hq"] // c["hkv"], max(s.draft), len(s.draft)
    room = s.table.shape[1] * s.page
    at = s.table.clamp(min=0).long()
    k = s.k[at].view(n, room, c["hkv"], c["dk"]).permute(0, 2, 3, 1).float()
    v = s.v[at].view(n, room, c["hkv"], c["dv"]).permute(0, 2, 1, 3).float()
    q = torch.zeros(n, most, c["hq"], c["dk"], device=s.q.device)
    q[s.seq, s.num] = s.q.float()
    mask = torch.zeros(n, most, dtype=torch.int64, device=s.q.device)
    mask[s.seq, s.num] = s.mask
    past = torch.arange(room, device=s.q.device) - s.lens[:, None]  # place in the draft
    bit = (mask[:, :, None] >> past.clamp(0, 63)[:, None, :]) & 1
    sees = (past < 0)[:, None, :] | ((bit == 1) & (past < 64)[:, None, :])
    q = q.view(n, most, c["hkv"], groups, c["dk"]).permute(0, 2, 3, 1, 4).reshape(n, c["hkv"], groups * most, c["dk"])
    x = torch.matmul(q, k).mul_(s.scale).view(n, c["hkv"], groups, most, room)
    x = x.masked_fill_(~sees[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m.clamp(min=torch.finfo(torch.float32).min)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, c["hkv"], groups * most, room), v).view(n, c["hkv"], groups, most, c["dv"])
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(n, most, c["hq"], c["dv"])
    lse = (m + total.log()).permute(0, 3, 1, 2, 4).reshape(n, most, c["hq"])
    return [o[s.seq, s.num].to(s.q.dtype), lse[s.seq, s.num]]


def _accept(s):
    page, cols = s.page, torch.arange(s.table.shape[1], device=s.table.device, dtype=torch.int32)
    # room for the drafted tokens: pages off the top of the free ones, sequence by sequence
    more = ((s.lens + s.need + page - 1) // page - s.held).clamp(min=0)
    first = torch.cumsum(more, 0) - more
    new = (cols >= s.held[:, None]) & (cols < (s.held + more)[:, None])
    which = (s.n_free - 1 - first[:, None] - (cols - s.held[:, None])).clamp(min=0, max=s.free.numel() - 1)
    s.table.copy_(torch.where(new, s.free[which.long()], s.table))
    s.refs.index_add_(0, s.table.clamp(min=0).flatten().long(), new.flatten().to(torch.int32))
    s.held.add_(more)
    s.n_free.sub_(more.sum())
    # their keys and values
    to = s.lens[s.seq] + s.num
    at, off = s.table[s.seq, to // page].long(), to % page
    s.k[:, at, off] = s.new_k
    s.v[:, at, off] = s.new_v
    # the accepted ones move up behind the sequence
    src, dst = s.lens[s.taken_seq] + s.taken, s.lens[s.taken_seq] + s.taken_num
    from_at, to_at = s.table[s.taken_seq, (src // page).long()].long(), s.table[s.taken_seq, dst // page].long()
    moved_k, moved_v = s.k[:, from_at, (src % page).long()], s.v[:, from_at, (src % page).long()]
    s.k[:, to_at, dst % page] = moved_k
    s.v[:, to_at, dst % page] = moved_v
    return [s.k, s.v, s.table, s.held, s.refs, s.free, s.n_free, s.lens + s.cu_taken.diff()]


def _drop(s):
    """The children give back their pages; those that nobody holds any more are free."""
    rows = s.children.long()
    cols = torch.arange(s.table.shape[1], device=s.table.device, dtype=torch.int32)
    held = (cols < s.held[rows][:, None]).flatten()
    ids = s.table[rows].clamp(min=0).flatten().long()
    s.refs.index_add_(0, ids, -held.to(torch.int32))
    place = torch.arange(ids.numel(), device=ids.device)
    none = ids.numel()
    first = torch.full_like(s.refs, none, dtype=torch.int64)
    first.scatter_reduce_(0, ids, torch.where(held, place, none), "amin")
    freed = held & (s.refs[ids] == 0) & (first[ids] == place)  # a page that two of them held counts once
    to = s.n_free + torch.cumsum(freed, 0) - 1
    spare = torch.cat([s.free, s.free[:1]])  # one place more, for those that free nothing
    spare[torch.where(freed, to, s.free.numel())] = ids.to(torch.int32)
    s.free.copy_(spare[:-1])
    s.n_free.add_(freed.sum())
    s.table[rows] = -1
    s.held[rows] = 0
    s.lens[rows] = 0


def _fork(s):
    _drop(s)
    page, src, dst = s.page, s.src.long(), s.children.long()
    cols = torch.arange(s.table.shape[1], device=s.table.device, dtype=torch.int32)
    full, used = s.lens[src] // page, s.lens[src] % page
    part = used > 0
    rank = torch.cumsum(part, 0) - part.long()
    fresh = s.free[(s.n_free - 1 - rank).clamp(min=0)]
    s.n_free.sub_(part.sum())
    own_page = (cols == full[:, None]) & part[:, None]
    rows = torch.where(own_page, fresh[:, None], torch.where(cols < full[:, None], s.table[src], -1))
    s.refs.index_add_(0, rows.clamp(min=0).flatten().long(), (rows >= 0).flatten().to(torch.int32))
    # what the last page holds; the rest of the fresh page stays as it was
    last = s.table[src].gather(1, full.long().clamp(max=cols.numel() - 1)[:, None])[:, 0].clamp(min=0).long()
    to = torch.where(part, fresh.long(), last)
    keep = (torch.arange(page, device=cols.device) < used[:, None])[None, :, :, None, None]
    s.k[:, to] = torch.where(keep, s.k[:, last], s.k[:, to])
    s.v[:, to] = torch.where(keep, s.v[:, last], s.v[:, to])
    s.table[dst] = rows
    s.lens[dst] = s.lens[src]
    s.held[dst] = full + part.to(torch.int32)
    return [s.k, s.v, s.table, s.held, s.refs, s.free, s.n_free, s.lens]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _run_own(s):
    import gated_delta_rule_60_amd as kda

    if s.kind == "prompt":
        return list(kda.attn_prefill_t(s.q, s.k, s.v, s.cu, scale=s.scale))
    if s.kind == "train":
        o, lse = kda.attn_prefill_t(s.q, s.k, s.v, s.cu, scale=s.scale)
        return [o, *kda.attn_prefill_backward_t(s.q, s.k, s.v, o, lse, s.do, s.cu, scale=s.scale)]
    if s.kind == "tree":
        return list(kda.attn_tree_decode_t(s.q, s.k, s.v, s.table, s.lens, s.cu, s.mask, scale=s.scale))
    pages = kda.KVPages(table=s.table, lens=s.lens, held=s.held, refs=s.refs, free=s.free, n_free=s.n_free,
                        page_size=s.page)
    if s.kind == "accept":
        kda.kv_reserve_t(pages, s.rows, s.need)
        kda.kv_append_t(s.new_k, s.new_v, s.k, s.v, s.table, s.lens, s.cu)
        lens = kda.kv_compact_t(s.k, s.v, s.table, s.lens, s.taken, s.cu_taken)
        return [s.k, s.v, s.table, s.held, s.refs, s.free, s.n_free, lens]
    kda.kv_free_t(pages, s.children)
    kda.kv_fork_t(pages, s.src, s.children, s.k, s.v)
    return [s.k, s.v, s.table, s.held, s.refs, s.free, s.n_free, s.lens]


def run(s):
    if own:
        return _run_own(s)
    if s.kind in ("prompt", "train"):
        return _prompt(s, s.kind == "train")
    return {"tree": _tree, "accept": _accept, "fork": _fork}[s.kind](s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_prompt(s):
    groups = s.case["hq"] // s.case["hkv"]
    train = s.kind == "train"
    t = sum(s.lens)
    f64 = dict(dtype=torch.float64, device=s.q.device)
    o, lse = torch.empty(t, s.case["hq"], s.case["dv"], **f64), torch.empty(t, s.case["hq"], **f64)
    d_q, d_k, d_v = torch.zeros(s.q.shape, **f64), torch.zeros(s.k.shape, **f64), torch.zeros(s.v.shape, **f64)
    a = 0
    for n in s.lens:
        seen = torch.tril(torch.ones(n, n, dtype=torch.bool, device=s.q.device))
        for h in range(s.case["hq"] if n else 0):
            g = h // groups
            q, k, v = (x[a:a + n, i].double().requires_grad_(train) for x, i in ((s.q, h), (s.k, g), (s.v, g)))
            x = torch.where(seen, (q @ k.T) * s.scale, -math.inf)
            lse[a:a + n, h] = torch.logsumexp(x, -1).detach()
            y = torch.softmax(x, -1) @ v
            o[a:a + n, h] = y.detach()
            if train:
                grads = torch.autograd.grad(y, (q, k, v), s.do[a:a + n, h].double())
                d_q[a:a + n, h] += grads[0]
                d_k[a:a + n, g] += grads[1]
                d_v[a:a + n, g] += grads[2]
        a += n
    return [o, d_q, d_k, d_v] if train else [o, lse]


def _exact_tree(s):
    c, a = s.case, 0
    o = torch.zeros(s.q.shape[0], c["hq"], c["dv"], dtype=torch.float64, device=s.q.device)
    lse = torch.full((s.q.shape[0], c["hq"]), -math.inf, dtype=torch.float64, device=s.q.device)
    for n, d in enumerate(s.draft):
        ctx = int(s.lens[n])
        at = s.table[n][: -(-(ctx + d) // s.page)].long()
        k = s.k[at].flatten(0, 1)[: ctx + d].double().repeat_interleave(c["hq"] // c["hkv"], 1)
        v = s.v[at].flatten(0, 1)[: ctx + d].double().repeat_interleave(c["hq"] // c["hkv"], 1)
        for j in range(d):
            m = int(s.mask[a]) & ((1 << 64) - 1)
            use = list(range(ctx)) + [ctx + i for i in range(d) if m >> i & 1] if ctx < 64 else None
            if use is None:
                use = torch.cat([torch.arange(ctx), torch.tensor([ctx + i for i in range(d) if m >> i & 1],
                                                                 dtype=torch.int64)])
            use = torch.as_tensor(use, dtype=torch.int64, device=s.q.device)
            if use.numel():
                x = (k[use] * s.q[a].double()).sum(-1) * s.scale
                lse[a] = torch.logsumexp(x, 0)
                o[a] = (torch.softmax(x, 0)[..., None] * v[use]).sum(0)
            a += 1
    return [o, lse]


class _Book:
    """The bookkeeping of the pages, one request after another on the host."""

    def __init__(self, s):
        self.table, self.held, self.refs = s.table.tolist(), s.held.tolist(), s.refs.tolist()
        self.lens, self.free, self.n = s.lens.tolist(), s.free.tolist(), int(s.n_free)

    def pop(self):
        self.n -= 1
        self.refs[self.free[self.n]] = 1
        return self.free[self.n]

    def outputs(self, s, k, v, lens):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=s.k.device)  # noqa: E731
        return [k, v, i32(self.table), i32(self.held), i32(self.refs), i32(self.free), i32([self.n]), i32(lens)]


def _exact_accept(s):
    b, k, v = _Book(s), s.k.double(), s.v.double()
    need, taken, lens = s.need.tolist(), s.taken.tolist(), []
    cu, cu_taken = s.cu.tolist(), s.cu_taken.tolist()
    for n, length in enumerate(b.lens):
        while b.held[n] * s.page < length + need[n]:
            b.table[n][b.held[n]] = b.pop()
            b.held[n] += 1
        accepted = taken[cu_taken[n]:cu_taken[n + 1]]
        final = {length + j: cu[n] + j for j in range(need[n])}  # where each drafted place ends
        final.update({length + i: cu[n] + j for i, j in enumerate(accepted)})
        for place, token in final.items():
            k[:, b.table[n][place // s.page], place % s.page] = s.new_k[:, token].double()
            v[:, b.table[n][place // s.page], place % s.page] = s.new_v[:, token].double()
        lens.append(length + len(accepted))
    return b.outputs(s, k, v, lens)


def _exact_fork(s):
    b, k, v = _Book(s), s.k.double(), s.v.double()
    gone = [p for r in s.children.tolist() for p in b.table[r][:b.held[r]]]
    for p in gone:
        b.refs[p] -= 1
    for p in dict.fromkeys(gone):
        if b.refs[p] == 0:
            b.free[b.n] = p
            b.n += 1
    for r in s.children.tolist():
        b.table[r], b.held[r], b.lens[r] = [-1] * len(b.table[r]), 0, 0
    for a, r in zip(s.src.tolist(), s.children.tolist()):
        b.lens[r], b.held[r] = b.lens[a], b.held[a]
        full, used = divmod(b.lens[a], s.page)
        for p in range(full):
            b.table[r][p] = b.table[a][p]
            b.refs[b.table[a][p]] += 1
        if used:
            b.table[r][full] = b.pop()
            k[:, b.table[r][full], :used] = k[:, b.table[a][full], :used]
            v[:, b.table[r][full], :used] = v[:, b.table[a][full], :used]
    return b.outputs(s, k, v, b.lens)


def exact(case, seed):
    s = prepare(case, seed)
    if s.kind in ("prompt", "train"):
        return _exact_prompt(s)
    return {"tree": _exact_tree, "accept": _exact_accept, "fork": _exact_fork}[s.kind](s)
