"""Attention that looks at a bounded part of the past, and the cache that keeps no more than that, as a program uses them.

Six kinds of pass:

  window   causal attention over packed prompts where a token sees the last ``window`` positions and the first ``sinks``
  train    the same with its backward pass: the gradients of q, k and v
  decode   the same for new tokens over a paged cache
  weights  how much attention every position of a prompt has drawn from the prompt's (last) rows
  weighed  a decode step that adds its own attention weights to those
  evict    sequences that outgrew their share of the cache keep their first and last positions and, of the others, the
           ones with the most weight, by layer and key head

Where ``own`` is false the passes are elementary torch operations in 32 bits; where it is true they are the calls of
gated_delta_rule_60_amd.
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
    r = random.Random(7)
    batch = _text(int(math.exp(r.uniform(math.log(300), math.log(4000)))) for _ in range(256))
    rows = _text(int(math.exp(r.uniform(math.log(700), math.log(4000)))) for _ in range(32))
    return [
        # a short prompt of a small fp32 model: a launch is all it should cost
        dict(name="window_t256_h2_d32_f32", kind="window", dtype="f32", lens="256", hq=2, hkv=2, dk=32, dv=32, window=50,
             sinks=3),
        # the packed batch of eight prompts that the delta-attention prefill is measured on, grouped heads
        dict(name="window_varlen8_32k_h32_d128", kind="window", dtype="bf16",
             lens="5416,2822,7999,7811,1485,2381,2454,2309", hq=32, hkv=8, dk=128, dv=128, window=1024, sinks=4),
        # a gradient check's or small fp32 model's step, ragged down to one token
        dict(name="train_ragged_h8_d64_f32", kind="train", dtype="f32", lens="1,77,300,33,513", hq=8, hkv=2, dk=64, dv=64,
             window=100, sinks=5),
        # a training step's micro-batch: packed documents
        dict(name="train_varlen4_16k_h32_d128", kind="train", dtype="bf16", lens="4096,2822,7811,1485", hq=32, hkv=8,
             dk=128, dv=128, window=1024, sinks=4),
        # one user's next token, far into a long text: latency
        dict(name="decode_n1_16k_h32_d128", kind="decode", dtype="bf16", ctx="16383", draft="1", hq=32, hkv=8, dk=128,
             dv=128, page=16, window=1024, sinks=4),
        # a full serving batch, one token each
        dict(name="decode_n256_h32_d128", kind="decode", dtype="bf16", ctx=batch, draft=_text([1] * 256), hq=32, hkv=8,
             dk=128, dv=128, page=64, window=1024, sinks=4),
        # a short fp32 prompt, its last rows only
        dict(name="weights_t300_r32_h2_d32_f32", kind="weights", dtype="f32", lens="300", hq=2, hkv=2, dk=32, dv=32, last=32,
             width=512),
        # the packed batch again, every row of it
        dict(name="weights_varlen8_32k_h32_d128", kind="weights", dtype="bf16",
             lens="5416,2822,7999,7811,1485,2381,2454,2309", hq=32, hkv=8, dk=128, dv=128, last=8192, width=8192),
        # three users of a small fp32 model
        dict(name="weighed_n3_h8_d64_f32", kind="weighed", dtype="f32", ctx="33,640,0", hq=8, hkv=2, dk=64, dv=64, page=16),
        # a full serving batch
        dict(name="weighed_n256_h32_d128", kind="weighed", dtype="bf16", ctx=batch, hq=32, hkv=8, dk=128, dv=128, page=64),
        # one sequence of a small fp32 model, a little past its share
        dict(name="evict_n1_l4_d64_f32", kind="evict", dtype="f32", lens="300", layers=4, hkv=2, dk=64, dv=64, page=16,
             budget=256, recent=64, sinks=4),
        # a batch after its prompts: long ones cut down to their share, the ones within it left alone
        dict(name="evict_n32_l8_d128", kind="evict", dtype="bf16", lens=rows, layers=8, hkv=8, dk=128, dv=128, page=64,
             budget=1024, recent=256, sinks=4),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    kind = rng.choice(["window", "train", "decode", "weights", "weighed", "evict"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([g for g in (1, 2, 3, 4, 8) if hkv * g <= 32])
    c = dict(kind=kind, dtype=dtype, dk=rng.choice([32, 64, 128]), dv=rng.choice([32, 64, 128]), hkv=hkv)
    if kind in ("window", "train", "decode"):
        c.update(window=_spread(rng, 16, 4096), sinks=rng.choice([0, 1, 4, rng.randint(2, 64)]))
    if kind in ("window", "train", "weights"):
        c.update(hq=hq, lens=_text(_spread(rng, 2 if kind == "train" else 1, 8192) for _ in range(_spread(rng, 1, 16))))
        if kind == "weights":
            c.update(last=rng.choice([_spread(rng, 1, 256), 8192]), width=rng.choice([8192, 8200]))
    elif kind == "evict":
        lens = [_spread(rng, 64, 4000) for _ in range(_spread(rng, 1, 32))]
        sinks, recent = rng.choice([0, 1, 4, 16]), _spread(rng, 1, min(512, max(lens) // 4))
        budget = sinks + recent + _spread(rng, 1, max(lens) - sinks - recent) - 1  # the longest, at least, is over it
        c.update(lens=_text(lens), layers=rng.randint(1, 8), page=rng.choice([16, 32, 64]), sinks=sinks, recent=recent,
                 budget=budget)
    else:
        n = _spread(rng, 1, 128)
        c.update(hq=hq, ctx=_text(_spread(rng, 1, 16000) - 1 for _ in range(n)), page=rng.choice([16, 32, 64, 128]))
        if kind == "decode":
            most = rng.choice([1, 1, 8, 64])
            c.update(draft=_text(rng.randint(1, most) for _ in range(n)))
    return c


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        old = most.get(c["kind"], (0, 0))
        most[c["kind"]] = (max(old[0], w["flops"] * (16 if c["dtype"] == "f32" else 1)), max(old[1], _held(c)))
    while True:
        c = _draw(rng)
        if work(c)["flops"] * (16 if c["dtype"] == "f32" else 1) <= most[c["kind"]][0] and _held(c) <= most[c["kind"]][1]:
            return c


def _seen(p, c):
    """How many positions a token at position p sees."""
    return p + 1 - max(0, p + 1 - c["window"] - c["sinks"])


def _pairs(c):
    if c["kind"] == "decode":
        return sum(_seen(a + j, c) for a, d in zip(_ints(c["ctx"]), _ints(c["draft"])) for j in range(d))
    if c["kind"] == "weights":  # the last rows, each with all keys up to itself
        return sum(x * (x + 1) // 2 - max(0, x - c["last"]) * (max(0, x - c["last"]) + 1) // 2 for x in _ints(c["lens"]))
    full = c["window"] + c["sinks"]
    return sum(x * (x + 1) // 2 if x <= full else full * (full + 1) // 2 + (x - full) * full for x in _ints(c["lens"]))


def _held(c):
    """Bytes that the inputs (for prompts also the plain form's largest score matrix) take."""
    row = c["hkv"] * (c["dk"] + c["dv"])
    if c["kind"] in ("window", "train", "weights"):
        lens = _ints(c["lens"])
        inputs = sum(lens) * (c["hq"] + c["hkv"]) * (c["dk"] + c["dv"]) * _SIZE[c["dtype"]]
        if c["kind"] == "weights":
            return max(lens) ** 2 * c["hq"] * 4 + inputs + len(lens) * c["hkv"] * c["width"] * 4
        return min(max(lens), 4096) * max(lens) * c["hq"] * 4 + inputs
    if c["kind"] == "evict":
        lens = _ints(c["lens"])
        return c["layers"] * (sum(lens) * row * _SIZE[c["dtype"]] + 8 * len(lens) * max(lens) * c["hkv"])
    ctx = _ints(c["ctx"])
    draft = _ints(c.get("draft", _text([1] * len(ctx))))
    room = max(a + b for a, b in zip(ctx, draft)) * len(ctx)  # the plain form pads to the longest
    return room * row * 4 + max(draft) * room * c["hq"] * 4


def _fills(c, length):
    """Positions that come from behind to a place given up in front, at even odds; and the last ones, which move up."""
    if length <= c["budget"]:
        return 0
    chosen, front = c["budget"] - c["recent"] - c["sinks"], c["budget"] - c["recent"]
    return (length - c["recent"] - front) * chosen // (length - c["recent"] - c["sinks"]) + c["recent"]


def work(c):
    es, d = _SIZE[c["dtype"]], c["dk"] + c["dv"]
    if c["kind"] in ("window", "train"):
        t, pairs = sum(_ints(c["lens"])), _pairs(c)
        q_like, kv = c["hq"] * d, c["hkv"] * d
        fwd_b, fwd_f = t * (q_like + kv) * es, 2 * pairs * c["hq"] * d
        if c["kind"] == "window":
            return {"bytes": fwd_b + 4 * t * c["hq"], "flops": fwd_f}
        # d_o is read too, d_q, d_k and d_v are written; five products a pair
        return {"bytes": fwd_b + t * (q_like + kv) * es,
                "flops": fwd_f + 2 * pairs * c["hq"] * (3 * c["dk"] + 2 * c["dv"])}
    if c["kind"] == "weights":
        lens = _ints(c["lens"])
        rows = sum(min(x, c["last"]) for x in lens)
        return {"bytes": rows * c["hq"] * (c["dk"] * es + 4) + sum(lens) * c["hkv"] * c["dk"] * es
                + len(lens) * c["hkv"] * c["width"] * 4, "flops": 2 * _pairs(c) * c["hq"] * c["dk"]}
    if c["kind"] == "decode":
        ctx, draft = _ints(c["ctx"]), _ints(c["draft"])
        tokens, kv = sum(draft), c["hkv"] * d * es
        read = sum(min(a + n, c["window"] + c["sinks"] + n - 1) for a, n in zip(ctx, draft))
        return {"bytes": read * kv + tokens * c["hq"] * (d * es + 4), "flops": 2 * _pairs(c) * c["hq"] * d}
    if c["kind"] == "weighed":
        ctx = _ints(c["ctx"])
        seen = sum(ctx) + len(ctx)
        return {"bytes": seen * c["hkv"] * (d * es + 8) + len(ctx) * c["hq"] * (d * es + 4), "flops": 2 * seen * c["hq"] * d}
    lens, heads = _ints(c["lens"]), c["layers"] * c["hkv"]
    over = [x for x in lens if x > c["budget"]]
    return {"bytes": heads * (2 * d * es * sum(_fills(c, x) for x in over) + 4 * sum(x + c["budget"] for x in over)),
            "flops": 0}


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
    s.window, s.sinks = case.get("window"), case.get("sinks")
    if s.kind in ("window", "train", "weights"):
        s.lens = _ints(case["lens"])
        t = sum(s.lens)
        s.cu = _i32(_offsets(s.lens), dev)
        s.q, s.k = rand(t, case["hq"], dk), rand(t, hkv, dk)
        if s.kind == "weights":  # the prompt pass leaves its row statistics; the rows of the table are made once
            s.lse = torch.cat([_row_statistics(s.q[a:a + n], s.k[a:a + n], s.scale)
                               for a, n in zip(_offsets(s.lens), s.lens)])
            s.weights = torch.empty(len(s.lens), hkv, case["width"], device=dev)
            return s
        s.v = rand(t, hkv, dv)
        s.do = rand(t, case["hq"], dv) if s.kind == "train" else None
        return s
    s.page = case["page"]
    lens = _ints(case["lens" if s.kind == "evict" else "ctx"])
    draft = _ints(case["draft"]) if s.kind == "decode" else [0 if s.kind == "evict" else 1] * len(lens)
    held = [-(-(a + d) // s.page) for a, d in zip(lens, draft)]
    total, wide = sum(held) + 3, max(held) + 1
    ids = list(range(total))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (wide - h))
        at += h
    if s.kind != "evict":
        s.lens, s.table = _i32(lens, dev), torch.tensor(table, dtype=torch.int32, device=dev)
        s.k, s.v = rand(total, s.page, hkv, dk), rand(total, s.page, hkv, dv)
        s.draft = draft
        s.q = rand(sum(draft), case["hq"], dk)
        # which sequence a new token belongs to, and its number in the draft
        s.seq = torch.tensor([n for n, d in enumerate(draft) for _ in range(d)], device=dev)
        s.num = torch.tensor([j for d in draft for j in range(d)], device=dev)
        s.cu = _i32(_offsets(draft), dev)
        if s.kind == "weighed":  # what the steps before have added up
            s.weights = torch.rand(len(lens), hkv, wide * s.page, generator=gen, device=dev)
            s.weights *= torch.arange(wide * s.page, device=dev) < s.lens[:, None, None]
        return s
    s.k, s.v = rand(case["layers"], total, s.page, hkv, dk), rand(case["layers"], total, s.page, hkv, dv)
    # the bookkeeping in one tensor, so that a pass can put it back with one copy
    free = ids[at:]
    sizes = [len(lens) * wide, len(lens), len(lens), total, total, 1]
    refs = [0] * total
    for p in ids[:at]:
        refs[p] = 1
    s.book0 = _i32([x for row in table for x in row] + lens + held + refs + ids[at:] + [0] * at + [total - at], dev)
    s.book = s.book0.clone()
    table, s.lens, s.held, s.refs, s.free, s.n_free = s.book.split(sizes)
    s.table = table.view(len(lens), wide)
    s.rows = _i32(range(len(lens)), dev)
    # heavy-tailed, as accumulated weights are; some positions have drawn none
    shape = (case["layers"], len(lens), hkv, wide * s.page)
    s.weights0 = torch.randn(shape, generator=gen, device=dev).mul_(2).exp_()
    s.weights0 *= torch.rand(shape, generator=gen, device=dev) > 0.05
    s.weights0 *= torch.arange(wide * s.page, device=dev) < s.lens[:, None, None]
    s.weights = s.weights0.clone()
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


def _row_statistics(q, k, scale):
    """ln sum_j exp(s_ij) of causal attention over one sequence, [L, H]."""
    n, groups = q.shape[0], q.shape[1] // k.shape[1]
    x = torch.matmul(_heads_first(q, groups), _heads_first(k, 1).transpose(1, 2)).mul_(scale)
    later = torch.ones(n, n, dtype=torch.bool, device=q.device).triu_(1)
    x.view(x.shape[0], -1, n, n).masked_fill_(later, float("-inf"))
    m = x.amax(-1, keepdim=True)
    return _tokens_first(m + x.sub_(m).exp_().sum(-1, keepdim=True).log(), n)[..., 0]


def _blocks(s):
    """Rows [a, b) of a sequence [beg, end), and the keys they see: the first ones and a range up to b."""
    for beg, n in zip(_offsets(s.lens), s.lens):
        step = max(s.window, 512)
        for a in range(0, n, step):
            b = min(a + step, n)
            lo = max(0, a - s.window + 1)
            head = min(s.sinks, lo)
            yield beg, a, b, lo, head


def _window(s, backward):
    c = s.case
    groups = c["hq"] // c["hkv"]
    o = torch.empty(s.q.shape[0], c["hq"], c["dv"], dtype=s.q.dtype, device=s.q.device)
    lse = torch.empty(s.q.shape[0], c["hq"], device=s.q.device)
    if backward:
        d_q, d_k, d_v = torch.empty_like(s.q), torch.zeros_like(s.k, dtype=torch.float), torch.zeros_like(s.v, dtype=torch.float)
    for beg, a, b, lo, head in _blocks(s):
        at = torch.cat([torch.arange(head, device=s.q.device), torch.arange(lo, b, device=s.q.device)])
        i = torch.arange(a, b, device=s.q.device)[:, None]
        hidden = (at > i) | ((at <= i - s.window) & (at >= s.sinks))
        q, k, v = _heads_first(s.q[beg + a:beg + b], groups), _heads_first(s.k[beg + at], 1), _heads_first(s.v[beg + at], 1)
        p = torch.matmul(q, k.transpose(1, 2)).mul_(s.scale)
        p.view(p.shape[0], groups, b - a, -1).masked_fill_(hidden, float("-inf"))
        m = p.amax(-1, keepdim=True)
        p = p.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        p = p.div_(total)
        x = torch.matmul(p, v)
        o[beg + a:beg + b] = _tokens_first(x, b - a).to(o.dtype)
        lse[beg + a:beg + b] = _tokens_first(m + total.log(), b - a)[..., 0]
        if backward:
            do = _heads_first(s.do[beg + a:beg + b], groups)
            ds = torch.matmul(do, v.transpose(1, 2)).sub_((do * x).sum(-1, keepdim=True)).mul_(p)
            d_q[beg + a:beg + b] = _tokens_first(torch.matmul(ds, k).mul_(s.scale), b - a).to(d_q.dtype)
            d_k.index_add_(0, beg + at, torch.matmul(ds.transpose(1, 2), q).mul_(s.scale).transpose(0, 1))
            d_v.index_add_(0, beg + at, torch.matmul(p.transpose(1, 2), do).transpose(0, 1))
    return [o, d_q, d_k.to(s.k.dtype), d_v.to(s.v.dtype)] if backward else [o, lse]


def _decode(s):
    c = s.case
    n, groups, most = len(s.draft), c["hq"] // c["hkv"], max(s.draft)
    room = s.table.shape[1] * s.page
    if s.kind == "weighed":
        at = torch.arange(room, device=s.q.device).expand(n, room)
        sees = (at <= s.lens[:, None])[:, None]
    else:  # the first positions, and the ones that any of the sequence's new tokens has in its window
        lo = (s.lens - s.window + 1).clamp(min=s.sinks)[:, None]
        wide = min(s.window - 1 + most, room)
        at = torch.cat([torch.arange(min(s.sinks, room), device=s.q.device).expand(n, -1),
                        lo + torch.arange(wide, device=s.q.device)], 1)
        own_place = (s.lens[:, None] + torch.arange(most, device=s.q.device))[:, :, None]
        sees = (at[:, None] <= own_place) & ((at[:, None] > own_place - s.window) | (at[:, None] < s.sinks))
        at = at.clamp(max=room - 1)
    page = s.table.gather(1, at // s.page).clamp(min=0).long()
    k = s.k[page, at % s.page].permute(0, 2, 3, 1).float()
    v = s.v[page, at % s.page].permute(0, 2, 1, 3).float()
    q = torch.zeros(n, most, c["hq"], c["dk"], device=s.q.device)
    q[s.seq, s.num] = s.q.float()
    q = q.view(n, most, c["hkv"], groups, c["dk"]).permute(0, 2, 3, 1, 4).reshape(n, c["hkv"], groups * most, c["dk"])
    x = torch.matmul(q, k).mul_(s.scale).view(n, c["hkv"], groups, most, -1)
    x = x.masked_fill_(~sees[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, c["hkv"], groups * most, -1), v).view(n, c["hkv"], groups, most, c["dv"])
    o = (o / total).permute(0, 3, 1, 2, 4).reshape(n, most, c["hq"], c["dv"])
    lse = (m + total.log()).permute(0, 3, 1, 2, 4).reshape(n, most, c["hq"])
    out = [o[s.seq, s.num].to(s.q.dtype), lse[s.seq, s.num]]
    if s.kind == "weighed":
        s.weights.add_((p / total).sum((2, 3)))
        out.append(s.weights)
    return out


def _weights(s):
    groups = s.case["hq"] // s.case["hkv"]
    for n, (beg, length) in enumerate(zip(_offsets(s.lens), s.lens)):
        first = max(0, length - s.case["last"])
        q, k = _heads_first(s.q[beg + first:beg + length], groups), _heads_first(s.k[beg:beg + length], 1)
        x = torch.matmul(q, k.transpose(1, 2)).mul_(s.scale)
        x.sub_(_heads_first(s.lse[beg + first:beg + length, :, None], groups)).exp_()
        later = torch.ones(length - first, length, dtype=torch.bool, device=q.device).triu_(1 + first)
        x.view(x.shape[0], groups, length - first, length).masked_fill_(later, 0)
        s.weights[n, :, :length] = x.sum(1)
        s.weights[n, :, length:] = 0
    return [s.weights]


def _evict(s):
    c = s.case
    layers, n, hkv, room = s.weights.shape
    budget, recent, sinks = c["budget"], c["recent"], c["sinks"]
    front, chosen = budget - recent, budget - recent - sinks
    pos = torch.arange(room, device=s.k.device)
    length = s.lens[:, None]
    shrinks = length > budget
    # the ones to choose from, by weight, the lower position first where weights are equal
    among = ((pos >= sinks) & (pos < length - recent) & shrinks)[None, :, None]
    order = torch.where(among, s.weights, -1.0).sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(s.weights, dtype=torch.bool).scatter_(-1, order[..., :chosen], True) & among
    gone, come = among & ~kept & (pos < front), kept & (pos >= front)
    gone, come = (torch.where(x, pos, room).sort(-1).values for x in (gone, come))  # in rising order, the others last
    # what comes to each place: itself; one from behind; the last ones
    source = torch.cat([pos, pos[:1]]).expand(layers, n, hkv, -1).clone()
    source.scatter_(-1, gone, torch.where(gone < room, come, 0))
    source = source[..., :min(budget, room)]
    pos = pos[:min(budget, room)]
    source = torch.where((shrinks & (pos >= front))[None, :, None], (pos + length - budget)[None, :, None].long(), source)
    stays = (pos >= length) & ~shrinks  # places behind a short sequence: its first position onto itself
    source, place = source.masked_fill_(stays[None, :, None], 0), pos.expand(n, -1).masked_fill(stays, 0)
    slot = lambda t: t % s.page  # noqa: E731
    src_page = s.table.gather(1, (source // s.page).permute(1, 0, 2, 3).reshape(n, -1)).view(n, layers, hkv, -1).permute(1, 0, 2, 3).long()
    dst_page = s.table.gather(1, place // s.page).long()[None, :, None]
    lay = torch.arange(layers, device=pos.device)[:, None, None, None]
    head = torch.arange(hkv, device=pos.device)[None, None, :, None]
    for cache in (s.k, s.v):
        cache[lay, dst_page, slot(place)[None, :, None], head] = cache[lay, src_page, slot(source), head]
    moved = s.weights.gather(-1, source)
    s.weights[..., :pos.numel()] = torch.where((shrinks | (pos < length))[None, :, None], moved, s.weights[..., :pos.numel()])
    s.weights.masked_fill_((shrinks & (torch.arange(room, device=pos.device) >= budget))[None, :, None], 0)
    # pages that hold nothing any more
    need = torch.where(shrinks[:, 0], -(-budget // s.page), s.held)
    cols = torch.arange(s.table.shape[1], device=pos.device)
    back = (cols >= need[:, None]) & (cols < s.held[:, None])
    ids = torch.where(back, s.table, 0).flatten().long()
    spare = torch.cat([s.free, s.free[:1]])  # one place more, for entries that give nothing back
    to = s.n_free + torch.cumsum(back.flatten(), 0) - 1
    spare[torch.where(back.flatten(), to, s.free.numel())] = ids.to(torch.int32)
    s.free.copy_(spare[:-1])
    s.refs.index_add_(0, ids, -back.flatten().to(torch.int32))
    s.n_free.add_(back.sum())
    s.table.masked_fill_(back, -1)
    s.held.copy_(need)
    s.lens.clamp_(max=budget)
    return [s.k, s.v, s.weights, s.table, s.lens, s.held, s.refs, s.free, s.n_free]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _run_own(s):
    import gated_delta_rule_60_amd as kda

    if s.kind == "window":
        return list(kda.attn_window_prefill_t(s.q, s.k, s.v, s.cu, window=s.window, sinks=s.sinks, scale=s.scale))
    if s.kind == "train":
        o, lse = kda.attn_window_prefill_t(s.q, s.k, s.v, s.cu, window=s.window, sinks=s.sinks, scale=s.scale)
        return [o, *kda.attn_window_prefill_backward_t(s.q, s.k, s.v, o, lse, s.do, s.cu, window=s.window, sinks=s.sinks,
                                                       scale=s.scale)]
    if s.kind == "decode":
        return list(kda.attn_window_decode_t(s.q, s.k, s.v, s.table, s.lens, s.cu, window=s.window, sinks=s.sinks,
                                             scale=s.scale))
    if s.kind == "weights":
        return [kda.attn_prefill_weights_t(s.q, s.k, s.lse, s.cu, rows=s.case["last"], weights=s.weights, scale=s.scale)]
    if s.kind == "weighed":
        return [*kda.attn_weighed_decode_t(s.q, s.k, s.v, s.table, s.lens, s.weights, scale=s.scale), s.weights]
    pages = kda.KVPages(table=s.table, lens=s.lens, held=s.held, refs=s.refs, free=s.free, n_free=s.n_free,
                        page_size=s.page)
    kda.kv_evict_t(pages, s.rows, s.k, s.v, s.weights, budget=s.case["budget"], recent=s.case["recent"], sinks=s.sinks)
    return [s.k, s.v, s.weights, s.table, s.lens, s.held, s.refs, s.free, s.n_free]


def run(s):
    if s.kind == "evict":
        # where the prompt or the steps since the last eviction have left the rows, in place of those steps
        s.book.copy_(s.book0)
        s.weights.copy_(s.weights0)
    if own:
        return _run_own(s)
    if s.kind in ("window", "train"):
        return _window(s, s.kind == "train")
    return {"decode": _decode, "weighed": _decode, "weights": _weights, "evict": _evict}[s.kind](s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_window(s):
    groups = s.case["hq"] // s.case["hkv"]
    train = s.kind == "train"
    t = sum(s.lens)
    f64 = dict(dtype=torch.float64, device=s.q.device)
    o, lse = torch.empty(t, s.case["hq"], s.case["dv"], **f64), torch.empty(t, s.case["hq"], **f64)
    d_q, d_k, d_v = torch.zeros(s.q.shape, **f64), torch.zeros(s.k.shape, **f64), torch.zeros(s.v.shape, **f64)
    a = 0
    for n in s.lens:
        at = torch.arange(n, device=s.q.device)
        back = at[:, None] - at  # how far a key lies behind the row
        seen = (back >= 0) & ((back < s.window) | (at < s.sinks))
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


def _exact_decode(s):
    c, a = s.case, 0
    groups = c["hq"] // c["hkv"]
    f64 = dict(dtype=torch.float64, device=s.q.device)
    o = torch.zeros(s.q.shape[0], c["hq"], c["dv"], **f64)
    lse = torch.full((s.q.shape[0], c["hq"]), -math.inf, **f64)
    weights = s.weights.double() if s.kind == "weighed" else None
    for n, d in enumerate(s.draft):
        ctx = int(s.lens[n])
        at = s.table[n][: -(-(ctx + d) // s.page)].long()
        k = s.k[at].flatten(0, 1)[: ctx + d].double()
        v = s.v[at].flatten(0, 1)[: ctx + d].double()
        for j in range(d):
            here = ctx + j
            use = torch.arange(here + 1, device=s.q.device)
            if s.kind == "decode":
                use = use[(use < s.sinks) | (use > here - s.window)]
            kk, vv = (x[use].repeat_interleave(groups, 1) for x in (k, v))
            x = (kk * s.q[a].double()).sum(-1) * s.scale
            lse[a] = torch.logsumexp(x, 0)
            p = torch.softmax(x, 0)
            o[a] = (p[..., None] * vv).sum(0)
            if weights is not None:
                weights[n, :, use] += p.view(len(use), c["hkv"], groups).sum(-1).T
            a += 1
    return [o, lse] if weights is None else [o, lse, weights]


def _exact_weights(s):
    groups = s.case["hq"] // s.case["hkv"]
    out = torch.zeros(s.weights.shape, dtype=torch.float64, device=s.q.device)
    a = 0
    for n, length in enumerate(s.lens):
        first = max(0, length - s.case["last"])
        seen = torch.tril(torch.ones(length, length, dtype=torch.bool, device=s.q.device))[first:]
        for h in range(s.case["hq"]):
            q, k = s.q[a + first:a + length, h].double(), s.k[a:a + length, h // groups].double()
            x = q @ k.T * s.scale - s.lse[a + first:a + length, h, None].double()
            out[n, h // groups, :length] += torch.where(seen, torch.exp(x), 0.0).sum(0)
        a += length
    return [out]


def _exact_evict(s):
    c = s.case
    k, v, weights = s.k.double(), s.v.double(), s.weights0.double()
    sizes = [s.table.numel(), s.lens.numel(), s.held.numel(), s.refs.numel(), s.free.numel(), 1]
    table, lens, held, refs, free, n_free = (x.tolist() for x in s.book0.split(sizes))
    wide = s.table.shape[1]
    table, n_free = [table[i * wide:(i + 1) * wide] for i in range(len(lens))], n_free[0]
    ranked = s.weights0.cpu().numpy()
    for n, length in enumerate(lens):
        if length <= c["budget"]:
            continue
        places = torch.tensor([table[n][p // s.page] * s.page + p % s.page for p in range(length)], device=s.k.device)
        last = list(range(length - c["recent"], length))
        front = c["budget"] - c["recent"]
        for layer in range(c["layers"]):
            for h in range(c["hkv"]):
                w = ranked[layer, n, h].tolist()
                best = sorted(range(c["sinks"], length - c["recent"]), key=lambda p: (-w[p], p))[:front - c["sinks"]]
                kept = set(best)
                late = iter(sorted(p for p in best if p >= front))
                src = [p if p < c["sinks"] or p in kept else next(late) for p in range(front)] + last
                src = torch.tensor(src, device=s.k.device)
                for x in (k, v):
                    rows = x[layer].view(-1, c["hkv"], x.shape[-1])[:, h]
                    rows[places[:c["budget"]]] = rows[places[src]]
                weights[layer, n, h, :c["budget"]] = weights[layer, n, h, src]
        weights[:, n, :, c["budget"]:] = 0
        for j in range(-(-c["budget"] // s.page), held[n]):
            free[n_free], refs[table[n][j]], table[n][j] = table[n][j], 0, -1
            n_free += 1
        lens[n], held[n] = c["budget"], -(-c["budget"] // s.page)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=s.k.device)  # noqa: E731
    return [k, v, weights, i32(table), i32(lens), i32(held), i32(refs), i32(free), i32([n_free])]


def exact(case, seed):
    s = prepare(case, seed)
    if s.kind in ("window", "train"):
        return _exact_window(s)
    return {"decode": _exact_decode, "weighed": _exact_decode, "weights": _exact_weights, "evict": _exact_evict}[s.kind](s)
