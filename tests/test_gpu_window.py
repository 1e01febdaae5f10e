"""Windowed attention over prompts and its backward pass against a 64-bit
reference, at the sizes, windows and layouts where they can go wrong."""
import math

import pytest
import torch

import attn_ref
import gated_delta_rule_60_amd as kda
import window_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAMES = ("o", "lse", "d_q", "d_k", "d_v")
# Batches that fill the device run whole 128-row blocks; small ones split their keys (or rows) over the
# waves of a block.  These sequences behind the ones under test make a batch full.
FILL = [64] * 150


def _make(lens, hq, hkv, dk, dv, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    t = sum(lens)
    r = lambda h, d: (spread * torch.randn(t, h, d, generator=g)).to(DT[dtype]).cuda()  # noqa: E731
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32).cuda()
    return r(hq, dk), r(hkv, dk), r(hkv, dv), r(hq, dv) / spread, cu


def _run(q, k, v, d_o, cu, **kw):
    o, lse = kda.attn_window_prefill_t(q, k, v, cu, **kw)
    return (o, lse, *kda.attn_window_prefill_backward_t(q, k, v, o, lse, d_o, cu, **kw))


def _check_all(lens, hq, hkv, dk, dv, dtype, seed, window, sinks, scale=None, spread=1.0):
    q, k, v, d_o, cu = _make(lens, hq, hkv, dk, dv, dtype, seed, spread)
    got = _run(q, k, v, d_o, cu, window=window, sinks=sinks, scale=scale)
    torch.cuda.synchronize()
    want = window_ref.prefill(q, k, v, lens, window, sinks, 1 / math.sqrt(dk) if scale is None else scale, d_o)
    for name, x in zip(NAMES, got):
        attn_ref.check(x, want[name], f"{dtype} {name}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("full", [False, True])
def test_head_sizes(dtype, dk, dv, full):
    _check_all([70, 331] + ([131] * 60 if full else []), 4, 4 if full else 2, dk, dv, dtype, 100 + dk + dv, 90, 5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 63, 64, 65, 100, 128, 129, 200, 400, 1 << 30])
@pytest.mark.parametrize("sinks", [0, 1, 4, 33, 64, 100])
def test_windows_and_sinks(dtype, window, sinks):
    _check_all([391, 1, 130, 0, 64], 2, 1, 64, 32, dtype, window % 1000 + sinks, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (17, 0), (40, 4), (64, 32), (100, 70), (129, 33), (250, 256), (300, 1),
                                          (1 << 30, 9)])
def test_windows_and_sinks_of_a_full_batch(dtype, window, sinks):
    _check_all([391, 1, 130, 0, 64, 515] + FILL, 4, 2, 32, 64, dtype, window % 1000 + sinks, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (8, 2), (6, 2), (5, 1), (9, 9)])
@pytest.mark.parametrize("full", [False, True])
def test_head_groups(dtype, hq, hkv, full):
    _check_all([40, 265] + (FILL if full else []), hq, hkv, 32, 64, dtype, 7 * hq + hkv, 50, 4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [2], [31, 32, 33], [63, 64, 65], [127, 128, 129], [1, 0, 0, 5, 1], [0, 300, 0],
                                  [257, 256, 255], [1] * 70, [3, 130] * 40, [60, 200] * 50])
def test_lengths(dtype, lens):
    _check_all(lens, 2, 1, 64, 64, dtype, len(lens) + sum(lens), 48, 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(256, 4), (700, 40)])
@pytest.mark.parametrize("hq,hkv", [(2, 1), (16, 8)])
def test_longer_sequences(dtype, window, sinks, hq, hkv):
    """Many pieces of the rows behind the sinks' window."""
    _check_all([2100, 777], hq, hkv, 128, 128, dtype, 5, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(200, 4), (80, 40), (75, 4), (600, 130), (2000, 4)])
@pytest.mark.parametrize("before", [0, 37])
def test_long_sequences_among_many_short_ones(dtype, window, sinks, before):
    """A full batch in which few sequences have rows past their window, some of them by one, and more sequences than
    can have any."""
    lens = [64] * 70 + [701] + [65] * 3 + [64] * 100 + [201, 1, 0, 200, 601, 513]
    t = sum(lens)
    assert len(lens) > (t + before) // (window + 1)
    q, k, v, d_o, _ = _make([before + t], 4, 2, 32, 64, dtype, window)
    cu = torch.tensor([before, *(before + torch.tensor(lens).cumsum(0)).tolist()], dtype=torch.int32).cuda()
    got = _run(q, k, v, d_o, cu, window=window, sinks=sinks)
    torch.cuda.synchronize()
    want = window_ref.prefill(q[before:], k[before:], v[before:], lens, window, sinks, 1 / math.sqrt(32), d_o[before:])
    for name, x in zip(NAMES, got):
        attn_ref.check(x[before:], want[name], f"{dtype} {name}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,sinks", [([100] * 90 + [3000, 1, 1500], 40), ([2200, 1700] + [131] * 60, 4), ([2600] * 5, 100)])
def test_many_pieces_of_a_full_batch(dtype, lens, sinks):
    """Whole blocks, and several pieces of a sequence's rows behind the sinks' window to join."""
    _check_all(lens, 8, 4, 64, 128, dtype, sinks, 256, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale,spread", [(1.0, 1.0), (1e-3, 1.0), (0.3, 3.0)])
def test_scales(dtype, scale, spread):
    """Peaked rows (scores of tens) and flat ones."""
    _check_all([200, 33], 2, 2, 64, 32, dtype, 11, 70, 2, scale, spread)


@pytest.mark.parametrize("full", [False, True])
def test_the_maximum_leaves_the_window(full):
    """A key whose score lies at 200 is seen by the rows of its window, not by later ones."""
    lens = [300] + (FILL if full else [])
    q, k, v, d_o, cu = _make(lens, 2, 1, 64, 64, "f32", 3)
    k[150] = 25.0 * q[0, 0] / q[0, 0].norm()
    q[151:300] = 0.2 * q[151:300] + 8.0 * q[0] / q[0].norm(dim=-1, keepdim=True)
    got = _run(q, k, v, d_o, cu, window=60, sinks=2, scale=1.0)
    want = window_ref.prefill(q, k, v, lens, 60, 2, 1.0, d_o)
    assert float(want["lse"][0][200:205].max()) > 100 and float(want["lse"][0][215:].max()) < 100
    for name, x in zip(NAMES, got):
        attn_ref.check(x, want[name], name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_window_as_long_as_the_sequence(dtype):
    """The plain attention, within both kernels' bounds."""
    lens = [300, 77]
    q, k, v, d_o, cu = _make(lens, 4, 2, 64, 64, dtype, 8)
    plain = attn_ref.prefill(q, k, v, lens, 1 / 8, d_o)
    for window, sinks in ((300, 0), (44, 256), (1 << 30, 0)):
        for name, x in zip(NAMES, _run(q, k, v, d_o, cu, window=window, sinks=sinks)):
            attn_ref.check(x, plain[name], name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_of_a_fused_projection(dtype):
    """q, k and v as views of one [T, (H_q + 2 H_kv) d] tensor: the same bits as from contiguous copies."""
    hq, hkv, d = 4, 2, 64
    g = torch.Generator().manual_seed(1)
    fused = torch.randn(237, (hq + 2 * hkv) * d, generator=g).to(DT[dtype]).cuda()
    q, k, v = fused.split([hq * d, hkv * d, hkv * d], 1)
    q, k, v = q.view(237, hq, d), k.view(237, hkv, d), v.view(237, hkv, d)
    cu = torch.tensor([0, 200, 237], dtype=torch.int32).cuda()
    d_o = torch.randn(237, hq, d, generator=g).to(DT[dtype]).cuda()
    for x, y in zip(_run(q, k, v, d_o, cu, window=50, sinks=3),
                    _run(q.contiguous(), k.contiguous(), v.contiguous(), d_o, cu, window=50, sinks=3)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("full", [False, True])
def test_rows_before_and_behind_the_sequences_stay(dtype, full):
    lens = [60, 230] + (FILL if full else [])
    t = sum(lens)
    q, k, v, d_o, _ = _make([50 + t + 40], 2, 1, 32, 32, dtype, 9)
    cu = torch.tensor([50, *(50 + torch.tensor(lens).cumsum(0)).tolist()], dtype=torch.int32).cuda()
    for x in (q, k, v, d_o):
        x[:50] = x[50 + t:] = float("nan")  # padding holds anything
    kw = dict(window=45, sinks=4, scale=1 / math.sqrt(32))
    st = torch.cuda.current_stream().cuda_stream
    outs = [torch.full(s, 7.0, dtype=d, device="cuda") for s, d in
            ((q.shape, q.dtype), (q.shape[:2], torch.float32), (q.shape, q.dtype), (k.shape, q.dtype), (v.shape, q.dtype))]
    o, lse = kda.attn_window_prefill_t(q, k, v, cu, o=outs[0], lse=outs[1], **kw)
    T, N, code = q.shape[0], len(lens), kda.KDA_DTYPE_BF16 if dtype == "bf16" else kda.KDA_DTYPE_F32
    ws = torch.empty(kda.attn_window_prefill_backward_workspace_size(N, T, 2, 1, 32, 32, 45, 4, code), dtype=torch.uint8, device="cuda")
    assert kda.attn_window_prefill_backward(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), d_o.data_ptr(), cu.data_ptr(), N, T, 2, 1, 32, 32,
        64, 32, 32, 45, 4, kw["scale"], code, *(x.data_ptr() for x in outs[2:]), ws.data_ptr(), ws.numel(), st) == kda.KDA_OK
    want = window_ref.prefill(q[50:50 + t], k[50:50 + t], v[50:50 + t], lens, 45, 4, kw["scale"], d_o[50:50 + t])
    for name, x in zip(NAMES, outs):
        attn_ref.check(x[50:50 + t], want[name], name)
        assert (x[:50] == 7).all() and (x[50 + t:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 3, 4, 5, 31, 32, 63, 64, 130, 199])
@pytest.mark.parametrize("dv", [32, 128])
@pytest.mark.parametrize("full", [False, True])
def test_rows_that_do_not_see_a_token(dtype, at, dv, full):
    """NaN and infinite keys and values of token `at`: the rows that do not see it keep their bits, the
    others turn NaN (or infinite)."""
    n, window, sinks = 200, 50, 4
    q, k, v, _, cu = _make([n] + (FILL if full else []), 2, 1, 64, dv, dtype, 17)
    want, lse_want = kda.attn_window_prefill_t(q, k, v, cu, window=window, sinks=sinks)
    sees = torch.zeros(q.shape[0], dtype=torch.bool)
    sees[:n] = window_ref.seen(n, window, sinks)[:, at]
    sees = sees.cuda()
    for bad in (float("nan"), float("inf"), -float("inf")):
        v2 = v.clone()
        v2[at, 0, 3] = bad
        o, lse = kda.attn_window_prefill_t(q, k, v2, cu, window=window, sinks=sinks)
        assert torch.equal(o[~sees], want[~sees]) and torch.equal(lse, lse_want)
        if bad != bad:
            assert torch.isnan(o[sees][:, :, 3]).all()
        else:
            assert (o[sees][:, :, 3].float() == bad).all()
        rest = [i for i in range(dv) if i != 3]
        assert torch.equal(o[..., rest], want[..., rest])
        k2 = k.clone()
        k2[at, 0, 7] = bad
        o, lse = kda.attn_window_prefill_t(q, k2, v, cu, window=window, sinks=sinks)
        assert torch.equal(o[~sees], want[~sees]) and torch.equal(lse[~sees], lse_want[~sees])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("full", [False, True])
def test_a_sequence_does_not_see_its_neighbours(dtype, full):
    q, k, v, d_o, cu = _make([170, 50, 190] + (FILL if full else []), 2, 1, 64, 64, dtype, 13)
    kw = dict(window=60, sinks=5)
    want = _run(q, k, v, d_o, cu, **kw)
    k[170:220], v[170:220] = float("nan"), float("inf")
    for x, y in zip(_run(q, k, v, d_o, cu, **kw), want):
        assert torch.equal(x[:170], y[:170]) and torch.equal(x[220:], y[220:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_outside_the_batch_are_clamped(dtype):
    q, k, v, _, _ = _make([100], 2, 1, 32, 32, dtype, 2)
    o = torch.full((100, 2, 32), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((100, 2), 7.0, device="cuda")
    bad = torch.tensor([-5, 40, 30, 2 ** 30], dtype=torch.int32).cuda()
    kda.attn_window_prefill_t(q, k, v, bad, o=o, lse=lse, window=16, sinks=4)
    good, _ = kda.attn_window_prefill_t(q, k, v, torch.tensor([0, 40], dtype=torch.int32).cuda(), window=16, sinks=4)
    torch.cuda.synchronize()
    assert torch.equal(o[:30], good[:30])  # rows that one sequence alone covers


def test_overlapping_offsets_touch_nothing_else():
    """Offsets that fall are not allowed, and what they give is not defined: but no row outside the batch's
    offsets is written, and every call ends."""
    q, k, v, d_o, _ = _make([300], 2, 1, 32, 32, "f32", 2)
    bad = torch.tensor([30, 200, 20, 290, 25, 290], dtype=torch.int32).cuda()
    o, lse = torch.full((300, 2, 32), 7.0, device="cuda"), torch.full((300, 2), 7.0, device="cuda")
    kda.attn_window_prefill_t(q, k, v, bad, o=o, lse=lse, window=16, sinks=4)
    kda.attn_window_prefill_backward_t(q, k, v, o, lse, d_o, bad, window=16, sinks=4)
    torch.cuda.synchronize()
    for x in (o, lse):
        assert (x[:20] == 7).all() and (x[290:] == 7).all()


@pytest.mark.parametrize("hq,hkv", [(8, 2), (32, 32)])
def test_the_same_bits_every_time(hq, hkv):
    x = _make([1900, 40, 333], hq, hkv, 128, 128, "bf16", 4)
    first = None
    for _ in range(4):
        r = _run(*x, window=200, sinks=4)
        torch.cuda.synchronize()
        first = first or r
        assert all(torch.equal(a, b) for a, b in zip(first, r))


@pytest.mark.parametrize("window,sinks", [(12, 0), (12, 3)])
def test_gradients_against_differences(window, sinks):
    """fp32: L(x + h d) - L(x - h d) over 2 h, L summed in 64 bits from the kernel's own fp32 outputs; bounds
    as in the plain attention's test: third derivatives, h^2 / 6 of the gradient's scale times |d|^2 a row
    (32 entries), and 2^-13 for the outputs' rounding over h."""
    q, k, v, d_o, cu = _make([50, 33], 4, 2, 32, 32, "f32", 21)
    grads = _run(q, k, v, d_o, cu, window=window, sinks=sinks)[2:]
    g = torch.Generator().manual_seed(2)
    for i in range(3):
        d = torch.randn(grads[i].shape, generator=g).cuda()
        want = float((grads[i].double() * d.double()).sum())
        h = 2.0 ** -7
        loss = []
        for sign in (1, -1):
            x = [q, k, v]
            x[i] = x[i] + sign * h * d
            loss.append(float((kda.attn_window_prefill_t(*x, cu, window=window, sinks=sinks)[0].double() * d_o.double()).sum()))
        got = (loss[0] - loss[1]) / (2 * h)
        size = float(grads[i].norm() * d.norm())
        print(f"    input {i}: differences {got:.6f}, gradient {want:.6f}, size {size:.3f}", flush=True)
        assert abs(got - want) <= size * (2.0 ** -14 * 32 / 6 + 2.0 ** -13)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("full", [False, True])
def test_another_stream_and_graph_replays(dtype, full):
    kw = dict(window=70, sinks=3)
    q, k, v, d_o, cu = _make([200, 161] + (FILL if full else []), 4, 2, 64, 64, dtype, 31)
    first = _run(q, k, v, d_o, cu, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = _run(q, k, v, d_o, cu, stream=side, **kw)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, second))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = _run(q, k, v, d_o, cu, **kw)
    for n in range(3):
        q.mul_(1.0 + n / 4)
        for x in kept:
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        eager = _run(q, k, v, d_o, cu, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(kept, eager)), f"replay {n}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_tokens(dtype):
    q, k, v, d_o, _ = _make([0], 4, 2, 64, 32, dtype, 1)
    for cu in (None, torch.zeros(4, dtype=torch.int32).cuda()):
        got = _run(q, k, v, d_o, cu, window=5, sinks=1)
        assert [tuple(x.shape) for x in got] == [(0, 4, 32), (0, 4), (0, 4, 64), (0, 2, 64), (0, 2, 32)]
    torch.cuda.synchronize()


def test_two_calls_at_once():
    kw = dict(window=100, sinks=6)
    a, b = _make([900, 33], 8, 2, 64, 64, "bf16", 1), _make([700, 7], 8, 2, 64, 64, "bf16", 2)
    want = [_run(*x, **kw) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, x in enumerate((a, b)):
            got[i].append(_run(*x, stream=streams[i], **kw))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(p, q) for g in got[i] for p, q in zip(g, want[i]))


def test_offsets_past_32_bits():
    """Token rows 2^31 elements and more into a wide fused buffer."""
    stride, t = 1 << 16, 33100  # 2.17e9 elements, 4.3 GB
    fused = torch.zeros(t, stride, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    fused[:, :512] = torch.randn(t, 512, generator=g, device="cuda")
    q, k, v = fused[:, :256].view(t, 2, 128), fused[:, 256:384].view(t, 1, 128), fused[:, 384:512].view(t, 1, 128)
    cu = torch.tensor([0, 32800, 33100], dtype=torch.int32).cuda()
    d_o = torch.randn(t, 2, 128, generator=g, device="cuda").bfloat16()
    got = _run(q, k, v, d_o, cu, window=100, sinks=4)
    tail = [x[32800:].contiguous() for x in (q, k, v)]
    want = window_ref.prefill(*tail, [300], 100, 4, 1 / math.sqrt(128), d_o[32800:])
    for name, x in zip(NAMES, got):
        attn_ref.check(x[32800:], want[name], name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("full", [False, True])
def test_scores_below_the_range_weigh_nothing(dtype, full):
    """Finite queries and keys whose products pass -2^128, for every sink and the first keys of the window:
    -infinity in 32 bits, and a weight of zero by the formula."""
    gone, n = 100, 300
    q, k, v, d_o, cu = _make([n] + (FILL if full else []), 2, 1, 64, 64, dtype, 23)
    q[:n, :, 0], k[:gone, :, 0], k[gone:n, :, 0] = 1e20, -1e20, 0.0
    got = _run(q, k, v, d_o, cu, window=80, sinks=4)
    torch.cuda.synchronize()
    q, k, v, d_o = (x[:n].cpu().double() for x in (q, k, v, d_o))
    seen = window_ref.seen(n, 80, 4, gone)
    seen[:, :gone] = False
    for h in range(2):
        r = attn_ref.attend(q[gone:, h], k[:, 0], v[:, 0], seen, 1 / 8, DT[dtype], d_o[gone:, h])
        for name, x in zip(NAMES[:3], got):
            attn_ref.check(x[gone:n, h], r[name], f"{name} head {h}")


@pytest.mark.parametrize("lens", [[40, 9], [300] * 60])
def test_the_row_statistics_may_be_left_out(lens):
    q, k, v, _, cu = _make(lens, 4, 2, 64, 32, "bf16", 6)
    want, _ = kda.attn_window_prefill_t(q, k, v, cu, window=30, sinks=2)
    o = torch.empty_like(want)
    rc = kda.attn_window_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu.data_ptr(), len(lens), sum(lens), 4, 2, 64, 32, 256,
                                 128, 64, 30, 2, 1 / 8, kda.KDA_DTYPE_BF16, o.data_ptr(), None,
                                 torch.cuda.current_stream().cuda_stream)
    assert rc == kda.KDA_OK
    torch.cuda.synchronize()
    assert torch.equal(o, want)


def test_torch_helper_refusals():
    q, k, v, d_o, cu = _make([20], 4, 2, 32, 32, "f32", 1)
    with pytest.raises(TypeError, match="window"):
        kda.attn_window_prefill_t(q, k, v, cu)
    with pytest.raises(ValueError, match="shape"):
        kda.attn_window_prefill_t(q, k[:10], v, cu, window=4)
    with pytest.raises(kda.KDAError, match="window"):
        kda.attn_window_prefill_t(q, k, v, cu, window=0)
    with pytest.raises(kda.KDAError, match="sinks"):
        kda.attn_window_prefill_t(q, k, v, cu, window=4, sinks=257)
    o, lse = kda.attn_window_prefill_t(q, k, v, cu, window=4)
    with pytest.raises(kda.KDAError, match="workspace smaller"):
        kda.attn_window_prefill_backward_t(q, k, v, o, lse, d_o, cu, window=4,
                                           workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
