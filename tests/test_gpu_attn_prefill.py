"""Prompt attention and its backward pass against a 64-bit reference, at the
sizes and layouts where they can go wrong."""
import math

import pytest
import torch

import attn_ref
import gated_delta_rule_60_amd as kda

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _make(lens, hq, hkv, dk, dv, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    t = sum(lens)
    r = lambda h, d: (spread * torch.randn(t, h, d, generator=g)).to(DT[dtype]).cuda()  # noqa: E731
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32).cuda()
    return r(hq, dk), r(hkv, dk), r(hkv, dv), r(hq, dv) / spread, cu


def _check_all(lens, hq, hkv, dk, dv, dtype, seed, scale=None, spread=1.0):
    q, k, v, d_o, cu = _make(lens, hq, hkv, dk, dv, dtype, seed, spread)
    s = 1 / math.sqrt(dk) if scale is None else scale
    o, lse = kda.attn_prefill_t(q, k, v, cu, scale=scale)
    grads = kda.attn_prefill_backward_t(q, k, v, o, lse, d_o, cu, scale=scale)
    torch.cuda.synchronize()
    want = attn_ref.prefill(q, k, v, lens, s, d_o)
    for name, got in zip(("o", "lse", "d_q", "d_k", "d_v"), (o, lse, *grads)):
        attn_ref.check(got, want[name], f"{dtype} {name}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_head_sizes(dtype, dk, dv):
    _check_all([70, 131], 2, 1, dk, dv, dtype, 100 + dk + dv)


# Batches that fill the device run whole 128-row blocks; the small ones above and below split their
# keys (or rows) over the waves of a block.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_head_sizes_of_a_full_batch(dtype, dk, dv):
    _check_all([70, 131] * 30, 4, 4, dk, dv, dtype, 200 + dk + dv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,hq,hkv", [([1, 0, 300, 129, 128, 127, 65, 64, 63, 33, 32, 31] * 8, 6, 3), ([200] * 90, 6, 3),
                                         ([1] * 300, 1, 1), ([700, 1, 513], 40, 40), ([1000], 66, 33)])
def test_lengths_and_groups_of_a_full_batch(dtype, lens, hq, hkv):
    _check_all(lens, hq, hkv, 64, 64, dtype, len(lens))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (8, 2), (6, 2), (5, 1), (9, 9)])
def test_head_groups(dtype, hq, hkv):
    _check_all([40, 65], hq, hkv, 32, 64, dtype, 7 * hq + hkv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [2], [31, 32, 33], [63, 64, 65], [127, 128, 129], [1, 0, 0, 5, 1], [0, 300, 0],
                                  [257, 256, 255], [1] * 70, [3, 130] * 40])
def test_lengths(dtype, lens):
    _check_all(lens, 2, 1, 64, 64, dtype, len(lens) + sum(lens))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_longer_sequences(dtype):
    _check_all([1500, 777], 2, 1, 128, 128, dtype, 5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale,spread", [(1.0, 1.0), (1e-3, 1.0), (0.3, 3.0)])
def test_scales(dtype, scale, spread):
    """Peaked rows (scores of tens) and flat ones."""
    _check_all([200, 33], 2, 2, 64, 32, dtype, 11, scale, spread)


def test_a_score_far_above_the_rest_moves_the_maximum():
    """The running maximum moves late and far: the first keys' scores are near
    zero, one key in the middle lies at 200, the last again near zero."""
    q, k, v, d_o, cu = _make([300], 2, 1, 64, 64, "f32", 3)
    k[150] = 25.0 * q[0, 0] / q[0, 0].norm()
    q[151:] = 0.2 * q[151:] + 8.0 * q[0] / q[0].norm(dim=-1, keepdim=True)
    o, lse = kda.attn_prefill_t(q, k, v, cu, scale=1.0)
    grads = kda.attn_prefill_backward_t(q, k, v, o, lse, d_o, cu, scale=1.0)
    want = attn_ref.prefill(q, k, v, [300], 1.0, d_o)
    assert float(want["lse"][0][200:].max()) > 100
    for name, got in zip(("o", "lse", "d_q", "d_k", "d_v"), (o, lse, *grads)):
        attn_ref.check(got, want[name], name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_of_a_fused_projection(dtype):
    """q, k and v as views of one [T, (H_q + 2 H_kv) d] tensor: the same bits
    as from contiguous copies."""
    lens, hq, hkv, d = [100, 37], 4, 2, 64
    g = torch.Generator().manual_seed(1)
    fused = torch.randn(137, (hq + 2 * hkv) * d, generator=g).to(DT[dtype]).cuda()
    q, k, v = fused.split([hq * d, hkv * d, hkv * d], 1)
    q, k, v = q.view(137, hq, d), k.view(137, hkv, d), v.view(137, hkv, d)
    cu = torch.tensor([0, 100, 137], dtype=torch.int32).cuda()
    d_o = torch.randn(137, hq, d, generator=g).to(DT[dtype]).cuda()
    o, lse = kda.attn_prefill_t(q, k, v, cu)
    grads = kda.attn_prefill_backward_t(q, k, v, o, lse, d_o, cu)
    c = [x.contiguous() for x in (q, k, v)]
    o2, lse2 = kda.attn_prefill_t(*c, cu)
    grads2 = kda.attn_prefill_backward_t(*c, o2, lse2, d_o, cu)
    for x, y in zip((o, lse, *grads), (o2, lse2, *grads2)):
        assert torch.equal(x, y)
    attn_ref.check(o, attn_ref.prefill(q, k, v, lens, 1 / 8)["o"], "o")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_last_sequence_stay(dtype):
    q, k, v, d_o, _ = _make([150], 2, 1, 32, 32, dtype, 9)
    cu = torch.tensor([0, 60, 90], dtype=torch.int32).cuda()
    for x in (q, k, v, d_o):
        x[90:] = float("nan")  # padding holds anything
    o = torch.full((150, 2, 32), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((150, 2), 7.0, device="cuda")
    kda.attn_prefill_t(q, k, v, cu, o=o, lse=lse)
    assert (o[90:] == 7).all() and (lse[90:] == 7).all()
    grads = kda.attn_prefill_backward_t(q, k, v, o, lse, d_o, cu)
    want = attn_ref.prefill(q[:90], k[:90], v[:90], [60, 30], 1 / math.sqrt(32), d_o[:90])
    for name, got in zip(("o", "lse", "d_q", "d_k", "d_v"), (o, lse, *grads)):
        attn_ref.check(got[:90], want[name], name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_sequence_does_not_see_its_neighbours_values(dtype):
    """Non-finite keys and values of one sequence stay there."""
    q, k, v, d_o, cu = _make([70, 50, 90], 2, 1, 64, 64, dtype, 13)
    want = kda.attn_prefill_t(q, k, v, cu)
    gw = kda.attn_prefill_backward_t(q, k, v, *want, d_o, cu)
    k[70:120], v[70:120] = float("nan"), float("inf")
    o, lse = kda.attn_prefill_t(q, k, v, cu)
    grads = kda.attn_prefill_backward_t(q, k, v, o, lse, d_o, cu)
    for x, y in zip((o, lse, *grads), (*want, *gw)):
        assert torch.equal(x[:70], y[:70]) and torch.equal(x[120:], y[120:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 5, 31, 32, 63, 64, 130, 199])
@pytest.mark.parametrize("dv", [32, 128])
@pytest.mark.parametrize("full", [False, True])
def test_earlier_rows_do_not_see_a_later_token(dtype, at, dv, full):
    """NaN and infinite keys and values of token `at`: the rows before it keep
    their bits, its own and the later ones turn NaN (or infinite)."""
    q, k, v, _, cu = _make([200] + [64] * (150 if full else 0), 2, 1, 64, dv, dtype, 17)
    n = 200  # the rows that may change
    want, lse_want = kda.attn_prefill_t(q, k, v, cu)
    for bad in (float("nan"), float("inf"), -float("inf")):
        v2 = v.clone()
        v2[at, 0, 3] = bad
        o, lse = kda.attn_prefill_t(q, k, v2, cu)
        assert torch.equal(o[:at], want[:at]) and torch.equal(o[n:], want[n:]) and torch.equal(lse, lse_want)
        if bad != bad:
            assert torch.isnan(o[at:n, :, 3]).all()
        else:
            assert (o[at:n, :, 3].float() == bad).all()
        rest = [i for i in range(dv) if i != 3]
        assert torch.equal(o[..., rest], want[..., rest])
        k2 = k.clone()
        k2[at, 0, 7] = bad
        o, lse = kda.attn_prefill_t(q, k2, v, cu)
        assert torch.equal(o[:at], want[:at]) and torch.equal(lse[:at], lse_want[:at])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_outside_the_batch_are_clamped(dtype):
    q, k, v, _, _ = _make([100], 2, 1, 32, 32, dtype, 2)
    o = torch.full((100, 2, 32), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((100, 2), 7.0, device="cuda")
    bad = torch.tensor([-5, 40, 30, 2 ** 30], dtype=torch.int32).cuda()
    kda.attn_prefill_t(q, k, v, bad, o=o, lse=lse)
    good, _ = kda.attn_prefill_t(q, k, v, torch.tensor([0, 40], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert torch.equal(o[:30], good[:30])  # rows that one sequence alone covers


def test_the_same_bits_every_time():
    q, k, v, d_o, cu = _make([900, 40, 333], 8, 2, 128, 128, "bf16", 4)
    first = None
    for _ in range(4):
        o, lse = kda.attn_prefill_t(q, k, v, cu)
        r = (o, lse, *kda.attn_prefill_backward_t(q, k, v, o, lse, d_o, cu))
        torch.cuda.synchronize()
        first = first or r
        assert all(torch.equal(x, y) for x, y in zip(first, r))


def test_gradients_against_differences():
    """fp32: L(x + h d) - L(x - h d) over 2 h, L summed in 64 bits from the
    kernel's own fp32 outputs.  The outputs are within 2^-20 of exact here
    (|o| < 4), so the quotient is off by at most sqrt-free 2^-20 |d_o|_1 / h
    from rounding (in practice far less: errors average), and by h^2 terms."""
    q, k, v, d_o, cu = _make([50, 33], 4, 2, 32, 32, "f32", 21)
    o, lse = kda.attn_prefill_t(q, k, v, cu)
    grads = kda.attn_prefill_backward_t(q, k, v, o, lse, d_o, cu)
    g = torch.Generator().manual_seed(2)
    for i in range(3):
        d = torch.randn(grads[i].shape, generator=g).cuda()
        want = float((grads[i].double() * d.double()).sum())
        h = 2.0 ** -7
        loss = []
        for sign in (1, -1):
            x = [q, k, v]
            x[i] = x[i] + sign * h * d
            loss.append(float((kda.attn_prefill_t(*x, cu)[0].double() * d_o.double()).sum()))
        got = (loss[0] - loss[1]) / (2 * h)
        size = float(grads[i].norm() * d.norm())
        print(f"    input {i}: differences {got:.6f}, gradient {want:.6f}, size {size:.3f}", flush=True)
        # third derivatives: h^2 / 6 of the same scale as the gradient times |d|^2 a row (d_k entries): 2^-14 * 32 / 6
        assert abs(got - want) <= size * (2.0 ** -14 * 32 / 6 + 2.0 ** -13)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_another_stream_and_graph_replays(dtype):
    q, k, v, d_o, cu = _make([200, 61], 4, 2, 64, 64, dtype, 31)
    o0, lse0 = kda.attn_prefill_t(q, k, v, cu)
    g0 = kda.attn_prefill_backward_t(q, k, v, o0, lse0, d_o, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o1, lse1 = kda.attn_prefill_t(q, k, v, cu, stream=side)
    g1 = kda.attn_prefill_backward_t(q, k, v, o1, lse1, d_o, cu, stream=side)
    side.synchronize()
    for x, y in zip((o0, lse0, *g0), (o1, lse1, *g1)):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, lse2 = kda.attn_prefill_t(q, k, v, cu)
        g2 = kda.attn_prefill_backward_t(q, k, v, o2, lse2, d_o, cu)
    for n in range(3):
        q.mul_(1.0 + n / 4)
        for x in (o2, lse2, *g2):
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        o3, lse3 = kda.attn_prefill_t(q, k, v, cu)
        g3 = kda.attn_prefill_backward_t(q, k, v, o3, lse3, d_o, cu)
        torch.cuda.synchronize()
        for x, y in zip((o2, lse2, *g2), (o3, lse3, *g3)):
            assert torch.equal(x, y), f"replay {n}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_tokens(dtype):
    q, k, v, d_o, _ = _make([0], 4, 2, 64, 32, dtype, 1)
    for cu in (None, torch.zeros(4, dtype=torch.int32).cuda()):
        o, lse = kda.attn_prefill_t(q, k, v, cu)
        assert o.shape == (0, 4, 32) and lse.shape == (0, 4)
        grads = kda.attn_prefill_backward_t(q, k, v, o, lse, d_o, cu)
        assert [tuple(x.shape) for x in grads] == [(0, 4, 64), (0, 2, 64), (0, 2, 32)]
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("full", [False, True])
def test_rows_before_the_first_sequence_stay(dtype, full):
    lens = [40, 100] + [64] * (150 if full else 0)
    q, k, v, d_o, _ = _make([50] + lens, 2, 1, 64, 64, dtype, 19)
    cu = torch.tensor([50, *(50 + torch.tensor(lens).cumsum(0)).tolist()], dtype=torch.int32).cuda()
    for x in (q, k, v, d_o):
        x[:50] = float("nan")
    o = torch.full((q.shape[0], 2, 64), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((q.shape[0], 2), 7.0, device="cuda")
    kda.attn_prefill_t(q, k, v, cu, o=o, lse=lse)
    assert (o[:50] == 7).all() and (lse[:50] == 7).all()
    grads = kda.attn_prefill_backward_t(q, k, v, o, lse, d_o, cu)
    want = attn_ref.prefill(q[50:], k[50:], v[50:], lens, 1 / 8, d_o[50:])
    for name, got in zip(("o", "lse", "d_q", "d_k", "d_v"), (o, lse, *grads)):
        attn_ref.check(got[50:], want[name], name)


def test_a_captured_call_without_offsets():
    q, k, v, _, cu = _make([150], 4, 2, 64, 32, "bf16", 9)
    kda.attn_prefill_t(q, k, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = kda.attn_prefill_t(q, k, v)
    for n in range(3):
        v.mul_(1.0 + n / 4)
        o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = kda.attn_prefill_t(q, k, v, cu)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), f"replay {n}"


@pytest.mark.parametrize("lens", [[40, 9], [300] * 60])
def test_the_row_statistics_may_be_left_out(lens):
    q, k, v, _, cu = _make(lens, 4, 2, 64, 32, "bf16", 6)
    want, _ = kda.attn_prefill_t(q, k, v, cu)
    o = torch.empty_like(want)
    st = torch.cuda.current_stream().cuda_stream
    rc = kda.attn_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu.data_ptr(), len(lens), sum(lens), 4, 2, 64, 32, 256, 128, 64,
                          1 / 8, kda.KDA_DTYPE_BF16, o.data_ptr(), None, st)
    assert rc == kda.KDA_OK
    torch.cuda.synchronize()
    assert torch.equal(o, want)


def test_two_backward_calls_at_once():
    a, b = _make([500, 33], 8, 2, 64, 64, "bf16", 1), _make([300, 7], 8, 2, 64, 64, "bf16", 2)
    fwd = [kda.attn_prefill_t(*x[:3], x[4]) for x in (a, b)]
    want = [kda.attn_prefill_backward_t(*x[:3], *f, x[3], x[4]) for x, f in zip((a, b), fwd)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, (x, f) in enumerate(zip((a, b), fwd)):
            got[i].append(kda.attn_prefill_backward_t(*x[:3], *f, x[3], x[4], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(p, q) for g in got[i] for p, q in zip(g, want[i]))


def test_offsets_past_32_bits():
    """Token rows 2^31 elements and more into a wide fused buffer."""
    stride, t = 1 << 16, 33000  # 2.16e9 elements, 4.3 GB
    fused = torch.zeros(t, stride, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    fused[:, :512] = torch.randn(t, 512, generator=g, device="cuda")
    q, k, v = fused[:, :256].view(t, 2, 128), fused[:, 256:384].view(t, 1, 128), fused[:, 384:512].view(t, 1, 128)
    cu = torch.tensor([0, 32800, 33000], dtype=torch.int32).cuda()
    d_o = torch.randn(t, 2, 128, generator=g, device="cuda").bfloat16()
    o, lse = kda.attn_prefill_t(q, k, v, cu)
    grads = kda.attn_prefill_backward_t(q, k, v, o, lse, d_o, cu)
    tail = [x[32800:].contiguous() for x in (q, k, v)]
    want = attn_ref.prefill(*tail, [200], 1 / math.sqrt(128), d_o[32800:])
    for name, got in zip(("o", "lse", "d_q", "d_k", "d_v"), (o, lse, *grads)):
        attn_ref.check(got[32800:], want[name], name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("full", [False, True])
def test_scores_below_the_range_weigh_nothing(dtype, full):
    """Finite queries and keys whose products pass -2^128, for every key of the first tiles: -infinity in
    32 bits, and a weight of e^-10^39 = 0 by the formula.  The later rows are those of the later keys alone."""
    gone, n = 100, 300
    q, k, v, d_o, cu = _make([n] + [64] * (150 if full else 0), 2, 1, 64, 64, dtype, 23)
    q[:n, :, 0], k[:gone, :, 0], k[gone:n, :, 0] = 1e20, -1e20, 0.0
    o, lse = kda.attn_prefill_t(q, k, v, cu)
    grads = kda.attn_prefill_backward_t(q, k, v, o, lse, d_o, cu)
    torch.cuda.synchronize()
    q, k, v, d_o = (x[:n].cpu().double() for x in (q, k, v, d_o))
    seen = torch.tril(torch.ones(n, n, dtype=torch.bool))[gone:]
    seen[:, :gone] = False
    parts = []
    for h in range(2):
        r = attn_ref.attend(q[gone:, h], k[:, 0], v[:, 0], seen, 1 / 8, DT[dtype], d_o[gone:, h])
        for name, got in (("o", o), ("lse", lse), ("d_q", grads[0])):
            attn_ref.check(got[gone:n, h], r[name], f"{name} head {h}")
        parts.append(r)
    for name, got in (("d_k", grads[1]), ("d_v", grads[2])):
        value, bound = (sum(r[name][i][gone:] for r in parts) for i in range(2))
        attn_ref.check(got[gone:n, 0], (value, bound), name)


def test_torch_helper_refusals():
    q, k, v, d_o, cu = _make([20], 4, 2, 32, 32, "f32", 1)
    with pytest.raises(ValueError, match="shape"):
        kda.attn_prefill_t(q, k[:10], v, cu)
    with pytest.raises(TypeError, match="k must be"):
        kda.attn_prefill_t(q, k.bfloat16(), v, cu)
    with pytest.raises(TypeError):
        kda.attn_prefill_t(q.half(), k.half(), v.half(), cu)
    with pytest.raises(ValueError, match="is on cpu"):
        kda.attn_prefill_t(q, k.cpu(), v, cu)
    with pytest.raises(kda.KDAError, match="multiple of H_kv"):
        kda.attn_prefill_t(q[:, :3], k, v, cu)
    with pytest.raises(kda.KDAError, match="scale"):
        kda.attn_prefill_t(q, k, v, cu, scale=-1.0)
    o, lse = kda.attn_prefill_t(q, k, v, cu)
    with pytest.raises(kda.KDAError, match="workspace smaller"):
        kda.attn_prefill_backward_t(q, k, v, o, lse, d_o, cu, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
