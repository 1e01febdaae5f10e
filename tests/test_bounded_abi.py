"""The entry points of windowed attention on the CPU: every refusal comes
before any HIP call (no kernel is launched here)."""
import pytest

import gated_delta_rule_60_amd as kda
from test_attn_abi import BAD, BF16, COMMON, F32, FAKE, NOT


def _prefill(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, cu_seqlens=FAKE, N=1, T_tot=64, H_q=4, H_kv=2, d_k=64, d_v=32, q_stride=256,
             k_stride=128, v_stride=64, window=16, sinks=4, scale=0.125, dtype=BF16, o=FAKE, lse=FAKE, stream=None)
    a.update(kw)
    return kda.attn_window_prefill(**a)


def _backward(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, d_o=FAKE, cu_seqlens=FAKE, N=1, T_tot=64, H_q=4, H_kv=2,
             d_k=64, d_v=32, q_stride=256, k_stride=128, v_stride=64, window=16, sinks=4, scale=0.125, dtype=BF16,
             d_q=FAKE, d_k_out=FAKE, d_v_out=FAKE, workspace=FAKE, workspace_bytes=1 << 40, stream=None)
    a.update(kw)
    return kda.attn_window_prefill_backward(**a)


WINDOW = [
    (dict(window=0), BAD, "window"),
    (dict(window=-3), BAD, "window"),
    (dict(window=(1 << 30) + 1), BAD, "window"),
    (dict(sinks=-1), BAD, "sinks"),
    (dict(sinks=257), BAD, "sinks"),
]


@pytest.mark.parametrize("kw,status,needle", COMMON + WINDOW)
def test_window_prefill_refuses(kw, status, needle):
    assert _prefill(**kw) == status
    assert needle in kda.kda_last_error()


@pytest.mark.parametrize("kw,status,needle", COMMON + WINDOW + [
    (dict(lse=None), BAD, "lse"),
    (dict(d_o=None), BAD, "d_o"),
    (dict(d_k_out=None), BAD, "must not be NULL"),
    (dict(d_v_out=FAKE + 8), BAD, "16-byte aligned"),
    (dict(workspace=None), BAD, "workspace must not be NULL"),
    (dict(workspace=FAKE + 16), BAD, "256-byte aligned"),
    (dict(workspace_bytes=64 * 4 * 8), BAD, "workspace smaller"),
    (dict(N=1 << 21, T_tot=300, sinks=256, H_q=2, H_kv=1), BAD, "ceil(sinks / 32)"),
])
def test_window_backward_refuses(kw, status, needle):
    assert _backward(**kw) == status
    assert needle in kda.kda_last_error()


def test_window_backward_workspace():
    size = kda.attn_window_prefill_backward_workspace_size
    plain = kda.attn_prefill_backward_workspace_size(2, 100000, 8, 8, 64, 64, BF16)
    assert size(2, 100000, 8, 8, 64, 64, 512, 0, BF16) == plain  # no sinks: nothing past a window
    assert size(2, 100000, 8, 8, 64, 64, 100000, 4, BF16) == plain  # a window that holds everything
    assert size(2, 100000, 8, 8, 64, 64, 512, 4, BF16) > plain
    assert size(2, 100000, 8, 8, 64, 64, 512, 33, F32) > size(2, 100000, 8, 8, 64, 64, 512, 32, F32)
    for kw in ((0, 10, 1, 1, 64, 64, 5, 1, BF16), (1, -1, 1, 1, 64, 64, 5, 1, BF16), (1, 10, 3, 2, 64, 64, 5, 1, BF16),
               (1, 10, 1, 1, 48, 64, 5, 1, BF16), (1, 10, 1, 1, 64, 64, 0, 1, BF16), (1, 10, 1, 1, 64, 64, 5, 300, BF16),
               (1, 10, 1, 1, 64, 64, 5, 1, 7)):
        assert size(*kw) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_window_backward_workspace_of_short_sequences(dtype):
    """What the sinks' rows take goes by the sequences that can be longer than the window, T_tot / (window + 1), not by
    all: 4096 sequences of 64 tokens with a window of 1024 took 2.2 GB."""
    size = kda.attn_window_prefill_backward_workspace_size
    for n, t, window, sinks in ((4096, 4096 * 64, 1024, 4), (4096, 4096 * 64, 1024, 32), (100000, 400000, 8000, 64)):
        plain = kda.attn_prefill_backward_workspace_size(n, t, 32, 8, 128, 128, dtype)
        blocks, bands = (sinks + 31) // 32, t // (window + 1)
        part = 32 * blocks * 8 * 256 * 4  # of a piece or a sequence
        assert size(n, t, 32, 8, 128, 128, window, sinks, dtype) <= plain + part * (2 * bands + 64)
    # one sequence can be longer than the window, however many there are
    assert size(1000, 2000, 8, 8, 64, 64, 1500, 4, dtype) <= size(1, 2000, 8, 8, 64, 64, 1500, 4, dtype) + 2 * 32 * 8 * 128 * 4
    # a batch of as many long ones as fit
    assert size(16, 16 * 1025, 32, 8, 128, 128, 1024, 4, dtype) >= 16 * 2 * 32 * 8 * 256 * 4


def test_window_backward_cuts_long_sequences_whatever_stands_beside_them():
    """Pieces of the rows behind the sinks' windows, as the workspace has places for them: workgroups for at
    least half of 256 compute units, also beside many sequences and with many sinks.  (One piece a sequence from 31
    sequences on, or with 256 sinks from 4, left a long one's rows to 8 workgroups.)"""
    for n, t, sinks in ((32, 8192 + 31 * 256, 4), (32, 8192 + 31 * 256, 64), (4, 16214, 64), (4, 16214, 256), (64, 40000, 4)):
        plain = kda.attn_prefill_backward_workspace_size(n, t, 32, 8, 128, 128, BF16)
        blocks, bands = (sinks + 31) // 32, min(n, t // 1025)
        part = 32 * blocks * 8 * 256 * 4
        pieces = (kda.attn_window_prefill_backward_workspace_size(n, t, 32, 8, 128, 128, 1024, sinks, BF16) - plain) // part - bands
        assert pieces >= 256 // (blocks * 8) // 2, (n, t, sinks, pieces)
    # the largest numbers: no overflow on the way
    assert kda.attn_window_prefill_backward_workspace_size(1, 1 << 30, 4096, 4096, 32, 32, 1, 256, BF16) > 0


def _window_decode(**kw):
    a = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, block_table=FAKE, ctx_lens=FAKE, cu_q=FAKE, N=2, T_q=3, H_q=4, H_kv=2, d_k=64,
             d_v=32, n_pages=100, page_size=16, max_pages=50, q_stride=256, window=64, sinks=4, scale=0.125, dtype=BF16, o=FAKE,
             lse=FAKE, workspace=FAKE, workspace_bytes=1 << 40, stream=None)
    a.update(kw)
    return kda.attn_window_decode(**a)


def _weighed(**kw):
    a = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, block_table=FAKE, ctx_lens=FAKE, N=2, H_q=4, H_kv=2, d_k=64, d_v=32, n_pages=100,
             page_size=16, max_pages=50, q_stride=256, scale=0.125, dtype=BF16, o=FAKE, lse=FAKE, weights=FAKE, workspace=FAKE,
             workspace_bytes=1 << 40, stream=None)
    a.update(kw)
    return kda.attn_weighed_decode(**a)


DECODE = [
    (dict(N=0), BAD, "N >= 1"),
    (dict(H_q=3), BAD, "multiple of H_kv"),
    (dict(d_k=48), NOT, "d_k and d_v"),
    (dict(dtype=2), NOT, "dtype"),
    (dict(page_size=24), BAD, "page_size"),
    (dict(page_size=8192), BAD, "page_size"),
    (dict(n_pages=0), BAD, "n_pages"),
    (dict(n_pages=1 << 28), BAD, "2^31"),
    (dict(max_pages=0), BAD, "max_pages"),
    (dict(max_pages=1 << 27), BAD, "2^30"),
    (dict(q_stride=248), BAD, "q_stride"),
    (dict(scale=0.0), BAD, "scale"),
    (dict(q=None), BAD, "must not be NULL"),
    (dict(v_cache=None), BAD, "must not be NULL"),
    (dict(o=None), BAD, "must not be NULL"),
    (dict(block_table=None), BAD, "must not be NULL"),
    (dict(ctx_lens=None), BAD, "must not be NULL"),
    (dict(k_cache=FAKE + 8), BAD, "16-byte aligned"),
    (dict(ctx_lens=FAKE + 2), BAD, "4-byte aligned"),
    (dict(workspace=None), BAD, "workspace must not be NULL"),
    (dict(workspace=FAKE + 16), BAD, "256-byte aligned"),
    (dict(workspace_bytes=64), BAD, "workspace smaller"),
]


@pytest.mark.parametrize("kw,status,needle", DECODE + WINDOW + [
    (dict(T_q=-1), BAD, "T_q"),
    (dict(T_q=(1 << 24) + 1), BAD, "T_q"),
    (dict(cu_q=None), BAD, "cu_q"),
    (dict(cu_q=FAKE + 2), BAD, "4-byte aligned"),
])
def test_window_decode_refuses(kw, status, needle):
    assert _window_decode(**kw) == status
    assert needle in kda.kda_last_error()


@pytest.mark.parametrize("kw,status,needle", DECODE + [
    (dict(weights=None), BAD, "weights"),
    (dict(weights=FAKE + 2), BAD, "weights"),
    (dict(N=(1 << 24) + 1), BAD, "2^24"),
    (dict(N=1 << 20, page_size=4096, max_pages=1 << 10), BAD, "for sequences this long"),
])
def test_weighed_decode_refuses(kw, status, needle):
    assert _weighed(**kw) == status
    assert needle in kda.kda_last_error()


def test_decode_workspaces():
    size = kda.attn_window_decode_workspace_size
    assert 0 < size(1, 1, 32, 8, 128, 16, 8192, 1000, 4) <= kda.attn_tree_decode_workspace_size(1, 1, 32, 8, 128, 16, 8192)
    assert size(1, 1, 32, 8, 128, 16, 8192, 1 << 30, 4) == kda.attn_tree_decode_workspace_size(1, 1, 32, 8, 128, 16, 8192)
    weighed = kda.attn_weighed_decode_workspace_size(3, 8, 2, 64, 16, 10)
    assert weighed >= kda.attn_tree_decode_workspace_size(3, 3, 8, 2, 64, 16, 10) + 3 * 8 * (160 + 1) * 4
    for kw in ((0, 1, 1, 1, 64, 16, 10, 5, 1), (1, -1, 1, 1, 64, 16, 10, 5, 1), (1, 1, 3, 2, 64, 16, 10, 5, 1),
               (1, 1, 1, 1, 48, 16, 10, 5, 1), (1, 1, 1, 1, 64, 15, 10, 5, 1), (1, 1, 1, 1, 64, 16, 0, 5, 1),
               (1, 1, 1, 1, 64, 16, 10, 0, 1), (1, 1, 1, 1, 64, 16, 10, 5, 257)):
        assert size(*kw) == 0
    for kw in ((0, 1, 1, 64, 16, 10), (1, 3, 2, 64, 16, 10), (1, 1, 1, 48, 16, 10), (1, 1, 1, 64, 15, 10), (1, 1, 1, 64, 16, 0)):
        assert kda.attn_weighed_decode_workspace_size(*kw) == 0


def _weights(**kw):
    a = dict(q=FAKE, k=FAKE, lse=FAKE, cu_seqlens=FAKE, N=1, T_tot=64, H_q=4, H_kv=2, d_k=64, q_stride=256, k_stride=128, rows=32,
             scale=0.125, dtype=BF16, weights=FAKE, width=64, workspace=FAKE, workspace_bytes=1 << 40, stream=None)
    a.update(kw)
    return kda.attn_prefill_weights(**a)


@pytest.mark.parametrize("kw,status,needle", [c for c in COMMON if not {"v", "o", "d_v", "v_stride"} & set(c[0])] + [
    (dict(lse=None), BAD, "lse"),
    (dict(rows=0), BAD, "rows"),
    (dict(rows=-1), BAD, "rows"),
    (dict(width=0), BAD, "width"),
    (dict(width=(1 << 30) + 1), BAD, "width"),
    (dict(weights=None), BAD, "weights"),
    (dict(weights=FAKE + 2), BAD, "weights"),
    (dict(width=1 << 30, N=2, H_q=4, H_kv=2), BAD, "ceil(width / 256)"),
    (dict(T_tot=2000, rows=2000, workspace=None), BAD, "workspace must not be NULL"),
    (dict(T_tot=2000, rows=2000, workspace=FAKE + 16), BAD, "256-byte aligned"),
    (dict(T_tot=2000, rows=2000, workspace_bytes=2000 * 2 * 4), BAD, "workspace smaller"),
])
def test_prefill_weights_refuses(kw, status, needle):
    assert _weights(**kw) == status
    assert needle in kda.kda_last_error()


def test_prefill_weights_workspace():
    size = kda.attn_prefill_weights_workspace_size
    assert size(1, 300, 2, 2, 32) == 0  # a few rows: one part
    assert size(1, 4000, 8, 2, 4000) >= 2 * 2 * 4000 * 4
    for kw in ((0, 10, 1, 1, 5), (1, -1, 1, 1, 5), (1, 10, 3, 2, 5), (1, 10, 1, 1, 0)):
        assert size(*kw) == 0


def _evict(**kw):
    a = dict(block_table=FAKE, lens=FAKE + (1 << 20), held=FAKE + (2 << 20), refs=FAKE + (3 << 20), free_list=FAKE, n_free=FAKE,
             n_rows=8, n_pages=100, page_size=16, max_pages=50, rows=FAKE + (4 << 20), n=4, k_cache=FAKE, v_cache=FAKE, n_layers=2,
             H_kv=2, d_k=64, d_v=32, dtype=BF16, weights=FAKE, budget=64, recent=16, sinks=4, status=FAKE + (5 << 20), stream=None)
    a.update(kw)
    return kda.kv_evict(**a)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(n_rows=0), BAD, "n_rows"),
    (dict(page_size=24), BAD, "page_size"),
    (dict(n_pages=0), BAD, "n_pages"),
    (dict(max_pages=0), BAD, "max_pages"),
    (dict(n=-1), BAD, "1024"),
    (dict(n=1025), BAD, "1024"),
    (dict(rows=None), BAD, "must not be NULL"),
    (dict(status=None), BAD, "must not be NULL"),
    (dict(refs=None), BAD, "must not be NULL"),
    (dict(rows=FAKE + 2), BAD, "4-byte aligned"),
    (dict(k_cache=None), BAD, "must not be NULL"),
    (dict(v_cache=FAKE + 8), BAD, "16-byte aligned"),
    (dict(n_layers=0), BAD, "n_layers"),
    (dict(H_kv=0), BAD, "H_kv"),
    (dict(d_k=48), NOT, "d_k and d_v"),
    (dict(dtype=3), NOT, "dtype"),
    (dict(weights=FAKE + 2), BAD, "weights"),
    (dict(weights=None), BAD, "without weights"),
    (dict(budget=0, recent=0, sinks=0), BAD, "budget"),
    (dict(budget=(1 << 30) + 1), BAD, "budget"),
    (dict(recent=-1), BAD, "recent"),
    (dict(sinks=-1), BAD, "sinks"),
    (dict(recent=61), BAD, "recent + sinks"),
    (dict(recent=2 ** 31 - 1, sinks=2 ** 31 - 1), BAD, "recent + sinks"),
    (dict(n=1024, n_layers=64, H_kv=64), BAD, "n * n_layers * H_kv"),
    (dict(status=FAKE + (4 << 20) + 12), BAD, "status"),
    (dict(status=FAKE + (1 << 20) + 28), BAD, "status"),
    (dict(status=FAKE + 396), BAD, "status"),
])
def test_evict_refuses(kw, status, needle):
    assert _evict(**kw) == status
    assert needle in kda.kda_last_error()


@pytest.mark.parametrize("kw", [dict(n_free=FAKE + (5 << 20)), dict(n_free=FAKE + (5 << 20) + 12), dict(free_list=FAKE + (5 << 20) - 396)])
def test_evict_refuses_a_status_over_the_free_pages(kw):
    """The pages are given back by a second launch, which reads their number and list after status is written."""
    assert _evict(**kw) == BAD
    assert "status" in kda.kda_last_error()


@pytest.mark.parametrize("call,kw,name", [
    (_prefill, dict(window=(1 << 32) + 5), "window"), (_prefill, dict(sinks=1 << 32), "sinks"),
    (_backward, dict(window=(1 << 32) + 5), "window"), (_window_decode, dict(window=(1 << 32) + 5), "window"),
    (_window_decode, dict(sinks=-(1 << 32)), "sinks"), (_weights, dict(rows=(1 << 32) + 1), "rows"),
    (_weights, dict(width=(1 << 32) + 64), "width"), (_evict, dict(budget=(1 << 32) + 64), "budget"),
    (_evict, dict(recent=(1 << 32) + 16), "recent"), (_evict, dict(sinks=1 << 40), "sinks")])
def test_numbers_past_32_bits_are_not_cut(call, kw, name):
    """ctypes takes the lowest 32 bits of a number: a window of 2^32 + 5 would have been one of 5."""
    with pytest.raises(ValueError, match=name):
        call(**kw)


def test_workspaces_of_numbers_past_32_bits():
    assert kda.attn_window_prefill_backward_workspace_size(1, 1000, 4, 2, 64, 64, (1 << 32) + 5, 4, BF16) == 0
    assert kda.attn_window_decode_workspace_size(1, 1, 4, 2, 64, 16, 100, 64, 1 << 32) == 0
    assert kda.attn_prefill_weights_workspace_size(1, 4000, 8, 2, (1 << 32) + 4000) == 0
