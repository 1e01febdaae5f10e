"""The attention and cache entry points on the CPU: every symbol declared in
include/kda.h is exported and bound, and every refusal comes before any HIP
call (no kernel is launched here)."""
import os
import re

import pytest

import gated_delta_rule_60_amd as kda
from gated_delta_rule_60_amd import _lib

_ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 256-byte aligned, never dereferenced: validation fails first
BF16, F32 = kda.KDA_DTYPE_BF16, kda.KDA_DTYPE_F32
BAD, NOT = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED


def test_every_declared_symbol_is_exported_and_bound():
    text = open(os.path.join(_ROOT, "include", "kda.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b((?:attn|kv)_[a-z_]+)\s*\(", text)))
    assert "attn_prefill" in names and "attn_prefill_backward" in names
    lib = kda.load()
    for name in names:
        assert hasattr(lib, name), f"{name} declared in kda.h but not exported"
        assert name in _lib.SIGNATURES, f"{name} has no signature in _lib.py"
        assert hasattr(kda, name), f"{name} has no binding"


def _prefill(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, cu_seqlens=FAKE, N=1, T_tot=64, H_q=4, H_kv=2, d_k=64, d_v=32, q_stride=256,
             k_stride=128, v_stride=64, scale=0.125, dtype=BF16, o=FAKE, lse=FAKE, stream=None)
    a.update(kw)
    return kda.attn_prefill(**a)


def _backward(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, d_o=FAKE, cu_seqlens=FAKE, N=1, T_tot=64, H_q=4, H_kv=2,
             d_k=64, d_v=32, q_stride=256, k_stride=128, v_stride=64, scale=0.125, dtype=BF16, d_q=FAKE,
             d_k_out=FAKE, d_v_out=FAKE, workspace=FAKE, workspace_bytes=1 << 40, stream=None)
    a.update(kw)
    return kda.attn_prefill_backward(**a)


COMMON = [
    (dict(N=0), BAD, "N >= 1"),
    (dict(T_tot=-1), BAD, "T_tot"),
    (dict(T_tot=(1 << 30) + 1), BAD, "2^30"),
    (dict(H_q=3), BAD, "multiple of H_kv"),
    (dict(H_kv=0), BAD, "multiple of H_kv"),
    (dict(H_q=0), BAD, "multiple of H_kv"),
    (dict(H_q=4098, q_stride=4098 * 64), BAD, "4096"),
    (dict(d_k=48), NOT, "d_k and d_v"),
    (dict(d_v=256), NOT, "d_k and d_v"),
    (dict(dtype=2), NOT, "dtype"),
    (dict(q_stride=248), BAD, "q_stride"),
    (dict(k_stride=132), BAD, "k_stride"),
    (dict(v_stride=(1 << 22) + 8), BAD, "v_stride"),
    (dict(scale=0.0), BAD, "scale"),
    (dict(scale=-1.0), BAD, "scale"),
    (dict(scale=float("inf")), BAD, "scale"),
    (dict(scale=float("nan")), BAD, "scale"),
    (dict(q=None), BAD, "must not be NULL"),
    (dict(v=None), BAD, "must not be NULL"),
    (dict(o=None), BAD, "must not be NULL"),
    (dict(cu_seqlens=None), BAD, "cu_seqlens"),
    (dict(k=FAKE + 8), BAD, "16-byte aligned"),
    (dict(lse=FAKE + 2), BAD, "4-byte aligned"),
    (dict(T_tot=1 << 30, H_q=2048, q_stride=2048 * 64), BAD, "too large"),
    (dict(T_tot=1 << 24, N=1 << 23), BAD, "too large"),  # 2^32 work items and more
]


@pytest.mark.parametrize("kw,status,needle", COMMON)
def test_prefill_refuses(kw, status, needle):
    assert _prefill(**kw) == status
    assert needle in kda.kda_last_error()


@pytest.mark.parametrize("kw,status,needle", COMMON + [
    (dict(lse=None), BAD, "lse"),
    (dict(d_o=None), BAD, "d_o"),
    (dict(d_k_out=None), BAD, "must not be NULL"),
    (dict(d_v_out=FAKE + 8), BAD, "16-byte aligned"),
    (dict(workspace=None), BAD, "workspace must not be NULL"),
    (dict(workspace=FAKE + 16), BAD, "256-byte aligned"),
    (dict(workspace_bytes=64 * 4 * 8 - 1), BAD, "workspace smaller"),
])
def test_backward_refuses(kw, status, needle):
    assert _backward(**kw) == status
    assert needle in kda.kda_last_error()


@pytest.mark.parametrize("N,T_tot,H_q", [
    (4095, 1, 4096),             # the one token makes a piece of its own: 4096 pieces of 4096 heads
    (4095, 127, 4096),
    (4094, 129, 4096),
    (4096, 0, 4096),
    (1, 128 * 32766 + 1, 512),   # 32767 pieces and one a sequence
])
def test_the_last_short_piece_of_rows_counts(N, T_tot, H_q):
    """2^32 work items: one more than a launch can count, refused before it."""
    kw = dict(N=N, T_tot=T_tot, H_q=H_q, H_kv=1, q_stride=H_q * 64)
    assert ((T_tot + 127) // 128 + N) * H_q * 256 == 1 << 32
    for call in (_prefill, _backward):
        assert call(**kw) == BAD
        assert "too large" in kda.kda_last_error()


def test_backward_workspace():
    size = kda.attn_prefill_backward_workspace_size
    big = size(8, 32677, 32, 8, 128, 128, BF16)  # the batch fills the device: two floats a row and head
    assert big == (32677 * 32 * 8 + 255) // 256 * 256
    few = size(5, 924, 8, 2, 64, 64, F32)        # a part of dk and dv for every query head of a key head
    assert few == 924 * 8 * 8 + 4 * 924 * 2 * 128 * 4
    assert size(5, 924, 2, 2, 64, 64, F32) == (924 * 2 * 8 + 255) // 256 * 256  # one head: one part
    for bad in ((0, 9, 4, 2, 64, 64, BF16), (1, -1, 4, 2, 64, 64, BF16), (1, 9, 3, 2, 64, 64, BF16),
                (1, 9, 4, 2, 48, 64, BF16), (1, 9, 4, 2, 64, 64, 5)):
        assert size(*bad) == 0


def _tree(**kw):
    a = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, block_table=FAKE, ctx_lens=FAKE, cu_q=FAKE, tree_mask=FAKE, N=4, T_q=16,
             H_q=8, H_kv=2, d_k=64, d_v=128, n_pages=100, page_size=16, max_pages=32, q_stride=512, scale=0.1,
             dtype=BF16, o=FAKE, lse=FAKE, workspace=FAKE, workspace_bytes=1 << 40, stream=None)
    a.update(kw)
    return kda.attn_tree_decode(**a)


CACHE = [
    (dict(page_size=12), BAD, "page_size"),
    (dict(page_size=0), BAD, "page_size"),
    (dict(page_size=-16), BAD, "page_size"),
    (dict(page_size=8192), BAD, "page_size"),
    (dict(n_pages=0), BAD, "n_pages"),
    (dict(n_pages=1 << 27), BAD, "2^31"),
    (dict(max_pages=0), BAD, "max_pages"),
    (dict(max_pages=(1 << 26) + 1), BAD, "2^30"),
]


@pytest.mark.parametrize("kw,status,needle", CACHE + [
    (dict(N=0), BAD, "N >= 1"),
    (dict(T_q=-1), BAD, "T_q"),
    (dict(T_q=(1 << 24) + 1), BAD, "T_q"),
    (dict(H_q=7), BAD, "multiple of H_kv"),
    (dict(d_k=16), NOT, "d_k and d_v"),
    (dict(dtype=3), NOT, "dtype"),
    (dict(q_stride=504), BAD, "q_stride"),
    (dict(scale=0.0), BAD, "scale"),
    (dict(block_table=None), BAD, "must not be NULL"),
    (dict(ctx_lens=None), BAD, "must not be NULL"),
    (dict(q=None), BAD, "must not be NULL"),
    (dict(o=None), BAD, "must not be NULL"),
    (dict(k_cache=FAKE + 8), BAD, "16-byte aligned"),
    (dict(tree_mask=FAKE + 4), BAD, "8-byte aligned"),
    (dict(cu_q=FAKE + 1), BAD, "4-byte aligned"),
    (dict(workspace_bytes=64), BAD, "workspace smaller"),
    (dict(workspace=None), BAD, "workspace must not be NULL"),
    (dict(workspace=FAKE + 128), BAD, "256-byte aligned"),
    (dict(T_q=1 << 24, max_pages=1 << 26), BAD, "too many drafted tokens"),
    (dict(T_q=1 << 24, H_q=256, q_stride=256 * 64), BAD, "too many drafted tokens"),
    (dict(T_q=1 << 24, N=1 << 24), BAD, "too many drafted tokens"),
    (dict(scale=3e38), BAD, "scale"),
])
def test_tree_refuses(kw, status, needle):
    assert _tree(**kw) == status
    assert needle in kda.kda_last_error()


def test_tree_workspace():
    size = kda.attn_tree_decode_workspace_size
    assert size(4, 16, 8, 2, 128, 16, 8) == 0        # one block of keys: nothing to join
    assert size(4, 16, 8, 2, 128, 16, 32) > 0
    assert size(4, 0, 8, 2, 128, 16, 32) == 0
    assert size(4, 16, 8, 2, 128, 16, 64) >= size(4, 16, 8, 2, 128, 16, 32)
    for bad in ((0, 16, 8, 2, 128, 16, 32), (4, -1, 8, 2, 128, 16, 32), (4, 16, 8, 3, 128, 16, 32),
                (4, 16, 8, 2, 48, 16, 32), (4, 16, 8, 2, 128, 12, 32), (4, 16, 8, 2, 128, 16, 0)):
        assert size(*bad) == 0


def test_tree_masks():
    torch = pytest.importorskip("torch")
    m = kda.attn_tree_masks([[-1, 0, 0, 1, -1], [], [-1] + list(range(63))])
    assert m.dtype == torch.int64 and m.tolist()[:5] == [1, 3, 5, 11, 16]
    assert m[5 + 63] == -1 and m[5 + 62] == (1 << 63) - 1
    with pytest.raises(ValueError, match="64"):
        kda.attn_tree_masks([[-1] * 65])
    for bad in ([0], [-1, 1], [-1, -2]):
        with pytest.raises(ValueError, match="parent"):
            kda.attn_tree_masks([bad])


_BOOK = dict(block_table=FAKE, lens=FAKE, held=FAKE, refs=FAKE, free_list=FAKE, n_free=FAKE, n_rows=8, n_pages=100,
             page_size=16, max_pages=32)
_LAYERS = dict(k_cache=FAKE, v_cache=FAKE, n_layers=2, H_kv=2, d_k=64, d_v=128, dtype=BF16)
_CALLS = {
    "kv_reserve": dict(_BOOK, rows=FAKE, n_tokens=FAKE, n=4, status=FAKE, stream=None),
    "kv_free": dict(_BOOK, rows=FAKE, n=4, stream=None),
    "kv_fork": dict(_BOOK, **_LAYERS, src=FAKE, dst=FAKE, n=4, status=FAKE, stream=None),
    "kv_append": dict(_LAYERS, k=FAKE, v=FAKE, block_table=FAKE, lens=FAKE, cu_new=FAKE, N=4, T_new=9, n_pages=100,
                      page_size=16, max_pages=32, stream=None),
    "kv_compact": dict(_LAYERS, block_table=FAKE, lens=FAKE, accepted=FAKE, cu_accepted=FAKE, N=4, A_tot=9, n_pages=100,
                       page_size=16, max_pages=32, new_lens=FAKE + 64, stream=None),
}
_SOME_ROWS = [(dict(n=-1), BAD, "1024"), (dict(n=1025), BAD, "1024"), (dict(n_rows=0), BAD, "n_rows"),
              (dict(held=None), BAD, "must not be NULL"), (dict(n_free=FAKE + 2), BAD, "4-byte aligned")]
_SOME_LAYERS = [(dict(n_layers=0), BAD, "n_layers"), (dict(n_layers=65536), BAD, "n_layers"), (dict(d_k=40), NOT, "d_k and d_v"),
                (dict(dtype=9), NOT, "dtype"), (dict(H_kv=0), BAD, "H_kv"), (dict(k_cache=None), BAD, "must not be NULL"),
                (dict(v_cache=FAKE + 8), BAD, "16-byte aligned")]


@pytest.mark.parametrize("call,kw,status,needle", [
    (call, *rest) for call in _CALLS for rest in
    CACHE + (_SOME_ROWS if "n" in _CALLS[call] else []) + (_SOME_LAYERS if "n_layers" in _CALLS[call] else [])] + [
    ("kv_reserve", dict(n_tokens=None), BAD, "must not be NULL"),
    ("kv_reserve", dict(status=None), BAD, "must not be NULL"),
    ("kv_free", dict(rows=None), BAD, "must not be NULL"),
    ("kv_free", dict(n=1024, max_pages=(1 << 19) + 1), BAD, "2^29"),
    ("kv_fork", dict(dst=None), BAD, "must not be NULL"),
    ("kv_append", dict(T_new=-1), BAD, "T_new"),
    ("kv_append", dict(T_new=(1 << 24) + 1), BAD, "T_new"),
    ("kv_append", dict(T_new=1 << 24), BAD, "T_new"),
    ("kv_compact", dict(N=1 << 24), BAD, "2^24"),
    ("kv_append", dict(N=0), BAD, "n_rows"),
    ("kv_append", dict(k=None), BAD, "must not be NULL"),
    ("kv_append", dict(v=FAKE + 8), BAD, "16-byte aligned"),
    ("kv_compact", dict(A_tot=-1), BAD, "A_tot"),
    ("kv_compact", dict(accepted=None), BAD, "must not be NULL"),
    ("kv_compact", dict(new_lens=FAKE), BAD, "must not be lens"),
])
def test_page_calls_refuse(call, kw, status, needle):
    assert getattr(kda, call)(**dict(_CALLS[call], **kw)) == status
    assert needle in kda.kda_last_error()


@pytest.mark.parametrize("call,kw,needle", [
    # N = 4: lens and new_lens are four numbers each; A_tot = 9; the table 4 x 32
    ("kv_compact", dict(lens=FAKE, new_lens=FAKE + 4), "must not be lens"),
    ("kv_compact", dict(lens=FAKE + 12, new_lens=FAKE), "must not be lens"),
    ("kv_compact", dict(accepted=FAKE + 4096, new_lens=FAKE + 4096 + 32), "accepted"),
    ("kv_compact", dict(cu_accepted=FAKE + 4096, new_lens=FAKE + 4096 + 16), "accepted"),
    ("kv_compact", dict(block_table=FAKE + 4096, new_lens=FAKE + 4096 + 4 * 127), "accepted"),
    ("kv_fork", dict(src=FAKE + 64, status=FAKE + 64), "status"),
    ("kv_fork", dict(dst=FAKE + 64, status=FAKE + 76), "status"),
    ("kv_fork", dict(dst=FAKE + 76, status=FAKE + 64), "status"),
])
def test_an_output_over_what_is_still_read_is_refused(call, kw, needle):
    """Other workgroups, or the call's second launch, read these lists while the output is written."""
    assert getattr(kda, call)(**dict(_CALLS[call], **kw)) == BAD
    assert needle in kda.kda_last_error()


def test_nothing_to_do_is_done():
    assert _prefill(T_tot=0, q=None, k=None, v=None, o=None, lse=None) == kda.KDA_OK
    assert kda.kda_last_error() == ""
    assert _tree(T_q=0, q=None, k_cache=None, v_cache=None, o=None, workspace=None, workspace_bytes=0) == kda.KDA_OK
    assert _backward(T_tot=0, q=None, k=None, v=None, o=None, lse=None, d_o=None, d_q=None, d_k_out=None, d_v_out=None,
                     workspace=None, workspace_bytes=0) == kda.KDA_OK


def test_torch_helpers_refuse_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 2, 32)
    with pytest.raises(ValueError, match="GPU"):
        kda.attn_prefill_t(x, x, x)
    with pytest.raises(ValueError, match="GPU"):
        kda.attn_prefill_backward_t(x, x, x, x, x[..., 0], x)


@pytest.mark.parametrize("shape,stride,want", [
    ((5, 2, 32), (64, 32, 1), 64),
    ((5, 2, 32), (200, 32, 1), 200),       # a slice of a wider projection
    ((1, 2, 32), (7, 32, 1), 64),          # one token: its stride says nothing
    ((5, 1, 32), (96, 5, 1), 96),          # one head: nor does the heads'
    ((0, 2, 32), (1, 1, 1), 64),
    ((5, 2, 32), (64, 1, 2), None),        # heads last
    ((5, 2, 32), (32, 160, 1), None),      # heads first
])
def test_token_strides(shape, stride, want):
    torch = pytest.importorskip("torch")
    from gated_delta_rule_60_amd import _attn
    t = torch.as_strided(torch.zeros(2000), shape, stride)
    if want is None:
        with pytest.raises(ValueError, match="contiguous"):
            _attn._tokens(t, "q", shape, t.dtype, t.device)
    else:
        assert _attn._tokens(t, "q", shape, t.dtype, t.device) == want
