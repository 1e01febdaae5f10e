"""The entry points of windowed attention on the CPU: every refusal comes
before any HIP call (no kernel is launched here)."""
import pytest

import gated_delta_rule_60_amd as kda
from test_attn_abi import BAD, BF16, COMMON, F32, FAKE


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
