"""Sizes that the kernels of the serving operators cannot take: refused on the
host before any HIP call (so these run without a GPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


A = 0x100000  # an aligned address; no call here gets as far as using it


def prefill(sq, **kw):
    d = dict(n_seq=1, n_tokens=1, n_heads=1, n_k_heads=1, d_k=4, d_v=4, dtype=1, rule=0, q=A, k=A, v=A, q_stride=4,
             k_stride=4, v_stride=4, alpha=A, beta=A, cu_seqlens=A, o=A, S=A, workspace=A, workspace_bytes=1 << 62)
    return sq._lib.sq_prefill(ctypes.byref(sq.SqPrefillDesc(**(d | kw))), None)


@pytest.mark.parametrize("n_tokens", [2 ** 31 - 1, 2 ** 31 - 16, 2 ** 31 - 64])
@pytest.mark.parametrize("kw", [{}, dict(dtype=0), dict(d_k=128, d_v=128, q_stride=128, k_stride=128, v_stride=128),
                                dict(d_k=128, d_v=128, q_stride=128, k_stride=128, v_stride=128, rule=1)])
def test_prompt_positions_are_32_bits(sq, n_tokens, kw):
    """Counting on by 16 or 64 tokens from the last would wrap."""
    assert prefill(sq, n_tokens=n_tokens, **kw) == sq.SQ_ERR_UNSUPPORTED
