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


def cache(sq, **kw):
    d = dict(k=A, v=A, n_pages=4, page_size=16, n_kv_heads=1, head_dim=32, dtype=1)
    return ctypes.byref(sq.SqKvCacheDesc(**(d | kw)))


# A launch has fewer than 2^32 threads: 2^24 workgroups of 256 are too many.

@pytest.mark.parametrize("dtype,n_tok,heads", [(1, 2 ** 30, 1), (1, 2 ** 28 - 64, 8), (0, 2 ** 29, 1)])
def test_append_of_too_many_tiles(sq, dtype, n_tok, heads):
    c = cache(sq, n_kv_heads=heads, dtype=dtype)
    assert sq._lib.sq_kv_append(c, A, A, heads * 32, heads * 32, A, n_tok, None) == sq.SQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("n_req,heads,kv,max_len", [
    (2 ** 24, 1, 1, 16),           # one split each
    (2 ** 19, 32, 32, 100),
    (2 ** 19, 17, 1, 2 ** 17),     # two tiles of query heads, 16 splits of 8,192 tokens
    (2 ** 21, 16, 1, 8193),        # the attention fits, the join of its two splits does not
    (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 30)])
def test_attention_of_too_many_requests(sq, n_req, heads, kv, max_len):
    c = cache(sq, n_kv_heads=kv)
    args = [c, A, heads * 32, n_req, heads, A, 2 ** 20, A, max_len, 1.0, 0, A, None, A, 1 << 62, None]
    assert sq._lib.sq_paged_attention(*args) == sq.SQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(n_seq=2 ** 20, n_heads=16, n_tokens=2 ** 20, d_k=4, d_v=4),                       # 2^24 workgroups
    dict(n_seq=2 ** 18, n_heads=16, n_tokens=2 ** 18, d_k=256, d_v=256, dtype=0),          # four for 256 columns
    dict(n_seq=2 ** 18, n_heads=32, n_tokens=13 * 2 ** 18, d_k=128, d_v=128),              # 768 threads each
    dict(n_seq=2 ** 18, n_heads=32, n_tokens=13 * 2 ** 18, d_k=128, d_v=128, rule=1)])
def test_prompts_of_too_many_tiles(sq, kw):
    H = kw["n_heads"]
    st = dict(n_k_heads=H, q_stride=H * kw["d_k"], k_stride=H * kw["d_k"], v_stride=H * kw["d_v"])
    assert prefill(sq, **kw, **st) == sq.SQ_ERR_UNSUPPORTED
