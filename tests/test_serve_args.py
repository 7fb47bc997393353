"""Argument checks of the serving operators, made on the host before any HIP
call (so these run without a GPU), and the workspace sizes."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


P = ctypes.c_void_p
A = 0x100000  # an aligned address; no call here gets as far as using it


def cache(sq, **kw):
    d = dict(k=A, v=A, n_pages=4, page_size=16, n_kv_heads=2, head_dim=64, dtype=1) | kw
    return sq.SqKvCacheDesc(**d)


BAD_CACHE = [(dict(k=None), -1), (dict(v=A + 8), -1), (dict(n_pages=0), -1), (dict(n_kv_heads=0), -1),
             (dict(dtype=2), -1), (dict(page_size=8), -2), (dict(page_size=48), -2), (dict(page_size=512), -2),
             (dict(head_dim=48), -2), (dict(head_dim=512), -2)]


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_cache_is_checked(sq, kw, status):
    c = ctypes.byref(cache(sq, **kw))
    assert sq._lib.sq_kv_append(c, A, A, 128, 128, A, 1, None) == status
    assert sq._lib.sq_paged_attention(c, A, 256, 1, 4, A, 1, A, 16, 1.0, 0, A, None, None, 0, None) == status
    assert sq._lib.sq_paged_attention_workspace(c, 1, 4, 10 ** 6) == 0


@pytest.mark.parametrize("at,bad,status", [
    (0, None, -1), (1, None, -1), (1, A + 2, -1), (2, None, -1), (3, 127, -1), (3, 132, -1), (4, 64, -1), (5, None, -1),
    (5, A + 4, -1), (6, -1, -1)])
def test_append_is_checked(sq, at, bad, status):
    args = [ctypes.byref(cache(sq)), A, A, 128, 128, A, 3, None]
    args[at] = bad
    assert sq._lib.sq_kv_append(*args) == status


def test_nothing_to_do_is_fine(sq):
    c = ctypes.byref(cache(sq))
    assert sq._lib.sq_kv_append(c, None, None, 0, 0, None, 0, None) == 0
    assert sq._lib.sq_paged_attention(c, None, 0, 0, 4, None, 0, None, 0, 1.0, 0, None, None, None, 0, None) == 0
    d = sq.SqPrefillDesc(n_heads=2, n_k_heads=2, d_k=8, d_v=8)
    assert sq._lib.sq_prefill(ctypes.byref(d), None) == 0


@pytest.mark.parametrize("at,bad,status", [
    (0, None, -1), (1, None, -1), (1, A + 8, -1), (2, 255, -1), (2, 260, -1), (3, -1, -1), (4, 0, -1), (4, 5, -1),
    (5, None, -1), (6, -1, -1), (7, None, -1), (8, -1, -1), (9, float("nan"), -1), (9, float("inf"), -1), (10, -1, -1),
    (11, None, -1), (11, A + 4, -1), (12, A + 2, -1), (13, None, -1), (13, A + 4, -1), (14, 100, -1)])
def test_attention_is_checked(sq, at, bad, status):
    # 5000 tokens are split, so the call needs its workspace
    args = [ctypes.byref(cache(sq)), A, 256, 2, 4, A, 400, A, 5000, 0.125, 0, A, None, A, 1 << 30, None]
    args[at] = bad
    assert sq._lib.sq_paged_attention(*args) == status


@pytest.mark.parametrize("at,bad,status", [
    (0, None, -1), (1, A + 2, -1), (2, -1, -1), (3, 0, -2), (3, 24, -2), (4, None, -1), (5, -1, -1), (6, None, -1),
    (7, -1, -1), (8, None, -1), (9, None, -1), (10, A + 1, -1), (11, None, -1), (11, A + 4, -1), (12, -1, -1),
    (12, 2 ** 31, -1), (13, None, -1)])
def test_tables_are_checked(sq, at, bad, status):
    args = [A, A, 3, 16, A, 9, A, 5, A, A, A, A, 40, A, None]
    args[at] = bad
    assert sq._lib.sq_block_tables(*args) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n_seq=-1), -1), (dict(n_tokens=-1), -1), (dict(n_heads=0), -1), (dict(n_k_heads=0), -1),
    (dict(n_k_heads=3), -1), (dict(dtype=3), -1), (dict(rule=2), -1), (dict(d_k=6), -2), (dict(d_v=260), -2),
    (dict(d_k=0), -2), (dict(q=None), -1), (dict(k=A + 1), -1), (dict(v=None), -1), (dict(q_stride=511), -1),
    (dict(k_stride=0), -1), (dict(v_stride=511), -1), (dict(alpha=None), -1), (dict(beta=A + 2), -1),
    (dict(cu_seqlens=None), -1), (dict(o=None), -1), (dict(S0=A + 4), -1), (dict(S=A + 8), -1)])
def test_prefill_is_checked(sq, kw, status):
    d = dict(n_seq=2, n_tokens=100, n_heads=4, n_k_heads=4, d_k=128, d_v=128, dtype=1, rule=0, q=A, k=A, v=A,
             q_stride=512, k_stride=512, v_stride=512, alpha=A, beta=A, cu_seqlens=A, S0=A, o=A, S=A, workspace=A,
             workspace_bytes=1 << 40)
    assert sq._lib.sq_prefill(ctypes.byref(sq.SqPrefillDesc(**(d | kw))), None) == status


def test_null_descriptors(sq):
    assert sq._lib.sq_prefill(None, None) == -1
    assert sq._lib.sq_paged_attention_workspace(None, 1, 1, 1) == 0


def test_prefill_workspace_is_enforced_and_grows(sq):
    for dtype in (torch.bfloat16, torch.float32):
        for rule in (0, 1):
            f = lambda *a: sq.sq_prefill_workspace(*a, 128, 128, dtype, rule)  # noqa: E731
            assert f(1, 64, 2) <= f(2, 64, 2) <= f(2, 500, 2) <= f(2, 500, 5)
            sizes = [(1, 64, 2), (1, 1984, 2), (1, 1985, 2), (1, 5000, 2), (2, 5000, 2), (2, 5000, 40), (2, 5000, 90),
                     (300, 5000, 90), (300, 500000, 90)]
            for a, b in zip(sizes, sizes[1:]):
                assert f(*a) <= f(*b)
    # a long plain decay of few heads is cut into segments, through the workspace
    d = dict(n_seq=1, n_tokens=5000, n_heads=4, n_k_heads=4, d_k=128, d_v=128, dtype=1, rule=1, q=A, k=A, v=A,
             q_stride=512, k_stride=512, v_stride=512, alpha=A, beta=A, cu_seqlens=A, o=A)
    nb = sq.sq_prefill_workspace(1, 5000, 4, 128, 128, torch.bfloat16, 1)
    assert nb > 0
    for ws, size in ((None, nb), (A, 1 << 16), (A + 16, nb)):
        x = sq.SqPrefillDesc(**d, workspace=ws, workspace_bytes=size)
        assert sq._lib.sq_prefill(ctypes.byref(x), None) == -1
    assert sq.sq_prefill_workspace(1, 10, 1, 6, 128, torch.bfloat16) == 0
    with pytest.raises(TypeError):
        sq.sq_prefill_workspace(1, 10, 1, 64, 128, torch.float16)


def test_attention_workspace_grows(sq):
    c = ctypes.byref(cache(sq))
    f = lambda n, m: sq._lib.sq_paged_attention_workspace(c, n, 4, m)  # noqa: E731
    for n in (1, 3, 50, 700, 5000):
        for m in (0, 1, 100, 128, 129, 1000, 5000, 20000, 100000):
            assert f(n, m) <= f(n + 1, m) and f(n, m) <= f(n, m + 1)


def test_binding_checks(sq, monkeypatch):
    monkeypatch.setattr(sq, "_DEVICE_TYPES", ("cpu",))
    bf = torch.bfloat16
    with pytest.raises(sq.SqError):
        sq.SqKvCache(torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 16, 64))  # values not transposed
    with pytest.raises(TypeError):
        sq.SqKvCache(torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 64, 16, dtype=bf))
    with pytest.raises(TypeError):
        sq.SqKvCache(torch.zeros(2, 1, 16, 64, dtype=torch.float16), torch.zeros(2, 1, 64, 16, dtype=torch.float16))
    c = sq.SqKvCache(torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 64, 16))
    slots = torch.zeros(3, dtype=torch.int64)
    x = torch.zeros(3, 1, 64)
    with pytest.raises(TypeError):
        sq.sq_kv_append(c, x.to(bf), x, slots)
    with pytest.raises(TypeError):
        sq.sq_kv_append(c, x, x, slots.int())
    with pytest.raises(sq.SqError):
        sq.sq_kv_append(c, x, torch.zeros(2, 1, 64), slots)
    with pytest.raises(sq.SqError):
        sq.sq_kv_append(c, x, torch.zeros(3, 1, 128)[:, :, ::2], slots)
    q, o = torch.zeros(2, 2, 64), torch.zeros(2, 2, 64)
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(sq.SqError):
        sq.sq_paged_attention(c, q, table[:1], lens, 16, o)
    with pytest.raises(TypeError):
        sq.sq_paged_attention(c, q, table, lens.long(), 16, o)
    with pytest.raises(TypeError):
        sq.sq_paged_attention(c, q, table, lens, 16, o.to(bf))
    with pytest.raises(sq.SqError):
        sq.sq_paged_attention(c, torch.zeros(2, 2, 32), table, lens, 16, o)
    with pytest.raises(sq.SqError):
        sq.sq_paged_attention(c, q, table, lens, 16, o, lse=torch.zeros(3))
    i = torch.zeros(2, dtype=torch.int32)
    i3, i1 = torch.zeros(3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(sq.SqError):
        sq.sq_block_tables(i, i, 16, i, table, i, i, i3, slots, i1)
    with pytest.raises(sq.SqError):
        sq.sq_block_tables(i, i, 16, i, table[:1], i, i3, i3, slots, i1)
    with pytest.raises(TypeError):
        sq.sq_block_tables(i, i, 16, i, table, i, i3, i3, slots.int(), i1)
    N, H, d = 5, 2, 8
    t = torch.zeros(N, H, d)
    g, cu = torch.zeros(N, H), torch.tensor([0, 5], dtype=torch.int32)
    ok = dict(q=t, k=t, v=t, alpha=g, beta=g, cu_seqlens=cu, o=torch.zeros(N, H, d))
    for kw, err in ((dict(q=t.to(bf)), TypeError), (dict(alpha=g[:4]), sq.SqError), (dict(alpha=g.to(bf)), TypeError),
                    (dict(cu_seqlens=cu.long()), TypeError), (dict(o=torch.zeros(N, H, d + 4)), sq.SqError),
                    (dict(k=torch.zeros(N, H, d + 4)), sq.SqError), (dict(S=torch.zeros(1, H, d, d + 4)), sq.SqError),
                    (dict(S0=torch.zeros(1, H, d, d, dtype=bf)), TypeError), (dict(q=t[0]), sq.SqError),
                    (dict(v=torch.zeros(N, d, H).transpose(1, 2)), sq.SqError), (dict(rule=5), sq.SqError),
                    (dict(workspace=[1]), TypeError), (dict(q=t.to(torch.float16)), TypeError)):
        with pytest.raises(err):
            sq.sq_prefill(**(ok | kw))


def test_attention_longer_than_its_positions(sq):
    """Token positions are 32 bits: what a row can hold decides, not max_len alone."""
    most = 2 ** 31 - 1
    args = [ctypes.byref(cache(sq)), A, 256, 1, 4, A, most, A, most, 0.125, 0, A, None, A, 1 << 60, None]
    assert sq._lib.sq_paged_attention(*args) == -2
    args[8] = 2 ** 30 + 1
    assert sq._lib.sq_paged_attention(*args) == -2
    args[10] = 128  # a window does not shorten the row
    assert sq._lib.sq_paged_attention(*args) == -2
