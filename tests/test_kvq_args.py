"""Argument checks of the 8-bit cache's calls, made on the host before any HIP
call (so these run without a GPU), its workspace sizes and the Python binding's checks."""
import ctypes

import pytest
import torch

A = 0x100000  # an aligned address; no call here gets as far as using it
BIG = [2 ** 31, 2 ** 32, 2 ** 32 + 16, -2 ** 31 - 1, 2 ** 40]


@pytest.fixture()
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


def cache(sq, **kw):
    d = dict(k=A, v=A, scales=A, n_pages=4, page_size=16, n_kv_heads=2, head_dim=64, format=0) | kw
    return ctypes.byref(sq.SqKvqCacheDesc(**d))


def append_args(sq, **kw):
    #     0 cache    1 k 2 v 3 ks 4 vs 5 dtype 6 n_tok 7 ctx 8 cu 9 n_req 10 table 11 stride 12 stream
    return [cache(sq, **kw), A, A, 128, 128, 1, 5, A, A, 2, A, 3, None]


def load_args(sq, **kw):
    #     0 cache    1 first 2 cu 3 n_req 4 table 5 stride 6 k 7 v 8 ks 9 vs 10 dtype 11 n_tok 12 stream
    return [cache(sq, **kw), A, A, 2, A, 3, A, A, 128, 128, 1, 5, None]


def attend_args(sq, **kw):
    # 0 cache 1 q 2 qs 3 dtype 4 n_q 5 n_heads 6 cu 7 n_req 8 table 9 stride 10 lens 11 max_len 12 scale 13 window
    # 14 o 15 lse 16 ws 17 bytes 18 stream; 5000 tokens are split, so the call needs its workspace
    return [cache(sq, **kw), A, 256, 1, 2, 4, None, 2, A, 400, A, 5000, 0.125, 0, A, None, A, 1 << 30, None]


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(scales=None), -1), (dict(k=A + 8), -1), (dict(v=A + 4), -1),
    (dict(scales=A + 8), -1), (dict(n_pages=0), -1), (dict(n_kv_heads=0), -1), (dict(format=2), -1), (dict(format=-1), -1),
    (dict(page_size=8), -2), (dict(page_size=48), -2), (dict(page_size=512), -2), (dict(head_dim=48), -2),
    (dict(head_dim=512), -2), (dict(head_dim=0), -2)])
def test_cache_is_checked(sq, kw, status):
    assert sq._lib.sq_kvq_append(*append_args(sq, **kw)) == status
    assert sq._lib.sq_kvq_load(*load_args(sq, **kw)) == status
    assert sq._lib.sq_kvq_attention(*attend_args(sq, **kw)) == status
    assert sq._lib.sq_kvq_attention_workspace(cache(sq, **kw), 1, 1, 4, 10 ** 6) == 0


@pytest.mark.parametrize("at,bad", [
    (0, None), (1, None), (1, A + 8), (2, None), (2, A + 2), (3, 127), (3, 132), (4, 64), (5, 2), (5, -1), (6, -1),
    (7, None), (7, A + 2), (8, None), (8, A + 1), (9, -1), (10, None), (10, A + 2), (11, -1)])
def test_append_is_checked(sq, at, bad):
    args = append_args(sq)
    args[at] = bad
    assert sq._lib.sq_kvq_append(*args) == sq.SQ_ERR_INVALID


@pytest.mark.parametrize("at,bad", [
    (0, None), (1, A + 2), (2, None), (2, A + 1), (3, -1), (4, None), (4, A + 2), (5, -1), (6, A + 8), (7, A + 4),
    (8, 127), (8, 132), (9, 0), (10, 2), (11, -1)])
def test_load_is_checked(sq, at, bad):
    args = load_args(sq)
    args[at] = bad
    assert sq._lib.sq_kvq_load(*args) == sq.SQ_ERR_INVALID
    args = load_args(sq)
    args[6] = args[7] = None
    assert sq._lib.sq_kvq_load(*args) == sq.SQ_ERR_INVALID


@pytest.mark.parametrize("at,bad,status", [
    (0, None, -1), (1, None, -1), (1, A + 8, -1), (2, 255, -1), (2, 260, -1), (3, 2, -1), (4, -1, -1), (4, 3, -1),
    (5, 0, -1), (5, 5, -1), (6, A + 2, -1), (7, -1, -1), (7, 1, -1), (8, None, -1), (8, A + 2, -1), (9, -1, -1),
    (10, None, -1), (10, A + 1, -1), (11, -1, -1), (12, float("nan"), -1), (12, float("inf"), -1), (13, -1, -1),
    (14, None, -1), (14, A + 4, -1), (15, A + 2, -1), (16, None, -1), (16, A + 4, -1), (17, 100, -1)])
def test_attention_is_checked(sq, at, bad, status):
    args = attend_args(sq)
    args[at] = bad
    assert sq._lib.sq_kvq_attention(*args) == status


def test_nothing_to_do_is_fine(sq):
    c = cache(sq)
    assert sq._lib.sq_kvq_append(c, None, None, 0, 0, 0, 0, None, None, 3, None, 0, None) == 0
    assert sq._lib.sq_kvq_append(c, A, A, 128, 128, 0, 5, None, None, 0, None, 0, None) == 0
    assert sq._lib.sq_kvq_load(c, None, None, 0, None, 0, None, None, 0, 0, 0, 5, None) == 0
    assert sq._lib.sq_kvq_attention(c, None, 0, 0, 0, 4, None, 0, None, 0, None, 0, 1.0, 0, None, None, None, 0, None) == 0
    assert sq._lib.sq_kvq_attention(c, None, 0, 0, 0, 4, A, 3, None, 0, None, 0, 1.0, 0, None, None, None, 0, None) == 0


@pytest.mark.parametrize("n_tok,n_req,heads", [(2 ** 31 - 1, 1, 2), (5, 2 ** 25, 1), (2 ** 28, 1, 4)])
def test_rows_of_too_many_blocks(sq, n_tok, n_req, heads):
    """A launch has fewer than 2^32 threads, a wave for each block and head, keys and values."""
    args = append_args(sq, n_kv_heads=heads)
    args[3] = args[4] = heads * 64
    args[6], args[9] = n_tok, n_req
    assert sq._lib.sq_kvq_append(*args) == sq.SQ_ERR_UNSUPPORTED
    args = load_args(sq, n_kv_heads=heads)
    args[8] = args[9] = heads * 64
    args[11], args[3] = n_tok, n_req
    assert sq._lib.sq_kvq_load(*args) == sq.SQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("n_q,n_req,heads,kv,max_len", [
    (2 ** 24, 2 ** 24, 1, 1, 16), (2 ** 30, 2 ** 30, 1, 1, 16), (2 ** 31 - 1, 1, 1, 1, 16), (2 ** 29, 3, 4, 2, 100),
    (2 ** 19, 2 ** 19, 32, 32, 100), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 30)])
@pytest.mark.parametrize("cu", [None, A])
def test_attention_of_too_much(sq, n_q, n_req, heads, kv, max_len, cu):
    if cu is None and n_q != n_req:
        return
    args = attend_args(sq, n_kv_heads=kv)
    args[2], args[4], args[5], args[6], args[7], args[9], args[11], args[17] = heads * 64, n_q, heads, cu, n_req, 2 ** 27, max_len, 1 << 62
    assert sq._lib.sq_kvq_attention(*args) == sq.SQ_ERR_UNSUPPORTED


def test_more_tokens_than_positions(sq):
    args = attend_args(sq)
    args[9], args[11], args[17] = 2 ** 28, 2 ** 30 + 1, 1 << 62
    assert sq._lib.sq_kvq_attention(*args) == sq.SQ_ERR_UNSUPPORTED
    assert sq._lib.sq_kvq_attention_workspace(cache(sq), 2, 2, 4, 2 ** 30 + 1) == 0


def test_workspace_grows_with_its_arguments(sq):
    c = cache(sq)
    size = sq._lib.sq_kvq_attention_workspace
    assert size(c, 0, 1, 4, 100) == size(c, 1, 0, 4, 100) == size(c, 1, 1, 3, 100) == size(c, 1, 1, 4, -1) == 0
    last = 0
    for n in (1, 3, 64, 1000):
        for m in (1, 255, 256, 257, 8192, 10 ** 5, 10 ** 6):
            assert size(c, n, n, 4, m) >= (last if m > 1 else 0)
            assert size(c, n, 2 * n, 4, m) >= size(c, n, n, 4, m)
            last = size(c, n, n, 4, m)


# ---------------------------------------------------------------- the binding

@pytest.fixture()
def called(sq, monkeypatch):
    monkeypatch.setattr(sq, "_DEVICE_TYPES", ("cpu",))
    names = []
    for n in ("sq_kvq_append", "sq_kvq_load", "sq_kvq_attention", "sq_kvq_attention_workspace"):
        monkeypatch.setattr(sq._lib, n, lambda *a, n=n: names.append(n) or 0)
    return names


def host_cache(sq, fmt=0):
    return sq.SqKvqCache(torch.zeros(4, 2, 32, 64, dtype=torch.uint8), torch.zeros(4, 2, 2, 64, 16, dtype=torch.uint8),
                         torch.zeros(4, 2, 2, 2), fmt)


def test_cache_tensors_are_checked(sq, called):
    k, v, s = torch.zeros(4, 2, 32, 64, dtype=torch.uint8), torch.zeros(4, 2, 2, 64, 16, dtype=torch.uint8), torch.zeros(4, 2, 2, 2)
    for bad in ((k[0], v, s), (k, v.view(4, 2, 64, 32), s), (k, v, s.view(4, 2, 4)), (k, v[:3], s), (k, v, s[:3]),
                (k.transpose(1, 2), v, s), (k, v, s, 2)):
        with pytest.raises(sq.SqError):
            sq.SqKvqCache(*bad)
    for bad in ((k.to(torch.int8), v, s), (k, v.to(torch.int8), s), (k, v, s.double())):
        with pytest.raises(TypeError):
            sq.SqKvqCache(*bad)
    c = sq.SqKvqCache(k, v, s, sq.SQ_KVQ_E4M3)
    assert (c.n_pages, c.n_kv_heads, c.page_size, c.head_dim, c.format) == (4, 2, 32, 64, 1)


def test_binding_checks_rows(sq, called):
    c = host_cache(sq)
    i2, i3 = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    t, x = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(5, 2, 64)
    sq.sq_kvq_append(c, x, x, i2, i3, t)
    sq.sq_kvq_load(c, t, i3, x, x, first=i2)
    sq.sq_kvq_load(c, t, i3, v=x)
    assert called == ["sq_kvq_append", "sq_kvq_load", "sq_kvq_load"]
    del called[:]
    for args in ((x[:, :1], x, i2, i3, t), (x, x[:4], i2, i3, t), (x, x, i2, i2, t), (x, x, i2, i3, t[:1]),
                 (x, x, i2, i3, t.view(-1)), (x.transpose(1, 2).contiguous().transpose(1, 2), x, i2, i3, t)):
        with pytest.raises(sq.SqError):
            sq.sq_kvq_append(c, *args)
    for args in ((x.bfloat16(), x, i2, i3, t), (x.double(), x.double(), i2, i3, t), (x, x, i2.long(), i3, t),
                 (x, x, i2, i3, t.long())):
        with pytest.raises(TypeError):
            sq.sq_kvq_append(c, *args)
    for kw in (dict(), dict(k=x, first=i3), dict(k=x, v=x[:4])):
        with pytest.raises(sq.SqError):
            sq.sq_kvq_load(c, t, i3, **kw)
    with pytest.raises(TypeError):
        sq.sq_kvq_load(c, t, i3, x, x.bfloat16())
    assert not called


def test_binding_checks_attention(sq, called):
    c = host_cache(sq)
    i2, i3, t = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    q, o = torch.zeros(5, 4, 64), torch.zeros(5, 4, 64)
    sq.sq_kvq_attention(c, q, t, i2, 50, o, cu_q=i3, lse=torch.zeros(5, 4))
    assert called.pop() == "sq_kvq_attention"
    for args, kw in (((q[0], t, i2, 50, o), {}), ((q, t[:1], i2, 50, o), dict(cu_q=i3)), ((q, t, i2, 50, o[:4]), dict(cu_q=i3)),
                     ((q, t, i2, 50, o), dict(cu_q=i2)), ((q[..., :32], t, i2, 50, o), dict(cu_q=i3)),
                     ((q, t, i2, 50, o), dict(cu_q=i3, lse=torch.zeros(4)))):
        with pytest.raises(sq.SqError):
            sq.sq_kvq_attention(c, *args, **kw)
    for args, kw in (((q, t, i2, 50, o.bfloat16()), dict(cu_q=i3)), ((q, t, i2.long(), 50, o), dict(cu_q=i3)),
                     ((q, t, i2, 50, o), dict(cu_q=i3.long()))):
        with pytest.raises(TypeError):
            sq.sq_kvq_attention(c, *args, **kw)
    for big in BIG:
        for args, kw in (((big, o), {}), ((16, o), dict(window=big))):
            with pytest.raises(sq.SqError):
                sq.sq_kvq_attention(c, q, t, i2, *args, cu_q=i3, **kw)
        for sizes in ((big, 2, 4, 16), (2, big, 4, 16), (2, 2, big, 16), (2, 2, 4, big)):
            with pytest.raises(sq.SqError):
                sq.sq_kvq_attention_workspace(c, *sizes)
    assert not called
