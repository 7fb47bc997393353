"""Sizes past 32 bits are refused by the Python binding, not cut to their low
32 bits (2^32 + 16 tokens at most is not 16 tokens at most).  No GPU is used."""
import pytest
import torch

BIG = [2 ** 31, 2 ** 32, 2 ** 32 + 16, -2 ** 31 - 1, 2 ** 40]


@pytest.fixture()
def sq(monkeypatch):
    from quantized_recurrent_state_gated_amd import sq as m
    monkeypatch.setattr(m, "_DEVICE_TYPES", ("cpu",))
    return m


@pytest.fixture()
def called(sq, monkeypatch):
    """Names of the library's functions that were called in spite of it."""
    names = []
    for n in ("sq_prefill", "sq_paged_attention", "sq_block_tables", "sq_prefill_workspace",
              "sq_paged_attention_workspace"):
        monkeypatch.setattr(sq._lib, n, lambda *a, n=n: names.append(n) or 0)
    return names


@pytest.mark.parametrize("big", BIG)
def test_attention(sq, called, big):
    c = sq.SqKvCache(torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 64, 16))
    q, o = torch.zeros(2, 2, 64), torch.zeros(2, 2, 64)
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for args, kw in (((big,), {}), ((16,), dict(window=big))):
        with pytest.raises(sq.SqError) as e:
            sq.sq_paged_attention(c, q, table, lens, *args, o, **kw)
        assert e.value.status == sq.SQ_ERR_INVALID
    for n, heads, most in ((big, 2, 16), (2, big, 16), (2, 2, big)):
        with pytest.raises(sq.SqError):
            sq.sq_paged_attention_workspace(c, n, heads, most)
    assert not called
    sq.sq_paged_attention(c, q, table, lens, 2 ** 31 - 1, o, window=2 ** 31 - 1)
    assert called == ["sq_paged_attention"]


@pytest.mark.parametrize("big", BIG)
def test_tables(sq, called, big):
    i = torch.zeros(2, dtype=torch.int32)
    i3, i1 = torch.zeros(3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(sq.SqError):
        sq.sq_block_tables(i, i, big, i, torch.zeros(2, 1, dtype=torch.int32), i, i3, i3,
                           torch.zeros(2, dtype=torch.int64), i1)
    assert not called


@pytest.mark.parametrize("big", BIG)
def test_prompts(sq, called, big):
    t, g = torch.zeros(5, 2, 8), torch.zeros(5, 2)
    with pytest.raises(sq.SqError):
        sq.sq_prefill(t, t, t, g, g, torch.tensor([0, 5], dtype=torch.int32), torch.zeros(5, 2, 8), rule=big)
    for at in range(5):
        sizes = [1, 5, 2, 8, 8]
        sizes[at] = big
        with pytest.raises(sq.SqError):
            sq.sq_prefill_workspace(*sizes, torch.float32)
    assert not called


def test_more_tokens_than_32_bits(sq, called):
    """2^32 + 5 tokens of views that repeat one row: not five tokens."""
    N = 2 ** 32 + 5
    row = torch.zeros(1, 1, 4)
    q = row.expand(N, 1, 4)
    with pytest.raises(sq.SqError):
        sq.sq_prefill(q, q, q, 64, 64, torch.tensor([0, 5], dtype=torch.int32), 64)  # device pointers for the rest
    assert not called
